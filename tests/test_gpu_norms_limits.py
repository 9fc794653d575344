"""The norms at the far ends of what they take.

Tolerance as in test_gpu_norms.py (128 units of 2^-24 of the size of a value's
terms, 192 for sums over rows, half a bf16 step), the reference in fp64 by torch
on the GPU, for its size.
"""
import pytest
import torch

import selective_state_space_27_amd as mss

pytestmark = pytest.mark.gpu

U, UROWS, EPS24 = 128, 192, 2.0 ** -24


def test_gradient_of_more_columns_than_a_launch_holds():
    """The sums over rows take 64 threads a column; a launch has fewer than 2^32
    along an axis, which 2^26 columns would need."""
    rows, groups, width = 2, 4098, 16384
    cols = groups * width
    assert cols > 1 << 26
    g = torch.Generator(device="cuda:0")
    g.manual_seed(1)
    y = torch.randn(rows, cols, generator=g, device="cuda:0").bfloat16()
    do = torch.randn(rows, cols, generator=g, device="cuda:0").bfloat16()
    w = 1.0 + 0.2 * torch.randn(cols, generator=g, device="cuda:0")
    got = mss.gated_norm_bwd(do, y, None, w, ngroups=groups)

    v, d = (t.double().view(rows, groups, width) for t in (y, do))
    wd = w.double().view(groups, width)
    rstd = 1.0 / torch.sqrt((v * v).mean(2, keepdim=True) + 1e-5)
    t = d * v * rstd
    off = (got["dweight"].double().view(groups, width) - t.sum(0)).abs() - UROWS * EPS24 * t.abs().sum(0)
    assert off.max() <= 0
    gw = d * wd
    ref = rstd * gw - v * rstd ** 3 * (gw * v).mean(2, keepdim=True)
    size = rstd * gw.abs() + v.abs() * rstd ** 3 * (gw * v).abs().mean(2, keepdim=True)
    tol = U * EPS24 * size
    tol = tol + torch.exp2(torch.floor(torch.log2((ref.abs() + tol).clamp_min(2.0 ** -126))) - 8)
    assert ((got["dy"].double().view(rows, groups, width) - ref).abs() - tol).max() <= 0
