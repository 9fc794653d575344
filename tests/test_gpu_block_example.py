"""The example block (examples/mamba2_block.py): norms, 8-bit checkpoints and
mixer used together, against a plain fp64 block with autograd.

Tolerances, relative in the 2-norm.  A checkpoint's step is at most max/63.75 of
its 32 columns, about 2.5 sigma / 63.75 = 0.04 sigma: an rms error of 0.04 /
sqrt(12) = 1.2%; six of them reach a gradient, and about ten bf16 roundings of
2^-9 each: 6 * 1.2% + 10 * 0.2% = 9.2% were they to add up.  Outputs see only the
bf16 roundings (u, p, g, out; weights are given) and the mixer's products: 1.5%.
"""
import importlib.util
import os

import pytest
import torch
import torch.nn.functional as F

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "mamba2_block.py")
OUT, GRAD = 0.015, 0.092


def load():
    spec = importlib.util.spec_from_file_location("mamba2_block", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def plain(p, x, residual, heads, groups, dstate):
    """The block in fp64 on the CPU, its recurrence step by step."""
    b, length, _ = x.shape
    inner = p["w_out"].shape[1]
    rms = lambda v: v / torch.sqrt(v.square().mean(-1, keepdim=True) + 1e-5)  # noqa: E731
    r = residual + x
    z, xs, bs, cs, dt = (rms(r) * p["norm"] @ p["w_in"].t()).split(
        [inner, inner, groups * dstate, groups * dstate, heads], dim=-1)
    xs = xs.view(b, length, heads, -1)
    bs, cs = (t.view(b, length, groups, dstate).repeat_interleave(heads // groups, 2) for t in (bs, cs))
    delta, a = F.softplus(dt + p["dt_bias"]), -torch.exp(p["a_log"])
    h, ys = torch.zeros(b, heads, xs.shape[3], dstate, dtype=torch.float64), []
    for t in range(length):
        h = torch.exp(delta[:, t] * a)[..., None, None] * h + (
            delta[:, t, :, None, None] * xs[:, t, :, :, None] * bs[:, t, :, None, :])
        ys.append((h * cs[:, t, :, None, :]).sum(-1) + p["d"][:, None] * xs[:, t])
    y = torch.stack(ys, 1).reshape(b, length, inner)
    return rms(y * F.silu(z)) * p["gate_norm"] @ p["w_out"].t(), r


def rel(got, ref):
    got = got.detach().double().cpu()
    return float((got - ref).norm() / ref.norm())


@pytest.mark.parametrize("b,length,width,heads,groups", [(2, 100, 96, 2, 1), (1, 65, 136, 4, 2)])
def test_training_step(b, length, width, heads, groups):
    m = load()
    torch.manual_seed(3)
    block = m.Mamba2Block(width, heads, groups=groups, dstate=64)
    x = torch.randn(b, length, width).bfloat16()
    residual, do, dr = torch.randn(b, length, width), torch.randn(b, length, width).bfloat16(), torch.randn(b, length, width)
    ref_p = {k: v.detach().double().cpu().requires_grad_(True) for k, v in block.named_parameters()}
    rx, rr = x.double().requires_grad_(True), residual.double().requires_grad_(True)
    ro, rres = plain(ref_p, rx, rr, heads, groups, 64)
    ((ro * do.double()).sum() + (rres * dr.double()).sum()).backward()

    gx, gr = x.cuda().requires_grad_(True), residual.cuda().requires_grad_(True)
    out, res = block(gx, gr)
    assert rel(out, ro.detach()) <= OUT and rel(res, rres.detach()) <= 1e-6
    torch.autograd.backward([out, res], [do.cuda(), dr.cuda()])
    assert rel(gx.grad, rx.grad) <= GRAD and rel(gr.grad, rr.grad) <= GRAD
    for k, v in block.named_parameters():
        assert rel(v.grad, ref_p[k].grad) <= GRAD, k


def test_generation_follows_the_chunked_pass():
    m = load()
    torch.manual_seed(4)
    b, length, width, heads = 2, 20, 128, 2
    block = m.Mamba2Block(width, heads, dstate=64)
    x = torch.randn(b, length, width, device="cuda").bfloat16()
    residual = torch.randn(b, length, width, device="cuda")
    with torch.no_grad():
        out, res = block(x, residual)
    h = block.state(b)
    for t in range(length):
        y, r = block.step(x[:, t], residual[:, t], h)
        assert torch.equal(r, res[:, t])
        # both differ from the exact value by the bf16 roundings; y is one more here
        assert rel(y, out[:, t].double().cpu()) <= 2 * OUT
