"""GPU parity of the norms around the mixer against the fp64 reference.

Tolerance, per element: U * 2^-24 * size, size the sum of the magnitudes of the
terms the value is made of (oracle/block.py), plus half a bf16 step of the value
itself where it is stored in bf16.  U counts fp32 roundings: a row's sums have
at most 16 sequential terms per thread and 10 levels over lanes and waves, which
move rstd and the means by at most 26; the gate's sigmoid is off by |z| + 4 units
of 2^-23 (the exponent's argument is rounded, two hardware functions of one unit
each), |z| < 12 here: 32; a dozen further products.  U = 128 covers their sum.
Sums over rows: a thread's rows in order, then at most 64 slices: U = 128 + the
rows a workgroup can see here (at most 64).  The 8-bit forms are exact: bit for
bit.
"""
import numpy as np
import pytest
import torch

import selective_state_space_27_amd as mss
from block_util import half_step
from gpu_util import host64
from oracle import block as ob

pytestmark = pytest.mark.gpu

U, UROWS, EPS24 = 128, 192, 2.0 ** -24
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
PAIRS = [("bf16", "fp32"), ("bf16", "bf16"), ("fp32", "fp32")]  # io, wide


def close(got, ref, size, what, u=U):
    got_dtype, got = got.dtype, host64(got)
    ref, size = np.broadcast_to(ref, got.shape), np.broadcast_to(size, got.shape)
    tol = u * EPS24 * size + 1e-37
    tol = tol + (half_step(np.abs(ref) + tol) if got_dtype == torch.bfloat16 else 0.0)
    off = np.abs(got - ref) - tol
    assert np.isfinite(got).all() and off.max() <= 0, (
        f"{what}: {np.abs(got - ref).max():.3e} off at {np.unravel_index(off.argmax(), off.shape)}, tol there "
        f"{tol.reshape(-1)[off.argmax()]:.3e}")


def gen(seed):
    g = torch.Generator(device="cuda:0")
    g.manual_seed(seed)
    return g


def act(g, rows, cols, dtype, scale=1.0, pad=0):
    """Values of unlike sizes; pad > 0: a slice of wider rows, off every alignment."""
    v = torch.randn(rows, cols, generator=g, device="cuda:0") * torch.exp(
        0.7 * torch.randn(1, cols, generator=g, device="cuda:0")) * scale
    if pad == 0:
        return v.to(dtype)
    wide = torch.full((rows, cols + 2 * pad), float("nan"), dtype=dtype, device="cuda:0")
    wide[:, pad:pad + cols] = v.to(dtype)
    return wide[:, pad:pad + cols]


def weight(g, cols):
    return 1.0 + 0.2 * torch.randn(cols, generator=g, device="cuda:0")


def cols_of():
    # every layout of a row over lanes and both sides of its borders; odd sizes
    return [1, 7, 8, 33, 128, 129, 255, 256, 257, 511, 512, 513, 1001, 2560, 5120, 8191, 8192, 8193, 10240, 16384]


@pytest.mark.parametrize("cols", cols_of())
def test_add_norm_fwd_sizes(cols):
    g = gen(cols)
    io, wide = PAIRS[cols % 3]
    rows = 5 if cols > 512 else 37
    x, res, w = act(g, rows, cols, DT[io]), act(g, rows, cols, DT[wide], 3.0), weight(g, cols)
    out, r, p = mss.add_norm_fwd(x, res, w, pack_out=True)
    ro, rr = ob.add_norm(host64(x), host64(res), host64(w))
    so, sr = ob.add_norm_sizes(host64(x), host64(res), host64(w))
    close(out, ro, so, "out")
    close(r, rr, sr, "residual_out")
    q, e = ob.pack8(host64(out))
    assert np.array_equal(p.q.cpu().numpy(), q) and np.array_equal(p.scale.cpu().numpy(), e)
    assert torch.equal(mss.pack8(out).q, p.q) and torch.equal(mss.pack8(out).scale, p.scale)


@pytest.mark.parametrize("io,wide", PAIRS)
@pytest.mark.parametrize("post,gamma", [(False, False), (False, True), (True, False), (True, True)])
@pytest.mark.parametrize("rows,cols,pad", [(1, 2560, 0), (3, 100, 3), (70, 768, 5), (9, 9000, 1), (4, 15001, 0)])
def test_add_norm_fwd_options(io, wide, post, gamma, rows, cols, pad):
    g = gen(rows)
    x, res, w = act(g, rows, cols, DT[io], pad=pad), act(g, rows, cols, DT[wide], 3.0, pad=pad), weight(g, cols)
    pw, gm = weight(g, cols) if post else None, weight(g, cols) if gamma else None
    out, r = mss.add_norm_fwd(x, res, w, post_weight=pw, gamma=gm, scale=0.25, eps=1e-3)
    args = (host64(x), host64(res), host64(w), None if pw is None else host64(pw), None if gm is None else host64(gm),
            0.25, 1e-3)
    (ro, rr), (so, sr) = ob.add_norm(*args), ob.add_norm_sizes(*args)
    close(out, ro, so, "out")
    close(r, rr, sr, "residual_out")


def test_add_norm_without_residual_and_residual_dtype():
    g = gen(1)
    x, w = act(g, 6, 320, torch.bfloat16), weight(g, 320)
    out, r = mss.add_norm_fwd(x, None, w, residual_dtype=torch.float32, scale=2.0)
    assert r.dtype == torch.float32 and torch.equal(r, 2.0 * x.float())
    zero = torch.zeros(6, 320, device="cuda:0")
    out0, r0 = mss.add_norm_fwd(x, zero, w, scale=2.0)
    assert torch.equal(out, out0) and torch.equal(r, r0)
    assert mss.add_norm_fwd(x, None, w)[1].dtype == torch.bfloat16


def add_bwd_case(g, rows, cols, io, wide, post, gamma, packed=False, pad=0, dres=True):
    x, r, w = act(g, rows, cols, DT[io], pad=pad), act(g, rows, cols, DT[wide], 3.0, pad=pad), weight(g, cols)
    do = act(g, rows, cols, DT[io], 1e-2, pad=pad)
    e = act(g, rows, cols, DT[wide], 1e-2, pad=pad) if dres else None
    pw, gm = weight(g, cols) if post else None, weight(g, cols) if gamma else None
    xin, rin, x64, r64 = x, r, host64(x), host64(r)
    if packed:
        xin, rin = mss.pack8(x), mss.pack8(r)
        x64, r64 = host64(mss.unpack8(xin, torch.float32)), host64(mss.unpack8(rin, torch.float32))
    got = mss.add_norm_bwd(do, rin, w, dresidual_out=e, x=xin if post or gamma else None, post_weight=pw, gamma=gm,
                           scale=0.5, eps=1e-4)
    h = lambda t: None if t is None else host64(t)  # noqa: E731
    ref = ob.add_norm_bwd(host64(do), r64, h(w), h(e), x64, h(pw), h(gm), 0.5, 1e-4)
    assert got["dx"].dtype == DT[io] and got["dresidual"].dtype == DT[wide]
    for name, key in (("dx", "dx"), ("dresidual", "dresidual"), ("dweight", "dweight"), ("dpost_weight", "dpost"),
                      ("dgamma", "dgamma")):
        if key not in ref:
            assert got[name] is None
            continue
        close(got[name], *ref[key], name, UROWS if name[:2] == "dw" or name[:2] in ("dp", "dg") else U)


@pytest.mark.parametrize("cols", cols_of())
def test_add_norm_bwd_sizes(cols):
    io, wide = PAIRS[(cols + 1) % 3]
    add_bwd_case(gen(cols), 5 if cols > 512 else 150, cols, io, wide, False, False)


@pytest.mark.parametrize("io,wide", PAIRS)
@pytest.mark.parametrize("post,gamma", [(False, False), (False, True), (True, False), (True, True)])
@pytest.mark.parametrize("rows,cols,pad,packed", [(1, 1001, 0, False), (33, 100, 3, True), (600, 200, 0, False),
                                                  (70, 768, 5, False), (6, 12000, 0, True), (1500, 513, 1, False),
                                                  (3, 16000, 0, False), (300, 12999, 1, True)])
def test_add_norm_bwd_options(io, wide, post, gamma, rows, cols, pad, packed):
    add_bwd_case(gen(rows), rows, cols, io, wide, post, gamma, packed, pad, dres=rows != 70)


def test_add_norm_bwd_wanted_outputs():
    g = gen(5)
    do, r, w = act(g, 4, 96, torch.bfloat16), act(g, 4, 96, torch.float32), weight(g, 96)
    both = mss.add_norm_bwd(do, r, w)
    assert torch.equal(both["dx"], both["dresidual"].bfloat16())
    a, b = mss.add_norm_bwd(do, r, w, want_dx=False), mss.add_norm_bwd(do, r, w, want_dresidual=False)
    assert a["dx"] is None and torch.equal(a["dresidual"], both["dresidual"])
    assert b["dresidual"] is None and torch.equal(b["dx"], both["dx"])
    with pytest.raises(ValueError):
        mss.add_norm_bwd(do, r, w, gamma=w)  # x is missing


def test_add_norm_gradient_by_differences():
    """The kernels' gradient against central differences of the fp32 forward:
    one step of a random direction, the loss summed in fp64.  The forward's
    error (2^-24 of values of order 1, 4 * 96 of them, random signs) over the
    step 2 * 2^-7 bounds what the difference can resolve: 2^-24 * 128 * 20 /
    2^-6 < 1e-2; the third-order term is (2^-7)^2 relative."""
    g = gen(9)
    rows, cols = 4, 96
    t = {k: act(g, rows, cols, torch.float32) for k in ("x", "res", "do", "de")}
    v = {k: weight(g, cols) for k in ("w", "p", "g")}

    def loss(d, s):
        out, r = mss.add_norm_fwd(t["x"] + s * d["x"], t["res"] + s * d["res"], v["w"] + s * d["w"],
                                  post_weight=v["p"] + s * d["p"], gamma=v["g"] + s * d["g"], scale=0.5)
        return float((host64(out) * host64(t["do"])).sum() + (host64(r) * host64(t["de"])).sum())

    _, r = mss.add_norm_fwd(t["x"], t["res"], v["w"], post_weight=v["p"], gamma=v["g"], scale=0.5)
    got = mss.add_norm_bwd(t["do"], r, v["w"], dresidual_out=t["de"], x=t["x"], post_weight=v["p"], gamma=v["g"],
                           scale=0.5)
    grads = {"x": got["dx"], "res": got["dresidual"], "w": got["dweight"], "p": got["dpost_weight"], "g": got["dgamma"]}
    h = 2.0 ** -7
    for name, grad in grads.items():
        zero = {k: 0.0 for k in grads}
        d = torch.randn(grad.shape, generator=g, device="cuda:0")
        num = (loss(zero | {name: d}, h) - loss(zero | {name: d}, -h)) / (2 * h)
        ana = float((host64(grad) * host64(d)).sum())
        scale = float(np.sqrt((host64(grad) ** 2).sum()))
        assert abs(num - ana) <= 1e-2 + 1e-2 * scale, (name, num, ana)


# -------------------------------------------------------- norm after a mixer
MODES = [("none", False), ("gate", False), ("gate", True)]


def gated_case(g, rows, cols, io, wide, gate, norm_first, ngroups, packed=False, pad=0):
    y, w = act(g, rows, cols, DT[wide], pad=pad), weight(g, cols)
    z = None
    if gate:
        z = act(g, rows, cols, DT[io], 0.7, pad=pad).clamp_(-12, 12)
    od = DT[io]
    args = dict(ngroups=ngroups, norm_first=norm_first, eps=1e-4)
    out = mss.gated_norm_fwd(y, z, w, out_dtype=od, pack_inputs=packed, pack_out=packed, **args)
    y64, z64 = host64(y), None if z is None else host64(z)
    if packed:
        out, y8, z8, out8 = out
        for p, t in ((y8, y), (z8, z), (out8, out)):
            if t is None:
                assert p is None
                continue
            q, e = ob.pack8(host64(t))
            assert np.array_equal(p.q.cpu().numpy(), q) and np.array_equal(p.scale.cpu().numpy(), e)
    ro = ob.gated_norm(y64, z64, host64(w), ngroups, norm_first, 1e-4)
    close(out, ro, np.abs(ro), "out")
    do = act(g, rows, cols, od, 1e-2, pad=pad)
    yin, zin = y, z
    if packed:
        yin, zin = y8, z8
        y64 = host64(mss.unpack8(y8, torch.float32))
        z64 = None if z is None else host64(mss.unpack8(z8, torch.float32))
    got = mss.gated_norm_bwd(do, yin, zin, w, **args)
    ref = ob.gated_norm_bwd(host64(do), y64, z64, host64(w), ngroups, norm_first, 1e-4)
    assert got["dy"].dtype == DT[wide]
    close(got["dy"], *ref["dy"], "dy")
    close(got["dweight"], *ref["dweight"], "dweight", UROWS)
    if gate:
        close(got["dz"], *ref["dz"], "dz")
    else:
        assert got["dz"] is None


@pytest.mark.parametrize("cols", cols_of())
def test_gated_norm_sizes(cols):
    io, wide = PAIRS[cols % 3]
    gate, first = MODES[cols % 2 + 1]
    gated_case(gen(cols), 5 if cols > 512 else 150, cols, io, wide, gate == "gate", first, 1)


@pytest.mark.parametrize("io,wide", PAIRS)
@pytest.mark.parametrize("gate,first", MODES)
@pytest.mark.parametrize("rows,cols,ngroups,packed,pad", [
    (1, 5120, 1, False, 0), (1, 5120, 8, True, 0), (40, 96, 3, True, 0), (33, 1536, 8, False, 3), (5, 100, 1, True, 1),
    (300, 60, 5, False, 0), (4, 10000, 1, True, 0), (3, 20480, 2, True, 0), (2, 65, 65, False, 0),
    (5, 16384, 1, True, 0), (300, 14001, 1, False, 1)])
def test_gated_norm_options(io, wide, gate, first, rows, cols, ngroups, packed, pad):
    gated_case(gen(rows), rows, cols, io, wide, gate == "gate", first, ngroups, packed, pad)


def test_gated_norm_gradient_by_differences():
    """As for add_norm."""
    g = gen(10)
    rows, cols = 4, 96
    y, z, do, w = (act(g, rows, cols, torch.float32), act(g, rows, cols, torch.float32),
                   act(g, rows, cols, torch.float32), weight(g, cols))
    for first in (False, True):
        got = mss.gated_norm_bwd(do, y, z, w, ngroups=3, norm_first=first)
        h = 2.0 ** -7
        for i, name in enumerate(("dy", "dz", "dweight")):
            d = torch.randn(got[name].shape, generator=g, device="cuda:0")

            def loss(s):
                a = [y, z, w]
                a[i] = a[i] + s * d
                return float((host64(mss.gated_norm_fwd(*a, ngroups=3, norm_first=first)) * host64(do)).sum())

            num, ana = (loss(h) - loss(-h)) / (2 * h), float((host64(got[name]) * host64(d)).sum())
            assert abs(num - ana) <= 1e-2 + 1e-2 * float(np.sqrt((host64(got[name]) ** 2).sum())), (first, name)


# ------------------------------------------------------------------ behaviour
def test_rows_do_not_see_each_other():
    """NaN and infinities stay in their row; a row of zeros gives zeros and
    finite gradients; the type's lowest value in a row does not become NaN in
    the others."""
    g = gen(11)
    for cols in (100, 2000):
        y, z, w = act(g, 8, cols, torch.float32), act(g, 8, cols, torch.bfloat16), weight(g, cols)
        do = act(g, 8, cols, torch.bfloat16)
        good = mss.gated_norm_fwd(y, z, w)
        goodb = mss.gated_norm_bwd(do, y, z, w)
        y2, z2 = y.clone(), z.clone()
        y2[1, 3], y2[2, 5], z2[3, 7] = float("nan"), float("inf"), torch.finfo(torch.bfloat16).min
        y2[4] = 0
        out, back = mss.gated_norm_fwd(y2, z2, w), mss.gated_norm_bwd(do, y2, z2, w)
        keep = [0, 5, 6, 7]
        assert torch.equal(out[keep], good[keep]) and torch.equal(back["dy"][keep], goodb["dy"][keep])
        assert torch.isnan(out[1]).any() and not torch.isfinite(out[2]).all()
        assert not out[4].any() and torch.isfinite(back["dy"][4]).all() and not back["dz"][4].any()
        assert torch.isfinite(out[3]).all()  # silu of the lowest value is 0
        x, r = act(g, 8, cols, torch.bfloat16), act(g, 8, cols, torch.float32)
        x2, r2 = x.clone(), r.clone()
        x2[1, 3] = float("nan")
        x2[4], r2[4] = 0, 0
        a, b = mss.add_norm_fwd(x, r, w)[0], mss.add_norm_fwd(x2, r2, w)[0]
        assert torch.equal(a[keep], b[keep]) and torch.isnan(b[1]).all() and not b[4].any()


def test_repeatable_and_strided_outputs():
    g = gen(12)
    rows, cols = 3000, 640
    y, z, w = act(g, rows, cols, torch.float32), act(g, rows, cols, torch.bfloat16), weight(g, cols)
    do = act(g, rows, cols, torch.bfloat16)
    a = mss.gated_norm_bwd(do, y, z, w)
    wide = torch.full((rows, 2 * cols + 9), 7.0, dtype=torch.bfloat16, device="cuda:0")
    b = mss.gated_norm_bwd(do, y, z, w, dz=wide[:, 9:9 + cols])
    assert all(torch.equal(a[k], b[k]) for k in a)
    assert torch.equal(wide[:, 9:9 + cols], a["dz"]) and (wide[:, :9] == 7).all() and (wide[:, 9 + cols:] == 7).all()
    out = torch.full((rows, cols + 3), 7.0, dtype=torch.bfloat16, device="cuda:0")
    ref = mss.gated_norm_fwd(y, z, w)
    mss.gated_norm_fwd(y, z, w, out=out[:, :cols])
    assert torch.equal(out[:, :cols], ref) and (out[:, cols:] == 7).all()


def test_leading_dimensions_and_single_token():
    g = gen(13)
    x, res, w = act(g, 12, 256, torch.bfloat16), act(g, 12, 256, torch.float32), weight(g, 256)
    out, r = mss.add_norm_fwd(x, res, w)
    o3, r3 = mss.add_norm_fwd(x.view(3, 4, 256), res.view(3, 4, 256), w)
    assert o3.shape == (3, 4, 256) and torch.equal(o3.view(12, 256), out) and torch.equal(r3.view(12, 256), r)
    for i in (0, 7):
        o1, r1 = mss.add_norm_fwd(x[i], res[i], w)
        assert o1.shape == (256,) and torch.equal(o1, out[i]) and torch.equal(r1, r[i])


def test_other_stream():
    g = gen(14)
    x, res, w = act(g, 512, 2560, torch.bfloat16), act(g, 512, 2560, torch.float32), weight(g, 2560)
    do = act(g, 512, 2560, torch.bfloat16)
    ref, refb = mss.add_norm_fwd(x, res, w), mss.add_norm_bwd(do, res, w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = mss.add_norm_fwd(x, res, w, stream=s)
    gotb = mss.add_norm_bwd(do, res, w, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(ref, got))
    assert torch.equal(refb["dweight"], gotb["dweight"]) and torch.equal(refb["dx"], gotb["dx"])


def test_rows_past_32_bit_offsets():
    """Rows 2^20 elements apart: the last ones lie past 2^32 elements."""
    rows, cols, pitch = 4100, 64, 1 << 20
    big = torch.empty(rows * pitch, dtype=torch.bfloat16, device="cuda:0")
    x = big.view(rows, pitch)[:, 16:16 + cols]
    g = gen(15)
    x.copy_(act(g, rows, cols, torch.bfloat16))
    w = weight(g, cols)
    dense = x.contiguous()
    assert torch.equal(mss.gated_norm_fwd(x, None, w), mss.gated_norm_fwd(dense, None, w))
    a, b = mss.gated_norm_bwd(x, x, None, w), mss.gated_norm_bwd(dense, dense, None, w)
    assert torch.equal(a["dy"], b["dy"]) and torch.equal(a["dweight"], b["dweight"])
    p, q = mss.pack8(x), mss.pack8(dense)
    assert torch.equal(p.q, q.q) and torch.equal(p.scale, q.scale)
    mss.unpack8(p, out=x)
    assert torch.equal(x, mss.unpack8(q))


def test_graph_replays():
    """A token's two norms in a captured graph, replayed with new inputs between eager work."""
    g = gen(16)
    x, res, w = act(g, 4, 2560, torch.bfloat16), act(g, 4, 2560, torch.float32), weight(g, 2560)
    y, z = act(g, 4, 2560, torch.bfloat16), act(g, 4, 2560, torch.bfloat16)
    outs = (torch.empty_like(x), torch.empty_like(res), torch.empty_like(y))

    def step():
        mss.add_norm_fwd(x, res, w, out=outs[0], residual_out=outs[1])
        mss.gated_norm_fwd(y, z, w, out=outs[2])

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        for t in (x, res, y, z):
            t.copy_(act(g, *t.shape, t.dtype))
        want = mss.add_norm_fwd(x, res, w) + (mss.gated_norm_fwd(y, z, w),)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want)), i


def test_binding_refusals():
    g = gen(17)
    x, res, w = act(g, 4, 96, torch.bfloat16), act(g, 4, 96, torch.float32), weight(g, 96)
    with pytest.raises(TypeError):
        mss.add_norm_fwd(x.half(), res, w)
    with pytest.raises(TypeError):
        mss.add_norm_fwd(x, res, w.bfloat16())
    with pytest.raises(ValueError):
        mss.add_norm_fwd(x, res[:3], w)
    with pytest.raises(ValueError):
        mss.add_norm_fwd(x, res, w[:95])
    with pytest.raises(ValueError):
        mss.add_norm_fwd(x[:0], res[:0], w)
    with pytest.raises(mss.MambaScanError) as e:
        mss.add_norm_fwd(x.float(), x, w)        # a residual narrower than x
    assert e.value.status == 5
    with pytest.raises(mss.MambaScanError) as e:
        mss.add_norm_fwd(x, res, w, residual_out=res)
    assert e.value.status == 7
    with pytest.raises(mss.MambaScanError) as e:
        mss.gated_norm_fwd(res, x, w, ngroups=2, pack_out=True)  # 48 columns a group
    assert e.value.status == 5
    with pytest.raises(mss.MambaScanError):
        mss.gated_norm_bwd(x, mss.pack8(res), x, w)  # y in 8 bits, z not
    with pytest.raises(ValueError):
        mss.gated_norm_fwd(res, x.cpu(), w)
