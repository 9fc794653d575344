"""Refusals of the operators around the mixer, all on the host before any HIP
call (fake, never-dereferenced pointers; CPU only)."""
import ctypes

import pytest
import torch

import selective_state_space_27_amd as mss

OK, NULL, SHAPE, DTYPE, ALIGN, UNSUP, WS, ALIAS = 0, 1, 2, 3, 4, 5, 6, 7
FP32, BF16 = 0, 1
BASE = 0x7F0000000000
GB = 1 << 32


def P(i, off=0):
    return ctypes.c_void_p(BASE + i * GB + off)


def call(fn, defaults, order, **kw):
    a = dict(defaults)
    unknown = set(kw) - set(a)
    assert not unknown, unknown
    a.update(kw)
    return getattr(mss.lib(), fn)(*(a[k] for k in order))


def add_fwd(**kw):
    d = dict(x=P(0), xs=96, res=P(1), rs=96, w=P(2), post=P(3), gamma=P(4), scale=1.0, eps=1e-5, out=P(5), os=96,
             rout=P(6), ros=96, q=P(7), qs=P(8), rows=4, cols=96, io=BF16, rdt=FP32, flags=0, stream=None)
    return call("mss_add_norm_fwd", d, list(d), **kw)


def test_add_norm_fwd_refusals():
    for k in ("x", "w", "out", "rout", "q", "qs"):
        assert add_fwd(**{k: None}) == NULL, k
    assert add_fwd(rows=0) == SHAPE
    assert add_fwd(cols=0) == SHAPE
    assert add_fwd(rows=-1) == SHAPE
    assert add_fwd(rows=1 << 42) == SHAPE
    for k in ("xs", "rs", "os", "ros"):
        assert add_fwd(**{k: 95}) == SHAPE, k
        assert add_fwd(**{k: 1 << 46}) == SHAPE, k
    assert add_fwd(io=7) == DTYPE
    assert add_fwd(rdt=-1) == DTYPE
    assert add_fwd(io=FP32, rdt=BF16) == UNSUP
    assert add_fwd(flags=1) == UNSUP
    wide = dict(xs=16385, rs=16385, os=16385, ros=16385)
    assert add_fwd(cols=16385, **wide) == UNSUP
    for eps in (0.0, -1.0, float("inf"), float("nan")):
        assert add_fwd(eps=eps) == UNSUP
    assert add_fwd(x=P(0, 1)) == ALIGN
    assert add_fwd(res=P(1, 2)) == ALIGN
    assert add_fwd(w=P(2, 2)) == ALIGN
    assert add_fwd(q=P(7, 8)) == ALIGN
    assert add_fwd(out=P(0)) == ALIAS
    assert add_fwd(rout=P(1)) == ALIAS
    assert add_fwd(rout=P(5, 64)) == ALIAS
    assert add_fwd(qs=P(7, 64)) == ALIAS
    assert add_fwd(out=P(2)) == ALIAS
    assert add_fwd(q=P(6)) == ALIAS


def test_slices_of_one_buffer_may_interleave():
    """Rows of equal stride overlap exactly when their columns do: these two
    differ only in where `out` starts within x's wide rows.  The refusal tells
    them apart; the accepted one gets past the alias check to the next
    argument's (a null q with a given scale is looked at before, so a bad
    alias of the scale is used as the marker)."""
    clear = dict(xs=400, os=400, out=P(0, 192 * 2))
    assert add_fwd(**clear, qs=P(2)) == ALIAS          # the marker
    assert add_fwd(xs=400, os=400, out=P(0, 95 * 2)) == ALIAS
    assert add_fwd(xs=400, os=400, out=P(0, (400 - 95) * 2)) == ALIAS
    assert add_fwd(xs=400, os=404, out=P(0, 192 * 2)) == ALIAS  # other strides: by their spans


def add_bwd(**kw):
    d = dict(dout=P(0), ds=96, dres=P(1), es=96, r=P(2), rs=96, rsc=None, x=P(3), xs=96, xsc=None, w=P(4), post=P(5),
             gamma=P(6), scale=1.0, eps=1e-5, dx=P(7), dxs=96, dr=P(8), drs=96, dw=P(9), dpost=P(10), dgamma=P(11),
             rows=4, cols=96, io=BF16, rdt=FP32, flags=0, ws=P(12),
             wsb=mss.lib().mss_add_norm_bwd_workspace_size(4, 96, 3), stream=None)
    return call("mss_add_norm_bwd", d, list(d), **kw)


def test_add_norm_bwd_refusals():
    for k in ("dout", "r", "w", "dw", "dpost", "dgamma", "x", "post", "gamma"):
        assert add_bwd(**{k: None}) == NULL, k
    assert add_bwd(rows=0) == SHAPE
    for k in ("ds", "es", "rs", "xs", "dxs", "drs"):
        assert add_bwd(**{k: 95}) == SHAPE, k
    assert add_bwd(io=3) == DTYPE
    assert add_bwd(io=FP32, rdt=BF16) == UNSUP
    assert add_bwd(rsc=P(13)) == UNSUP   # r in 8 bits, x not
    assert add_bwd(xsc=P(13)) == UNSUP
    assert add_bwd(flags=2) == UNSUP
    assert add_bwd(eps=0.0) == UNSUP
    assert add_bwd(dout=P(0, 1)) == ALIGN
    assert add_bwd(rsc=P(13), xsc=P(14), r=P(2, 8)) == ALIGN
    assert add_bwd(ws=P(12, 8)) == ALIGN
    assert add_bwd(ws=None) == WS
    assert add_bwd(wsb=300) == WS
    assert add_bwd(dx=P(0)) == ALIAS
    assert add_bwd(dr=P(1)) == ALIAS
    assert add_bwd(dgamma=P(9)) == ALIAS
    assert add_bwd(dw=P(12)) == ALIAS
    size = mss.lib().mss_add_norm_bwd_workspace_size
    assert size(4, 96, 0) == 0 and size(4, 96, 4) == 0 and size(0, 96, 1) == 0 and size(4, 16385, 1) == 0
    assert size(4, 96, 1) > 0


def gated_fwd(**kw):
    d = dict(y=P(0), ys=96, z=P(1), zs=96, w=P(2), eps=1e-5, out=P(3), os=96, yq=P(4), yqs=P(5), zq=P(6), zqs=P(7),
             oq=P(8), oqs=P(9), rows=4, cols=96, groups=1, ydt=FP32, io=BF16, flags=0, stream=None)
    return call("mss_gated_norm_fwd", d, list(d), **kw)


def test_gated_norm_fwd_refusals():
    for k in ("y", "w", "out", "yq", "yqs", "zq", "zqs", "oq", "oqs"):
        assert gated_fwd(**{k: None}) == NULL, k
    assert gated_fwd(z=None) == NULL                      # z's form wanted without z
    assert gated_fwd(yq=None, yqs=None) == NULL           # z's form without y's
    assert gated_fwd(groups=0) == SHAPE
    for k in ("ys", "zs", "os"):
        assert gated_fwd(**{k: 95}) == SHAPE, k
    assert gated_fwd(ydt=9) == DTYPE
    assert gated_fwd(ydt=BF16, io=FP32) == UNSUP
    assert gated_fwd(groups=5) == UNSUP                   # does not divide
    assert gated_fwd(groups=2) == UNSUP                   # 48 columns: blocks of 32 would straddle
    assert gated_fwd(flags=1) == UNSUP
    assert gated_fwd(eps=0.0) == UNSUP
    assert gated_fwd(z=P(1, 1)) == ALIGN
    assert gated_fwd(zq=P(6, 4)) == ALIGN
    assert gated_fwd(out=P(0)) == ALIAS
    assert gated_fwd(zq=P(4, 64)) == ALIAS
    assert gated_fwd(oqs=P(9, -1), oq=P(9)) == ALIAS
    big = dict(ys=16385 * 2, zs=16385 * 2, os=16385 * 2, cols=16385 * 2)
    assert gated_fwd(**big) == UNSUP


def gated_bwd(**kw):
    d = dict(dout=P(0), ds=96, y=P(1), ys=96, ysc=None, z=P(2), zs=96, zsc=None, w=P(3), eps=1e-5, dy=P(4), dys=96,
             dz=P(5), dzs=96, dw=P(6), rows=4, cols=96, groups=1, ydt=FP32, io=BF16, flags=0, ws=P(7),
             wsb=mss.lib().mss_gated_norm_bwd_workspace_size(4, 96, 1), stream=None)
    return call("mss_gated_norm_bwd", d, list(d), **kw)


def test_gated_norm_bwd_refusals():
    for k in ("dout", "y", "w", "dy", "dw", "z", "dz"):
        assert gated_bwd(**{k: None}) == NULL, k
    assert gated_bwd(rows=0) == SHAPE
    for k in ("ds", "ys", "zs", "dys", "dzs"):
        assert gated_bwd(**{k: 95}) == SHAPE, k
    assert gated_bwd(ysc=P(8)) == UNSUP
    assert gated_bwd(zsc=P(8)) == UNSUP
    assert gated_bwd(ysc=P(8), zsc=P(9), groups=2) == UNSUP
    assert gated_bwd(flags=0x40) == UNSUP
    assert gated_bwd(ysc=P(8), zsc=P(9), y=P(1, 8)) == ALIGN
    assert gated_bwd(ws=P(7, 4)) == ALIGN
    assert gated_bwd(ws=None) == WS
    assert gated_bwd(wsb=256) == WS
    assert gated_bwd(dz=P(0)) == ALIAS
    assert gated_bwd(dy=P(5)) == ALIAS
    assert gated_bwd(dw=P(7, 256)) == ALIAS
    size = mss.lib().mss_gated_norm_bwd_workspace_size
    assert size(4, 96, 5) == 0 and size(4, 0, 1) == 0 and size(4, 96, 3) > 0


def pack(fn="mss_pack8", **kw):
    d = dict(x=P(0), xs=96, q=P(1), s=P(2), rows=4, cols=96, dt=BF16, stream=None)
    order = list(d) if fn == "mss_pack8" else ["q", "s", "x", "xs", "rows", "cols", "dt", "stream"]
    return call(fn, d, order, **kw)


@pytest.mark.parametrize("fn", ["mss_pack8", "mss_unpack8"])
def test_pack8_refusals(fn):
    for k in ("x", "q", "s"):
        assert pack(fn, **{k: None}) == NULL, k
    assert pack(fn, rows=0) == SHAPE
    assert pack(fn, cols=0) == SHAPE
    assert pack(fn, xs=95) == SHAPE
    assert pack(fn, cols=1 << 30, xs=1 << 30) == SHAPE
    assert pack(fn, rows=1 << 31) == SHAPE               # more than 2^32 threads
    assert pack(fn, dt=2) == DTYPE
    assert pack(fn, x=P(0, 1)) == ALIGN
    assert pack(fn, q=P(1, 8)) == ALIGN
    assert pack(fn, q=P(0)) == ALIAS
    assert pack(fn, s=P(0, 100)) == ALIAS


def test_pack8_outputs_apart():
    assert pack("mss_pack8", s=P(1, 100)) == ALIAS


def wgrad(**kw):
    d = dict(dy=P(0), ds=48, q=P(1), s=P(2), dw=P(3), tokens=100, outs=48, ins=40, dydt=BF16, dwdt=FP32, flags=0,
             ws=P(4), wsb=mss.lib().mss_wgrad8_workspace_size(P(0), 48, 100, 48, 40), stream=None)
    return call("mss_wgrad8", d, list(d), **kw)


def test_wgrad8_refusals():
    for k in ("dy", "q", "s", "dw"):
        assert wgrad(**{k: None}) == NULL, k
    for k in ("tokens", "outs", "ins"):
        assert wgrad(**{k: 0}) == SHAPE, k
    assert wgrad(ds=47) == SHAPE
    assert wgrad(ins=(1 << 20) + 1) == SHAPE
    assert wgrad(outs=1 << 20, ins=1 << 20, ds=1 << 20) == SHAPE
    assert wgrad(dydt=5) == DTYPE
    assert wgrad(dwdt=5) == DTYPE
    assert wgrad(dydt=FP32) == UNSUP
    assert wgrad(flags=1) == UNSUP
    assert wgrad(dy=P(0, 1)) == ALIGN
    assert wgrad(q=P(1, 8)) == ALIGN
    assert wgrad(dw=P(3, 4)) == ALIGN
    assert wgrad(ws=None) == WS
    assert wgrad(wsb=0) == WS
    assert wgrad(dw=P(0)) == ALIAS
    assert wgrad(dw=P(4)) == ALIAS
    assert wgrad(tokens=1 << 31, ds=48) == SHAPE            # more than 2^32 threads of the copy
    size = mss.lib().mss_wgrad8_workspace_size
    assert size(P(0), 1, 0, 1, 1) == 0
    # rows that cannot be read as they lie need room for their copy
    apart = [size(P(0, 2), 48, 100, 48, 40), size(P(0), 52, 100, 48, 40), size(P(0), 1 << 24, 100, 48, 40)]
    assert all(n == size(P(0), 48, 100, 48, 40) + 100 * 48 * 2 for n in apart)
    assert wgrad(dy=P(0, 2)) == WS                          # sized for aligned rows


def test_binding_refuses_cpu_tensors_and_empty_shapes():
    x, w = torch.zeros(2, 32), torch.ones(32)
    with pytest.raises(ValueError):
        mss.add_norm_fwd(x, None, w)
    with pytest.raises(ValueError):
        mss.gated_norm_fwd(x, x, w)
    with pytest.raises(ValueError):
        mss.pack8(x)
    p = mss.Packed8(torch.zeros(2, 32, dtype=torch.int8), torch.ones(2, 1, dtype=torch.uint8), (2, 32), torch.float32)
    with pytest.raises(ValueError):
        mss.unpack8(p)
    with pytest.raises(ValueError):
        mss.wgrad8(x.bfloat16(), p)
    with pytest.raises(TypeError):
        mss.unpack8(x)
    with pytest.raises(ValueError):
        mss.Packed8(p.q, p.scale, (2, 33), torch.float32)    # another pitch
    with pytest.raises(ValueError):
        mss.Packed8(p.q, p.scale, (0, 32), torch.float32)
    with pytest.raises(TypeError):
        mss.Packed8(p.q, p.scale, (2, 32), torch.float16)


def test_row_strides_of_leading_dimensions():
    from selective_state_space_27_amd import norms

    dev = torch.device("cpu")

    def rows(t):
        return norms._rows(t, "t", t.shape, t.dtype, dev)[1]

    wide = torch.zeros(3, 4, 50)
    assert rows(wide) == 50 and rows(wide[:, :, 10:42]) == 50
    assert rows(wide[0]) == 50 and rows(wide[:1, :, :32]) == 50 and rows(wide[:, :1, :32]) == 200
    assert rows(torch.zeros(32)) == 32 and rows(wide[0, 0, 5:6]) == 1
    assert rows(torch.zeros(7, 1)) == 1
    with pytest.raises(ValueError):
        rows(wide[:, :2])                       # rows of two strides
    with pytest.raises(ValueError):
        rows(wide.transpose(1, 2))              # columns not contiguous
    with pytest.raises(ValueError):
        rows(torch.zeros(1, 8).expand(4, 8))    # rows on top of each other
