"""Refusals of the gated recurrence and of beam search, all on the host before
any HIP call (fake, never-dereferenced pointers; CPU only)."""
import ctypes

import pytest
import torch

import selective_state_space_27_amd as mss
from test_abi_block import ALIAS, ALIGN, BF16, DTYPE, FP32, NULL, SHAPE, UNSUP, WS, P, call


def fwd(**kw):
    d = dict(x=P(0), xs=96, ga=P(1), gas=96, gx=P(2), gxs=96, lam=P(3), c=8.0, h0=P(4), starts=P(5), y=P(6), ys=96,
             last=P(7), states=P(8), batch=2, seqlen=100, dim=96, io=BF16, flags=0, ws=P(9),
             wsb=mss.lib().mss_gated_recurrence_workspace_size(2, 100, 96, BF16), stream=None)
    return call("mss_gated_recurrence_fwd", d, list(d), **kw)


SIZES = [dict(batch=0), dict(seqlen=0), dict(dim=0), dict(batch=-1), dict(batch=1 << 40), dict(seqlen=1 << 40),
         dict(batch=1 << 23), dict(seqlen=1 << 29), dict(batch=1 << 22, seqlen=65),
         dict(dim=1 << 29, xs=1 << 29, gas=1 << 29, gxs=1 << 29, ys=1 << 29, ds=1 << 29, dxs=1 << 29, das=1 << 29,
              dgs=1 << 29)]


STRIDES = {fwd: ("xs", "gas", "gxs", "ys")}


def only(f, kw):
    """The sizes, and the strides that f takes."""
    return {k: v for k, v in kw.items() if k in ("batch", "seqlen", "dim") or k in STRIDES[f]}


def test_fwd_refusals():
    for k in ("x", "ga", "gx", "lam", "y"):
        assert fwd(**{k: None}) == NULL, k
    for kw in SIZES:
        assert fwd(**only(fwd, kw)) == SHAPE, kw
    for k in ("xs", "gas", "gxs", "ys"):
        assert fwd(**{k: 95}) == SHAPE, k
        assert fwd(**{k: 1 << 46}) == SHAPE, k
    assert fwd(io=2) == DTYPE
    assert fwd(flags=1) == UNSUP
    for c in (0.0, -8.0, float("inf"), float("nan")):
        assert fwd(c=c) == UNSUP
    for k, i in (("x", 0), ("ga", 1), ("gx", 2), ("y", 6)):
        assert fwd(**{k: P(i, 1)}) == ALIGN, k
        assert fwd(**{k: P(i, 2)}, io=FP32) == ALIGN, k
    for k, i in (("lam", 3), ("h0", 4), ("last", 7), ("states", 8)):
        assert fwd(**{k: P(i, 2)}) == ALIGN, k
    assert fwd(ws=P(9, 8)) == ALIGN
    assert fwd(ws=None) == WS
    assert fwd(wsb=8) == WS
    for i in (0, 1, 2, 3, 4, 5, 9):
        assert fwd(y=P(i)) == ALIAS, i
        assert fwd(last=P(i)) == ALIAS, i
        assert fwd(states=P(i)) == ALIAS, i
    assert fwd(last=P(6, 4)) == ALIAS
    assert fwd(states=P(6, 4)) == ALIAS
    assert fwd(states=P(7, 4)) == ALIAS
    # Slices of one buffer may interleave; a shared column may not.
    wide = dict(xs=400, ys=400)
    assert fwd(**wide, y=P(0, 95 * 2)) == ALIAS
    assert fwd(**wide, y=P(0, 96 * 2), last=P(4)) == ALIAS  # the marker: y itself was accepted
    size = mss.lib().mss_gated_recurrence_workspace_size
    assert size(0, 1, 1, 0) == 0 and size(1, 1, 1, 7) == 0 and size(1 << 23, 1, 1, 0) == 0 and size(1, 1, 1, 0) > 0


def bwd(**kw):
    d = dict(dy=P(0), ds=96, x=P(1), xs=96, ga=P(2), gas=96, gx=P(3), gxs=96, lam=P(4), c=8.0, starts=P(5), states=P(6),
             dlast=P(7), dx=P(8), dxs=96, da=P(9), das=96, dg=P(10), dgs=96, dlam=P(11), dh0=P(12), batch=2, seqlen=100,
             dim=96, io=BF16, flags=0, ws=P(13), wsb=mss.lib().mss_gated_recurrence_bwd_workspace_size(2, 100, 96, BF16),
             stream=None)
    return call("mss_gated_recurrence_bwd", d, list(d), **kw)


STRIDES[bwd] = ("ds", "xs", "gas", "gxs", "dxs", "das", "dgs")


def test_bwd_refusals():
    for k in ("dy", "x", "ga", "gx", "lam", "states", "dx", "da", "dg", "dlam"):
        assert bwd(**{k: None}) == NULL, k
    for kw in SIZES:
        assert bwd(**only(bwd, kw)) == SHAPE, kw
    for k in ("ds", "xs", "gas", "gxs", "dxs", "das", "dgs"):
        assert bwd(**{k: 95}) == SHAPE, k
        assert bwd(**{k: 1 << 46}) == SHAPE, k
    assert bwd(io=-1) == DTYPE
    assert bwd(flags=2) == UNSUP
    assert bwd(c=0.0) == UNSUP
    for k, i in (("dy", 0), ("x", 1), ("ga", 2), ("gx", 3), ("dx", 8), ("da", 9), ("dg", 10)):
        assert bwd(**{k: P(i, 1)}) == ALIGN, k
    for k, i in (("lam", 4), ("states", 6), ("dlast", 7), ("dlam", 11), ("dh0", 12)):
        assert bwd(**{k: P(i, 2)}) == ALIGN, k
    assert bwd(ws=P(13, 4)) == ALIGN
    assert bwd(ws=None) == WS
    assert bwd(wsb=256) == WS
    for out in ("dx", "da", "dg", "dlam", "dh0"):
        for i in (0, 1, 2, 3, 4, 5, 6, 7, 13):
            assert bwd(**{out: P(i)}) == ALIAS, (out, i)
    assert bwd(da=P(8, 64)) == ALIAS
    assert bwd(dlam=P(10, 64)) == ALIAS
    size = mss.lib().mss_gated_recurrence_bwd_workspace_size
    assert size(1, 0, 1, 0) == 0 and size(1, 1, 1, -1) == 0 and size(1, 1, 1, 1) > 0


def step(**kw):
    d = dict(h=P(0), parents=P(1), x=P(2), xs=96, ga=P(3), gas=96, gx=P(4), gxs=96, lam=P(5), c=8.0, out=P(6), y=P(7),
             ys=96, batch=2, beams=3, dim=96, io=BF16, flags=0, stream=None)
    return call("mss_gated_recurrence_step", d, list(d), **kw)


def test_step_refusals():
    for k in ("h", "x", "ga", "gx", "lam", "out", "y"):
        assert step(**{k: None}) == NULL, k
    for kw in (dict(batch=0), dict(beams=0), dict(dim=0), dict(batch=1 << 31), dict(beams=1 << 62),
               dict(batch=1 << 20, beams=1 << 10), dict(dim=1 << 40)):
        assert step(**kw) == SHAPE, kw
    for k in ("xs", "gas", "gxs", "ys"):
        assert step(**{k: 95}) == SHAPE, k
    assert step(io=5) == DTYPE
    assert step(flags=4) == UNSUP
    assert step(c=float("inf")) == UNSUP
    assert step(parents=P(1, 4)) == ALIGN
    assert step(h=P(0, 2)) == ALIGN
    assert step(x=P(2, 1)) == ALIGN
    assert step(out=P(0)) == ALIAS                          # in place with parents
    assert step(out=P(0, 4), parents=None) == ALIAS         # not the same rows
    for i in (1, 2, 3, 4, 5):
        assert step(out=P(i)) == ALIAS, i
        assert step(y=P(i)) == ALIAS, i
    assert step(y=P(0)) == ALIAS
    assert step(y=P(6, 8)) == ALIAS


def select(**kw):
    d = dict(logits=P(0), ls=1000, scores=P(1), fin=P(2), eos=3, best=P(3), parents=P(4), tokens=P(5), done=P(6), batch=2,
             beams=4, vocab=1000, n=8, io=BF16, flags=0, ws=P(7),
             wsb=mss.lib().mss_beam_select_workspace_size(2, 4, 1000, 8), stream=None)
    return call("mss_beam_select", d, list(d), **kw)


def test_select_refusals():
    for k in ("logits", "scores", "best", "parents", "tokens"):
        assert select(**{k: None}) == NULL, k
    for kw in (dict(batch=0), dict(beams=0), dict(vocab=0), dict(n=0), dict(batch=65536),
               dict(vocab=(1 << 24) + 1, ls=1 << 25), dict(ls=999), dict(ls=1 << 46),
               dict(batch=65535, beams=64, vocab=1 << 16, ls=1 << 16)):
        assert select(**kw) == SHAPE, kw
    assert select(io=3) == DTYPE
    for kw in (dict(beams=65), dict(n=65), dict(vocab=1, eos=0, n=5), dict(flags=1), dict(eos=1000), dict(eos=-2),
               dict(eos=-1), dict(eos=-1, fin=None), dict(eos=-1, done=None)):
        assert select(**kw) == UNSUP, kw
    for k, i, off in (("logits", 0, 1), ("scores", 1, 2), ("best", 3, 2), ("parents", 4, 4), ("tokens", 5, 4), ("ws", 7, 8)):
        assert select(**{k: P(i, off)}) == ALIGN, k
    assert select(ws=None) == WS
    assert select(wsb=100) == WS
    for out in ("best", "parents", "tokens", "done"):
        for i in (0, 1, 2, 7):
            assert select(**{out: P(i)}) == ALIAS, (out, i)
    assert select(tokens=P(4, 8)) == ALIAS
    size = mss.lib().mss_beam_select_workspace_size
    assert size(2, 65, 10, 3) == 0 and size(2, 2, 2, 5) == 0 and size(0, 1, 1, 1) == 0 and size(1, 1, 1, 1) > 0


def reorder(states, sizes, parents=P(50), batch=2, beams=4, count=None):
    n = len(states)
    return mss.lib().mss_reorder_states((ctypes.c_void_p * n)(*states), (ctypes.c_int64 * n)(*sizes),
                                        n if count is None else count, parents, batch, beams, None)


def test_reorder_refusals():
    a, b = P(0), P(1)
    assert mss.lib().mss_reorder_states(None, (ctypes.c_int64 * 1)(4), 1, P(50), 2, 4, None) == NULL
    assert mss.lib().mss_reorder_states((ctypes.c_void_p * 1)(a), None, 1, P(50), 2, 4, None) == NULL
    assert reorder([a], [4], parents=None) == NULL
    assert reorder([a, None], [4, 4]) == NULL
    for kw in (dict(count=0), dict(batch=0), dict(batch=65536), dict(beams=0), dict(beams=-4)):
        assert reorder([a], [4], **kw) == SHAPE, kw
    assert reorder([a, b], [4, 0]) == SHAPE
    assert reorder([a], [(1 << 30) + 1]) == SHAPE
    assert reorder([a], [4], beams=65) == UNSUP
    assert reorder([a], [4], parents=P(50, 4)) == ALIGN
    assert reorder([a, a], [4, 4]) == ALIAS
    assert reorder([a, P(0, 31)], [4, 4]) == ALIAS
    assert reorder([P(50, 8)], [4]) == ALIAS


def test_no_cpu_path():
    t = torch.zeros(1, 2, 4)
    lam = torch.zeros(4)
    with pytest.raises(ValueError):
        mss.gated_recurrence_fwd(t, t, t, lam)
    with pytest.raises(ValueError):
        mss.gated_recurrence_bwd(t, t, t, t, lam, t)
    with pytest.raises(ValueError):
        mss.gated_recurrence_step(t[0], t[0], t[0], t[0], lam)
    with pytest.raises(ValueError):
        mss.beam_select(t, t[..., 0].contiguous())
    with pytest.raises(ValueError):
        mss.reorder_states([t], torch.zeros(1, 2, dtype=torch.int64))


def test_chunk_matches_the_header():
    import os
    import re

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    with open(os.path.join(root, "include", "mambascan.h")) as f:
        assert int(re.search(r"#define MSS_RECURRENCE_CHUNK (\d+)", f.read()).group(1)) == mss.RECURRENCE_CHUNK
