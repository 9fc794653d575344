"""Python binding of the gated linear recurrence (``include/mambascan.h``): a
mixer with one state per channel, scanned over whole sequences, its gradient,
and its one-token step.

    r = sigmoid(gate_a), i = sigmoid(gate_x), a = exp(-c softplus(lam) r)
    h_t = a h_{t-1} + sqrt(1 - a^2) i x_t,   y = h

Activations, checks, streams and errors are as in norms.py: tensors whose
leading dimensions collapse to rows of one stride (x and the gates may be
slices of one projection's output), outputs new and contiguous unless given.

As everywhere in the package there is no autograd: results require no gradient
whatever the inputs do, and a training step calls gated_recurrence_bwd itself (in
a torch.autograd.Function around the layer, say).  Nor does autograd notice what
is written in place (the step's state, given outputs): what a graph still needs of
those has to be kept apart.
"""
from __future__ import annotations

import torch

import selective_state_space_27_amd as _mss

from .norms import _code, _on, _result, _rows, _vec, _workspace_size

# Steps between two of the states that the forward keeps for the backward.
RECURRENCE_CHUNK = 64


def _sequences(x, name):
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if x.dim() != 3 or x.numel() == 0:
        raise ValueError(f"{name} has shape {tuple(x.shape)}: [batch, seqlen, dim], none of them empty")
    return x.shape


def _state(t, name, shape, device):
    """Pointer of a dense float32 tensor, or None."""
    if t is None:
        return None
    if not (isinstance(t, torch.Tensor) and t.dtype == torch.float32 and t.shape == shape and t.device == device and
            t.is_contiguous()):
        _mss._check(t, name, shape, torch.float32, device)
    return t.data_ptr()


def _address(t):
    return None if t is None else t.data_ptr()


def _marks(t, name, shape, device):
    """Pointer of a bool or uint8 tensor, or None."""
    if t is None:
        return None
    dtype = torch.uint8 if isinstance(t, torch.Tensor) and t.dtype == torch.uint8 else torch.bool
    _mss._check(t, name, shape, dtype, device)
    return t.data_ptr()


def _chunks(seqlen):
    return (seqlen + RECURRENCE_CHUNK - 1) // RECURRENCE_CHUNK


def gated_recurrence_fwd(x, gate_a, gate_x, lam, *, c=8.0, h0=None, starts=None, return_last_state=False,
                         keep_states=False, out=None, stream=None, check_waits=False):
    """Gated linear recurrence over whole sequences.

    x, gate_a, gate_x: [batch, seqlen, dim] float32 or bfloat16 (one type); lam:
    [dim] float32; h0: [batch, dim] float32, the state before the first step
    (None: zero); starts: [batch, seqlen] bool or uint8, true where a sequence
    packed into the row begins (the state before that step counts as zero).
    Returns y (x's shape and type), and after it, as asked for, the last state
    ([batch, dim] float32) with ``return_last_state`` and, with ``keep_states``,
    the states that gated_recurrence_bwd needs ([batch, ceil(seqlen /
    RECURRENCE_CHUNK), dim] float32).  ``check_waits`` waits for the call and
    raises if a wait between workgroups gave up."""
    b, length, dim = shape = _sequences(x, "x")
    dev = _mss._device_of(x)
    io = _code(x.dtype)
    xp, xs = _rows(x, "x", shape, x.dtype, dev)
    ap, as_ = _rows(gate_a, "gate_a", shape, x.dtype, dev)
    ip, is_ = _rows(gate_x, "gate_x", shape, x.dtype, dev)
    lp = _vec(lam, "lam", dim, dev)
    hp, sp = _state(h0, "h0", (b, dim), dev), _marks(starts, "starts", (b, length), dev)
    handle, here = _on(stream, dev)
    with here:
        out, op, os = _result(out, "out", shape, x.dtype, dev, x)
        last = torch.empty((b, dim), dtype=torch.float32, device=dev) if return_last_state else None
        states = torch.empty((b, _chunks(length), dim), dtype=torch.float32, device=dev) if keep_states else None
        need = _workspace_size("mss_gated_recurrence_workspace_size", b, length, dim, io)
        if need == 0:
            _mss._raise(2, "gated_recurrence_fwd")
        ws = torch.empty(need, dtype=torch.uint8, device=dev)
        st = _mss.lib().mss_gated_recurrence_fwd(xp, xs, ap, as_, ip, is_, lp, c, hp, sp, op, os, _address(last),
                                                 _address(states), b, length, dim, io, 0, ws.data_ptr(), need, handle)
        _mss._raise(st, "mss_gated_recurrence_fwd")
        if check_waits:
            _mss._check_waits(ws, stream, "mss_gated_recurrence_fwd")
    got = [t for t in (out, last, states) if t is not None]
    return got[0] if len(got) == 1 else tuple(got)


def gated_recurrence_bwd(dy, x, gate_a, gate_x, lam, states, *, c=8.0, starts=None, dh_last=None, want_dh0=False,
                         dx=None, dgate_a=None, dgate_x=None, stream=None, check_waits=False):
    """Gradients of gated_recurrence_fwd, given dy (x's shape and type) and
    dh_last ([batch, dim] float32; None: zero), at the forward's inputs and the
    ``states`` it kept.  Returns a dict: dx, dgate_a, dgate_x (x's type; the
    given tensors, slices of a projection's gradient for instance, or new ones),
    dlam ([dim] float32) and dh0 ([batch, dim] float32; None unless
    ``want_dh0``)."""
    b, length, dim = shape = _sequences(dy, "dy")
    dev = _mss._device_of(dy)
    io = _code(dy.dtype)
    dp, ds = _rows(dy, "dy", shape, dy.dtype, dev)
    if x is None or gate_a is None or gate_x is None or states is None:
        raise TypeError("x, gate_a, gate_x and states are needed")
    xp, xs = _rows(x, "x", shape, dy.dtype, dev)
    ap, as_ = _rows(gate_a, "gate_a", shape, dy.dtype, dev)
    ip, is_ = _rows(gate_x, "gate_x", shape, dy.dtype, dev)
    lp = _vec(lam, "lam", dim, dev)
    tp = _state(states, "states", (b, _chunks(length), dim), dev)
    hp, sp = _state(dh_last, "dh_last", (b, dim), dev), _marks(starts, "starts", (b, length), dev)
    handle, here = _on(stream, dev)
    with here:
        dx, dxp, dxs = _result(dx, "dx", shape, dy.dtype, dev, dy)
        dgate_a, dap, das = _result(dgate_a, "dgate_a", shape, dy.dtype, dev, dy)
        dgate_x, dip, dis = _result(dgate_x, "dgate_x", shape, dy.dtype, dev, dy)
        dlam = torch.empty_like(lam)
        dh0 = torch.empty((b, dim), dtype=torch.float32, device=dev) if want_dh0 else None
        need = _workspace_size("mss_gated_recurrence_bwd_workspace_size", b, length, dim, io)
        if need == 0:
            _mss._raise(2, "gated_recurrence_bwd")
        ws = torch.empty(need, dtype=torch.uint8, device=dev)
        st = _mss.lib().mss_gated_recurrence_bwd(dp, ds, xp, xs, ap, as_, ip, is_, lp, c, sp, tp, hp, dxp, dxs, dap, das,
                                                 dip, dis, dlam.data_ptr(), _address(dh0), b, length, dim, io, 0,
                                                 ws.data_ptr(), need, handle)
        _mss._raise(st, "mss_gated_recurrence_bwd")
        if check_waits:
            _mss._check_waits(ws, stream, "mss_gated_recurrence_bwd")
    return {"dx": dx, "dgate_a": dgate_a, "dgate_x": dgate_x, "dlam": dlam, "dh0": dh0}


def gated_recurrence_step(h, x, gate_a, gate_x, lam, *, c=8.0, parents=None, h_out=None, out=None, stream=None):
    """One token of the gated linear recurrence: returns y ([rows, dim], x's
    type) and the new state.

    h: [rows, dim] float32; x, gate_a, gate_x: [rows, dim] float32 or bfloat16.
    parents ([batch, beams] int64, batch * beams rows): row (b, k) continues from
    the state of beam parents[b, k] of its sequence.  The new state is written to
    ``h_out``; None: in place, or to a new tensor with parents (which h itself
    cannot be)."""
    if not isinstance(x, torch.Tensor) or x.dim() != 2 or x.numel() == 0:
        raise ValueError("x must be a [rows, dim] tensor, neither of them empty")
    dev = _mss._device_of(x)
    rows, dim = shape = x.shape
    io = _code(x.dtype)
    if h is None:
        raise TypeError("h must be a torch.Tensor")
    hp = _state(h, "h", shape, dev)
    xp, xs = _rows(x, "x", shape, x.dtype, dev)
    ap, as_ = _rows(gate_a, "gate_a", shape, x.dtype, dev)
    ip, is_ = _rows(gate_x, "gate_x", shape, x.dtype, dev)
    lp = _vec(lam, "lam", dim, dev)
    batch, beams, pp = rows, 1, None
    if parents is not None:
        if not isinstance(parents, torch.Tensor) or parents.dim() != 2 or parents.numel() != rows:
            raise ValueError(f"parents must be [batch, beams] with batch * beams = {rows} rows")
        _mss._check(parents, "parents", parents.shape, torch.int64, dev)
        (batch, beams), pp = parents.shape, parents.data_ptr()
    handle, here = _on(stream, dev)
    with here:
        if h_out is None:
            h_out = h if parents is None else torch.empty_like(h)
        np_ = _state(h_out, "h_out", shape, dev)
        out, op, os = _result(out, "out", shape, x.dtype, dev, x)
        st = _mss.lib().mss_gated_recurrence_step(hp, pp, xp, xs, ap, as_, ip, is_, lp, c, np_, op, os, batch, beams, dim,
                                                  io, 0, handle)
    _mss._raise(st, "mss_gated_recurrence_step")
    return out, h_out
