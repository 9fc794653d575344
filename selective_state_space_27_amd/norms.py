"""Python binding of the operators around the mixer (``include/mambascan.h``):
the norm before a block with its residual, the norm after a mixer with its
gate, 8-bit activation checkpoints, and the weight gradient from one.

Activations are [..., cols] tensors whose leading dimensions collapse to rows
of one stride (a slice of a wider tensor's columns does); outputs are new
contiguous tensors of the same shape unless given.  Everything else is as in
the package's other functions: checks here and in the library, no CPU path,
outputs and workspaces allocated by PyTorch on the stream that the call runs
on (``stream``, default the current one; as inside ``torch.cuda.stream``,
tensors of another stream have to be ready, and results are ordered with that
stream).
"""
from __future__ import annotations

import contextlib
import functools

import torch

import selective_state_space_27_amd as _mss

_CODES = {torch.float32: 0, torch.bfloat16: 1}
_HERE = contextlib.nullcontext()
# The current stream's handle without a Stream object around it (1 us of a
# call of 9); the public way where this torch lacks it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


class Packed8:
    """The 8-bit form of a tensor (``pack8``): ``q`` int8 [rows, pitch] and
    ``scale`` uint8 [rows, pitch // 32], the exponents of the blocks' powers of
    two; pitch is cols rounded up to a multiple of 32.  ``shape`` and ``dtype``
    are the packed tensor's."""

    __slots__ = ("q", "scale", "shape", "dtype")

    def __init__(self, q, scale, shape, dtype):
        shape = torch.Size(shape)
        rows, cols = _rows_cols(shape, "shape")
        pitch = -(-cols // 32) * 32
        if dtype not in _CODES:
            raise TypeError(f"unsupported dtype {dtype} (float32 or bfloat16)")
        _mss._check(q, "q", (rows, pitch), torch.int8, q.device)
        _mss._check(scale, "scale", (rows, pitch // 32), torch.uint8, q.device)
        self.q, self.scale, self.shape, self.dtype = q, scale, shape, dtype

    @property
    def device(self):
        return self.q.device

    def nbytes(self) -> int:
        """Bytes held."""
        return self.q.numel() + self.scale.numel()


def _rows_cols(shape, name):
    cols = shape[-1] if len(shape) else 0
    rows = shape.numel() // cols if cols else 0
    if rows == 0:
        raise ValueError(f"{name} has shape {tuple(shape)}: at least one dimension, none of them empty")
    return rows, cols


def _rows(t, name, shape, dtype, device):
    """(pointer, row stride) of an activation."""
    if t is None:
        return None, 0
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    cols = shape[-1]
    if t.is_contiguous():
        return t.data_ptr(), cols
    strides = t.stride()
    if cols > 1 and strides[-1] != 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    rows, stride = 1, cols
    for n, s in zip(reversed(shape[:-1]), reversed(strides[:-1])):
        if n == 1:
            continue
        if rows == 1:
            stride = s
        elif s != rows * stride:
            raise ValueError(f"{name}: leading dimensions of {tuple(shape)} with strides {tuple(strides)} "
                             "are not rows of one stride")
        rows *= n
    if stride < cols:
        raise ValueError(f"{name}: rows overlap (stride {stride} of {cols} columns)")
    return t.data_ptr(), stride


def _packed(p, name, shape, dtype, device):
    """(q pointer, scale pointer) of a Packed8."""
    if p.device != device:
        raise ValueError(f"{name} is on {p.device}, expected {device}")
    if p.dtype != dtype:
        raise TypeError(f"{name} holds {p.dtype}, expected {dtype}")
    if p.shape != shape:
        raise ValueError(f"{name} has shape {tuple(p.shape)}, expected {tuple(shape)}")
    return p.q.data_ptr(), p.scale.data_ptr()


def _source(t, name, shape, dtype, device):
    """(pointer, stride, scale pointer) of a tensor or Packed8."""
    if isinstance(t, Packed8):
        q, s = _packed(t, name, shape, dtype, device)
        return q, 0, s
    p, stride = _rows(t, name, shape, dtype, device)
    return p, stride, None


def _vec(t, name, cols, device):
    if t is None:
        return None
    if not (isinstance(t, torch.Tensor) and t.dtype == torch.float32 and t.shape == (cols,) and t.device == device and
            t.is_contiguous()):
        _mss._check(t, name, (cols,), torch.float32, device)
    return t.data_ptr()


def _code(dtype) -> int:
    try:
        return _CODES[dtype]
    except KeyError:
        raise TypeError(f"unsupported dtype {dtype} (float32 or bfloat16)") from None


def _on(stream, device):
    """(stream handle, context) of a call: allocations inside the context belong
    to the stream, launches to the device."""
    if stream is None:
        index = device.index
        return _raw_stream(index), _HERE if index == torch.cuda.current_device() else torch.cuda.device(device)
    if stream.device != device:
        raise ValueError(f"stream is on {stream.device}, expected {device}")
    return stream.cuda_stream, torch.cuda.stream(stream)


def _empty_packed(rows, cols, shape, dtype, device):
    blocks = (cols + 31) // 32
    p = Packed8.__new__(Packed8)  # of the right make: nothing to check
    p.q = torch.empty((rows, blocks * 32), dtype=torch.int8, device=device)
    p.scale = torch.empty((rows, blocks), dtype=torch.uint8, device=device)
    p.shape, p.dtype = shape, dtype
    return p


def _pq(p):
    return (None, None) if p is None else (p.q.data_ptr(), p.scale.data_ptr())


def _result(given, name, shape, dtype, device, like=None):
    """(tensor, pointer, row stride) of an output, allocated unless given; `like`
    an input of its shape, which makes that quicker where it fits."""
    if given is None:
        if isinstance(like, torch.Tensor) and like.dtype == dtype and like.is_contiguous():
            t = torch.empty_like(like)
        else:
            t = torch.empty(shape, dtype=dtype, device=device)
        return t, t.data_ptr(), shape[-1]
    p, stride = _rows(given, name, shape, dtype, device)
    return given, p, stride


@functools.lru_cache(maxsize=256)
def _workspace_size(query, *sizes):
    return getattr(_mss.lib(), query)(*sizes)


# ------------------------------------------------------- norm before a block
def add_norm_fwd(x, residual, weight, *, post_weight=None, gamma=None, scale=1.0, eps=1e-5, residual_dtype=None,
                 pack_out=False, out=None, residual_out=None, stream=None):
    """r = residual + scale*gamma*x', out = RMS(r)*weight, with x' = x, or
    RMS(x)*post_weight when that is given; RMS(v) = v / sqrt(mean(v^2) + eps)
    over the last dimension.

    x: [..., cols] float32 or bfloat16; residual: the same shape, or None (zero),
    in ``residual_dtype`` (default its own dtype, or x's): float32, or x's
    dtype; weight, post_weight, gamma: [cols] float32.  Returns out (x's dtype)
    and residual_out (residual_dtype), and with ``pack_out`` a Packed8 of out.
    The form for a generated token is a call with its row(s)."""
    dev = _mss._device_of(x)
    shape = x.shape
    rows, cols = _rows_cols(shape, "x")
    rdt = residual_dtype if residual_dtype is not None else x.dtype if residual is None else residual.dtype
    io, res = _code(x.dtype), _code(rdt)
    xp, xs = _rows(x, "x", shape, x.dtype, dev)
    rp, rs = _rows(residual, "residual", shape, rdt, dev)
    wp, pp, gp = (_vec(weight, "weight", cols, dev), _vec(post_weight, "post_weight", cols, dev),
                  _vec(gamma, "gamma", cols, dev))
    handle, here = _on(stream, dev)
    with here:
        out, op, os = _result(out, "out", shape, x.dtype, dev, x)
        residual_out, qp, qs = _result(residual_out, "residual_out", shape, rdt, dev, residual)
        packed = _empty_packed(rows, cols, shape, x.dtype, dev) if pack_out else None
        st = _mss.lib().mss_add_norm_fwd(xp, xs, rp, rs, wp, pp, gp, scale, eps, op, os, qp, qs, *_pq(packed), rows,
                                         cols, io, res, 0, handle)
    _mss._raise(st, "mss_add_norm_fwd")
    return (out, residual_out, packed) if pack_out else (out, residual_out)


def add_norm_bwd(dout, residual_out, weight, *, dresidual_out=None, x=None, post_weight=None, gamma=None, scale=1.0,
                 eps=1e-5, want_dx=True, want_dresidual=True, dx=None, dresidual=None, stream=None):
    """Gradients of add_norm_fwd at its stored ``residual_out`` (a tensor or
    its Packed8), given dout and dresidual_out (None: zero).  ``x`` (a tensor,
    or a Packed8 when residual_out is one) is needed with post_weight or gamma.

    Returns a dict: dx (dout's dtype), dresidual (residual_out's dtype; either
    None when not wanted), dweight, dpost_weight, dgamma ([cols] float32; None
    without the weight)."""
    dev = _mss._device_of(dout)
    shape = dout.shape
    rows, cols = _rows_cols(shape, "dout")
    rdt = residual_out.dtype
    io, res = _code(dout.dtype), _code(rdt)
    dp, ds = _rows(dout, "dout", shape, dout.dtype, dev)
    ep, es = _rows(dresidual_out, "dresidual_out", shape, rdt, dev)
    rp, rs, rsc = _source(residual_out, "residual_out", shape, rdt, dev)
    wp, pp, gp = (_vec(weight, "weight", cols, dev), _vec(post_weight, "post_weight", cols, dev),
                  _vec(gamma, "gamma", cols, dev))
    xp = xs = xsc = None
    if pp is not None or gp is not None:
        if x is None:
            raise ValueError("x is needed with post_weight or gamma")
        xp, xs, xsc = _source(x, "x", shape, dout.dtype, dev)
    ngrads = 1 + (pp is not None) + (gp is not None)
    handle, here = _on(stream, dev)
    with here:
        dxp = dxs = drp = drs = None
        if want_dx:
            dx, dxp, dxs = _result(dx, "dx", shape, dout.dtype, dev, dout)
        if want_dresidual:
            dresidual, drp, drs = _result(dresidual, "dresidual", shape, rdt, dev, residual_out)
        dw = torch.empty_like(weight)
        dpost, dgamma = (None if p is None else torch.empty_like(dw) for p in (pp, gp))
        need = _workspace_size("mss_add_norm_bwd_workspace_size", rows, cols, ngrads)
        if need == 0:
            _mss._raise(5, "add_norm_bwd")
        ws = torch.empty(need, dtype=torch.uint8, device=dev)
        st = _mss.lib().mss_add_norm_bwd(dp, ds, ep, es, rp, rs, rsc, xp, xs or 0, xsc, wp, pp, gp, scale, eps, dxp,
                                         dxs or 0, drp, drs or 0, dw.data_ptr(), _mss._ptr(dpost), _mss._ptr(dgamma),
                                         rows, cols, io, res, 0, ws.data_ptr(), need, handle)
    _mss._raise(st, "mss_add_norm_bwd")
    return {"dx": dx if want_dx else None, "dresidual": dresidual if want_dresidual else None, "dweight": dw,
            "dpost_weight": dpost, "dgamma": dgamma}


# -------------------------------------------------------- norm after a mixer
def gated_norm_fwd(y, z, weight, *, ngroups=1, norm_first=False, eps=1e-5, out_dtype=None, pack_inputs=False,
                   pack_out=False, out=None, stream=None):
    """RMS(y*silu(z))*weight, or RMS(y)*weight*silu(z) with ``norm_first``, or
    RMS(y)*weight without z (None); RMS over each of ``ngroups`` groups of columns.

    y: [..., cols] float32 or bfloat16 (ssd_chunk_fwd's y with its heads
    flattened); z: the same shape, y's dtype or bfloat16; weight: [cols] float32.
    out has z's dtype (without z: ``out_dtype``, default y's).  Returns out, and
    after it, as asked for, Packed8 forms: y's and z's with ``pack_inputs`` (z's
    None without z), out's with ``pack_out``."""
    dev = _mss._device_of(y)
    shape = y.shape
    rows, cols = _rows_cols(shape, "y")
    odt = z.dtype if z is not None else out_dtype if out_dtype is not None else y.dtype
    if out_dtype is not None and out_dtype != odt:
        raise TypeError(f"out has z's dtype {odt}, not {out_dtype}")
    wide, io = _code(y.dtype), _code(odt)
    yp, ys = _rows(y, "y", shape, y.dtype, dev)
    zp, zs = _rows(z, "z", shape, odt, dev)
    wp = _vec(weight, "weight", cols, dev)
    handle, here = _on(stream, dev)
    with here:
        out, op, os = _result(out, "out", shape, odt, dev, y)
        y8 = _empty_packed(rows, cols, shape, y.dtype, dev) if pack_inputs else None
        z8 = _empty_packed(rows, cols, shape, odt, dev) if pack_inputs and z is not None else None
        out8 = _empty_packed(rows, cols, shape, odt, dev) if pack_out else None
        st = _mss.lib().mss_gated_norm_fwd(yp, ys, zp, zs, wp, eps, op, os, *_pq(y8), *_pq(z8), *_pq(out8), rows, cols,
                                           ngroups, wide, io, _mss.MSS_FLAG_NORM_FIRST if norm_first else 0, handle)
    _mss._raise(st, "mss_gated_norm_fwd")
    if not pack_inputs and not pack_out:
        return out
    return (out,) + ((y8, z8) if pack_inputs else ()) + ((out8,) if pack_out else ())


def gated_norm_bwd(dout, y, z, weight, *, ngroups=1, norm_first=False, eps=1e-5, dy=None, dz=None, stream=None):
    """Gradients of gated_norm_fwd, given dout.  y and z are the forward's
    tensors, or both their Packed8 forms (the gradient at the values these
    stand for).  Returns a dict: dy (y's dtype), dz (dout's dtype; None without
    z), dweight ([cols] float32)."""
    dev = _mss._device_of(dout)
    shape = dout.shape
    rows, cols = _rows_cols(shape, "dout")
    wide, io = _code(y.dtype), _code(dout.dtype)
    dp, ds = _rows(dout, "dout", shape, dout.dtype, dev)
    yp, ys, ysc = _source(y, "y", shape, y.dtype, dev)
    zp, zs, zsc = _source(z, "z", shape, dout.dtype, dev)
    wp = _vec(weight, "weight", cols, dev)
    handle, here = _on(stream, dev)
    with here:
        dy, dyp, dys = _result(dy, "dy", shape, y.dtype, dev, y)
        dzp = dzs = None
        if z is not None:
            dz, dzp, dzs = _result(dz, "dz", shape, dout.dtype, dev, dout)
        dw = torch.empty_like(weight)
        need = _workspace_size("mss_gated_norm_bwd_workspace_size", rows, cols, ngroups)
        if need == 0:
            _mss._raise(5, "gated_norm_bwd")
        ws = torch.empty(need, dtype=torch.uint8, device=dev)
        st = _mss.lib().mss_gated_norm_bwd(dp, ds, yp, ys, ysc, zp, zs, zsc, wp, eps, dyp, dys, dzp, dzs or 0,
                                           dw.data_ptr(), rows, cols, ngroups, wide, io,
                                           _mss.MSS_FLAG_NORM_FIRST if norm_first else 0, ws.data_ptr(), need, handle)
    _mss._raise(st, "mss_gated_norm_bwd")
    return {"dy": dy, "dz": dz if z is not None else None, "dweight": dw}


# ---------------------------------------------------------- 8-bit checkpoints
def pack8(x, *, stream=None) -> Packed8:
    """The 8-bit form of x ([..., cols], float32 or bfloat16): 8.25 bits an
    element, within half a step of a block of 32 columns' power-of-two scale
    (max|x| / 127 of the block at most; fp32 magnitudes above 127.5 * 2^121
    saturate, off by up to a step)."""
    dev = _mss._device_of(x)
    rows, cols = _rows_cols(x.shape, "x")
    code = _code(x.dtype)
    xp, xs = _rows(x, "x", x.shape, x.dtype, dev)
    handle, here = _on(stream, dev)
    with here:
        p = _empty_packed(rows, cols, x.shape, x.dtype, dev)
        st = _mss.lib().mss_pack8(xp, xs, *_pq(p), rows, cols, code, handle)
    _mss._raise(st, "mss_pack8")
    return p


def unpack8(p, dtype=None, *, out=None, stream=None):
    """The values a Packed8 stands for, in its dtype or ``dtype`` (exact in both)."""
    if not isinstance(p, Packed8):
        raise TypeError("p must be a Packed8")
    dev = _mss._device_of(p.q)
    dtype = dtype if dtype is not None else p.dtype
    code = _code(dtype)
    rows, cols = _rows_cols(p.shape, "p")
    handle, here = _on(stream, dev)
    with here:
        out, op, os = _result(out, "out", p.shape, dtype, dev)
        st = _mss.lib().mss_unpack8(*_pq(p), op, os, rows, cols, code, handle)
    _mss._raise(st, "mss_unpack8")
    return out


def wgrad8(dy, x8, *, out=None, out_dtype=torch.float32, accumulate=False, stream=None):
    """Weight gradient dY^T X ([outs, ins], float32 or bfloat16) of a linear layer
    whose input x8 ([..., ins]) is a Packed8; dy: [..., outs] bfloat16.
    ``accumulate``: added to ``out``, which then has to be given."""
    if not isinstance(x8, Packed8):
        raise TypeError("x8 must be a Packed8")
    dev = _mss._device_of(dy)
    tokens, outs = _rows_cols(dy.shape, "dy")
    if x8.shape[:-1] != dy.shape[:-1]:
        raise ValueError(f"dy of shape {tuple(dy.shape)} and x8 of shape {tuple(x8.shape)} differ in their rows")
    ins = x8.shape[-1]
    dp, ds = _rows(dy, "dy", dy.shape, dy.dtype, dev)
    q, s = _packed(x8, "x8", x8.shape, x8.dtype, dev)
    code = _code(dy.dtype)
    if accumulate and out is None:
        raise ValueError("accumulate needs out")
    dtype = out.dtype if out is not None else out_dtype
    dcode = _code(dtype)
    handle, here = _on(stream, dev)
    with here:
        if out is None:
            out = torch.empty((outs, ins), dtype=dtype, device=dev)
        _mss._check(out, "out", (outs, ins), dtype, dev)
        need = _mss.lib().mss_wgrad8_workspace_size(dp, ds, tokens, outs, ins)
        if need == 0:
            _mss._raise(2, "wgrad8")
        ws = torch.empty(need, dtype=torch.uint8, device=dev)
        st = _mss.lib().mss_wgrad8(dp, ds, q, s, out.data_ptr(), tokens, outs, ins, code, dcode,
                                   _mss.MSS_FLAG_ACCUMULATE if accumulate else 0, ws.data_ptr(), need, handle)
    _mss._raise(st, "mss_wgrad8")
    return out
