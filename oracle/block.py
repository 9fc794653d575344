"""fp64 reference of the operators around the mixer: norm before a block with
its residual, norm after a mixer with its gate, the 8-bit checkpoint form, and
the weight gradient from one.  Plain numpy from the formulas; shares no code
with the GPU path.  Test infrastructure only.

Each gradient comes with a "size" array of the same shape: the sum of the
magnitudes of the terms it is made of, which is what a rounding error of its
fp32 evaluation is relative to.
"""
from __future__ import annotations

import numpy as np


def _f(a):
    return None if a is None else np.asarray(a, dtype=np.float64)


def _groups(v, ngroups):
    return v.reshape(v.shape[0], ngroups, -1)


def rstd(v, eps, ngroups=1):
    """1 / sqrt(mean(v^2) + eps) over each group of columns, shaped to multiply v."""
    g = _groups(v, ngroups)
    r = 1.0 / np.sqrt(np.mean(g * g, axis=2, keepdims=True) + eps)
    return np.broadcast_to(r, g.shape).reshape(v.shape)


def _mean(a, ngroups=1):
    g = _groups(a, ngroups)
    return np.broadcast_to(np.mean(g, axis=2, keepdims=True), g.shape).reshape(a.shape)


def _norm_grad(g, gsize, v, eps, ngroups=1):
    """d<g, v rstd(v)>/dv and its size."""
    r = rstd(v, eps, ngroups)
    grad = r * g - v * r ** 3 * _mean(g * v, ngroups)
    return grad, r * gsize + np.abs(v) * r ** 3 * _mean(gsize * np.abs(v), ngroups)


def silu(z):
    return z / (1.0 + np.exp(-z))


def silu_grad(z):
    s = 1.0 / (1.0 + np.exp(-z))
    return s * (1.0 + z * (1.0 - s))


# ------------------------------------------------------- norm before a block
def add_norm(x, residual, weight, post=None, gamma=None, scale=1.0, eps=1e-5):
    """(out, r) of r = residual + scale gamma x', out = r rstd(r) weight."""
    x, residual, weight, post, gamma = map(_f, (x, residual, weight, post, gamma))
    xp = x if post is None else x * rstd(x, eps) * post
    r = scale * (1.0 if gamma is None else gamma) * xp + (0.0 if residual is None else residual)
    return r * rstd(r, eps) * weight, r


def add_norm_sizes(x, residual, weight, post=None, gamma=None, scale=1.0, eps=1e-5):
    """Sizes of (out, r)."""
    x, residual, weight, post, gamma = map(_f, (x, residual, weight, post, gamma))
    _, r = add_norm(x, residual, weight, post, gamma, scale, eps)
    xp = x if post is None else x * rstd(x, eps) * post
    size = np.abs(scale * (1.0 if gamma is None else gamma) * xp) + (0.0 if residual is None else np.abs(residual))
    q = rstd(r, eps)
    # an error in r moves out by itself and through rstd
    return (size * q + np.abs(r) * q ** 3 * _mean(np.abs(r) * size)) * np.abs(weight), size


def add_norm_bwd(dout, r, weight, dresidual_out=None, x=None, post=None, gamma=None, scale=1.0, eps=1e-5):
    """Gradients at the stored r: {name: (gradient, size)} with dresidual, dx,
    dweight, and dpost, dgamma where post, gamma are given."""
    dout, r, weight, e, x, post, gamma = map(_f, (dout, r, weight, dresidual_out, x, post, gamma))
    g = dout * weight
    dr, drs = _norm_grad(g, np.abs(g), r, eps)
    if e is not None:
        dr, drs = dr + e, drs + np.abs(e)
    out = {"dresidual": (dr, drs)}
    t = dout * r * rstd(r, eps)
    out["dweight"] = (t.sum(0), np.abs(t).sum(0))
    m = scale * (np.ones_like(weight) if gamma is None else gamma)
    if gamma is not None:
        xp = x if post is None else x * rstd(x, eps) * post
        out["dgamma"] = (scale * (dr * xp).sum(0), np.abs(scale) * (drs * np.abs(xp)).sum(0))
    dxp, dxps = m * dr, np.abs(m) * drs
    if post is None:
        out["dx"] = (dxp, dxps)
        return out
    n = x * rstd(x, eps)
    out["dpost"] = ((dxp * n).sum(0), (dxps * np.abs(n)).sum(0))
    out["dx"] = _norm_grad(dxp * post, dxps * np.abs(post), x, eps)
    return out


# -------------------------------------------------------- norm after a mixer
def gated_norm(y, z, weight, ngroups=1, norm_first=False, eps=1e-5):
    y, z, weight = map(_f, (y, z, weight))
    if z is None:
        return y * rstd(y, eps, ngroups) * weight
    if norm_first:
        return y * rstd(y, eps, ngroups) * weight * silu(z)
    v = y * silu(z)
    return v * rstd(v, eps, ngroups) * weight


def gated_norm_bwd(dout, y, z, weight, ngroups=1, norm_first=False, eps=1e-5):
    """{name: (gradient, size)} with dy, dweight, and dz where z is given."""
    dout, y, z, weight = map(_f, (dout, y, z, weight))
    g = dout * weight
    if z is None or norm_first:
        s = 1.0 if z is None else silu(z)
        dy = _norm_grad(g * s, np.abs(g * s), y, eps, ngroups)
        n = y * rstd(y, eps, ngroups)
        t = dout * n * s
        out = {"dy": dy, "dweight": (t.sum(0), np.abs(t).sum(0))}
        if z is not None:
            dz = g * n * silu_grad(z)
            out["dz"] = (dz, np.abs(g * n) * (np.abs(silu_grad(z)) + 1.0 / (1.0 + np.exp(-np.abs(z)))))
        return out
    s, ds = silu(z), silu_grad(z)
    v = y * s
    dv, dvs = _norm_grad(g, np.abs(g), v, eps, ngroups)
    t = dout * v * rstd(v, eps, ngroups)
    # silu' is a sum of terms of the size of 1 near its zero
    return {"dy": (dv * s, dvs * np.abs(s)), "dz": (dv * y * ds, dvs * np.abs(y) * (np.abs(ds) + 1.0)),
            "dweight": (t.sum(0), np.abs(t).sum(0))}


# ---------------------------------------------------------- 8-bit checkpoints
# A block's maximum is below this many steps: the form's definition, 127.5's lower neighbour in fp32 (mss_pack8 in
# include/mambascan.h).
TOP = 127.5 - 2.0 ** -17


def pack8(x):
    """(q int8 [rows, pitch], exponent bytes uint8 [rows, pitch / 32])."""
    x = _f(x)
    rows, cols = x.shape
    pitch = -(-cols // 32) * 32
    v = np.zeros((rows, pitch))
    v[:, :cols] = x
    v = v.reshape(rows, -1, 32)
    finite = np.isfinite(v).all(axis=2)
    top = np.where(finite, np.abs(np.where(np.isfinite(v), v, 0.0)).max(axis=2), 0.0)
    e = np.full(top.shape, 1, dtype=np.int64)
    for k in range(2, 249):  # the smallest power of two that holds the block
        e = np.where(top >= TOP * 2.0 ** (k - 1 - 127), k, e)
    q = np.clip(np.rint(np.where(finite[:, :, None], v, 0.0) / 2.0 ** (e - 127.0)[:, :, None]), -127, 127)
    return q.astype(np.int8).reshape(rows, pitch), np.where(finite, e, 255).astype(np.uint8)


def unpack8(q, e, cols):
    q, e = np.asarray(q), np.asarray(e)
    s = np.where(e == 255, np.nan, 2.0 ** (e.astype(np.float64) - 127.0))
    return (q.astype(np.float64).reshape(q.shape[0], -1, 32) * s[:, :, None]).reshape(q.shape[0], -1)[:, :cols]


def wgrad8(dy, q, e, cols):
    """(dY^T X, size)."""
    x, dy = unpack8(q, e, cols), _f(dy)
    return dy.T @ x, np.abs(dy).T @ np.abs(x)
