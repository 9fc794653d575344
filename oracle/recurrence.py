"""fp64 reference of the gated linear recurrence (a mixer with one state per
channel) and its gradient, step by step in plain numpy from the formulas; shares
no code with the GPU path.  Test infrastructure only.

Every result comes with a bound on what an fp32 evaluation may be off by (before
a rounding to the stored type), carried through the same steps.  In units of
u = 2^-24:
  sigmoid: the exponential's argument is rounded (2 |v| u with plain fp32, left
    out where that rounding is put back), two hardware functions of 2 u each, an
    addition, a correction: 8 u more;
  softplus: 4 u, its product with c and with the gate 4 u;
  m = 1 - exp(-s): the relative error of s is not amplified, 8 u for the
    polynomial or the exponential and the difference;
  sqrt(m (2 - m)): half of m's, 4 u;
  a = exp(-s): up to s = 1/2 as 1 - m, off by m's error; beyond it is the
    exponential itself, whose relative error is s times that of s, the rounding of
    the argument (2 s u, or left out as for the sigmoid) and 4 u.  (At s = 1/2 the
    first is the larger of the two whatever the gate, so it does not matter on
    which side a rounding of s falls.)  Below 2^-126 the exponential is 0;
  a step h + (b - m h) or a h + b: a's error on |h|, 4 u of the sum of magnitudes
    (the part of the state from before a piece of the sequence and the part from
    inside it are formed apart and added).
"""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24


def _f(a):
    return None if a is None else np.asarray(a, dtype=np.float64)


def sigmoid(v):
    return np.where(v >= 0, 1.0 / (1.0 + np.exp(-np.abs(v))), np.exp(-np.abs(v)) / (1.0 + np.exp(-np.abs(v))))


def softplus(v):
    return np.logaddexp(0.0, v)


class Parts:
    """What a step is made of, and the relative errors of an fp32 evaluation;
    ``exact``: the rounding of the sigmoids' arguments is put back."""

    def __init__(self, gate_a, gate_x, lam, c, exact):
        gate_a, gate_x, lam = _f(gate_a), _f(gate_x), _f(lam)
        self.r, self.i = sigmoid(gate_a), sigmoid(gate_x)
        self.rr, self.ri = sigmoid(-gate_a), sigmoid(-gate_x)
        self.s = c * softplus(lam) * self.r
        self.a, self.m = np.exp(-self.s), -np.expm1(-self.s)
        self.beta = np.sqrt(self.m * (2.0 - self.m))
        arg = 0.0 if exact else 2.0
        self.e_r, self.e_i = (8 + arg * np.abs(gate_a)) * U, (8 + arg * np.abs(gate_x)) * U
        self.e_s = self.e_r + 8 * U
        self.e_m = self.e_s + 8 * U
        beyond = self.a * (self.s * (self.e_s + arg * U) + 4 * U) + 2.0 ** -126
        self.d_a = np.where(self.s > 0.5001, beyond, self.e_m * self.m)  # of a, absolute
        self.rate = np.exp(-np.logaddexp(0.0, -lam) - np.log(softplus(lam)))  # sigmoid / softplus


def forward(x, gate_a, gate_x, lam, c=8.0, h0=None, starts=None, exact=True):
    """(h [batch, seqlen, dim], bound of h)."""
    x, h0 = _f(x), _f(h0)
    p = Parts(gate_a, gate_x, lam, c, exact)
    b = p.beta * p.i * x
    e_b = (p.e_m + p.e_i + 4 * U) * np.abs(b)
    h = np.zeros((x.shape[0], x.shape[2])) if h0 is None else h0.copy()
    size, err = np.abs(h), np.zeros_like(h)
    out, bound = np.empty_like(x), np.empty_like(x)
    for t in range(x.shape[1]):
        keep = np.ones((x.shape[0], 1)) if starts is None else (np.asarray(starts)[:, t, None] == 0).astype(float)
        a = keep * p.a[:, t]
        err = a * err + p.d_a[:, t] * keep * size
        size = a * size + np.abs(b[:, t])
        err = err + 4 * U * size + e_b[:, t]
        h = a * h + b[:, t]
        out[:, t], bound[:, t] = h, err
    return out, bound


def backward(dy, x, gate_a, gate_x, lam, c=8.0, h0=None, starts=None, dh_last=None, exact=True, adds=256):
    """{name: (gradient, bound)} of dx, dgate_a, dgate_x, dlam, dh0; ``adds``: units
    of the sums behind dlam."""
    dy, x, h0 = _f(dy), _f(x), _f(h0)
    p = Parts(gate_a, gate_x, lam, c, exact)
    h, e_h = forward(x, gate_a, gate_x, lam, c, h0, starts, exact)
    first = np.zeros((x.shape[0], 1, x.shape[2])) if h0 is None else h0[:, None]
    before = np.concatenate([first, h[:, :-1]], 1)
    e_before = np.concatenate([np.zeros_like(first), e_h[:, :-1]], 1)
    keep = np.ones(x.shape[:2]) if starts is None else (np.asarray(starts) == 0).astype(float)
    carry = np.zeros_like(first[:, 0]) if dh_last is None else _f(dh_last).copy()
    size, err = np.abs(carry), np.zeros_like(carry)
    g, gs, ge = np.empty_like(x), np.empty_like(x), np.empty_like(x)
    for t in reversed(range(x.shape[1])):
        g[:, t] = dy[:, t] + carry
        gs[:, t] = size + np.abs(dy[:, t])
        ge[:, t] = err + 4 * U * gs[:, t]
        k = keep[:, t, None]
        carry = k * p.a[:, t] * g[:, t]
        size = k * p.a[:, t] * gs[:, t]
        err = k * (p.a[:, t] * ge[:, t] + p.d_a[:, t] * gs[:, t] + 4 * U * size)
    bi = p.beta * p.i
    e_a = p.d_a + 2 * U * p.a
    with np.errstate(divide="ignore", invalid="ignore"):
        ratio = np.where(p.m > 0, p.s / p.beta, 0.0)
    ix, kb = np.abs(p.i * x), keep[:, :, None] * np.abs(before)
    first_term = p.a ** 2 * ratio * p.i * x
    second_term = keep[:, :, None] * p.s * p.a * before
    big = g * (first_term - second_term)
    e_big = ((np.abs(first_term) + np.abs(second_term)) * ge +
             gs * (2 * p.a * e_a * ratio * ix + np.abs(first_term) * (p.e_s + p.e_m + p.e_i + 8 * U) +
                   p.s * e_a * kb + np.abs(second_term) * (p.e_s + 6 * U) +
                   keep[:, :, None] * p.s * p.a * e_before))
    s_big = gs * (np.abs(first_term) + np.abs(second_term))
    dlam = big.sum((0, 1)) * p.rate
    return {
        "dx": (g * bi, bi * ge + gs * bi * (p.e_m + p.e_i + 6 * U)),
        "dgate_x": (g * bi * x * p.ri, np.abs(bi * x * p.ri) * (ge + gs * (p.e_m + 2 * p.e_i + 10 * U))),
        "dgate_a": (big * p.rr, p.rr * (e_big + s_big * (p.e_r + 6 * U))),
        "dlam": (dlam, p.rate * (e_big.sum((0, 1)) + (adds + 16) * U * s_big.sum((0, 1)))),
        "dh0": (carry, err),
    }
