"""Pins of the gated recurrence's and beam search's fp64 references (CPU)."""
import itertools

import numpy as np
import pytest

from oracle import beam as obeam
from oracle import recurrence as orec


def draw(batch, length, dim, seed):
    g = np.random.default_rng(seed)
    n = lambda *s: g.standard_normal(s)  # noqa: E731
    return {"x": n(batch, length, dim), "gate_a": n(batch, length, dim), "gate_x": n(batch, length, dim),
            "lam": n(dim) - 2.0, "h0": n(batch, dim)}


def test_constant_decay_is_a_geometric_sum():
    length, dim, c = 40, 3, 8.0
    lam = np.array([-4.0, -2.0, 1.0])
    shape = (1, length, dim)
    ga, gx, x = np.full(shape, 0.3), np.full(shape, -0.7), np.full(shape, 1.5)
    h, _ = orec.forward(x, ga, gx, lam, c)
    a = np.exp(-c * np.log1p(np.exp(lam)) / (1 + np.exp(-0.3)))
    b = np.sqrt(1 - a * a) / (1 + np.exp(0.7)) * 1.5
    want = b * (1 - a ** np.arange(1, length + 1)[:, None]) / (1 - a)
    assert np.allclose(h[0], want, rtol=1e-12)


def test_starts_split_a_row_into_its_sequences():
    d = draw(1, 30, 4, 1)
    starts = np.zeros((1, 30), np.uint8)
    starts[0, [7, 8, 21]] = 1
    h, _ = orec.forward(**d, starts=starts)
    for lo, hi in ((0, 7), (7, 8), (8, 21), (21, 30)):
        part, _ = orec.forward(*(d[k][:, lo:hi] for k in ("x", "gate_a", "gate_x")), d["lam"],
                               h0=d["h0"] if lo == 0 else None)
        assert np.allclose(part, h[:, lo:hi], rtol=1e-13)


def test_open_and_closed_gates():
    d = draw(1, 5, 2, 2)
    d["gate_a"][:] = -800.0  # closed: the state is kept, nothing comes in
    h, _ = orec.forward(**d)
    assert np.allclose(h, d["h0"][:, None])
    d["gate_a"][:] = 800.0
    d["lam"][:] = 50.0  # forgets everything: h = i x
    h, _ = orec.forward(**d)
    assert np.allclose(h, orec.sigmoid(d["gate_x"]) * d["x"])


@pytest.mark.parametrize("starts", [False, True])
def test_gradient_against_differences(starts):
    d = draw(2, 7, 3, 3)
    g = np.random.default_rng(4)
    dy, dl = g.standard_normal((2, 7, 3)), g.standard_normal((2, 3))
    marks = (g.random((2, 7)) < 0.3).astype(np.uint8) if starts else None

    def loss():
        h, _ = orec.forward(**d, starts=marks)
        return float((h * dy).sum() + (h[:, -1] * dl).sum())

    got = orec.backward(dy, **d, starts=marks, dh_last=dl)
    for name, key in (("x", "dx"), ("gate_a", "dgate_a"), ("gate_x", "dgate_x"), ("lam", "dlam"), ("h0", "dh0")):
        t, grad = d[name], got[key][0]
        for at in np.ndindex(t.shape):
            keep, eps = t[at], 1e-5
            t[at] = keep + eps
            up = loss()
            t[at] = keep - eps
            diff = (up - loss()) / (2 * eps)
            t[at] = keep
            assert abs(diff - grad[at]) < 1e-8 * max(1, abs(diff)), (name, at)


def test_bound_covers_an_fp32_evaluation():
    d = {k: v.astype(np.float32) for k, v in draw(2, 300, 5, 5).items()}
    want, bound = orec.forward(**{k: v.astype(np.float64) for k, v in d.items()}, exact=False)
    f = np.float32
    s = f(8) * np.log1p(np.exp(d["lam"])) * (f(1) / (f(1) + np.exp(-d["gate_a"])))
    m = -np.expm1(-s)
    b = np.sqrt(m * (f(2) - m)) * (f(1) / (f(1) + np.exp(-d["gate_x"]))) * d["x"]
    h = d["h0"]
    for t in range(300):
        h = (h - m[:, t] * h) + b[:, t]
        assert (np.abs(h - want[:, t]) <= bound[:, t]).all()


def test_selection_is_the_order_of_all_candidates():
    g = np.random.default_rng(6)
    logits = np.round(g.standard_normal((2, 3, 7)) * 2) / 2  # many ties
    scores = np.array([[-1.0, -1.0, -3.0], [-2.0, -np.inf, np.nan]])
    finished = np.array([[False, True, False], [False, False, False]])
    best, parents, tokens, done = obeam.select(logits, scores, 12, finished, 4)
    for b in range(2):
        every = []
        for k, v in itertools.product(range(3), range(7)):
            lse = np.log(sum(np.exp(logits[b, k, w]) for w in range(7)))
            total = scores[b, k] + logits[b, k, v] - lse if np.isfinite(scores[b, k]) else -np.inf
            if finished[b, k]:
                total = scores[b, k] if v == 4 else -np.inf
            every.append((-round(total, 9) if np.isfinite(total) else np.inf, k * 7 + v))
        every.sort()
        assert [p * 7 + t for p, t in zip(parents[b], tokens[b])] == [e[1] for e in every[:12]]
        assert np.allclose(best[b], [-e[0] for e in every[:12]], atol=1e-8)
    assert done[0].any() and (done == ((tokens == 4) | np.take_along_axis(finished, parents, 1))).all()
