"""The bound of the gated recurrence's fp64 reference where decays are strong (CPU): it
goes with the decay, so it holds for an evaluation that keeps the decay itself and not
for one that keeps it as 1 + n."""
import numpy as np
import pytest

from oracle import recurrence as orec

F = np.float32


def draw(length, lam, seed):
    g = np.random.default_rng(seed)
    n = lambda *s: g.standard_normal(s).astype(F)  # noqa: E731
    d = {"x": n(2, length, 70), "gate_a": n(2, length, 70) + F(2), "gate_x": n(2, length, 70),
         "lam": np.full(70, lam, F), "h0": n(2, 70)}
    return d, n(2, length, 70), n(2, 70)


@pytest.mark.parametrize("lam", [1.0, 2.0, 3.0])
@pytest.mark.parametrize("length", [1, 2, 3])
def test_the_bound_is_a_small_part_of_the_value(lam, length):
    """dgate_a and dh0 are products with the decay: a wrong sign or a zero must not pass.  16 u
    of the exponent, which is up to 24.4, and some 30 u more are below 3e-5 (without the arguments'
    roundings; with them 16 + 2 |gate| + 2 u of it, below 6e-5); sums that cancel to a third are let through."""
    d, dy, dl = draw(length, lam, length)
    for exact, most in ((True, 1e-4), (False, 2e-4)):
        got = orec.backward(dy, **d, dh_last=dl, exact=exact)
        for k in ("dgate_a", "dh0"):
            value, bound = got[k]
            assert np.mean(bound <= most * np.abs(value)) > 0.8, (k, exact)


@pytest.mark.parametrize("lam", [1.0, 2.0, 3.0])
def test_evaluations_of_one_step(lam):
    """h0's part of one step and its gradient, with the decay and with 1 + n."""
    d, dy, dl = draw(1, lam, 9)
    d["x"][:] = 0
    want, bound = orec.forward(**d, exact=False)
    grads = orec.backward(dy, **d, exact=False)
    s = F(8) * np.log1p(np.exp(d["lam"])) * (F(1) / (F(1) + np.exp(-d["gate_a"][:, 0])))
    kept, lost = np.exp(-s), F(1) + (np.exp(-s) - F(1))
    for a, holds in ((kept, True), (lost, False)):
        assert (np.abs(a * d["h0"] - want[:, 0]) <= bound[:, 0]).all() == holds
        assert (np.abs(a * dy[:, 0] - grads["dh0"][0]) <= grads["dh0"][1]).all() == holds
