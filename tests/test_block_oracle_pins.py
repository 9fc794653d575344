"""Pins of the fp64 reference of the operators around the mixer (CPU only):
hand-computed values, invariants, gradients against central differences, and
the 8-bit form's definition on its edges."""
import numpy as np
import pytest

from oracle import block as ob

RNG = np.random.default_rng


def central(f, x, h=1e-6):
    """Gradient of the scalar f at x by central differences."""
    g = np.zeros_like(x)
    it = np.nditer(x, flags=["multi_index"])
    for _ in it:
        i = it.multi_index
        keep = x[i]
        x[i] = keep + h
        hi = f()
        x[i] = keep - h
        lo = f()
        x[i] = keep
        g[i] = (hi - lo) / (2 * h)
    return g


def test_hand_values():
    # mean(v^2) = (9 + 16) / 2 = 12.5; with eps = 12.5 rstd = 1/5
    out, r = ob.add_norm([[1.0, 2.0]], [[2.0, 2.0]], [1.0, 10.0], eps=12.5)
    assert np.allclose(r, [[3.0, 4.0]], rtol=1e-15) and np.allclose(out, [[0.6, 8.0]], rtol=1e-15)
    # scale 0.5 and gamma halve each part of x
    out, r = ob.add_norm([[4.0, 8.0]], [[1.0, 0.0]], [1.0, 1.0], gamma=[1.0, 1.0], scale=0.5, eps=12.5)
    assert np.allclose(r, [[3.0, 4.0]], rtol=1e-15)
    # no gate: groups of one column give v / sqrt(v^2 + eps)
    out = ob.gated_norm([[3.0, -4.0]], None, [1.0, 1.0], ngroups=2, eps=16.0)
    assert np.allclose(out, [[0.6, -4.0 / np.sqrt(32.0)]], rtol=1e-15)
    # silu(0) = 0: a closed gate gives zeros, gate first (0 / sqrt(eps)) and norm first
    for first in (False, True):
        assert np.all(ob.gated_norm([[3.0, -4.0]], [[0.0, 0.0]], [1.0, 1.0], norm_first=first) == 0)


def test_scale_invariance_and_groups():
    r = RNG(0)
    y, z, w = r.standard_normal((3, 12)), r.standard_normal((3, 12)), r.standard_normal(12)
    # with eps = 0 the norm does not see a positive factor
    assert np.allclose(ob.gated_norm(7.0 * y, z, w, eps=0.0), ob.gated_norm(y, z, w, eps=0.0), rtol=1e-13)
    # a group is a norm of its own
    parts = [ob.gated_norm(y[:, i:i + 4], z[:, i:i + 4], w[i:i + 4]) for i in (0, 4, 8)]
    assert np.allclose(ob.gated_norm(y, z, w, ngroups=3), np.concatenate(parts, 1), rtol=1e-14)


@pytest.mark.parametrize("post,gamma", [(False, False), (False, True), (True, False), (True, True)])
def test_add_norm_gradients_by_differences(post, gamma):
    r = RNG(1)
    rows, cols = 3, 7
    x, res = r.standard_normal((rows, cols)), r.standard_normal((rows, cols))
    w, do, de = r.standard_normal(cols), r.standard_normal((rows, cols)), r.standard_normal((rows, cols))
    p = r.standard_normal(cols) if post else None
    g = r.standard_normal(cols) if gamma else None

    def loss():
        out, rr = ob.add_norm(x, res, w, p, g, 0.7, 1e-3)
        return float((out * do).sum() + (rr * de).sum())

    _, rr = ob.add_norm(x, res, w, p, g, 0.7, 1e-3)
    got = ob.add_norm_bwd(do, rr, w, de, x, p, g, 0.7, 1e-3)
    for name, t in (("dx", x), ("dresidual", res), ("dweight", w), ("dpost", p), ("dgamma", g)):
        if t is None:
            assert name not in got
            continue
        d = central(loss, t)
        assert np.allclose(got[name][0], d, rtol=0, atol=2e-8 * (1 + np.abs(d).max())), name
        assert np.all(got[name][1] >= np.abs(got[name][0]) * (1 - 1e-12))


@pytest.mark.parametrize("gate,norm_first,ngroups", [(False, False, 1), (True, False, 1), (True, True, 1),
                                                     (True, False, 3), (True, True, 2)])
def test_gated_norm_gradients_by_differences(gate, norm_first, ngroups):
    r = RNG(2)
    rows, cols = 3, 12
    y, w, do = r.standard_normal((rows, cols)), r.standard_normal(cols), r.standard_normal((rows, cols))
    z = 2 * r.standard_normal((rows, cols)) if gate else None

    def loss():
        return float((ob.gated_norm(y, z, w, ngroups, norm_first, 1e-3) * do).sum())

    got = ob.gated_norm_bwd(do, y, z, w, ngroups, norm_first, 1e-3)
    for name, t in (("dy", y), ("dz", z), ("dweight", w)):
        if t is None:
            assert name not in got
            continue
        d = central(loss, t)
        assert np.allclose(got[name][0], d, rtol=0, atol=2e-8 * (1 + np.abs(d).max())), name


def test_pack8_definition():
    r = RNG(3)
    x = r.standard_normal((5, 70)) * np.exp(3 * r.standard_normal((5, 70)))
    q, e = ob.pack8(x)
    assert q.shape == (5, 96) and e.shape == (5, 3) and np.all(q[:, 70:] == 0)
    s = 2.0 ** (e.astype(float) - 127)
    top = np.abs(np.pad(x, ((0, 0), (0, 26)))).reshape(5, 3, 32).max(2)
    assert np.all(top / s < ob.TOP) and np.all(top / (s / 2) >= ob.TOP)  # the smallest power of two
    back = ob.unpack8(q, e, 70)
    assert np.all(np.abs(back - x) <= np.repeat(s / 2, 32, axis=1)[:, :70])
    # packing what it stands for changes nothing
    q2, e2 = ob.pack8(back)
    assert np.array_equal(ob.unpack8(q2, e2, 70), back)


def test_pack8_edges():
    row = np.zeros((1, 32))
    q, e = ob.pack8(row)
    assert e[0, 0] == 1 and not q.any()
    for top in (127.5, 127.5 - 2.0 ** -17):  # the next power
        row[0, 3] = top
        q, e = ob.pack8(row)
        assert e[0, 0] == 128 and q[0, 3] == 64
    row[0, 3] = 127.5 - 2.0 ** -16
    q, e = ob.pack8(row)
    assert e[0, 0] == 127 and q[0, 3] == 127
    row[0, 4] = 2.5  # ties to even
    row[0, 5] = -3.5
    q, _ = ob.pack8(row)
    assert q[0, 4] == 2 and q[0, 5] == -4
    big = np.zeros((1, 32))
    big[0, 0] = -3.3895313892515355e38  # the lowest bf16
    q, e = ob.pack8(big)
    assert e[0, 0] == 248 and q[0, 0] == -127 and np.isfinite(ob.unpack8(q, e, 32).astype(np.float32)).all()
    small = np.full((1, 32), 2.0 ** -126)
    q, e = ob.pack8(small)
    assert e[0, 0] == 1 and np.all(q == 1)
    bad = np.ones((1, 64))
    bad[0, 40] = np.inf
    q, e = ob.pack8(bad)
    assert e[0, 1] == 255 and e[0, 0] != 255 and not q[0, 32:].any()
    back = ob.unpack8(q, e, 64)
    assert np.isnan(back[0, 32:]).all() and np.array_equal(back[0, :32], np.ones(32))


def test_wgrad_is_the_product():
    r = RNG(4)
    dy, x = r.standard_normal((9, 5)), r.standard_normal((9, 33))
    q, e = ob.pack8(x)
    assert np.allclose(ob.wgrad8(dy, q, e, 33)[0], np.einsum("to,ti->oi", dy, ob.unpack8(q, e, 33)))
