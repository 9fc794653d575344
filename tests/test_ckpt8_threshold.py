"""The 8-bit form's threshold, on the CPU and with its numbers written out: the
next power of two is taken from 127.5 - 2^-17 steps on (for bf16 values: from
127.5).  That is where max|x| times fp32's 1/127.5 reaches 1; a correctly rounded
division reaches it one fp32 unit later."""
import numpy as np

from oracle import block as ob

BOUND = 127.49999237060546875  # 127.5 - 2^-17


def exponents(tops):
    row = np.zeros((len(tops), 32))
    row[:, 7] = tops
    return ob.pack8(row)[1][:, 0].astype(int)


def by_reciprocal(tops):
    """The exponent byte as an fp32 evaluation with a reciprocal finds it."""
    ratio = np.asarray(tops, dtype=np.float32) * (np.float32(1) / np.float32(127.5))
    return np.clip(np.frexp(ratio)[1] + 127, 1, 248)


def test_the_bound():
    below, at = np.nextafter(np.float32(BOUND), np.float32(0)), np.float32(BOUND)
    assert float(at) == BOUND and np.nextafter(at, np.float32(200)) == np.float32(127.5)
    for p in (-100, -7, 0, 1, 100):
        s = 2.0 ** p
        assert list(exponents([below * s, at * s, 127.5 * s])) == [127 + p, 128 + p, 128 + p]
    q, _ = ob.pack8(np.full((1, 32), float(below)))
    assert (q == 127).all()


def test_an_evaluation_by_the_reciprocal_finds_the_same_scales():
    r = np.random.default_rng(0)
    near = [np.float32(127.5 - k * 2.0 ** -17) * np.float32(2.0 ** p) for k in range(-3, 5) for p in (-90, -1, 0, 5, 90)]
    tops = np.concatenate([np.exp(r.uniform(-60, 60, 20000)).astype(np.float32), np.array(near, dtype=np.float32)])
    assert np.array_equal(exponents(tops.astype(np.float64)), by_reciprocal(tops))


def test_a_division_differs_at_the_bound_alone():
    assert np.float32(BOUND) / np.float32(127.5) < 1.0 <= np.float32(BOUND) * (np.float32(1) / np.float32(127.5))
    below = np.nextafter(np.float32(BOUND), np.float32(0))
    assert below / np.float32(127.5) < 1.0 and below * (np.float32(1) / np.float32(127.5)) < 1.0


def test_bf16_values_do_not_see_the_difference():
    # eight significant bits: 127 and 127.5 are neighbours
    assert list(exponents([127.0, 127.5])) == [127, 128]


def test_the_error_and_where_it_saturates():
    r = np.random.default_rng(1)
    top = float(np.finfo(np.float32).max)
    x = np.concatenate([r.standard_normal((50, 32)) * np.exp(r.uniform(-60, 60, (50, 1))),
                        r.uniform(-1.0, 1.0, (50, 32)) * 127.5 * 2.0 ** 121, r.uniform(-1.0, 1.0, (50, 32)) * top,
                        np.full((1, 32), top)])
    x = x.astype(np.float32).astype(np.float64)
    q, e = ob.pack8(x)
    s = 2.0 ** (e.astype(float) - 127.0)
    off, tail = np.abs(ob.unpack8(q, e, 32) - x), np.abs(x) > 127.5 * 2.0 ** 121
    assert (off[~tail] <= np.broadcast_to(s / 2, x.shape)[~tail]).all()
    assert tail.any() and (off <= s).all() and (off > s / 2)[tail].all()
