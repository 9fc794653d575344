"""GPU parity of the 8-bit checkpoint form: exact, bit for bit, against the
fp64 reference; and the weight gradient from one.

Weight gradient's tolerance, per element: the products are exact in fp32, the
sum of T terms is held in fp32, 16 terms to a matrix instruction whose sum may
be cut rather than rounded, then the parts': (T / 16 + 64) * 2^-23 * sum |dY||X|,
plus half a bf16 step for a bf16 result.  Small whole numbers, whose sums stay
below 2^24, have to come out exactly.
"""
import numpy as np
import pytest
import torch

import selective_state_space_27_amd as mss
from block_util import half_step
from gpu_util import host64
from oracle import block as ob

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def gen(seed):
    g = torch.Generator(device="cuda:0")
    g.manual_seed(seed)
    return g


def act(g, rows, cols, dtype, spread=2.0):
    v = torch.randn(rows, cols, generator=g, device="cuda:0")
    return (v * torch.exp(spread * torch.randn(rows, cols, generator=g, device="cuda:0"))).to(dtype)


def same_form(p, x64):
    q, e = ob.pack8(x64)
    assert np.array_equal(p.q.cpu().numpy(), q)
    assert np.array_equal(p.scale.cpu().numpy(), e)


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 31), (1, 32), (3, 33), (7, 100), (1000, 1), (77, 1001), (5, 8192),
                                       (2, 70001), (33, 2560)])
def test_pack_and_unpack(io, rows, cols):
    x = act(gen(rows + cols), rows, cols, DT[io])
    p = mss.pack8(x)
    assert p.shape == x.shape and p.dtype == x.dtype
    same_form(p, host64(x))
    ref = ob.unpack8(p.q.cpu().numpy(), p.scale.cpu().numpy(), cols)
    for dt in DT.values():
        back = mss.unpack8(p, dt)
        assert back.dtype == dt and np.array_equal(host64(back), ref)


@pytest.mark.parametrize("io", ["bf16", "fp32"])
def test_slices_and_leading_dimensions(io):
    g = gen(1)
    wide = act(g, 6 * 5, 300, DT[io]).view(6, 5, 300)
    x = wide[:, :, 17:17 + 101]
    p = mss.pack8(x)
    assert p.shape == (6, 5, 101)
    same_form(p, host64(x.contiguous()).reshape(30, 101))
    keep = wide.clone()
    mss.unpack8(p, out=x)
    assert torch.equal(x.contiguous(), mss.unpack8(p))
    assert torch.equal(wide[:, :, :17], keep[:, :, :17]) and torch.equal(wide[:, :, 118:], keep[:, :, 118:])


@pytest.mark.parametrize("io", ["bf16", "fp32"])
def test_edges(io):
    dt = DT[io]
    tiny = torch.finfo(torch.float32).tiny
    rows = [torch.zeros(64), torch.full((64,), torch.finfo(dt).min), torch.full((64,), torch.finfo(dt).max),
            torch.full((64,), tiny), torch.full((64,), -tiny / 8), torch.full((64,), 127.5), torch.full((64,), 127.0),
            torch.arange(64) - 31.5, torch.cat([torch.full((32,), 1e-30), torch.full((32,), 1e30)]),
            torch.tensor([-0.0] * 64), torch.full((64,), 1.9921875 * 2.0 ** 20)]
    # around the threshold of a scale, at small, middle and large exponents
    rows += [torch.full((64,), (127.5 - k * 2.0 ** -17) * 2.0 ** p) for k in (-1, 0, 1, 2, 3) for p in (-100, 0, 100)]
    x = torch.stack([r.float() for r in rows]).to(dt).to("cuda:0")
    p = mss.pack8(x)
    same_form(p, host64(x))
    assert torch.isfinite(mss.unpack8(p)).all()


def test_non_finite_blocks_read_back_as_nan_and_stay_alone():
    x = act(gen(2), 4, 96, torch.float32)
    good = mss.unpack8(mss.pack8(x))
    for bad in (float("inf"), float("-inf"), float("nan")):
        y = x.clone()
        y[1, 40] = bad
        p = mss.pack8(y)
        same_form(p, host64(y))
        back = mss.unpack8(p)
        assert torch.isnan(back[1, 32:64]).all()
        back[1, 32:64] = good[1, 32:64]
        assert torch.equal(back, good)


def test_other_stream():
    x = act(gen(3), 3000, 512, torch.bfloat16)
    ref = mss.pack8(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    p = mss.pack8(x, stream=s)
    back = mss.unpack8(p, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(p.q, ref.q) and torch.equal(back, mss.unpack8(ref))


# ------------------------------------------------------- weight gradient
def wgrad_ref(dy, p, tokens, outs, ins):
    q, e = p.q.cpu().numpy(), p.scale.cpu().numpy()
    return ob.wgrad8(host64(dy), q, e, ins)


# One tile, its borders, several tiles, cut sums (few tiles, many tokens), both
# tile sizes; stages that end inside the tokens.
SHAPES = [(1, 1, 1), (1, 64, 64), (63, 40, 33), (64, 128, 128), (65, 129, 127), (200, 256, 320), (1000, 257, 100),
          (5000, 96, 160), (130, 1000, 31), (513, 768, 1536), (2048, 80, 2560), (31, 8, 1), (33, 16, 40), (191, 8, 8),
          (193, 72, 96), (385, 136, 64), (2051, 200, 136)]


@pytest.mark.parametrize("tokens,outs,ins", SHAPES)
def test_wgrad_whole_numbers(tokens, outs, ins):
    g = gen(tokens)
    dy = torch.randint(-3, 4, (tokens, outs), generator=g, device="cuda:0").bfloat16()
    x = torch.randint(-100, 101, (tokens, ins), generator=g, device="cuda:0").bfloat16()
    p = mss.pack8(x)
    assert torch.equal(mss.unpack8(p), x)
    got = mss.wgrad8(dy, p)
    assert np.array_equal(host64(got), host64(dy).T @ host64(x))


@pytest.mark.parametrize("dw", ["fp32", "bf16"])
@pytest.mark.parametrize("tokens,outs,ins", SHAPES)
def test_wgrad(tokens, outs, ins, dw):
    g = gen(tokens + 1)
    dy, p = act(g, tokens, outs, torch.bfloat16, 1.0), mss.pack8(act(g, tokens, ins, torch.bfloat16, 1.0))
    got = mss.wgrad8(dy, p, out_dtype=DT[dw])
    ref, size = wgrad_ref(dy, p, tokens, outs, ins)
    tol = (tokens / 16 + 64) * 2.0 ** -23 * size
    tol = tol + (half_step(np.abs(ref) + tol) if dw == "bf16" else 0.0)
    assert got.dtype == DT[dw] and np.all(np.abs(host64(got) - ref) <= tol)
    assert torch.equal(got, mss.wgrad8(dy, p, out_dtype=DT[dw]))  # repeatable


@pytest.mark.parametrize("tokens,outs,ins", [(300, 4112, 2050), (129, 3000, 4000), (1000, 5000, 2601),
                                             (70, 4001, 2050), (31, 2816, 3000), (1500, 4000, 3900),
                                             (1470, 4007, 3833), (32768, 1296, 1020), (32007, 1290, 1020)])
def test_wgrad_large_tiles(tokens, outs, ins):
    """Sizes for 256-wide tiles, whole and cut along the tokens, borders inside them."""
    g = gen(tokens)
    dy = torch.randint(-3, 4, (tokens, outs), generator=g, device="cuda:0").bfloat16()
    x = torch.randint(-100, 101, (tokens, ins), generator=g, device="cuda:0").bfloat16()
    got = mss.wgrad8(dy, mss.pack8(x))
    want = dy.double().t().contiguous() @ x.double()
    assert torch.equal(got.double(), want)


@pytest.mark.parametrize("tokens,outs,ins", [(300, 128, 160), (4000, 96, 64), (100, 4096, 2600)])
@pytest.mark.parametrize("dw", ["fp32", "bf16"])
def test_wgrad_accumulates(tokens, outs, ins, dw):
    g = gen(6)
    dy = torch.randint(-1, 2, (tokens, outs), generator=g, device="cuda:0").bfloat16()
    x = torch.randint(-1, 2, (tokens, ins), generator=g, device="cuda:0").bfloat16()
    p = mss.pack8(x)
    out = torch.randint(-50, 51, (outs, ins), generator=g, device="cuda:0").to(DT[dw])
    want = (host64(dy).T @ host64(x) + host64(out))
    assert mss.wgrad8(dy, p, out=out, accumulate=True) is out
    want_t = torch.from_numpy(want).to(DT[dw])  # rounded once, after the sum
    assert torch.equal(out.cpu(), want_t)
    with pytest.raises(ValueError):
        mss.wgrad8(dy, p, accumulate=True)


@pytest.mark.parametrize("off,extra", [(0, 8), (3, 5), (16, 48)])
@pytest.mark.parametrize("tokens,outs,ins", [(70, 100, 40), (130, 136, 300)])
def test_wgrad_of_a_slice_does_not_read_around_it(off, extra, tokens, outs, ins):
    """dY as columns of a wider buffer that holds NaN everywhere else, above
    and below too."""
    g = gen(7)
    wide = torch.full((tokens + 80, off + outs + extra), float("nan"), dtype=torch.bfloat16, device="cuda:0")
    dy = wide[8:8 + tokens, off:off + outs]
    dy.copy_(torch.randint(-3, 4, (tokens, outs), generator=g, device="cuda:0"))
    x = torch.randint(-100, 101, (tokens, ins), generator=g, device="cuda:0").bfloat16()
    got = mss.wgrad8(dy, mss.pack8(x))
    assert np.array_equal(host64(got), host64(dy.contiguous()).T @ host64(x))


@pytest.mark.parametrize("off", [0, 3])
def test_wgrad_past_32_bit_offsets(off):
    """Rows of dY 2^20 elements apart (aligned and not): the last ones lie past 2^32 elements."""
    tokens, outs, ins, pitch = 4100, 72, 64, 1 << 20
    g = gen(9)
    dy = torch.empty(tokens * pitch, dtype=torch.bfloat16, device="cuda:0").view(tokens, pitch)[:, off:off + outs]
    dy.copy_(torch.randint(-3, 4, (tokens, outs), generator=g, device="cuda:0"))
    p = mss.pack8(torch.randint(-100, 101, (tokens, ins), generator=g, device="cuda:0").bfloat16())
    assert torch.equal(mss.wgrad8(dy, p), mss.wgrad8(dy.contiguous(), p))


def test_wgrad_non_finite():
    """A block that reads back as NaN makes its 32 columns of dW NaN; an
    infinity in dY its row; nothing else."""
    g = gen(8)
    dy = act(g, 100, 64, torch.bfloat16, 0.5)
    x = act(g, 100, 96, torch.float32, 0.5)
    good = mss.wgrad8(dy, mss.pack8(x))
    bad = x.clone()
    bad[50, 33] = float("inf")
    got = mss.wgrad8(dy, mss.pack8(bad))
    assert torch.isnan(got[:, 32:64]).all()
    assert torch.equal(got[:, :32], good[:, :32]) and torch.equal(got[:, 64:], good[:, 64:])
    dy2 = dy.clone()
    dy2[7, 5] = float("inf")
    got = mss.wgrad8(dy2, mss.pack8(x))
    keep = [i for i in range(64) if i != 5]
    assert not torch.isfinite(got[5]).any() and torch.equal(got[keep], good[keep])


def test_wgrad_refusals():
    x = torch.ones(4, 32, device="cuda:0", dtype=torch.bfloat16)
    p = mss.pack8(x)
    with pytest.raises(mss.MambaScanError) as e:
        mss.wgrad8(x.float(), p)
    assert e.value.status == 5
    with pytest.raises(ValueError):
        mss.wgrad8(x[:3], p)
    with pytest.raises(ValueError):
        mss.wgrad8(x, p, out=torch.empty(32, 31, device="cuda:0"))
    with pytest.raises(TypeError):
        mss.wgrad8(x, x)
