"""Largest sizes of the gated recurrence and of beam search: offsets past 32 bits,
more rows than a grid's second axis holds.  A large call is compared bit for bit
with a small one on a part of its data (a channel's arithmetic does not depend on
where the channel lies), or with what was planted.  Long sequences of few streams
hand their states on by groups, with other roundings: the part's rows are repeated to
as many as are not few."""
import pytest
import torch

import selective_state_space_27_amd as mss

pytestmark = pytest.mark.gpu


def gen(seed):
    g = torch.Generator(device="cuda:0")
    g.manual_seed(seed)
    return g


def fill(t, g, scale=1.0):
    """Normal values written in place, a part at a time."""
    flat = t.view(-1)
    for i in range(0, flat.numel(), 1 << 28):
        part = flat[i:i + (1 << 28)]
        part.copy_((scale * torch.randn(part.numel(), generator=g, device=t.device)).to(t.dtype))
    return t


@pytest.mark.timeout(300)
@pytest.mark.parametrize("batch,length,dim", [(1, 1 << 20, 2200), (300, 8192, 960)])
def test_recurrence_past_32_bit_offsets(batch, length, dim):
    """Over 4 GB a tensor: the last channels, and the last rows of the batch, against a call of their own."""
    g = gen(1)
    x, a, i, dy = (fill(torch.empty(batch, length, dim, dtype=torch.bfloat16, device="cuda:0"), g) for _ in range(4))
    lam = torch.randn(dim, generator=g, device="cuda:0") - 4
    y, last, states = mss.gated_recurrence_fwd(x, a, i, lam, return_last_state=True, keep_states=True, check_waits=True)
    grads = mss.gated_recurrence_bwd(dy, x, a, i, lam, states, want_dh0=True, check_waits=True)
    rows, cols = slice(max(0, batch - 2), batch), slice(dim - 64, dim)
    n = min(2, batch)
    part = [t[rows, :, cols].repeat(17, 1, 1) for t in (x, a, i, dy)]
    z, zlast, zstates = mss.gated_recurrence_fwd(*part[:3], lam[cols].contiguous(), return_last_state=True,
                                                 keep_states=True)
    assert torch.equal(z[:n], y[rows, :, cols]) and torch.equal(zlast[-n:], last[rows, cols])
    assert torch.equal(zstates[:n], states[rows, :, cols])
    small = mss.gated_recurrence_bwd(part[3], *part[:3], lam[cols].contiguous(), zstates, want_dh0=True)
    for k in ("dx", "dgate_a", "dgate_x"):
        assert torch.equal(small[k][:n], grads[k][rows, :, cols]), k
    assert torch.equal(small["dh0"][-n:], grads["dh0"][rows, cols])


@pytest.mark.parametrize("io,batch,length,dim", [("fp32", 40, 3001, 161), ("bf16", 40, 6001, 161), ("fp32", 25, 130, 6011),
                                                 ("fp32", 60, 700, 33), ("bf16", 9, 200, 901), ("fp32", 70, 20, 515)])
def test_many_streams_of_rows_that_are_no_whole_lines(io, batch, length, dim):
    """Below and beyond the last-level cache, several pieces or one: the last batch rows against a call of their own."""
    g = gen(5)
    dtype = torch.float32 if io == "fp32" else torch.bfloat16
    x, a, i, dy = (torch.randn(batch, length, dim, generator=g, device="cuda:0").to(dtype) for _ in range(4))
    starts = torch.rand(batch, length, generator=g, device="cuda:0") < 0.002
    lam = torch.randn(dim, generator=g, device="cuda:0") - 3
    y, last, states = mss.gated_recurrence_fwd(x, a, i, lam, starts=starts, return_last_state=True, keep_states=True,
                                               check_waits=True)
    grads = mss.gated_recurrence_bwd(dy, x, a, i, lam, states, starts=starts, want_dh0=True, check_waits=True)
    for rows in (slice(0, 1), slice(batch // 2, batch // 2 + 2), slice(batch - 1, batch)):
        n, many = rows.stop - rows.start, lambda t: t[rows].repeat(17, *[1] * (t.dim() - 1))  # noqa: E731
        sx, sa, si, sdy, sstarts = (many(t) for t in (x, a, i, dy, starts))
        z, zlast, zstates = mss.gated_recurrence_fwd(sx, sa, si, lam, starts=sstarts, return_last_state=True,
                                                     keep_states=True)
        assert torch.equal(z[:n], y[rows]) and torch.equal(zlast[-n:], last[rows])
        assert torch.equal(zstates[:n], states[rows])
        small = mss.gated_recurrence_bwd(sdy, sx, sa, si, lam, zstates, starts=sstarts, want_dh0=True)
        for k in ("dx", "dgate_a", "dgate_x", "dh0"):
            assert torch.equal(small[k][-n:], grads[k][rows]), (k, rows)


@pytest.mark.parametrize("batch,length,dim", [(70001, 1, 1), (70001, 3, 2), (66000, 70, 3)])
def test_recurrence_of_many_rows(batch, length, dim):
    g = gen(2)
    x, a, i, dy = (torch.randn(batch, length, dim, generator=g, device="cuda:0") for _ in range(4))
    lam = torch.randn(dim, generator=g, device="cuda:0")
    y, states = mss.gated_recurrence_fwd(x, a, i, lam, keep_states=True)
    grads = mss.gated_recurrence_bwd(dy, x, a, i, lam, states)
    rows = slice(batch - 5, batch)
    z, zstates = mss.gated_recurrence_fwd(x[rows], a[rows], i[rows], lam, keep_states=True)
    small = mss.gated_recurrence_bwd(dy[rows], x[rows], a[rows], i[rows], lam, zstates)
    assert torch.equal(z, y[rows]) and all(torch.equal(small[k], grads[k][rows]) for k in ("dx", "dgate_a", "dgate_x"))


def test_step_past_32_bit_offsets():
    batch, beams, dim = 1 << 16, 8, 2081
    g = gen(3)
    rows = batch * beams
    h = fill(torch.empty(rows, dim, device="cuda:0"), g)
    x, a, i = (fill(torch.empty(rows, dim, dtype=torch.bfloat16, device="cuda:0"), g) for _ in range(3))
    lam = torch.randn(dim, generator=g, device="cuda:0")
    parents = torch.randint(0, beams, (batch, beams), generator=g, device="cuda:0")
    y, new = mss.gated_recurrence_step(h, x, a, i, lam, parents=parents)
    end = slice(rows - 24, rows)
    z, small = mss.gated_recurrence_step(h[end], x[end], a[end], i[end], lam, parents=parents[-3:])
    assert torch.equal(z, y[end]) and torch.equal(small, new[end])


def test_step_of_many_rows():
    g = gen(4)
    h, x, a, i = (torch.randn(1 << 22, 3, generator=g, device="cuda:0") for _ in range(4))
    lam = torch.randn(3, generator=g, device="cuda:0")
    y, new = mss.gated_recurrence_step(h.clone(), x, a, i, lam)
    z, small = mss.gated_recurrence_step(h[-7:].clone(), x[-7:], a[-7:], i[-7:], lam)
    assert torch.equal(z, y[-7:]) and torch.equal(small, new[-7:])


@pytest.mark.timeout(300)
def test_select_from_the_largest_vocabulary():
    """128 rows of 2^24 logits, over 4 GB: the best planted at known places."""
    batch, beams, vocab, n = 2, 64, 1 << 24, 48
    logits = torch.full((batch, beams, vocab), -30.0, dtype=torch.bfloat16, device="cuda:0")
    g = gen(5)
    scores = torch.full((batch, beams), -float("inf"), device="cuda:0")  # beams without any are not in use
    value = 1 + 0.25 * torch.arange(n, 0, -1, device="cuda:0").double()  # far above -30 from any other
    want = []
    for b in range(batch):
        places = torch.randint(0, beams * vocab, (n,), generator=g, device="cuda:0")
        places[:4] = torch.tensor([0, vocab - 1, (beams - 1) * vocab, beams * vocab - 1], device="cuda:0")
        assert places.unique().numel() == n
        logits[b].view(-1)[places] = value.bfloat16()
        scores[b, places // vocab] = 0.0
        want.append(places)
    best, parents, tokens = mss.beam_select(logits, scores, n)
    # Totals by the definition, in fp64: a row holds -30 everywhere but where planted.
    for b in range(batch):
        k = want[b] // vocab
        total = torch.empty(n, dtype=torch.float64, device="cuda:0")
        for r in k.unique():
            planted = value[k == r]
            top = planted.max()
            rest = (vocab - planted.numel()) * torch.exp(-30.0 - top)
            total[k == r] = planted - top - torch.log(torch.exp(planted - top).sum() + rest)
        by_place = torch.argsort(want[b])
        order = by_place[torch.argsort(-total[by_place], stable=True)]
        got = parents[b] * vocab + tokens[b]
        assert set(got.tolist()) == set(want[b].tolist())
        assert torch.allclose(best[b].double(), total[order], atol=1e-4)
        # The best of a beam with several planted is near 0, as all beams' are: compared where totals are apart.
        gap = (total[order][1:] - total[order][:-1]).abs() > 1e-6
        apart = torch.cat([gap[:1], gap[1:] & gap[:-1], gap[-1:]])
        assert apart.any() and torch.equal(got[apart], want[b][order][apart])


def test_select_of_many_sequences():
    g = gen(6)
    batch, beams, vocab, n = 65535, 3, 5, 4
    logits = torch.randn(batch, beams, vocab, generator=g, device="cuda:0")
    scores = torch.randn(batch, beams, generator=g, device="cuda:0")
    best, parents, tokens = mss.beam_select(logits, scores, n)
    total = (scores.double()[:, :, None] + torch.log_softmax(logits.double(), 2)).flatten(1)
    value, at = torch.sort(total, dim=1, descending=True, stable=True)
    apart = ((value[:, :n] - value[:, 1:n + 1]) > 1e-5).all(1)
    assert apart.float().mean() > 0.9
    assert torch.equal((parents * vocab + tokens)[apart], at[apart, :n])
    assert torch.allclose(best.double(), value[:, :n], atol=1e-4)
    wide = torch.randn(1200, 64, 3, generator=g, device="cuda:0")  # 76800 rows
    s = torch.randn(1200, 64, generator=g, device="cuda:0")
    best, parents, tokens = mss.beam_select(wide, s, 64)
    total = (s.double()[:, :, None] + torch.log_softmax(wide.double(), 2)).flatten(1)
    value, at = torch.sort(total, dim=1, descending=True, stable=True)
    apart = ((value[:, :64] - value[:, 1:65]) > 1e-5).all(1)
    assert apart.any() and torch.equal((parents * 3 + tokens)[apart], at[apart, :64])


@pytest.mark.timeout(300)
def test_reorder_past_32_bit_offsets():
    row, beams = 1 << 30, 5
    t = torch.zeros(1, beams, row, dtype=torch.uint8, device="cuda:0")
    for k in range(beams):
        t[0, k] = k + 1
        t[0, k, -1] = 100 + k
        t[0, k, 0] = 200 + k
    parents = torch.tensor([[4, 1, 0, 0, 3]], device="cuda:0")
    mss.reorder_states([t], parents)
    for k, from_ in enumerate(parents[0].tolist()):
        assert t[0, k, 0] == 200 + from_ and t[0, k, -1] == 100 + from_
        assert (t[0, k, 1:-1] == from_ + 1).all()


def test_reorder_of_many_sequences():
    g = gen(7)
    t = torch.randint(0, 1 << 30, (65535, 3, 7), generator=g, device="cuda:0")
    parents = torch.randint(0, 3, (65535, 3), generator=g, device="cuda:0")
    want = t[torch.arange(65535, device="cuda:0")[:, None], parents]
    mss.reorder_states([t], parents)
    assert torch.equal(t, want)
