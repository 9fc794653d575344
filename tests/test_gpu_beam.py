"""GPU parity of beam search's selection and of the states' reordering.

Parents, tokens and finished marks have to be equal.  Scores: a total is formed
in 64 bits from the log of a sum of terms exp(-d).  A term is within 4 units of 2^-24
(bf16 logits: 4 + 2 d, and on the softmax's own average d is below the log of the
vocabulary, 17), and has gone through at most 24 additions in fp32: under 140 units
in all, and its own rounding to fp32."""
import numpy as np
import pytest
import torch

import selective_state_space_27_amd as mss
from gpu_util import host64
from oracle import beam as obeam

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def gen(seed):
    g = torch.Generator(device="cuda:0")
    g.manual_seed(seed)
    return g


def check(logits, scores, n_out, finished=None, eos=None, apart=True):
    got = mss.beam_select(logits, scores, n_out, finished=finished, eos=eos)
    fin = None if finished is None else finished.cpu().numpy() != 0
    l64, s64 = host64(logits), host64(scores)
    best, parents, tokens, done = obeam.select(l64, s64, n_out, fin, eos)
    if apart:  # the reference itself: no two beams' candidates nearer than what rounding decides
        every = np.sort(obeam.totals(l64, s64, fin, eos).reshape(len(best), -1), axis=1)[:, ::-1][:, :n_out + 1]
        with np.errstate(invalid="ignore"):
            gaps = np.diff(every, axis=1)
        near = (gaps > -1e-6) & (gaps < 0)
        assert not near.any(), "inputs too near a tie to be compared"
    assert np.array_equal(got[1].cpu().numpy(), parents), np.argwhere(got[1].cpu().numpy() != parents)[:4]
    assert np.array_equal(got[2].cpu().numpy(), tokens), np.argwhere(got[2].cpu().numpy() != tokens)[:4]
    mine = host64(got[0])
    fine = np.isfinite(best)
    assert np.array_equal(mine[~fine], best[~fine])
    assert (np.abs(mine[fine] - best[fine]) <= np.abs(best[fine]) * U + 140 * U).all()
    if eos is not None:
        assert np.array_equal(got[3].cpu().numpy(), done)
    return got


def make(batch, beams, vocab, io, seed, pad=0):
    g = gen(seed)
    wide = torch.full((batch, beams, vocab + pad), float("nan"), dtype=DT[io], device="cuda:0")
    wide[..., pad // 2:pad // 2 + vocab] = (3 * torch.randn(batch, beams, vocab, generator=g, device="cuda:0")).to(DT[io])
    return wide[..., pad // 2:pad // 2 + vocab], -30 * torch.rand(batch, beams, generator=g, device="cuda:0")


SIZES = [(1, 1, 1, 1), (1, 3, 1, 3), (2, 2, 2, 4), (1, 1, 7, 7), (3, 4, 63, 4), (2, 5, 64, 10), (1, 8, 65, 16),
         (2, 3, 255, 6), (1, 16, 257, 32), (2, 64, 100, 64), (1, 2, 2047, 64), (1, 4, 4099, 8), (2, 6, 8191, 12),
         (1, 4, 8193, 33), (3, 8, 16385, 16), (1, 1, 32768, 64), (1, 12, 50277, 24), (2, 2, 131075, 5),
         (1, 1, 700001, 8), (40, 8, 1000, 8), (1, 7, 24, 64)]


@pytest.mark.parametrize("batch,beams,vocab,n_out", SIZES)
def test_sizes(batch, beams, vocab, n_out):
    for io in ("bf16", "fp32"):
        logits, scores = make(batch, beams, vocab, io, vocab + beams)
        check(logits, scores, n_out)


@pytest.mark.parametrize("pad", [1, 3, 6, 64])
@pytest.mark.parametrize("io", ["bf16", "fp32"])
def test_rows_of_any_stride_and_alignment(io, pad):
    logits, scores = make(3, 4, 5001, io, pad, pad)
    check(logits, scores, 8)


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("vocab", [9, 300, 5000, 40000])
def test_ties_go_to_the_lowest_place(io, vocab):
    g = gen(vocab)
    logits = torch.randint(-2, 3, (2, 4, vocab), generator=g, device="cuda:0").to(DT[io])  # nearly all tied
    logits[:, 3] = logits[:, 1]  # beams that tie with each other
    scores = torch.tensor([[-1.0, -2.0, -3.5, -2.0], [-4.0, -4.5, -4.25, -4.5]], device="cuda:0")
    check(logits, scores, 33 if vocab > 9 else 20)
    check(torch.zeros(2, 4, vocab, dtype=DT[io], device="cuda:0"), torch.zeros(2, 4, device="cuda:0"), 36)
    zeros = torch.zeros(1, 2, vocab, dtype=DT[io], device="cuda:0")
    zeros[0, :, ::2] = -0.0  # equal to +0
    check(zeros, torch.zeros(1, 2, device="cuda:0"), 16)


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("n_out", [1, 7, 64])
def test_many_nearly_equal_logits(io, n_out):
    """More candidates near the best than are ranked: equal ones of either sign, ones that differ in their last bits
    only, and ones a little above many equals."""
    vocab, g = 20011, gen(n_out)
    some = torch.rand(vocab, generator=g, device="cuda:0")
    negative = torch.full((vocab,), -1.1, device="cuda:0")
    above = torch.where(torch.arange(vocab, device="cuda:0") % 2500 == 77, 2.0 + some, 0.7)
    half = torch.where(some < 0.5, 3.3, -3.3)
    few = torch.where(some < 0.002, 5.0, -5.0)
    for row in (negative, above, -above, half, few, 1 + some / 128, -1 - some / 128, some * 1e-30, 100 + some,
                torch.where(some < 0.1, 1 + some / 128, negative)):
        check(row.expand(1, 2, vocab).to(DT[io]).contiguous(), torch.tensor([[-0.5, -40.0]], device="cuda:0"), n_out,
              apart=False)


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("n_out", [1, 8, 64])
def test_sorted_and_clustered_logits(io, n_out):
    """Orders in which the best lie side by side, far apart, or all in one thread's share."""
    vocab = 30011
    up = torch.linspace(-20, 20, vocab, device="cuda:0")
    rows = [up, up.flip(0), up.roll(7777), torch.where(torch.arange(vocab, device="cuda:0") % 512 == 5, up, up - 50),
            torch.where(torch.arange(vocab, device="cuda:0") < 100, up + 60, up), -up.abs()]
    logits = torch.stack(rows)[None].to(DT[io])
    scores = torch.tensor([[-0.5, -1.25, -2.0, -0.75, -1.0, -3.0]], device="cuda:0")
    check(logits, scores, n_out)
    for k in range(len(rows)):
        check(logits[:, k:k + 1], scores[:, :1].contiguous(), n_out)


@pytest.mark.parametrize("io", ["bf16", "fp32"])
def test_banned_tokens_and_the_types_lowest_value(io):
    logits, scores = make(2, 3, 9000, io, 5)
    logits[0, 0, 100:] = -float("inf")        # a long run
    logits[0, 1, ::2] = -float("inf")         # every other one
    logits[0, 2, :] = torch.finfo(DT[io]).min  # the lowest value: equal, not banned
    logits[1, 0, 3:] = -float("inf")          # three left
    logits[1, 1, :8999] = torch.finfo(DT[io]).min
    logits[1, 2, :] = -float("inf")           # none left
    check(logits, scores, 40, apart=False)
    few = torch.full((1, 2, 50), -float("inf"), dtype=DT[io], device="cuda:0")
    few[0, 1, 7] = 3.0
    check(few, torch.tensor([[-1.0, -2.0]], device="cuda:0"), 60)  # one candidate, 59 of none in order


def test_beams_without_candidates():
    logits, _ = make(2, 6, 3000, "fp32", 6)
    logits[0, 1, 17], logits[0, 2, 2999] = float("nan"), float("inf")
    scores = torch.tensor([[-1.0, 0.0, 0.0, float("nan"), float("inf"), -float("inf")], [-float("inf")] * 6],
                          device="cuda:0")
    got = check(logits, scores, 12)
    assert (got[1][0, :12] == 0).all() and (got[0][1] == -float("inf")).all()
    check(logits, scores, 3)


@pytest.mark.parametrize("io", ["bf16", "fp32"])
def test_more_lists_than_the_merge_holds(io):
    """Ordinary rows; ties beyond what is ranked; finished beams and beams without candidates."""
    for beams, vocab, n_out in ((64, 10001, 64), (32, 70001, 48), (3, 1000003, 64)):
        logits, scores = make(2, beams, vocab, io, vocab)
        check(logits, scores, n_out)
        finished = torch.arange(beams, device="cuda:0").expand(2, beams).contiguous() % 3 == 1
        logits[:, 1] = float("nan")  # finished: not looked at
        logits[0, 2, 17], scores[1, 0] = float("inf"), -float("inf")
        scores[:, 1] = -1.0
        check(logits, scores, n_out, finished, vocab - 1)
        check(torch.zeros(2, beams, vocab, dtype=DT[io], device="cuda:0"), torch.zeros(2, beams, device="cuda:0"), n_out,
              finished, 5)
        few = torch.full((1, beams, vocab), -float("inf"), dtype=DT[io], device="cuda:0")
        few[0, -1, vocab // 2], few[0, 0, vocab - 1] = 3.0, -7.0
        check(few, torch.zeros(1, beams, device="cuda:0"), n_out)


@pytest.mark.parametrize("io", ["bf16", "fp32"])
def test_finished_beams(io):
    for eos, n_out in ((0, 8), (2, 16), (699, 40)):
        logits, scores = make(4, 4, 700, io, eos, 3)
        finished = torch.tensor([[1, 0, 0, 1], [1, 1, 1, 1], [0, 0, 0, 0], [0, 1, 0, 0]], dtype=torch.bool,
                                device="cuda:0")
        logits[3, 1, 5] = float("nan")  # not looked at
        check(logits, scores, n_out, finished, eos)
        check(logits, scores, n_out, finished.to(torch.uint8) * 3, eos)
        scores[0, 0], scores[1, 2] = -float("inf"), float("nan")
        check(logits, scores, n_out, finished, eos)


def test_near_totals_far_from_zero():
    """Logits that differ in their last bits while totals are large: the order is that of the logits."""
    base = torch.full((1, 2, 4000), -8.0, device="cuda:0")
    base[0, 0, 1000:1064] = 1e-3 * (1 + torch.arange(64, device="cuda:0") * 2.0 ** -23)
    scores = torch.tensor([[-5000.0, -5100.0]], device="cuda:0")
    got = check(base, scores, 64, apart=False)
    assert got[2][0].tolist() == list(range(1063, 999, -1))


def test_same_call_same_bits_and_captured():
    logits, scores = make(3, 8, 50277, "bf16", 9, 27)
    finished = torch.rand(3, 8, generator=gen(1), device="cuda:0") < 0.3
    call = lambda: mss.beam_select(logits, scores, 16, finished=finished, eos=2)  # noqa: E731
    want = [t.clone() for t in call()]
    other = (logits.clone(), scores.clone(), finished.clone())
    logits2, scores2 = make(3, 8, 50277, "bf16", 10, 27)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    logits.copy_(logits2)
    scores.copy_(scores2)
    want2 = [t.clone() for t in call()]
    for i in (1, 0, 0, 1):
        logits.copy_((other[0], logits2)[i])
        scores.copy_((other[1], scores2)[i])
        graph.replay()
        eager = call()
        torch.cuda.synchronize()
        for a, b, c in zip(got, (want, want2)[i], eager):
            assert torch.equal(a, b) and torch.equal(c, b)


def test_two_streams_at_once():
    a, b = make(4, 8, 50277, "bf16", 11), make(2, 16, 30000, "fp32", 12)
    want = [mss.beam_select(*d, 16) for d in (a, b)]
    torch.cuda.synchronize()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    got = [[mss.beam_select(*d, 16, stream=s) for d, s in zip((a, b), streams)] for _ in range(5)]
    torch.cuda.synchronize()
    for pair in got:
        for g, w in zip(pair, want):
            assert all(torch.equal(x, y) for x, y in zip(g, w))


def test_workspace_status():
    """The workspace's status word is cleared like every call's, and a finished first beam does not keep it from that."""
    logits, scores = make(1, 2, 100, "fp32", 13)
    finished = torch.ones(1, 2, dtype=torch.uint8, device="cuda:0")
    need = mss.lib().mss_beam_select_workspace_size(1, 2, 100, 2)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda:0")
    out, at = torch.empty(1, 2, device="cuda:0"), torch.empty(2, 1, 2, dtype=torch.int64, device="cuda:0")
    torch.cuda.synchronize()
    st = mss.lib().mss_beam_select(logits.data_ptr(), 100, scores.data_ptr(), finished.data_ptr(), 3, out.data_ptr(),
                                   at[0].data_ptr(), at[1].data_ptr(), None, 1, 2, 100, 2, 0, 0, ws.data_ptr(), need, None)
    assert st == 0 and mss.lib().mss_workspace_status(ws.data_ptr(), None) == 0
    assert at[1].tolist() == [[3, 3]] and sorted(at[0][0].tolist()) == [0, 1]


def test_select_refusals():
    logits, scores = make(2, 3, 10, "fp32", 1)
    with pytest.raises(mss.MambaScanError):
        mss.beam_select(logits, scores, 31)
    with pytest.raises(mss.MambaScanError):
        mss.beam_select(logits, scores, 0)
    with pytest.raises(ValueError):
        mss.beam_select(logits, scores, 3, eos=10)
    with pytest.raises(ValueError):
        mss.beam_select(logits, scores, 3, finished=torch.zeros(2, 3, dtype=torch.bool, device="cuda:0"))
    with pytest.raises(ValueError):
        mss.beam_select(logits, scores[:, :2].contiguous(), 3)
    with pytest.raises(TypeError):
        mss.beam_select(logits.half(), scores, 3)
    with pytest.raises(ValueError):
        mss.beam_select(logits[:, :, ::2], scores, 3)
    wide, many = make(1, 65, 10, "fp32", 2)
    with pytest.raises(mss.MambaScanError):
        mss.beam_select(wide, many, 3)


# ------------------------------------------------------------------------------------------------- reordering
def bits(t):
    return t.contiguous().view(torch.uint8)


def random_state(g, batch, beams, shape, dtype):
    n = torch.empty(batch, beams, *shape, dtype=dtype, device="cuda:0")
    raw = torch.randint(0, 256, (n.numel() * n.element_size(),), generator=g, device="cuda:0").to(torch.uint8)
    return raw.view(dtype).view(n.shape)


@pytest.mark.parametrize("batch,beams", [(1, 1), (1, 2), (3, 4), (2, 5), (2, 16), (1, 33), (2, 64), (70, 3)])
def test_reorder(batch, beams):
    g = gen(batch * 100 + beams)
    shapes = [((16, 4), torch.float32), ((3, 7), torch.bfloat16), ((1,), torch.uint8), ((15,), torch.uint8),
              ((16,), torch.uint8), ((17,), torch.uint8), ((1023,), torch.uint8), ((1025,), torch.int8),
              ((5, 3, 2), torch.float32), ((1000, 16), torch.float32), ((2049,), torch.int64)]
    states = [random_state(g, batch, beams, s, t) for s, t in shapes]
    for parents in (torch.randint(0, beams, (batch, beams), generator=g, device="cuda:0"),
                    torch.arange(beams, device="cuda:0").flip(0).expand(batch, beams).contiguous(),  # swaps
                    torch.arange(beams, device="cuda:0").roll(1).expand(batch, beams).contiguous(),  # one long cycle
                    torch.zeros(batch, beams, dtype=torch.int64, device="cuda:0"),
                    torch.arange(beams, device="cuda:0").expand(batch, beams).contiguous()):
        at = torch.arange(batch, device="cuda:0")[:, None]
        want = [bits(t[at, parents]) for t in states]
        got = mss.reorder_states(states, parents)
        assert got is states
        assert all(torch.equal(bits(t), w) for t, w in zip(states, want))


def test_reorder_many_states_unaligned_and_their_surroundings():
    g = gen(3)
    batch, beams = 2, 4
    states, whole = [], []
    for i in range(75):  # more than one launch holds
        row = 1 + i * 13
        buf = torch.randint(0, 256, (batch * beams * row + 64,), generator=g, device="cuda:0").to(torch.uint8)
        whole.append(buf)
        states.append(buf[i % 17:i % 17 + batch * beams * row].view(batch, beams, row))
    parents = torch.tensor([[1, 1, 3, 2], [0, 3, 0, 1]], device="cuda:0")
    before = [w.clone() for w in whole]
    at = torch.arange(batch, device="cuda:0")[:, None]
    want = [t[at, parents].clone() for t in states]
    mss.reorder_states(states, parents)
    for i, (t, w, old, new) in enumerate(zip(states, want, before, whole)):
        assert torch.equal(t, w), i
        lo, hi = i % 17, i % 17 + t.numel()
        assert torch.equal(new[:lo], old[:lo]) and torch.equal(new[hi:], old[hi:]), i


def test_reorder_leaves_rows_with_bad_parents():
    t = random_state(gen(4), 2, 4, (100,), torch.float32)
    keep = t.clone()
    parents = torch.tensor([[-1, 4, 1 << 40, 0], [3, -(1 << 40), 2, 64]], device="cuda:0")
    mss.reorder_states([t], parents)
    fixed = torch.tensor([[0, 1, 2, 0], [3, 1, 2, 3]], device="cuda:0")
    assert torch.equal(bits(t), bits(keep[torch.arange(2, device="cuda:0")[:, None], fixed]))


def test_reorder_captured_and_replayed():
    g = gen(5)
    states = [random_state(g, 3, 4, (50, 16), torch.float32), random_state(g, 3, 4, (50, 3), torch.bfloat16)]
    parents = torch.randint(0, 4, (3, 4), generator=g, device="cuda:0")
    mss.reorder_states(states, parents)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mss.reorder_states(states, parents)
    for _ in range(4):
        parents.copy_(torch.randint(0, 4, (3, 4), generator=g, device="cuda:0"))
        at = torch.arange(3, device="cuda:0")[:, None]
        want = [bits(t[at, parents]) for t in states]
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(bits(t), w) for t, w in zip(states, want))


def test_reorder_refusals():
    parents = torch.zeros(2, 3, dtype=torch.int64, device="cuda:0")
    t = torch.zeros(2, 3, 5, device="cuda:0")
    assert mss.reorder_states([], parents) == []
    with pytest.raises(TypeError):
        mss.reorder_states([t], parents.int())
    with pytest.raises(ValueError):
        mss.reorder_states([t[:, :2]], parents)
    with pytest.raises(ValueError):
        mss.reorder_states([t.transpose(0, 1).contiguous().transpose(0, 1)], parents)
    with pytest.raises(ValueError):
        mss.reorder_states([t.cpu()], parents)
    with pytest.raises(mss.MambaScanError):
        mss.reorder_states([t, t], parents)
    with pytest.raises(mss.MambaScanError):
        mss.reorder_states([torch.zeros(1, 65, 2, device="cuda:0")], torch.zeros(1, 65, dtype=torch.int64, device="cuda:0"))
