"""How the operators around the mixer are called: on a stream of their own, and
on column slices of one buffer, inputs and outputs side by side."""
import pytest
import torch

import selective_state_space_27_amd as mss

pytestmark = pytest.mark.gpu


def gen(seed):
    g = torch.Generator(device="cuda:0")
    g.manual_seed(seed)
    return g


def randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda:0").to(dtype)


ROWS, COLS = 512, 1280


def operators(g):
    """{name: call of (x, stream) that returns its tensors}; x bf16 [ROWS, COLS] is the input that changes."""
    wide, w = randn(g, ROWS, COLS), 1.0 + 0.2 * randn(g, COLS)
    do = randn(g, ROWS, COLS, dtype=torch.bfloat16)

    def flat(v):
        if isinstance(v, mss.Packed8):
            return [v.q, v.scale]
        if isinstance(v, dict):
            v = list(v.values())
        return [t for u in v for t in flat(u)] if isinstance(v, (list, tuple)) else [] if v is None else [v]

    calls = {
        "add_norm_fwd": lambda x, s: mss.add_norm_fwd(x, wide, w, pack_out=True, stream=s),
        "add_norm_bwd": lambda x, s: mss.add_norm_bwd(x, wide, w, x=do, gamma=w, stream=s),
        "gated_norm_fwd": lambda x, s: mss.gated_norm_fwd(wide, x, w, pack_inputs=True, stream=s),
        "gated_norm_bwd": lambda x, s: mss.gated_norm_bwd(do, wide, x, w, stream=s),
        "pack8": lambda x, s: mss.pack8(x, stream=s),
        "unpack8": lambda x, s: mss.unpack8(mss.pack8(x, stream=s), stream=s),
        "wgrad8": lambda x, s: mss.wgrad8(x, packed, stream=s),
        "wgrad8 of unaligned rows": lambda x, s: mss.wgrad8(x[:, 3:], packed, stream=s),
    }
    packed = mss.pack8(wide)
    return {k: (lambda x, s, f=f: flat(f(x, s))) for k, f in calls.items()}


@pytest.mark.parametrize("name", ["add_norm_fwd", "add_norm_bwd", "gated_norm_fwd", "gated_norm_bwd", "pack8", "unpack8",
                                  "wgrad8", "wgrad8 of unaligned rows"])
def test_a_call_runs_on_the_stream_it_is_given(name):
    """The input is written on a side stream, behind work of some 100 ms, and the
    call follows on that stream alone: on any other it would read the old values."""
    g = gen(1)
    f = operators(g)[name]
    new = randn(g, ROWS, COLS, dtype=torch.bfloat16)
    want = f(new, None)
    x = torch.zeros_like(new)
    a = randn(g, 8192, 8192)
    f(x, None)  # everything that is set up once
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for _ in range(12):
            a = a @ a
        x.copy_(new)
    got = f(x, side)
    assert not side.query()  # the work in front was still running when the call was made
    side.synchronize()
    assert len(got) == len(want) and all(torch.equal(p, q) for p, q in zip(got, want))


def side_by_side(rows, cols, dtype, n, pad):
    """n column slices of one buffer of sevens, `pad` columns around each."""
    wide = torch.full((rows, n * (cols + pad) + pad), 7.0, dtype=dtype, device="cuda:0")
    return wide, [wide[:, pad + i * (cols + pad):][:, :cols] for i in range(n)]


def untouched(wide, slices):
    """Whether only the slices were written (they are reset)."""
    for s in slices:
        s.fill_(7.0)
    return bool((wide == 7.0).all())


@pytest.mark.parametrize("rows,cols,pad", [(5, 100, 0), (5, 100, 3), (300, 256, 0), (33, 1001, 1), (9, 2560, 0),
                                           (3, 9001, 0)])
def test_slices_of_one_buffer_side_by_side(rows, cols, pad):
    g = gen(cols)
    w = 1.0 + 0.2 * randn(g, cols)
    a, b, c = (randn(g, rows, cols, dtype=torch.bfloat16) for _ in range(3))
    d, e = (randn(g, rows, cols) for _ in range(2))

    # x beside out, the residual beside the stored one
    io, (x, out) = side_by_side(rows, cols, torch.bfloat16, 2, pad)
    res, (r, rout) = side_by_side(rows, cols, torch.float32, 2, pad)
    x.copy_(a), r.copy_(d)
    want = mss.add_norm_fwd(a, d, w)
    mss.add_norm_fwd(x, r, w, out=out, residual_out=rout)
    assert torch.equal(out, want[0]) and torch.equal(rout, want[1]) and torch.equal(x, a) and torch.equal(r, d)
    assert untouched(io, (x, out)) and untouched(res, (r, rout))

    # its backward: dout beside dx, the two residuals' gradients and the residual in one buffer
    io, (do, dx) = side_by_side(rows, cols, torch.bfloat16, 2, pad)
    res, (r, dr, dres) = side_by_side(rows, cols, torch.float32, 3, pad)
    do.copy_(a), r.copy_(d), dr.copy_(e)
    want = mss.add_norm_bwd(a, d, w, dresidual_out=e)
    got = mss.add_norm_bwd(do, r, w, dresidual_out=dr, dx=dx, dresidual=dres)
    assert all(torch.equal(got[k], want[k]) for k in ("dx", "dresidual", "dweight"))
    assert torch.equal(do, a) and torch.equal(r, d) and torch.equal(dr, e)
    assert untouched(io, (do, dx)) and untouched(res, (r, dr, dres))

    # gate, out and their gradients
    io, (z, out, do, dz) = side_by_side(rows, cols, torch.bfloat16, 4, pad)
    wide, (y, dy) = side_by_side(rows, cols, torch.float32, 2, pad)
    z.copy_(b), do.copy_(c), y.copy_(d)
    mss.gated_norm_fwd(y, z, w, out=out)
    want = mss.gated_norm_bwd(c, d, b, w)
    got = mss.gated_norm_bwd(do, y, z, w, dy=dy, dz=dz)
    assert torch.equal(out, mss.gated_norm_fwd(d, b, w))
    assert all(torch.equal(got[k], want[k]) for k in ("dy", "dz", "dweight"))
    assert torch.equal(z, b) and torch.equal(do, c) and torch.equal(y, d)
    assert untouched(io, (z, out, do, dz)) and untouched(wide, (y, dy))


def test_slices_that_share_a_column_are_refused():
    g = gen(2)
    w = torch.ones(96, device="cuda:0")
    wide, res = randn(g, 4, 400, dtype=torch.bfloat16), randn(g, 4, 96)
    for start in (0, 1, 95):
        with pytest.raises(mss.MambaScanError) as err:
            mss.add_norm_fwd(wide[:, :96], res, w, out=wide[:, start:start + 96])
        assert err.value.status == 7
    want = mss.add_norm_fwd(wide[:, :96].contiguous(), res, w)[0]
    assert torch.equal(mss.add_norm_fwd(wide[:, :96], res, w, out=wide[:, 96:192])[0], want)
