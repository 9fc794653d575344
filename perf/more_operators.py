"""What is measured of the gated linear recurrence (a mixer with one state per channel: scan over whole sequences, its
gradient, its one-token step) and of beam search on recurrent states (selection over beams and vocabulary, reordering
of the states).

``own`` false: the operators in their plain form, elementary torch operations in 32 bits, rounded once at the end (64
bits for the totals that beam search compares).  ``own`` true: the calls a user makes of this framework.

Definitions:
  recurrence  r = sigmoid(gate_a), i = sigmoid(gate_x), a = exp(-c softplus(lam) r),
              h_t = a h_{t-1} + sqrt(1 - a^2) i x_t; at the start of a packed sequence h_{t-1} counts as zero; y = h
  beam        total = score + log_softmax(logits); the largest over beams and vocabulary, ties to the lowest index;
              a finished beam has one candidate, the end token at its score
  reorder     state[b, k] = state[b, parent[b, k]], in place
"""
import math

import torch

own = False

C = 8.0
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------------------------------------------- the cases
def listed():
    return [
        # The smallest training call: a test's shape. Latency of a forward and a backward call.
        {"name": "rec_tiny_step", "op": "rec_train", "batch": 1, "seqlen": 64, "dim": 16, "io": "fp32", "h0": False,
         "starts": False},
        # A training step on the batch of the scan's headline shape; inputs are slices of one projection's output.
        {"name": "rec_train", "op": "rec_train", "batch": 4, "seqlen": 8192, "dim": 5120, "io": "bf16", "h0": False,
         "starts": False},
        # Odd sizes in fp32, several sequences packed into a row, a state carried in and its gradient out.
        {"name": "rec_packed", "op": "rec_train", "batch": 3, "seqlen": 4099, "dim": 1001, "io": "fp32", "h0": True,
         "starts": True},
        # One long prompt: few channels, so the sequence itself has to fill the card.
        {"name": "rec_prompt", "op": "rec_fwd", "batch": 1, "seqlen": 131072, "dim": 2560, "io": "bf16", "h0": True,
         "starts": False},
        # One generated token of one sequence. Latency.
        {"name": "rec_token", "op": "rec_step", "batch": 1, "beams": 1, "dim": 2560, "io": "bf16"},
        # One generated token of 32 sequences with 8 beams each, read from their parents' states.
        {"name": "rec_token_beams", "op": "rec_step", "batch": 32, "beams": 8, "dim": 5120, "io": "bf16"},
        # Beam search of one sequence. Latency.
        {"name": "beam_one", "op": "beam", "batch": 1, "beams": 4, "vocab": 32000, "pad": 0, "n_out": 4, "io": "bf16",
         "finished": False, "first": True},
        # A serving batch: odd vocabulary in padded rows, twice as many candidates as beams, some beams finished.
        {"name": "beam_batch", "op": "beam", "batch": 32, "beams": 8, "vocab": 50277, "pad": 27, "n_out": 16,
         "io": "bf16", "finished": True, "first": False},
        # Wide search over a large vocabulary, logits in fp32.
        {"name": "beam_wide", "op": "beam", "batch": 8, "beams": 16, "vocab": 250001, "pad": 0, "n_out": 32,
         "io": "fp32", "finished": False, "first": False},
        # The states of one layer of one search (scan state, convolution inputs, recurrence state). Latency.
        {"name": "reorder_one", "op": "reorder", "batch": 1, "beams": 4, "kept": 2, "dim": 5120, "dstate": 16,
         "layers": 1},
        # Four layers' states of a serving batch.
        {"name": "reorder_batch", "op": "reorder", "batch": 32, "beams": 8, "kept": 4, "dim": 5120, "dstate": 16,
         "layers": 4},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rec_train", "rec_train", "rec_fwd", "rec_step", "beam", "beam", "reorder"])
    if op in ("rec_train", "rec_fwd"):
        dim = _log(rng, 16, 5120)
        if rng.random() < 0.6:
            dim = max(16, dim // 16 * 16)
        seqlen = _log(rng, 1, 32768 if op == "rec_train" else 131072)
        batch = _log(rng, 1, 64)
        batch = max(1, min(batch, 4 * 8192 * 5120 // (dim * seqlen)))
        return {"op": op, "batch": batch, "seqlen": seqlen, "dim": dim, "io": rng.choice(["bf16", "bf16", "fp32"]),
                "h0": rng.random() < 0.5, "starts": rng.random() < 0.4}
    if op == "rec_step":
        dim = _log(rng, 16, 5120)
        return {"op": op, "batch": _log(rng, 1, 64), "beams": rng.choice([1, 1, 3, 4, 8]),
                "dim": max(16, dim // 16 * 16) if rng.random() < 0.6 else dim, "io": rng.choice(["bf16", "fp32"])}
    if op == "beam":
        beams, vocab = rng.choice([1, 2, 3, 4, 5, 8, 12, 16]), _log(rng, 256, 260000)
        batch = max(1, min(_log(rng, 1, 64), 32000000 // (beams * vocab)))
        return {"op": op, "batch": batch, "beams": beams, "vocab": vocab, "pad": rng.choice([0, 0, 5, 64]),
                "n_out": rng.choice([beams, beams, 2 * beams]), "io": rng.choice(["bf16", "bf16", "fp32"]),
                "finished": rng.random() < 0.4, "first": rng.random() < 0.2}
    beams = rng.choice([2, 3, 4, 5, 8, 16])
    c = {"op": op, "batch": _log(rng, 1, 64), "beams": beams, "kept": rng.randint(1, beams), "dim": _log(rng, 16, 5120),
         "dstate": rng.choice([16, 16, 32, 128]), "layers": rng.randint(1, 4)}
    while c["batch"] > 1 and _reorder_bytes(c) * c["batch"] * beams > 390e6:
        c["batch"] //= 2
    return c


def _reorder_bytes(c):
    """Bytes of one beam's states: scan state and recurrence state in fp32, three convolution inputs in bf16."""
    return c["layers"] * c["dim"] * (4 * c["dstate"] + 6 + 4)


def work(case):
    op = case["op"]
    if op == "reorder":  # only the rows that move: each read once however often it is copied
        moved = case["beams"] - case["kept"]
        rows = case["batch"] * (moved + min(moved, case["kept"]))
        return {"bytes": rows * _reorder_bytes(case) + 8 * case["batch"] * case["beams"], "flops": 0}
    io = 2 if case["io"] == "bf16" else 4
    if op == "beam":
        n = case["batch"] * case["beams"] * case["vocab"]
        return {"bytes": n * io + case["batch"] * (case["beams"] * 6 + case["n_out"] * 21), "flops": 4 * n}
    if op == "rec_step":
        n = case["batch"] * case["beams"] * case["dim"]
        return {"bytes": n * (4 * io + 8) + 4 * case["dim"] + 8 * case["batch"] * case["beams"], "flops": 25 * n}
    n, bd = case["batch"] * case["seqlen"] * case["dim"], case["batch"] * case["dim"]
    marks = case["batch"] * case["seqlen"] if case["starts"] else 0
    fwd = n * 4 * io + 4 * case["dim"] + 4 * bd * case["h0"] + marks
    if op == "rec_fwd":
        return {"bytes": fwd + 4 * bd, "flops": 25 * n}
    # The backward pass comes after the loss: it reads the inputs again, dy, and writes three gradients.
    return {"bytes": fwd + n * 7 * io + 8 * case["dim"] + 4 * bd * case["h0"] + marks, "flops": 85 * n}


# ------------------------------------------------------------------------------------------------------ the inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _rand(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda", dtype=torch.float32)


def _lam(g, dim):
    """Decays exp(-c softplus(lam)) of a fully open gate between 0.81 and 0.998, as such a layer starts out."""
    sp = -torch.log(0.81 + 0.188 * _rand(g, dim)) / C
    return torch.log(torch.expm1(sp))


def _projection(g, lead, dim, dtype):
    """x, gate_a and gate_x as slices of one projection's output: channels of unlike size, gates around zero."""
    p = torch.empty(*lead, 3 * dim, dtype=dtype, device="cuda")
    p[..., :dim] = (_randn(g, *lead, dim) * torch.exp(0.5 * _randn(g, dim))).to(dtype)
    p[..., dim:2 * dim] = (1.5 * _randn(g, *lead, dim)).to(dtype)
    p[..., 2 * dim:] = (1.5 * _randn(g, *lead, dim)).to(dtype)
    return p[..., :dim], p[..., dim:2 * dim], p[..., 2 * dim:]


def _parents(g, batch, beams, kept):
    """Survivors stay in their slots, each dropped beam becomes a copy of one of them (so that a second pass changes
    nothing and passes can be repeated on the same states)."""
    order = torch.argsort(_rand(g, batch, beams), dim=1)
    pick = torch.randint(0, kept, (batch, beams), generator=g, device="cuda")
    slot = torch.arange(beams, device="cuda").expand(batch, beams)
    parents = torch.empty_like(order)
    parents.scatter_(1, order, torch.where(slot < kept, order, torch.gather(order, 1, pick)))
    return parents


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = {"case": case}
    if op == "reorder":
        lead, dim = (case["batch"], case["beams"]), case["dim"]
        s["parents"] = _parents(g, *lead, case["kept"])
        s["states"] = []
        for _ in range(case["layers"]):
            s["states"] += [_randn(g, *lead, dim, case["dstate"]), _randn(g, *lead, dim, 3).bfloat16(),
                            _randn(g, *lead, dim)]
        return s
    if op == "beam":
        batch, beams, vocab = case["batch"], case["beams"], case["vocab"]
        logits = torch.empty(batch, beams, vocab + case["pad"], dtype=DT[case["io"]], device="cuda")
        common = 1.5 * _randn(g, vocab)  # frequent tokens are likely everywhere
        common[:: 97] = -math.inf  # tokens that the program bans
        for b in range(batch):
            logits[b, :, :vocab] = (2.0 * _randn(g, beams, vocab) + common).to(logits.dtype)
        s["logits"] = logits[:, :, :vocab]
        s["scores"] = -20.0 * _rand(g, batch, beams) - 1.0
        if case["first"]:  # the search begins with one beam
            s["scores"][:, 1:] = -math.inf
        s["finished"] = _rand(g, batch, beams) < 0.3 if case["finished"] else None
        s["eos"] = 2
        return s
    dim, io = case["dim"], DT[case["io"]]
    s["lam"] = _lam(g, dim)
    if op == "rec_step":
        rows = case["batch"] * case["beams"]
        s["x"], s["ga"], s["gx"] = _projection(g, (rows,), dim, io)
        s["h"] = _randn(g, rows, dim)
        s["h_out"] = torch.empty_like(s["h"])  # states in two buffers, in turn
        s["parents"] = None
        if case["beams"] > 1:
            s["parents"] = torch.randint(0, case["beams"], (case["batch"], case["beams"]), generator=g, device="cuda")
        return s
    batch, seqlen = case["batch"], case["seqlen"]
    s["x"], s["ga"], s["gx"] = _projection(g, (batch, seqlen), dim, io)
    s["h0"] = _randn(g, batch, dim) if case["h0"] else None
    s["starts"] = _rand(g, batch, seqlen) < 0.005 if case["starts"] else None
    if op == "rec_train":
        s["dy"] = (1e-3 * _randn(g, batch, seqlen, dim)).to(io)
    return s


# -------------------------------------------------------------------------------------------------- the plain forms
def _parts(x, ga, gx, lam):
    x, r, i = x.float(), torch.sigmoid(ga.float()), torch.sigmoid(gx.float())
    s = C * torch.log1p(torch.exp(lam)) * r
    return x, r, i, s, torch.exp(-s), torch.sqrt(-torch.expm1(-2 * s))


def _doubling(a, b):
    """h_t = a_t h_{t-1} + b_t over dim 1, from zero, in place: spans of 1, 2, 4, ... steps joined."""
    d = 1
    while d < a.shape[1]:
        b[:, d:] += a[:, d:] * b[:, :-d].clone()
        a[:, d:] *= a[:, :-d].clone()
        d *= 2
    return b


def _plain_rec(s):
    c = s["case"]
    x, r, i, sa, a, beta = _parts(s["x"], s["ga"], s["gx"], s["lam"])
    keep = a if s["starts"] is None else a * (~s["starts"])[:, :, None]
    b = beta * i * x
    if s["h0"] is not None:
        b[:, 0] += keep[:, 0] * s["h0"]
    h = _doubling(keep.clone(), b)
    got = {"y": h.to(s["x"].dtype)}
    if c["op"] == "rec_fwd":
        got["h_last"] = h[:, -1].clone()
        return got
    before = torch.cat([torch.zeros_like(h[:, :1]) if s["h0"] is None else s["h0"][:, None], h[:, :-1]], 1)
    after = torch.cat([keep[:, 1:], torch.zeros_like(keep[:, :1])], 1)
    g = _doubling(after.flip(1), s["dy"].float().flip(1)).flip(1)
    big = g * (a * a * (sa / beta) * i * x - sa * keep * before)
    sp = torch.log1p(torch.exp(s["lam"]))
    got |= {"dx": (g * beta * i).to(h.dtype), "dgate_x": g * beta * i * x * (1 - i), "dgate_a": big * (1 - r)}
    got = {k: v.to(s["x"].dtype) for k, v in got.items()}
    got["dlam"] = big.sum((0, 1)) * torch.sigmoid(s["lam"]) / sp
    if s["h0"] is not None:
        got["dh0"] = keep[:, 0] * g[:, 0]
    return got


def _plain_step(s):
    h = s["h"]
    if s["parents"] is not None:
        rows = torch.arange(s["case"]["batch"], device=h.device)[:, None] * s["case"]["beams"] + s["parents"]
        h = h[rows.flatten()]
    x, _, i, _, a, beta = _parts(s["x"], s["ga"], s["gx"], s["lam"])
    new = a * h + beta * i * x
    s["h_out"].copy_(new)
    return {"y": new.to(s["x"].dtype), "h": s["h_out"]}


def _plain_beam(s):
    c, eos, fin = s["case"], s["eos"], s["finished"]
    v = s["logits"].double()
    top = v.amax(2, keepdim=True)
    total = s["scores"].double()[:, :, None] + (v - top - torch.log(torch.exp(v - top).sum(2, keepdim=True)))
    if fin is not None:
        only = torch.full_like(total, -math.inf)
        only[:, :, eos] = s["scores"].double()
        total = torch.where(fin[:, :, None], only, total)
    best, at = torch.sort(total.flatten(1), dim=1, descending=True, stable=True)
    best, at = best[:, :c["n_out"]], at[:, :c["n_out"]]
    parents, tokens = at // c["vocab"], at % c["vocab"]
    done = tokens == eos
    if fin is not None:
        done = done | torch.gather(fin, 1, parents)
    return {"scores": best.float(), "parents": parents, "tokens": tokens, "finished": done}


def _plain_reorder(s):
    at = torch.arange(s["case"]["batch"], device="cuda")[:, None]
    for t in s["states"]:
        t.copy_(t[at, s["parents"]])
    return s["states"]


# ---------------------------------------------------------------------------------------------------- the framework
def _framework(s):
    import selective_state_space_27_amd as mss

    c, op = s["case"], s["case"]["op"]
    if op == "reorder":
        mss.reorder_states(s["states"], s["parents"])
        return s["states"]
    if op == "beam":
        scores, parents, tokens, done = mss.beam_select(s["logits"], s["scores"], c["n_out"], finished=s["finished"],
                                                        eos=s["eos"])
        return {"scores": scores, "parents": parents, "tokens": tokens, "finished": done}
    args = s["x"], s["ga"], s["gx"], s["lam"]
    if op == "rec_step":
        y, h = mss.gated_recurrence_step(s["h"], *args, c=C, parents=s["parents"], h_out=s["h_out"])
        return {"y": y, "h": h}
    if op == "rec_fwd":
        y, last = mss.gated_recurrence_fwd(*args, c=C, h0=s["h0"], starts=s["starts"], return_last_state=True)
        return {"y": y, "h_last": last}
    y, states = mss.gated_recurrence_fwd(*args, c=C, h0=s["h0"], starts=s["starts"], keep_states=True)
    g = mss.gated_recurrence_bwd(s["dy"], *args, states, c=C, starts=s["starts"], want_dh0=s["h0"] is not None)
    got = {"y": y, "dx": g["dx"], "dgate_x": g["dgate_x"], "dgate_a": g["dgate_a"], "dlam": g["dlam"]}
    if s["h0"] is not None:
        got["dh0"] = g["dh0"]
    return got


def run(state):
    if own:
        return _framework(state)
    op = state["case"]["op"]
    if op == "reorder":
        return _plain_reorder(state)
    if op == "beam":
        return _plain_beam(state)
    return _plain_step(state) if op == "rec_step" else _plain_rec(state)


# --------------------------------------------------------------------------------------------------------- 64 bits
def _exact_terms(s, lam):
    """Decay and input term of every step, from the definition."""
    open_a = 1 / (1 + torch.exp(-s["ga"].double()))
    open_x = 1 / (1 + torch.exp(-s["gx"].double()))
    log_a = -C * torch.nn.functional.softplus(lam) * open_a
    return open_a, open_x, log_a


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "reorder":
        parents = s["parents"].tolist()
        return [torch.stack([torch.stack([t[b, k] for k in row]) for b, row in enumerate(parents)]).double()
                for t in s["states"]]
    if op == "beam":
        got = {"scores": [], "parents": [], "tokens": [], "finished": []}
        for b in range(case["batch"]):
            total = s["scores"][b].double()[:, None] + torch.log_softmax(s["logits"][b].double(), 1)
            if s["finished"] is not None:
                for k in s["finished"][b].nonzero().flatten().tolist():
                    total[k] = -math.inf
                    total[k, s["eos"]] = s["scores"][b, k].double()
            flat = total.flatten()
            least = flat.topk(case["n_out"]).values[-1]
            # all at least as good as the last place, in order of index; Python's sort keeps that order for ties
            if math.isinf(least):
                at = (flat > least).nonzero().flatten().tolist()
                more = (flat[:at[-1] + 1 + 2 * case["n_out"] if at else 2 * case["n_out"]] == least).nonzero()
                at += more.flatten().tolist()
            else:
                at = (flat >= least).nonzero().flatten().tolist()
            value = dict(zip(at, flat[torch.tensor(at, device="cuda")].tolist()))
            at = sorted(sorted(at), key=lambda k: -value[k])[:case["n_out"]]
            got["scores"].append([value[k] for k in at])
            got["parents"].append([k // case["vocab"] for k in at])
            got["tokens"].append([k % case["vocab"] for k in at])
            fin = s["finished"][b].tolist() if s["finished"] is not None else [False] * case["beams"]
            got["finished"].append([fin[k // case["vocab"]] or k % case["vocab"] == s["eos"] for k in at])
        return {k: torch.tensor(v, device="cuda", dtype=torch.float64 if k == "scores" else None)
                for k, v in got.items()}
    lam = s["lam"].double()
    if op == "rec_step":
        _, open_x, log_a = _exact_terms(s, lam)
        h = s["h"].double()
        if s["parents"] is not None:
            h = torch.cat([h.view(case["batch"], case["beams"], -1)[b, s["parents"][b]] for b in range(case["batch"])])
        new = torch.exp(log_a) * h + torch.sqrt(-torch.expm1(2 * log_a)) * open_x * s["x"].double()
        return {"y": new, "h": new}
    # Step by step; the gradient backwards through the same steps, then by automatic differentiation through the
    # decay and the input term of each step.
    train = op == "rec_train"
    leaf = lambda t: t.detach().double().requires_grad_(train)  # noqa: E731
    d = {"x": leaf(s["x"]), "ga": leaf(s["ga"]), "gx": leaf(s["gx"])}
    lam = leaf(lam)
    _, open_x, log_a = _exact_terms(d, lam)
    a = torch.exp(log_a)
    if s["starts"] is not None:
        a = a.masked_fill(s["starts"][:, :, None], 0.0)
    b = torch.sqrt(-torch.expm1(2 * log_a)) * open_x * d["x"]
    zero = torch.zeros(case["batch"], case["dim"], dtype=torch.float64, device="cuda")
    h = zero if s["h0"] is None else s["h0"].double()
    av, bv = a.detach(), b.detach()
    y = torch.empty_like(av)
    for t in range(case["seqlen"]):
        y[:, t] = h = torch.addcmul(bv[:, t], av[:, t], h)
    if not train:
        return {"y": y, "h_last": h}
    first = zero if s["h0"] is None else s["h0"].double()
    da, db, carry = torch.empty_like(av), torch.empty_like(av), zero
    for t in reversed(range(case["seqlen"])):
        db[:, t] = carry = s["dy"][:, t].double() + carry
        da[:, t] = carry * (y[:, t - 1] if t else first)
        carry = carry * av[:, t]
    grads = torch.autograd.grad((a, b), (d["x"], d["gx"], d["ga"], lam), (da, db))
    got = {"y": y, **dict(zip(("dx", "dgate_x", "dgate_a", "dlam"), grads))}
    if s["h0"] is not None:
        got["dh0"] = carry
    return got
