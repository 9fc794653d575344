"""What is measured of the operators around the mixer: the norms before and after a Mamba-2 mixer (fused with
residual, scale and gate), forward and backward, and 8-bit activation checkpoints with the backward passes that
read them.

``own`` false: the operators in their plain form, elementary torch operations in 32 bits, rounded once at the end.
``own`` true: the calls a user makes of this framework.

Definitions (a row is one token; RMS(v) = v / sqrt(mean(v^2) + eps)):
  add_norm    r = residual + scale*gamma*x', x' = x or RMS(x)*post; out = RMS(r)*w; residual_out = r
  gated_norm  out = RMS(y*silu(z))*w, or RMS(y)*w*silu(z) (norm first); groups of columns are normed apart
  checkpoint  per row and block of 32 columns: s the smallest power of two with max|x|/s < 127.5, x ~ rint(x/s)*s
  wgrad       dW = dY^T X, X held as such a checkpoint
"""
import math

import torch

own = False

EPS = 1e-5
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------------------------------------------- the cases
def listed():
    return [
        # One generated token, one sequence: residual stream in fp32, block input in bf16. Latency.
        {"name": "add_norm_token", "op": "add_norm_fwd", "rows": 1, "cols": 2560, "io": "bf16", "res": "fp32",
         "post": False, "gamma": False, "pack": False},
        # A training batch of 32768 tokens, model width of an 80-head layer; the projection's input kept in 8 bits.
        {"name": "add_norm_batch", "op": "add_norm_fwd", "rows": 32768, "cols": 2560, "io": "bf16", "res": "fp32",
         "post": False, "gamma": False, "pack": True},
        # Its gradient.
        {"name": "add_norm_grad", "op": "add_norm_bwd", "rows": 32768, "cols": 2560, "io": "bf16", "res": "fp32",
         "post": False, "gamma": False},
        # Norms on both sides of the block and a learned residual scale, odd sizes, all in fp32.
        {"name": "sandwich_grad", "op": "add_norm_bwd", "rows": 4097, "cols": 1001, "io": "fp32", "res": "fp32",
         "post": True, "gamma": True},
        # One generated token for each of 128 sequences; z is a slice of the input projection's output.
        {"name": "gated_tokens", "op": "gated_norm_fwd", "rows": 128, "cols": 5120, "io": "bf16", "res": "bf16",
         "groups": 1, "norm_first": False},
        # The SSD layer's batch (2 x 16384 tokens, 80 heads of 64): y in fp32 as the SSD writes it.
        {"name": "gated_batch", "op": "gated_norm_fwd", "rows": 32768, "cols": 5120, "io": "bf16", "res": "fp32",
         "groups": 1, "norm_first": False},
        # A training step through the gated norm: the forward keeps y and z in 8 bits, the backward reads them.
        {"name": "gated_step_ckpt", "op": "gated_norm_step", "rows": 32768, "cols": 5120, "io": "bf16", "res": "fp32",
         "groups": 1, "norm_first": False},
        # A small layer's gradient, ragged rows, eight groups, the gate after the norm.
        {"name": "gated_grad_groups", "op": "gated_norm_bwd", "rows": 2049, "cols": 1536, "io": "fp32", "res": "fp32",
         "groups": 8, "norm_first": True},
        # A mixer input kept for the mixer's backward and taken back: a slice of the input projection's output.
        {"name": "ckpt_batch", "op": "ckpt", "rows": 32768, "cols": 5120, "io": "bf16", "slice": True},
        # The same for odd sizes in fp32 (the last block of 32 columns is partial).
        {"name": "ckpt_ragged", "op": "ckpt", "rows": 777, "cols": 1001, "io": "fp32", "slice": False},
        # Weight gradient of the input projection of an 80-head layer (2*5120 + 2*128 + 80 outputs).
        {"name": "wgrad_in_proj", "op": "wgrad", "tokens": 32768, "outs": 10576, "ins": 2560, "dw": "fp32"},
        # A small layer's output projection on a ragged number of tokens: few output tiles, a long sum.
        {"name": "wgrad_small", "op": "wgrad", "tokens": 8191, "outs": 768, "ins": 1536, "dw": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["add_norm_fwd", "add_norm_bwd", "gated_norm_fwd", "gated_norm_bwd", "gated_norm_step", "ckpt",
                     "wgrad"])
    if op == "wgrad":
        tokens, outs, ins = _log(rng, 64, 32768), _log(rng, 64, 10576), _log(rng, 64, 5120)
        if rng.random() < 0.6:  # projections are mostly whole multiples of a head's width
            outs, ins = max(64, outs // 64 * 64), max(64, ins // 64 * 64)
        while tokens * outs * ins > 32768 * 10576 * 2560:
            tokens //= 2
        return {"op": op, "tokens": tokens, "outs": outs, "ins": ins, "dw": rng.choice(["fp32", "bf16"])}
    cols = _log(rng, 96, 16384)
    rows = _log(rng, 1, 256) if op.endswith("_fwd") and rng.random() < 0.4 else _log(rng, 256, 32768)
    if rng.random() < 0.6:
        cols = cols // 32 * 32
    rows = max(1, min(rows, 32768 * 5120 // cols))
    io = rng.choice(["bf16", "bf16", "fp32"])
    c = {"op": op, "rows": rows, "cols": cols, "io": io}
    if op == "ckpt":
        c["slice"] = rng.random() < 0.5
        return c
    c["res"] = "fp32" if io == "fp32" else rng.choice(["bf16", "fp32"])
    if op.startswith("add_norm"):
        c["post"], c["gamma"] = rng.random() < 0.4, rng.random() < 0.4
        if op == "add_norm_fwd":
            c["pack"] = rng.random() < 0.3
        return c
    c["groups"] = rng.choice([1, 1, 2, 4, 8])
    if c["groups"] > 1:
        c["cols"] = max(1, cols // (32 * c["groups"])) * 32 * c["groups"]
    c["norm_first"] = rng.random() < 0.4
    return c


def work(case):
    if case["op"] == "wgrad":
        t, m, n = case["tokens"], case["outs"], case["ins"]
        blocks = -(-n // 32)
        return {"bytes": 2 * t * m + t * n + t * blocks + m * n * (4 if case["dw"] == "fp32" else 2),
                "flops": 2 * t * m * n}
    rows, cols = case["rows"], case["cols"]
    n, io = rows * cols, 2 if case["io"] == "bf16" else 4
    packed = n + rows * -(-cols // 32)
    op = case["op"]
    if op == "ckpt":  # written, then read for the backward
        return {"bytes": 2 * n * io + 2 * packed, "flops": 4 * n}
    res = 2 if case["res"] == "bf16" else 4
    if op == "add_norm_fwd":
        params = cols * 4 * (1 + case["post"] + case["gamma"])
        # With the checkpoint: written, and read and widened for its user in the backward.
        return {"bytes": n * (2 * io + 2 * res) + params + (2 * packed + n * 2 if case["pack"] else 0), "flops": 8 * n}
    if op == "add_norm_bwd":
        extra = case["post"] or case["gamma"]
        return {"bytes": n * (2 * io + 3 * res + (io if extra else 0)) + cols * 4 * 2 * (1 + case["post"] + case["gamma"]),
                "flops": 16 * n}
    if op == "gated_norm_fwd":
        return {"bytes": n * (res + 2 * io) + cols * 4, "flops": 10 * n}
    back = n * (2 * io + res) + cols * 8
    if op == "gated_norm_bwd":
        return {"bytes": n * (res + io) + back, "flops": 24 * n}
    return {"bytes": n * (res + 2 * io) + 4 * packed + back, "flops": 34 * n}  # gated_norm_step


# ------------------------------------------------------------------------------------------------------ the inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _act(g, rows, cols, dtype, scale=1.0):
    """Activations: channels of unlike size (a few stand out by 10 or more), tokens of unlike size."""
    ch = torch.exp(0.7 * _randn(g, 1, cols)) * scale
    ch[:, :: max(1, cols // 7)] *= 12.0
    tok = torch.exp(0.3 * _randn(g, rows, 1))
    return (_randn(g, rows, cols) * ch * tok).to(dtype)


def _grad(g, rows, cols, dtype):
    return (_randn(g, rows, cols) * 1e-3 * torch.exp(0.5 * _randn(g, 1, cols))).to(dtype)


def _sliced(make, g, rows, cols, dtype):
    """The same values as columns of a wider buffer, as a projection's output is cut into the mixer's inputs."""
    wide = torch.empty(rows, cols + 336, dtype=dtype, device="cuda")
    view = wide[:, 256:256 + cols]
    view.copy_(make(g, rows, cols, dtype))
    return view


def _weight(g, cols):
    return 1.0 + 0.1 * _randn(g, cols)


def _q8(x):
    """(q, scale) of a checkpoint, for the cases that start from one."""
    rows, cols = x.shape
    pitch = -(-cols // 32) * 32
    v = torch.nn.functional.pad(x.float(), (0, pitch - cols)).view(rows, pitch // 32, 32)
    e = torch.frexp(v.abs().amax(2) / 127.5).exponent
    e = torch.clamp(e + 127, 1, 248)
    inv = ((254 - e) << 23).view(torch.float32)
    q = torch.clamp(torch.round(v * inv[:, :, None]), -127, 127)
    return q.to(torch.int8).view(rows, pitch), e.to(torch.uint8)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = {"case": case}
    if op == "wgrad":
        x = _act(g, case["tokens"], case["ins"], torch.bfloat16)
        s["q"], s["qs"] = _q8(x)
        s["dy"] = _grad(g, case["tokens"], case["outs"], torch.bfloat16)
        return s
    rows, cols, io = case["rows"], case["cols"], DT[case["io"]]
    if op == "ckpt":
        s["x"] = _sliced(_act, g, rows, cols, io) if case["slice"] else _act(g, rows, cols, io)
        return s
    res = DT[case["res"]]
    s["w"] = _weight(g, cols)
    if op.startswith("add_norm"):
        s["post"] = _weight(g, cols) if case["post"] else None
        s["gamma"] = 0.5 + 0.1 * _randn(g, cols) if case["gamma"] else None
        s["x"] = _act(g, rows, cols, io)
        s["residual"] = _act(g, rows, cols, res, 3.0)
        if op == "add_norm_bwd":
            s["dout"] = _grad(g, rows, cols, io)
            s["dres"] = _grad(g, rows, cols, res)
        return s
    s["y"] = _act(g, rows, cols, res)
    s["z"] = _sliced(lambda g, r, c, d: (1.5 * _randn(g, r, c)).to(d), g, rows, cols, io)
    if op != "gated_norm_fwd":
        s["dout"] = _grad(g, rows, cols, io)
    return s


# -------------------------------------------------------------------------------------------------- the plain forms
def _rms(v, groups=1):
    u = v.view(v.shape[0], groups, -1)
    return (u * torch.rsqrt(u.square().mean(2, keepdim=True) + EPS)).view_as(v)


def _rms_grad(g, v, groups=1):
    """Gradient with respect to v of <g, RMS(v)>."""
    u, h = v.view(v.shape[0], groups, -1), g.view(v.shape[0], groups, -1)
    r = torch.rsqrt(u.square().mean(2, keepdim=True) + EPS)
    return (r * h - u * (r * r * r) * (h * u).mean(2, keepdim=True)).view_as(v)


def _dequant(q, scale, cols):
    s = (scale.int() << 23).view(torch.float32)
    return (q.float().view(q.shape[0], -1, 32) * s[:, :, None]).view(q.shape[0], -1)[:, :cols]


def _plain_gated(y, z, w, groups, norm_first):
    sz = z * torch.sigmoid(z)
    return _rms(y, groups) * w * sz if norm_first else _rms(y * sz, groups) * w


def _plain_gated_grad(dout, y, z, w, groups, norm_first):
    sg = torch.sigmoid(z)
    sz, dsz = z * sg, sg * (1 + z * (1 - sg))
    if norm_first:
        n = _rms(y, groups)
        return _rms_grad(dout * w * sz, y, groups), dout * w * n * dsz, (dout * n * sz).sum(0)
    v = y * sz
    dv = _rms_grad(dout * w, v, groups)
    return dv * sz, dv * y * dsz, (dout * _rms(v, groups)).sum(0)


def _plain(s):
    c, op = s["case"], s["case"]["op"]
    if op == "wgrad":
        return (s["dy"].float().t() @ _dequant(s["q"], s["qs"], c["ins"])).to(DT[c["dw"]])
    io = DT[c["io"]]
    if op == "ckpt":
        q, e = _q8(s["x"])
        return _dequant(q, e, c["cols"]).to(io)
    res, w = DT[c["res"]], s["w"]
    if op.startswith("add_norm"):
        x, m = s["x"].float(), s["gamma"] if s["gamma"] is not None else 1.0
        n = _rms(x) if c["post"] else x
        xp = n * s["post"] if c["post"] else n
        if op == "add_norm_fwd":
            r = s["residual"].float() + m * xp
            out = (_rms(r) * w).to(io)
            got = {"out": out, "residual": r.to(res)}
            if c["pack"]:
                q, e = _q8(out)
                got["ckpt"] = _dequant(q, e, c["cols"]).to(torch.bfloat16)
            return got
        r, dout = s["residual"].float(), s["dout"].float()
        dr = _rms_grad(dout * w, r) + s["dres"].float()
        got = {"dresidual": dr.to(res), "dweight": (dout * _rms(r)).sum(0)}
        if c["gamma"]:
            got["dgamma"] = (dr * xp).sum(0)
        dx = m * dr
        if c["post"]:
            got["dpost"] = (dx * n).sum(0)
            dx = _rms_grad(dx * s["post"], x)
        got["dx"] = dx.to(io)
        return got
    y, z, groups, first = s["y"].float(), s["z"].float(), c["groups"], c["norm_first"]
    got = {}
    if op != "gated_norm_bwd":
        got["out"] = _plain_gated(y, z, w, groups, first).to(io)
    if op == "gated_norm_step":
        y, z = _dequant(*_q8(y), c["cols"]), _dequant(*_q8(z), c["cols"])
    if op != "gated_norm_fwd":
        dy, dz, dw = _plain_gated_grad(s["dout"].float(), y, z, w, groups, first)
        got |= {"dy": dy.to(res), "dz": dz.to(io), "dweight": dw}
    return got


# ---------------------------------------------------------------------------------------------------- the framework
def _framework(s):
    import selective_state_space_27_amd as mss

    c, op = s["case"], s["case"]["op"]
    if op == "wgrad":
        x8 = mss.Packed8(s["q"], s["qs"], (c["tokens"], c["ins"]), torch.bfloat16)
        return mss.wgrad8(s["dy"], x8, out_dtype=DT[c["dw"]])
    if op == "ckpt":
        return mss.unpack8(mss.pack8(s["x"]))
    if op == "add_norm_fwd":
        got = mss.add_norm_fwd(s["x"], s["residual"], s["w"], post_weight=s["post"], gamma=s["gamma"], eps=EPS,
                               pack_out=c["pack"])
        d = {"out": got[0], "residual": got[1]}
        if c["pack"]:
            d["ckpt"] = mss.unpack8(got[2], torch.bfloat16)
        return d
    if op == "add_norm_bwd":
        g = mss.add_norm_bwd(s["dout"], s["residual"], s["w"], dresidual_out=s["dres"],
                             x=s["x"] if c["post"] or c["gamma"] else None, post_weight=s["post"], gamma=s["gamma"],
                             eps=EPS)
        d = {"dresidual": g["dresidual"], "dweight": g["dweight"], "dx": g["dx"]}
        if c["gamma"]:
            d["dgamma"] = g["dgamma"]
        if c["post"]:
            d["dpost"] = g["dpost_weight"]
        return d
    args = {"ngroups": c["groups"], "norm_first": c["norm_first"], "eps": EPS}
    if op == "gated_norm_fwd":
        return {"out": mss.gated_norm_fwd(s["y"], s["z"], s["w"], **args)}
    y, z, d = s["y"], s["z"], {}
    if op == "gated_norm_step":
        d["out"], y, z = mss.gated_norm_fwd(y, z, s["w"], pack_inputs=True, **args)
    g = mss.gated_norm_bwd(s["dout"], y, z, s["w"], **args)
    return d | {"dy": g["dy"], "dz": g["dz"], "dweight": g["dweight"]}


def run(state):
    return _framework(state) if own else _plain(state)


# --------------------------------------------------------------------------------------------------------- 64 bits
def _exact_norm(v, groups=1):
    """v / sqrt(mean(v^2) + eps), by groups of columns."""
    u = v.reshape(v.shape[0], groups, v.shape[1] // groups)
    return (u / torch.sqrt((u * u).sum(2, keepdim=True) / u.shape[2] + EPS)).reshape(v.shape)


def _exact_ckpt(x):
    """The values that a checkpoint of x stands for: exponents from log2, in 64 bits."""
    x = x.double()
    rows, cols = x.shape
    out = torch.zeros(rows, -(-cols // 32) * 32, dtype=torch.float64, device=x.device)
    out[:, :cols] = x
    blocks = out.reshape(rows, -1, 32)
    top = blocks.abs().max(2, keepdim=True).values
    step = torch.exp2(torch.floor(torch.log2(top / 127.5)) + 1)
    step = torch.where(top / step >= 127.5, step * 2, step)  # should log2 have rounded
    step = torch.where(top / (step / 2) < 127.5, step / 2, step)
    step = torch.where(top > 0, step, torch.ones_like(step)).clamp(2.0 ** -126, 2.0 ** 121)
    return (torch.round(blocks / step).clamp(-127, 127) * step).reshape(rows, -1)[:, :cols]


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "wgrad":
        x = s["q"].double() * torch.exp2(s["qs"].double() - 127).repeat_interleave(32, 1)
        return s["dy"].double().t().contiguous() @ x[:, :case["ins"]]
    if op == "ckpt":
        return _exact_ckpt(s["x"])
    leaf = lambda t: t.detach().double().requires_grad_(True)  # noqa: E731
    w = leaf(s["w"])
    if op.startswith("add_norm"):
        x = leaf(s["x"])
        post = leaf(s["post"]) if case["post"] else None
        gamma = leaf(s["gamma"]) if case["gamma"] else None
        part = _exact_norm(x) * post if case["post"] else x
        part = gamma * part if case["gamma"] else part
        if op == "add_norm_fwd":
            with torch.no_grad():
                r = s["residual"].double() + part
                got = {"out": _exact_norm(r) * w, "residual": r}
                if case["pack"]:  # of the output as it is stored
                    got["ckpt"] = _exact_ckpt(got["out"].to(DT[case["io"]]))
            return got
        # The gradient at the residual as it was stored, then through what was added to it.
        r = leaf(s["residual"])
        dr, dw = torch.autograd.grad(_exact_norm(r) * w, (r, w), s["dout"].double())
        dr = dr + s["dres"].double()
        names = {"dx": x, "dgamma": gamma, "dpost": post}
        names = {k: v for k, v in names.items() if v is not None}
        if part is x:
            return {"dresidual": dr, "dweight": dw, "dx": dr}
        return {"dresidual": dr, "dweight": dw,
                **dict(zip(names, torch.autograd.grad(part, list(names.values()), dr)))}

    def gated(y, z):
        gate = z / (1 + torch.exp(-z))
        if case["norm_first"]:
            return _exact_norm(y, case["groups"]) * w * gate
        return _exact_norm(y * gate, case["groups"]) * w

    got = {}
    if op != "gated_norm_bwd":
        with torch.no_grad():
            got["out"] = gated(s["y"].double(), s["z"].double())
    if op != "gated_norm_fwd":
        kept = _exact_ckpt if op == "gated_norm_step" else (lambda t: t)
        y, z = leaf(kept(s["y"])), leaf(kept(s["z"]))
        got |= dict(zip(("dy", "dz", "dweight"), torch.autograd.grad(gated(y, z), (y, z, w), s["dout"].double())))
    return got
