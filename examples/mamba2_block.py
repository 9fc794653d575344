"""A Mamba-2 block on libmambascan: norm with the residual, input projection, SSD
mixer, gated norm, output projection ("Mamba-1/2/3 visual guide", section 2
block diagram and section 3; the short convolution is left out).

Training keeps the wide activations that the backward pass reads in 8 bits: the
projections' inputs (their weight gradients come straight from that form), the
residual, the mixer's input and output and the gate; B and C (bfloat16) and the
step sizes (float32), a few percent of the rest, stay as they are.  Generation
runs one token at a time on the recurrent state.

    python examples/mamba2_block.py      # one training step and a few tokens
"""
from __future__ import annotations

import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import selective_state_space_27_amd as mss  # noqa: E402


class _Block(torch.autograd.Function):
    """(x, residual) -> (block output, residual with x added)."""

    @staticmethod
    def forward(ctx, x, residual, norm, w_in, dt_bias, a_log, d, gate_norm, w_out, heads, groups, dstate, grad):
        b, length, _ = x.shape
        inner = w_out.shape[1]
        keep = grad and any(ctx.needs_input_grad)  # a backward pass may follow
        u, r, *u8 = mss.add_norm_fwd(x, residual, norm, residual_dtype=torch.float32, pack_out=keep)
        p = u @ w_in.t()
        z, xs, bs, cs, dt = p.split([inner, inner, groups * dstate, groups * dstate, heads], dim=-1)
        xs = xs.reshape(b, length, heads, inner // heads)
        bs, cs = (t.reshape(b, length, groups, dstate) for t in (bs, cs))
        dt = dt.float() + dt_bias
        delta, a = F.softplus(dt), -torch.exp(a_log)
        y = mss.ssd_chunk_fwd(xs.contiguous(), delta, a, bs.contiguous(), cs.contiguous(), d)
        y = y.view(b, length, inner)
        if not keep:
            return mss.gated_norm_fwd(y, z, gate_norm) @ w_out.t(), r
        g, *gate8 = mss.gated_norm_fwd(y, z, gate_norm, pack_inputs=True, pack_out=True)
        packed = (*u8, mss.pack8(r), mss.pack8(xs.view(b, length, inner)), *gate8)
        # Through autograd, which frees them after the backward pass.
        ctx.save_for_backward(norm, w_in, a, d, gate_norm, w_out, bs.contiguous(), cs.contiguous(), dt,
                              *(t for p8 in packed for t in (p8.q, p8.scale)))
        ctx.forms, ctx.sizes = [(p8.shape, p8.dtype) for p8 in packed], (heads, groups, dstate)
        return g @ w_out.t(), r

    @staticmethod
    def kept(ctx):
        """What the backward pass reads: parameters, tensors, checkpoints."""
        saved = ctx.saved_tensors
        packed = [mss.Packed8(q, scale, *form) for q, scale, form in zip(saved[9::2], saved[10::2], ctx.forms)]
        return saved[:6], saved[6:9], packed

    @staticmethod
    def backward(ctx, dout, dr):
        if torch.is_grad_enabled():  # create_graph: what follows would drop its terms without a word
            raise RuntimeError("the block has first derivatives only (create_graph=True asks for second ones)")
        heads, groups, dstate = ctx.sizes
        (norm, w_in, a, d, gate_norm, w_out), (bs, cs, dt), (u8, r8, x8, y8, z8, g8) = _Block.kept(ctx)
        b, length, _ = dout.shape
        inner = w_out.shape[1]
        dout = dout.contiguous()
        dw_out = mss.wgrad8(dout, g8)
        dp = torch.empty(b, length, w_in.shape[0], dtype=dout.dtype, device=dout.device)
        dz, dxs, dbs, dcs, ddt = dp.split([inner, inner, groups * dstate, groups * dstate, heads], dim=-1)
        gate = mss.gated_norm_bwd(dout @ w_out, y8, z8, gate_norm, dz=dz)
        s = mss.ssd_chunk_bwd(mss.unpack8(x8).view(b, length, heads, -1), F.softplus(dt), a, bs, cs, d,
                              dy=gate["dy"].view(b, length, heads, -1), want_dh0=False)
        dxs.copy_(s["dx"].view(b, length, inner))
        dbs.copy_(s["dB"].flatten(2))
        dcs.copy_(s["dC"].flatten(2))
        graw = s["ddelta"] * torch.sigmoid(dt)
        ddt.copy_(graw)
        dw_in = mss.wgrad8(dp, u8)
        n = mss.add_norm_bwd(dp @ w_in, r8, norm, dresidual_out=None if dr is None else dr.contiguous())
        return (n["dx"], n["dresidual"], n["dweight"], dw_in.to(w_in.dtype), graw.sum((0, 1)), s["dA"] * a, s["dD"],
                gate["dweight"], dw_out.to(w_out.dtype), None, None, None, None)


class Mamba2Block(torch.nn.Module):
    def __init__(self, width, heads, headdim=64, groups=1, dstate=128, device="cuda"):
        super().__init__()
        self.sizes = heads, groups, dstate
        self.headdim, inner = headdim, heads * headdim
        outs = 2 * inner + 2 * groups * dstate + heads
        par = lambda t: torch.nn.Parameter(t.to(device))  # noqa: E731
        self.norm, self.gate_norm = par(torch.ones(width)), par(torch.ones(inner))
        self.w_in = par((torch.randn(outs, width) / width ** 0.5).bfloat16())
        self.w_out = par((torch.randn(width, inner) / inner ** 0.5).bfloat16())
        self.dt_bias = par(torch.log(torch.expm1(torch.exp(torch.empty(heads).uniform_(-6.9, -2.3)))))
        self.a_log, self.d = par(torch.log(torch.empty(heads).uniform_(1, 16))), par(torch.ones(heads))

    def forward(self, x, residual=None):
        """x: [b, L, width] bfloat16, the previous block's output; residual: [b, L, width] float32."""
        if residual is None:
            residual = torch.zeros_like(x, dtype=torch.float32)
        return _Block.apply(x, residual, self.norm, self.w_in, self.dt_bias, self.a_log, self.d, self.gate_norm,
                            self.w_out, *self.sizes, torch.is_grad_enabled())

    def state(self, batch):
        heads, _, dstate = self.sizes
        return torch.zeros(batch, heads, self.headdim, dstate, device=self.norm.device)

    @torch.no_grad()
    def step(self, x, residual, h):
        """One token per sequence: x, residual [b, width]; h, updated in place."""
        heads, groups, dstate = self.sizes
        b, inner = x.shape[0], heads * self.headdim
        u, r = mss.add_norm_fwd(x, residual, self.norm, residual_dtype=torch.float32)
        z, xs, bs, cs, dt = (u @ self.w_in.t()).split([inner, inner, groups * dstate, groups * dstate, heads], dim=-1)
        xs, bs, cs = xs.contiguous(), bs.contiguous(), cs.contiguous()
        y = mss.mamba3_state_update(h, xs.view(b, heads, 1, self.headdim), F.softplus(dt.float() + self.dt_bias),
                                    -torch.exp(self.a_log), bs.view(b, groups, 1, dstate), cs.view(b, groups, 1, dstate),
                                    self.d)
        return mss.gated_norm_fwd(y.view(b, inner), z, self.gate_norm) @ self.w_out.t(), r


def main():
    torch.manual_seed(0)
    width, heads, b, length = 2560, 80, 2, 4096
    block = Mamba2Block(width, heads)
    x = torch.randn(b, length, width, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    residual = torch.randn(b, length, width, device="cuda", requires_grad=True)
    out, r = block(x, residual)
    _, tensors, packed = _Block.kept(out.grad_fn)
    rest = sum(t.numel() * t.element_size() for t in tensors)
    held = rest + sum(p.nbytes() for p in packed)
    full = rest + sum(p.shape.numel() * p.dtype.itemsize for p in packed)
    del tensors, packed  # the graph's again, to be freed with it
    (out.float().square().mean() + r.square().mean()).backward()
    print(f"training step: activations held {held / 2**20:.0f} MiB (unpacked {full / 2**20:.0f}), "
          f"|dW_in| {block.w_in.grad.float().norm():.4g}, |dW_out| {block.w_out.grad.float().norm():.4g}")
    h = block.state(b)
    for t in range(4):
        y, _ = block.step(x[:, t].detach(), residual[:, t].detach(), h)
        off = (y.float() - out[:, t].float()).norm() / out[:, t].float().norm()
        print(f"token {t}: generation against the chunked pass, relative difference {off:.2e}")


if __name__ == "__main__":
    main()
