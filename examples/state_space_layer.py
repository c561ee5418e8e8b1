"""A state space layer from the library's sequence operators, as they are used
together: trained on a batch, then run over packed prompts of uneven length,
then token by token from the states the prompts left.

    python examples/state_space_layer.py

One layer, per row of the residual stream r:

    x, r   = block_norm(y_before, residual=r, scale)     before the block
    u, z   = x @ W_in                                    two halves of a projection
    u      = causal_conv(u)                              short convolution and SiLU
    dt,B,C = u @ W_x (dt @ W_dt)
    y      = selective_scan(u, dt, A, B, C, D)
    y      = block_norm(y, gate=z)                       after the block, gated
    y      = y @ W_out

The three torch.autograd functions below are all that training needs: each
calls an operator and, in backward, its gradient.
"""
from __future__ import annotations

import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import device_wide_prefix_gb300 as dwp  # noqa: E402


class Conv(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias):
        ctx.save_for_backward(x, weight, bias)
        return dwp.causal_conv(x, weight, bias)

    @staticmethod
    def backward(ctx, grad):
        g = dwp.causal_conv_backward(grad.contiguous(), *ctx.saved_tensors)
        return g["x"], g["weight"], g["bias"]


class Scan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, u, dt, A, B, C, D, dt_bias):
        out, points = dwp.selective_scan(u, dt, A, B, C, D=D, dt_bias=dt_bias, return_checkpoints=True)
        ctx.save_for_backward(u, dt, A, B, C, D, dt_bias, points)
        return out

    @staticmethod
    def backward(ctx, grad):
        u, dt, A, B, C, D, dt_bias, points = ctx.saved_tensors
        g = dwp.selective_scan_backward(grad.contiguous(), u, dt, A, B, C, points, D=D, dt_bias=dt_bias)
        return tuple(g[k] for k in ("u", "dt", "A", "B", "C", "D", "dt_bias"))


class ResidualNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, scale, weight):
        out, total = dwp.block_norm(x, weight, residual=residual, scale=scale)
        ctx.save_for_backward(x, total, scale, weight)
        return out, total

    @staticmethod
    def backward(ctx, grad, grad_total):
        x, total, scale, weight = ctx.saved_tensors
        g = dwp.block_norm_backward(grad.contiguous(), total, weight, x=x, scale=scale,
                                    grad_residual=grad_total.contiguous())
        return g["x"], g["residual"], g["scale"], g["weight"]


class GatedNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, gate, weight):
        ctx.save_for_backward(x, gate, weight)
        return dwp.block_norm(x, weight, gate=gate)[0]

    @staticmethod
    def backward(ctx, grad):
        x, gate, weight = ctx.saved_tensors
        g = dwp.block_norm_backward(grad.contiguous(), x, weight, gate=gate)
        return g["x"], g["gate"], g["weight"]


class Layer(torch.nn.Module):
    def __init__(self, width=256, inner=512, states=16, rank=16, taps=4, dtype=torch.bfloat16):
        super().__init__()
        self.inner, self.states, self.rank, self.taps = inner, states, rank, taps

        def matrix(rows, cols):
            return torch.nn.Parameter((torch.randn(rows, cols, device="cuda") / math.sqrt(rows)).to(dtype))

        def vector(v):
            return torch.nn.Parameter(v.float().cuda())

        self.w_in, self.w_x = matrix(width, 2 * inner), matrix(inner, rank + 2 * states)
        self.w_dt, self.w_out = matrix(rank, inner), matrix(inner, width)
        self.conv, self.conv_bias = vector(torch.randn(inner, taps) * 0.5), vector(torch.zeros(inner))
        self.log_a = vector(torch.log(torch.arange(1, states + 1).float()).repeat(inner, 1))
        step = torch.exp(torch.empty(inner).uniform_(math.log(1e-3), math.log(1e-1)))
        self.dt_bias, self.d = vector(torch.log(torch.expm1(step))), vector(torch.ones(inner))
        self.scale, self.norm, self.gate_norm = vector(torch.ones(width)), vector(torch.ones(width)), vector(torch.ones(inner))

    def project(self, u):
        low = u @ self.w_x
        return low[..., :self.rank] @ self.w_dt, *low[..., self.rank:].split(self.states, -1)

    def forward(self, y, residual):
        """Training: (batch, rows, width) of the block before and the residual stream."""
        x, residual = ResidualNorm.apply(y, residual, self.scale, self.norm)
        u, z = (x @ self.w_in).split(self.inner, -1)
        u = Conv.apply(u, self.conv, self.conv_bias)
        y = Scan.apply(u, *(lambda dt, B, C: (dt, -torch.exp(self.log_a), B, C))(*self.project(u)), self.d, self.dt_bias)
        return GatedNorm.apply(y, z, self.gate_norm) @ self.w_out, residual

    @torch.no_grad()
    def prompt(self, y, residual, offsets):
        """Packed prompts (rows, width) cut by CSR offsets: the output, and each prompt's (conv, scan) state."""
        x, residual = dwp.block_norm(y, self.norm, residual=residual, scale=self.scale)
        u, z = (x @ self.w_in).split(self.inner, -1)
        u, taps = dwp.causal_conv(u, self.conv, self.conv_bias, offsets=offsets, return_state=True)
        dt, B, C = self.project(u)
        y, state = dwp.selective_scan(u, dt, -torch.exp(self.log_a), B, C, D=self.d, dt_bias=self.dt_bias,
                                      offsets=offsets, return_state=True)
        return dwp.block_norm(y, self.gate_norm, gate=z)[0] @ self.w_out, residual, (taps, state)

    @torch.no_grad()
    def token(self, y, residual, cache, slots):
        """One new row of each sequence (batch, width); `cache` is updated in place at `slots`."""
        x, residual = dwp.block_norm(y, self.norm, residual=residual, scale=self.scale)
        u, z = (x @ self.w_in).split(self.inner, -1)
        u = dwp.causal_conv_step(u, cache[0], self.conv, self.conv_bias, slots=slots)
        dt, B, C = self.project(u)
        y = dwp.selective_scan_step(u, dt, -torch.exp(self.log_a), B, C, cache[1], D=self.d, dt_bias=self.dt_bias,
                                    slots=slots)
        return dwp.block_norm(y, self.gate_norm, gate=z)[0] @ self.w_out, residual


def train(steps=40):
    """Fits the layer to delay its input by three rows; returns the first and the last loss."""
    torch.manual_seed(0)
    layer = Layer()
    opt = torch.optim.Adam(layer.parameters(), lr=3e-3)
    losses = []
    for _ in range(steps):
        x = torch.randn(4, 128, 256, device="cuda").bfloat16()
        want = torch.nn.functional.pad(x, (0, 0, 3, 0))[:, :128].float()
        out, _ = layer(x, torch.zeros(4, 128, 256, device="cuda"))
        loss = (out.float() - want).square().mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.item())
    return layer, losses[0], losses[-1]


def generate(layer, lengths=(5, 0, 37, 130), tokens=6):
    """The largest difference between prompts run whole and prompts continued token by token, over the output's size."""
    total = sum(lengths)
    rows = torch.randn(total, 256, device="cuda").bfloat16()
    res = torch.randn(total, 256, device="cuda")
    cuts = [0]
    for n in lengths:
        cuts.append(cuts[-1] + n)
    more = torch.randn(len(lengths), tokens, 256, device="cuda").bfloat16()
    more_res = torch.randn(len(lengths), tokens, 256, device="cuda")

    def packed(extra):
        parts = [torch.cat([rows[a:b], more[i, :extra]]) for i, (a, b) in enumerate(zip(cuts[:-1], cuts[1:]))]
        rparts = [torch.cat([res[a:b], more_res[i, :extra]]) for i, (a, b) in enumerate(zip(cuts[:-1], cuts[1:]))]
        off = torch.tensor([c + i * extra for i, c in enumerate(cuts)], dtype=torch.int32).cuda()
        return torch.cat(parts), torch.cat(rparts), off

    whole, _, _ = layer.prompt(*packed(tokens))
    _, _, (taps, state) = layer.prompt(*packed(0))
    # the states go to a cache with other sequences' slots between them
    slots = torch.tensor([3 * i + 1 for i in range(len(lengths))], dtype=torch.int32).cuda()
    cache = [torch.zeros(3 * len(lengths) + 2, *s.shape[1:], dtype=s.dtype, device="cuda") for s in (taps, state)]
    for c, s in zip(cache, (taps, state)):
        c[slots.long()] = s
    far = 0.0
    for t in range(tokens):
        out, _ = layer.token(more[:, t], more_res[:, t], cache, slots)
        want = torch.stack([whole[cuts[i + 1] + i * tokens + t] for i in range(len(lengths))])
        far = max(far, (out.float() - want.float()).abs().max().item())
    return far / whole.float().abs().max().item()


def main():
    layer, first, last = train()
    print("training: loss %.4f -> %.4f in 40 steps" % (first, last))
    print("generation: token by token differs from the whole prompt by %.2g of the output's size" % generate(layer))


if __name__ == "__main__":
    main()
