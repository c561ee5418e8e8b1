"""A layer of the gated delta rule from the library's sequence operators, as
they are used together: trained on a batch, then run over packed prompts of
uneven length, then token by token from the states the prompts left.

    python examples/delta_rule_layer.py

One layer, per row of the residual stream r:

    x, r    = layer_norm(y_before, residual=r)          before the layer
    q, k, v = causal_conv(x @ W_qkv)                     short convolution and SiLU
    q, k    = block_norm(q), block_norm(k)               to length one, a head each
    g, beta = -rate softplus(x @ W_g), sigmoid(x @ W_b)  decay and strength of each head
    o       = gated_delta_rule(q, k, v, g, beta)
    y       = layer_norm(o, groups=heads) @ W_out        each head by itself

The torch.autograd functions below are all that training needs: each calls an
operator and, in backward, its gradient.
"""
from __future__ import annotations

import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import device_wide_prefix_gb300 as dwp  # noqa: E402
from examples.state_space_layer import Conv  # noqa: E402


class ResidualLayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, weight, bias):
        out, total = dwp.layer_norm(x, weight, bias, residual=residual)
        ctx.save_for_backward(total, weight, bias)
        return out, total

    @staticmethod
    def backward(ctx, grad, grad_total):
        total, weight, bias = ctx.saved_tensors
        g = dwp.layer_norm_backward(grad.contiguous(), total, weight, bias, grad_residual=grad_total.contiguous())
        return g["x"], g["residual"], g["weight"], g["bias"]


class HeadNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, groups):
        ctx.save_for_backward(x, weight, bias)
        ctx.groups = groups
        return dwp.layer_norm(x, weight, bias, groups=groups)[0]

    @staticmethod
    def backward(ctx, grad):
        g = dwp.layer_norm_backward(grad.contiguous(), *ctx.saved_tensors, groups=ctx.groups)
        return g["x"], g["weight"], g["bias"], None


class Unit(torch.autograd.Function):
    """Each of `groups` parts of a row to length one (up to eps)."""

    @staticmethod
    def forward(ctx, x, weight, groups):
        x = x.contiguous()
        ctx.save_for_backward(x, weight)
        ctx.groups = groups
        return dwp.block_norm(x, weight, groups=groups)[0]

    @staticmethod
    def backward(ctx, grad):
        return dwp.block_norm_backward(grad.contiguous(), *ctx.saved_tensors, groups=ctx.groups)["x"], None, None


class Delta(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, g, beta):
        out, points = dwp.gated_delta_rule(q, k, v, g, beta, return_checkpoints=True)
        ctx.save_for_backward(q, k, v, g, beta, points)
        return out

    @staticmethod
    def backward(ctx, grad):
        *args, points = ctx.saved_tensors
        grads = dwp.gated_delta_rule_backward(grad.contiguous(), *args, points)
        return tuple(grads[n] for n in ("q", "k", "v", "g", "beta"))


class Layer(torch.nn.Module):
    def __init__(self, width=256, key_heads=2, heads=4, keys=64, values=64, taps=4, dtype=torch.bfloat16):
        super().__init__()
        self.key_heads, self.heads, self.keys, self.values, self.taps = key_heads, heads, keys, values, taps
        inner = 2 * key_heads * keys + heads * values

        def matrix(rows, cols):
            return torch.nn.Parameter((torch.randn(rows, cols, device="cuda") / math.sqrt(rows)).to(dtype))

        def vector(v):
            return torch.nn.Parameter(v.float().cuda())

        self.w_qkv, self.w_gates, self.w_out = matrix(width, inner), matrix(width, 2 * heads), matrix(heads * values, width)
        self.conv, self.conv_bias = vector(torch.randn(inner, taps) * 0.5), vector(torch.zeros(inner))
        self.rate, self.step = vector(torch.empty(heads).uniform_(1, 16).log()), vector(torch.full((heads,), -4.0))
        self.norm, self.norm_bias = vector(torch.ones(width)), vector(torch.zeros(width))
        self.head_norm, self.head_bias = vector(torch.ones(heads * values)), vector(torch.zeros(heads * values))
        self.register_buffer("unit", torch.full((key_heads * keys,), keys ** -0.5, device="cuda"))

    def gates(self, x):
        """Log decay and strength of each row and head, f32."""
        a, b = (x @ self.w_gates).float().split(self.heads, -1)
        return -self.rate.exp() * torch.nn.functional.softplus(a + self.step), torch.sigmoid(b)

    def parts(self, u, unit):
        """Queries, keys and values of a convolved row, queries and keys of length one."""
        n = self.key_heads * self.keys
        q, k, v = u.split([n, n, self.heads * self.values], -1)
        q, k = (unit(t).unflatten(-1, (self.key_heads, self.keys)) for t in (q, k))
        return q, k, v.unflatten(-1, (self.heads, self.values))

    def forward(self, y, residual):
        """Training: (batch, rows, width) of the layer before and the residual stream."""
        x, residual = ResidualLayerNorm.apply(y, residual, self.norm, self.norm_bias)
        u = Conv.apply(x @ self.w_qkv, self.conv, self.conv_bias)
        q, k, v = self.parts(u, lambda t: Unit.apply(t, self.unit, self.key_heads))
        g, beta = self.gates(x)
        o = Delta.apply(q, k, v, g, beta).flatten(-2)
        return HeadNorm.apply(o, self.head_norm, self.head_bias, self.heads) @ self.w_out, residual

    @torch.no_grad()
    def prompt(self, y, residual, offsets):
        """Packed prompts (rows, width) cut by CSR offsets: the output, and each prompt's (conv, delta) state."""
        x, residual = dwp.layer_norm(y, self.norm, self.norm_bias, residual=residual)
        u, taps = dwp.causal_conv(x @ self.w_qkv, self.conv, self.conv_bias, offsets=offsets, return_state=True)
        q, k, v = self.parts(u, lambda t: dwp.block_norm(t, self.unit, groups=self.key_heads)[0])
        o, state = dwp.gated_delta_rule(q, k, v, *self.gates(x), offsets=offsets, return_state=True)
        o = dwp.layer_norm(o.flatten(-2), self.head_norm, self.head_bias, groups=self.heads)[0]
        return o @ self.w_out, residual, (taps, state)

    @torch.no_grad()
    def token(self, y, residual, cache, slots):
        """One new row of each sequence (batch, width); `cache` is updated in place at `slots`."""
        x, residual = dwp.layer_norm(y, self.norm, self.norm_bias, residual=residual)
        u = dwp.causal_conv_step(x @ self.w_qkv, cache[0], self.conv, self.conv_bias, slots=slots)
        q, k, v = self.parts(u, lambda t: dwp.block_norm(t, self.unit, groups=self.key_heads)[0])
        o = dwp.gated_delta_rule_step(q, k, v, *self.gates(x), cache[1], slots=slots)
        o = dwp.layer_norm(o.flatten(-2), self.head_norm, self.head_bias, groups=self.heads)[0]
        return o @ self.w_out, residual


def train(steps=40):
    """Fits the layer to delay its input by two rows; returns the layer, the first and the last loss."""
    torch.manual_seed(0)
    layer = Layer()
    opt = torch.optim.Adam(layer.parameters(), lr=3e-3)
    losses = []
    for _ in range(steps):
        x = torch.randn(4, 128, 256, device="cuda").bfloat16()
        want = torch.nn.functional.pad(x, (0, 0, 2, 0))[:, :128].float()
        out, _ = layer(x, torch.zeros(4, 128, 256, device="cuda"))
        loss = (out.float() - want).square().mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.item())
    return layer, losses[0], losses[-1]


def generate(layer, lengths=(5, 0, 37, 130), tokens=6):
    """The largest difference between prompts run whole and prompts continued token by token, over the output's size."""
    cuts = [sum(lengths[:i]) for i in range(len(lengths) + 1)]
    rows, res = torch.randn(cuts[-1], 256, device="cuda").bfloat16(), torch.randn(cuts[-1], 256, device="cuda")
    more = torch.randn(len(lengths), tokens, 256, device="cuda").bfloat16()
    more_res = torch.randn(len(lengths), tokens, 256, device="cuda")

    def packed(extra):
        join = lambda a, b: torch.cat([torch.cat([a[lo:hi], b[i, :extra]])  # noqa: E731
                                       for i, (lo, hi) in enumerate(zip(cuts[:-1], cuts[1:]))])
        off = torch.tensor([c + i * extra for i, c in enumerate(cuts)], dtype=torch.int32).cuda()
        return join(rows, more), join(res, more_res), off

    whole, _, _ = layer.prompt(*packed(tokens))
    _, _, states = layer.prompt(*packed(0))
    # the states go to a cache with other sequences' slots between them
    slots = torch.tensor([3 * i + 1 for i in range(len(lengths))], dtype=torch.int32).cuda()
    cache = [torch.zeros(3 * len(lengths) + 2, *s.shape[1:], dtype=s.dtype, device="cuda") for s in states]
    for c, s in zip(cache, states):
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
