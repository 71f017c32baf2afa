"""A stack of three hybrid layers run on the library's operators: a packed batch of prompts, then tokens one by one.

Each layer is   norm with the residual's addition (to e4m3 with a scale a row)  ->  projection  ->
mixing  ->  projection;   the mixing is a short causal convolution with the selective state space
scan in the first layer, one with the gated delta rule in the second, and attention over a paged
cache in the third.  The projections are plain torch products on the 8-bit values (bf16 holds them
exactly) with the rows' scales applied after.

    python examples/hybrid_layer.py      # compares a prompt continued token by token with the longer prompt
"""

import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from hybrid_linear_attention_prefill_gb300 import gdn  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32
I32 = torch.int32
HIDDEN, HK, HV, DK, DV, K = 512, 2, 4, 64, 64, 4
PAGE, WINDOW, SINKS = 16, 128, 4  # of the attention layer: tokens of a block, tokens looked back at, first tokens kept
EPS = 1e-6


def project(q, scales, w):
    """Rows of e4m3 values with a scale each, through a bf16 weight [out, in]."""
    return ((q.to(BF16) @ w.t()).float() * scales).to(BF16)


class Layer:
    """What all kinds share: the norm, and the projections in (`channels`, and some beside them) and out."""

    def __init__(self, gen, extra, conv=True):
        def w(*shape, scale):
            return (torch.randn(shape, generator=gen) * scale).to(BF16).cuda()

        self.channels = HV * DV + 2 * HK * DK
        self.norm = (1.0 + 0.1 * torch.randn(HIDDEN, generator=gen)).to(BF16).cuda()
        self.extra = extra
        width = -(-(self.channels + extra) // 8) * 8  # token strides are multiples of 8 elements
        self.w_in = w(width, HIDDEN, scale=HIDDEN ** -0.5)
        self.w_out = w(HIDDEN, HV * DV, scale=(HV * DV) ** -0.5)
        if conv:
            self.conv_w = w(self.channels, K, scale=K ** -0.5)
            self.conv_b = w(self.channels, scale=0.1)

    def enter(self, h, residual):
        q, scales, residual = gdn.add_norm(h, self.norm, residual, eps=EPS, e4m3=True)
        p = project(q, scales, self.w_in)
        return p[:, :self.channels], p[:, self.channels:self.channels + self.extra], residual

    def leave(self, y):
        return y.flatten(1) @ self.w_out.t()


class ScanLayer(Layer):
    """x, B, C through the convolution; a gate z and a step dt beside them."""

    def __init__(self, gen):
        super().__init__(gen, HV * DV + HV)
        step = torch.exp(torch.rand(HV, generator=gen) * math.log(100.0) + math.log(1e-3))
        self.dt_bias = (step + torch.log(-torch.expm1(-step))).cuda()
        self.A = -(1.0 + 15.0 * torch.rand(HV, generator=gen)).cuda()
        self.D = torch.ones(HV, device="cuda")

    def split(self, c, rest):
        n = HV * DV
        return dict(x=c[:, :n].unflatten(1, (HV, DV)), Bm=c[:, n:n + HK * DK].unflatten(1, (HK, DK)),
                    Cm=c[:, n + HK * DK:].unflatten(1, (HK, DK)), z=rest[:, :n].unflatten(1, (HV, DV)),
                    dt=rest[:, n:], A=self.A, D=self.D, dt_bias=self.dt_bias)

    def prompt(self, h, residual, cu):
        x, rest, residual = self.enter(h, residual)
        c, conv_state = gdn.causal_conv(x, self.conv_w, self.conv_b, cu)
        y, state = gdn.ssm_scan(**self.split(c, rest), cu_seqlens=cu)
        return self.leave(y), residual, (conv_state, state)

    def token(self, h, residual, states):
        x, rest, residual = self.enter(h, residual)
        c = gdn.causal_conv_step(x, self.conv_w, states[0], self.conv_b)
        return self.leave(gdn.ssm_step(**self.split(c, rest), state=states[1])), residual


class DeltaLayer(Layer):
    """q, k, v through the convolution; a log decay g and a write strength beta beside them."""

    def __init__(self, gen):
        super().__init__(gen, 2 * HV)

    def split(self, c, rest):
        n = HK * DK
        q, k, v = c[:, :n], c[:, n:2 * n], c[:, 2 * n:]
        q, k = (torch.nn.functional.normalize(t.unflatten(1, (HK, DK)).float(), dim=-1).to(BF16).contiguous()
                for t in (q, k))
        g = -torch.nn.functional.softplus(rest[:, :HV].float())
        beta = torch.sigmoid(rest[:, HV:].float())
        return q, k, v.unflatten(1, (HV, DV)).contiguous(), g.contiguous(), beta.contiguous()

    def prompt(self, h, residual, cu):
        x, rest, residual = self.enter(h, residual)
        c, conv_state = gdn.causal_conv(x, self.conv_w, self.conv_b, cu)
        y, state = gdn.prefill(*self.split(c, rest), cu_seqlens=cu)
        return self.leave(y), residual, (conv_state, state)

    def token(self, h, residual, states):
        x, rest, residual = self.enter(h, residual)
        c = gdn.causal_conv_step(x, self.conv_w, states[0], self.conv_b)
        q, k, v, g, beta = self.split(c, rest)
        y = torch.empty_like(v)
        gdn.check(gdn.gdn_decode(q, k, v, g, beta, states[1], y, x.shape[0], HK, HV, DK, DV))
        return self.leave(y), residual


class AttentionLayer(Layer):
    """HV query heads over HK key heads, within a window and the first tokens, over a paged cache."""

    def __init__(self, gen):
        super().__init__(gen, 0, conv=False)

    def split(self, c):
        n = HV * DK
        return [t.unflatten(1, (-1, DK)) for t in (c[:, :n], c[:, n:n + HK * DK], c[:, n + HK * DK:])]

    def prompt(self, h, residual, cu):
        x, _, residual = self.enter(h, residual)
        q, k, v = self.split(x)
        B, blocks = cu.numel() - 1, -(-x.shape[0] // PAGE) + 4 * cu.numel()
        table = torch.zeros(B, blocks, dtype=I32, device="cuda")
        free = torch.randperm(blocks, dtype=I32, device="cuda")
        slots, lens, count, refused = gdn.cache_plan(torch.zeros(B, dtype=I32, device="cuda"), table, free,
                                                     torch.tensor([blocks], dtype=I32, device="cuda"), cu, page=PAGE,
                                                     T=x.shape[0])
        cache = [torch.empty(blocks, HK, PAGE, DK, dtype=BF16, device="cuda") for _ in range(2)]
        gdn.cache_append(k, v, *cache, slots)
        y, _ = gdn.attention(q, k, v, cu, window=WINDOW, sinks=SINKS)
        return self.leave(y), residual, (lens, table, free, count, cache)

    def token(self, h, residual, states):
        lens, table, free, count, cache = states
        x, _, residual = self.enter(h, residual)
        q, k, v = self.split(x)
        slots = gdn.cache_plan(lens, table, free, count, page=PAGE, new_lens=lens, new_count=count)[0]
        gdn.cache_append(k, v, *cache, slots)
        y, _ = gdn.attention_step(q, *cache, table, lens, window=WINDOW, sinks=SINKS)
        return self.leave(y), residual


def prompt(layers, h, cu):
    """Hidden states after the layers (their residual added) for a packed batch, and the layers' states."""
    residual, states = torch.zeros_like(h), []
    for layer in layers:
        h, residual, s = layer.prompt(h, residual, cu)
        states.append(s)
    return h + residual, states


def token(layers, h, states):
    """The same for one token of every sequence; the states are updated in place."""
    residual = torch.zeros_like(h)
    for layer, s in zip(layers, states):
        h, residual = layer.token(h, residual, s)
    return h + residual


def compare(lens=(5, 130, 300), steps=6, seed=0):
    """Largest difference between prompts continued token by token and the longer prompts at once, over the
    largest value."""
    gen = torch.Generator().manual_seed(seed)
    layers = [ScanLayer(gen), DeltaLayer(gen), AttentionLayer(gen)]
    full = [torch.randn(n + steps, HIDDEN, generator=gen).to(BF16).cuda() for n in lens]

    def packed(parts):
        cu = torch.tensor([0] + [len(p) for p in parts]).cumsum(0).to(torch.int32).cuda()
        return torch.cat(parts), cu

    whole, _ = prompt(layers, *packed(full))
    ends = torch.tensor([n + steps for n in lens]).cumsum(0)
    _, states = prompt(layers, *packed([p[:n] for p, n in zip(full, lens)]))
    worst = 0.0
    for t in range(steps):
        got = token(layers, torch.stack([p[n + t] for p, n in zip(full, lens)]), states)
        want = whole[ends.cuda() - steps + t]
        worst = max(worst, float((got.float() - want.float()).abs().max()))
    return worst / float(whole.float().abs().max())


if __name__ == "__main__":
    print(f"prompts continued token by token against the longer prompts: {compare():.2e} of the largest value")
