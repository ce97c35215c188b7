"""A ternary decoder that serves a batch of prompts: norms that add and quantise, W2A8 products, rotary append to the paged int8
cache, prompt attention for the prefill and decode attention for every token after it, dense feed-forward parts or experts.

Weights are random (seeded), so the text is noise; what it shows is the order of the calls, and that tokens made one by
one through the cache agree with the same tokens run as one prompt.

    python examples/generate.py [--layers 4] [--hidden 2560] [--heads 20] [--kv-heads 5] [--new 16]
                               [--experts 8 --top 2 --ffn 1792]
"""
from __future__ import annotations

import argparse
import os
import sys

import numpy as np

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))


def _weight(rng, N, K, gain=1.0):
    """A random ternary matrix whose product keeps the scale of its input, times gain."""
    import bit_gemv_i2_amd as bn
    T = (rng.integers(0, 3, (N, K), dtype=np.int8) - 1).astype(np.int8)
    S = (rng.uniform(0.5, 1.5, (N, K // 128)) * gain / np.sqrt(K * 2 / 3)).astype(np.float32)
    return bn.PackedWeight.from_ternary(T, S)


EPS = 1e-6


class Experts:
    """A feed-forward part of which every token takes `top` of several."""

    def __init__(self, rng, hidden, ffn, experts, top):
        import torch

        import bit_gemv_i2_amd as bn
        self.top = top
        self.router = torch.from_numpy((rng.standard_normal((hidden, experts)) / np.sqrt(hidden)).astype(np.float32)).cuda()
        gate_up, down = _weight(rng, experts * 2 * ffn, hidden), _weight(rng, experts * hidden, ffn)
        self.gate_up = bn.PackedExperts(gate_up.packed, gate_up.scales, experts, 2 * ffn, hidden)
        self.down = bn.PackedExperts(down.packed, down.scales, experts, hidden, ffn)

    def __call__(self, x, pending):
        """The stream with what was pending, and what the experts add to it."""
        import torch

        import bit_gemv_i2_amd as bn
        h, x = bn.bitnet_add_norm(x, None, EPS, out_dtype=torch.float32, **pending)
        _, gates, starts, rows, slots = bn.bitnet_route(h @ self.router, self.top)
        g = self.gate_up.grouped(*bn.bitnet_quant_act(h), starts, rows=rows, act="relu2", gated=True, out_dtype=torch.float32)
        d = self.down.grouped(*bn.bitnet_quant_act(g), starts, out_dtype=torch.float32)
        return x, dict(add=d, slots=slots, gates=gates)


class Dense:
    def __init__(self, rng, hidden, ffn):
        self.gate_up = _weight(rng, 2 * ffn, hidden)
        self.down = _weight(rng, hidden, ffn)

    def __call__(self, x, pending):
        import torch

        import bit_gemv_i2_amd as bn
        q, s, x = bn.bitnet_add_norm_quant(x, None, EPS, **pending)
        h = self.gate_up.linear(q, s, act="relu2", gated=True, out_dtype=torch.float32)
        return x, dict(add=self.down.linear(*bn.bitnet_quant_act(h), out_dtype=torch.float32))


class Layer:
    """Takes the stream and what the layer before has still to add to it (the keywords of the norm that adds it), and gives both."""

    def __init__(self, rng, hidden, heads, kv_heads, dim, ffn, pages, page, experts, top):
        import bit_gemv_i2_amd as bn
        self.heads, self.kv_heads, self.dim = heads, kv_heads, dim
        self.qkv = _weight(rng, (heads + 2 * kv_heads) * dim, hidden)
        self.out = _weight(rng, hidden, heads * dim)
        self.ffn = Experts(rng, hidden, ffn, experts, top) if experts else Dense(rng, hidden, ffn)
        self.cache = bn.KVCache.empty(pages, kv_heads, dim, page)

    def prefill(self, x, pending, rope, table, starts, before, longest):
        """x fp32 [tokens][hidden] of packed prompts."""
        import bit_gemv_i2_amd as bn
        T = x.shape[0]
        q, s, x = bn.bitnet_add_norm_quant(x, None, EPS, **pending)
        qkv = self.qkv.gemm(q, s)
        q, k = self.cache.append(qkv, rope, table, starts, before, longest, self.heads, with_k=True)
        v = qkv[:, (self.heads + self.kv_heads) * self.dim:].unflatten(1, (self.kv_heads, self.dim))
        a = bn.bitnet_attn_prompt(q, k, v, starts, longest)
        return self.ffn(self.out.linear(*bn.bitnet_quant_act(a.view(T, -1)), residual=x), {})

    def decode(self, x, pending, rope, table, starts, before, lengths, longest):
        """x fp32 [batch][hidden], one token of each sequence."""
        import bit_gemv_i2_amd as bn
        B = x.shape[0]
        q, s, x = bn.bitnet_add_norm_quant(x, None, EPS, **pending)
        q, _ = self.cache.append(self.qkv.gemv(q, s), rope, table, starts, before, 1, self.heads)
        a = self.cache.attend(q, table, lengths, longest)
        return self.ffn(self.out.linear(*bn.bitnet_quant_act(a.view(B, -1)), residual=x), {})


class Decoder:
    def __init__(self, layers=4, hidden=2560, heads=20, kv_heads=5, ffn=6912, vocab=4096, page=64, pages=256, positions=4096,
                 seed=0, experts=0, top=2):
        import torch

        import bit_gemv_i2_amd as bn
        rng = np.random.default_rng(seed)
        self.page, self.pages = page, pages
        self.layers = [Layer(rng, hidden, heads, kv_heads, 128, ffn, pages, page, experts, top) for _ in range(layers)]
        self.embed = torch.from_numpy(rng.standard_normal((vocab, hidden)).astype(np.float32)).cuda()
        self.rope = torch.from_numpy(bn.bitnet_rope_table(positions, 128)).cuda()

    def table(self, longest, batch):
        """Pages for `batch` sequences of up to `longest` tokens, in turn."""
        import torch
        slots = -(-longest // self.page)
        if slots * batch > self.pages or slots * self.page > self.rope.shape[0]:
            raise ValueError("the cache or the rotary table is too small")
        return torch.arange(slots * batch, dtype=torch.int32, device="cuda").view(slots, batch).t().contiguous()

    def logits(self, x):
        import bit_gemv_i2_amd as bn
        return bn.bitnet_add_norm(x, None, EPS)[0] @ self.embed.t()

    def _settled(self, x, pending):
        """The stream with what the last layer adds."""
        import bit_gemv_i2_amd as bn
        return bn.bitnet_add_norm(x, None, EPS, **pending)[1]

    def prefill(self, prompts, table):
        """Runs packed prompts (lists of tokens), fills the cache; hidden states fp32 [tokens][hidden] and their starts."""
        import torch
        lens = [len(p) for p in prompts]
        starts = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
        before = torch.zeros(len(prompts), dtype=torch.int32, device="cuda")
        x = self.embed[torch.tensor([t for p in prompts for t in p], device="cuda")]
        pending = {}
        for layer in self.layers:
            x, pending = layer.prefill(x, pending, self.rope, table, starts, before, max(lens))
        return self._settled(x, pending), starts

    def generate(self, prompts, new):
        """Greedy tokens int64 [batch][new] and the hidden states fp32 [new][batch][hidden] that chose them."""
        import torch
        longest = max(len(p) for p in prompts) + new
        table = self.table(longest, len(prompts))
        x, starts = self.prefill(prompts, table)
        x = x[starts[1:].long() - 1].contiguous()
        each = torch.arange(len(prompts) + 1, dtype=torch.int32, device="cuda")
        before = starts[1:] - starts[:-1]
        states, tokens = [], []
        for _ in range(new):
            states.append(x)
            tokens.append(self.logits(x).argmax(-1))
            x = self.embed[tokens[-1]]
            after = before + 1
            pending = {}
            for layer in self.layers:
                x, pending = layer.decode(x, pending, self.rope, table, each, before, after, longest)
            x = self._settled(x, pending)
            before = after
        return torch.stack(tokens, 1), torch.stack(states)


def check(model, prompts, tokens, states):
    """The hidden states of the generated tokens, and the same tokens as whole prompts: the smallest cosine.
    They differ by the cache's 8 bits and by the activations' 8 bits around them."""
    import torch
    whole = [p + t for p, t in zip(prompts, tokens.tolist())]
    x, starts = model.prefill(whole, model.table(max(map(len, whole)), len(whole)))
    worst = 1.0
    for b, p in enumerate(prompts):
        for i in range(tokens.shape[1]):
            at = int(starts[b]) + len(p) - 1 + i
            worst = min(worst, float(torch.nn.functional.cosine_similarity(x[at], states[i][b], dim=0)))
    return worst


def main(argv=None):
    import time

    import torch
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, value in (("layers", 4), ("hidden", 2560), ("heads", 20), ("kv-heads", 5), ("ffn", 6912), ("new", 16), ("batch", 4),
                        ("experts", 0), ("top", 2)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args(argv)
    rng = np.random.default_rng(1)
    model = Decoder(a.layers, a.hidden, a.heads, a.kv_heads, a.ffn, experts=a.experts, top=a.top)
    prompts = [rng.integers(0, 4096, int(n)).tolist() for n in rng.integers(5, 200, a.batch)]
    model.generate(prompts, 2)
    torch.cuda.synchronize()
    t = time.perf_counter()
    tokens, states = model.generate(prompts, a.new)
    torch.cuda.synchronize()
    t = time.perf_counter() - t
    worst = check(model, prompts, tokens, states)
    print(f"{a.batch} prompts of {[len(p) for p in prompts]} tokens, {a.new} new each: {t * 1e3:.1f} ms; "
          f"smallest cosine between decode and prefill {worst:.4f}")
    return worst


if __name__ == "__main__":
    main()
