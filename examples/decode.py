"""A small decoder on the framework's decode path: attention over the 4-bit cache, then MoE.

    python examples/decode.py [--layers 4] [--prompts 3] [--beams 2] [--steps 32]

Each block projects its input to queries, keys and values, appends the keys and values to the paged
MXFP4 cache, attends, and sends the result through an MXFP8 MoE layer (``MoEDecodeLayer``).  Prompts go
in as one ragged chunk, then every prompt is forked into beams (whole pages shared), the beams are
decoded token by token, the losing beams are freed and the pool is compacted.  Weights are random: what
comes out are token numbers that mean nothing.
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import synth  # noqa: E402
from moe_decode_gate_gb300 import KVCache, MoEDecodeLayer  # noqa: E402


def norm(x):
    x32 = x.float()
    return (x32 * torch.rsqrt(x32.square().mean(-1, keepdim=True) + 1e-6)).to(x.dtype)


class Block:
    """Attention and MoE of one layer, with random weights."""

    def __init__(self, layer, wl, q_heads, kv_heads, head_dim, max_tokens, device, generator):
        def weight(out, into):
            return (torch.randn(out, into, generator=generator, device=device) /
                    math.sqrt(into)).bfloat16()

        self.layer, self.K = layer, wl.K
        self.q_heads, self.kv_heads, self.head_dim = q_heads, kv_heads, head_dim
        self.qkv = weight((q_heads + 2 * kv_heads) * head_dim, wl.H)
        self.out = weight(wl.H, q_heads * head_dim)
        self.router = weight(wl.E, wl.H)
        weights = synth.make_layer(wl, B=1, layer=layer)
        self.moe = MoEDecodeLayer(weights.gate_up, weights.gate_up_scale, weights.down,
                                  weights.down_scale, K=wl.K, max_batch=max_tokens, device=device)

    def __call__(self, x, cache, seqs, q_start=None, max_q=0):
        """x bf16 [tokens, H]: the new tokens of the sequences in slots `seqs`."""
        hq, hkv, D = self.q_heads, self.kv_heads, self.head_dim
        qkv = norm(x) @ self.qkv.t()
        q = qkv[:, :hq * D].unflatten(1, (hq, D))
        k = qkv[:, hq * D:(hq + hkv) * D].unflatten(1, (hkv, D))
        v = qkv[:, (hq + hkv) * D:].unflatten(1, (hkv, D))
        cache.append(self.layer, k, v, seqs, q_start)
        y = cache.attention(self.layer, q, seqs, q_start, max_q=max_q)
        x = x + y.flatten(1) @ self.out.t()
        h = norm(x)
        p, ids = torch.softmax((h @ self.router.t()).float(), -1).topk(self.K)
        return x + self.moe(h, ids.int(), (p / p.sum(-1, keepdim=True)).contiguous())


class Decoder:
    def __init__(self, layers=4, q_heads=8, kv_heads=2, head_dim=64, vocabulary=512, max_tokens=1024,
                 workload="tiny", device="cuda", seed=0):
        wl = synth.WORKLOADS[workload]
        g = torch.Generator(device=device).manual_seed(seed)
        self.device = torch.device(device, torch.cuda.current_device())
        self.kv_heads, self.head_dim = kv_heads, head_dim
        self.embedding = torch.randn(vocabulary, wl.H, generator=g, device=device).bfloat16()
        self.blocks = [Block(i, wl, q_heads, kv_heads, head_dim, max_tokens, device, g)
                       for i in range(layers)]

    def cache(self, num_pages, slots, columns, page_size=16):
        return KVCache(num_pages, slots, columns, len(self.blocks), self.kv_heads, self.head_dim,
                       page_size, device=self.device)

    def __call__(self, tokens, cache, seqs, q_start=None, max_q=0):
        """Logits [tokens, vocabulary] of new tokens whose places the cache has reserved."""
        x = self.embedding[tokens.long()]
        for block in self.blocks:
            x = block(x, cache, seqs, q_start, max_q)
        return (norm(x) @ self.embedding.t()).float() / math.sqrt(x.shape[1])


def ints(values, device):
    return torch.tensor(values, dtype=torch.int32, device=device)


def generate(model, prompts, beams, steps, cache, compact_after=None):
    """Beams of each prompt, decoded greedily (beam b starts with the b-th best token).

    Returns the tokens [prompts, beams, steps] and the slots of the beams."""
    dev, n = model.device, len(prompts)
    first = ints([i * beams for i in range(n)], dev)  # the slot of each prompt's first beam
    lens = [len(p) for p in prompts]
    start = ints([sum(lens[:i]) for i in range(n + 1)], dev)
    if not cache.reserve(ints(lens, dev), first).all():
        raise RuntimeError("the cache has too few pages for the prompts")
    logits = model(torch.cat([ints(p, dev) for p in prompts]), cache, first, start, max(lens))
    token = logits[start[1:].long() - 1].topk(beams).indices.flatten().int()
    # the other beams go on from the first one's pages
    others = [i * beams + b for i in range(n) for b in range(1, beams)]
    if others and not cache.fork(ints([s // beams * beams for s in others], dev),
                                 ints(others, dev)).all():
        raise RuntimeError("the cache has too few pages for the beams")
    slots = ints(list(range(n * beams)), dev)
    one = torch.ones_like(slots)
    out = [token]
    for step in range(steps - 1):
        if not cache.reserve(one, slots).all():
            raise RuntimeError("the cache is full")
        token = model(token, cache, slots).argmax(-1).int()
        out.append(token)
        if step == compact_after:
            cache.compact()
    return torch.stack(out, 1).view(n, beams, steps), slots


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--layers", type=int, default=4)
    ap.add_argument("--prompts", type=int, default=3)
    ap.add_argument("--beams", type=int, default=2)
    ap.add_argument("--steps", type=int, default=32)
    a = ap.parse_args()
    model = Decoder(a.layers)
    r = torch.Generator().manual_seed(1)
    prompts = [torch.randint(0, 512, (5 + 37 * i,), generator=r).tolist() for i in range(a.prompts)]
    cache = model.cache(num_pages=64 * a.prompts * a.beams, slots=a.prompts * a.beams, columns=64)
    tokens, slots = generate(model, prompts, a.beams, a.steps, cache)
    for i, p in enumerate(prompts):
        for b in range(a.beams):
            print(f"prompt {i} ({len(p)} tokens), beam {b}:", tokens[i, b, :12].tolist(), "...")
    used = int((cache.refs > 0).sum())
    losers = slots.view(a.prompts, a.beams)[:, 1:].flatten().contiguous()
    cache.free(losers)
    left = int((cache.compact() >= 0).sum())
    assert cache.read_error_flag() == 0
    print(f"pages in use {used}, after freeing {losers.numel()} beams {left}, at the front of the "
          f"pool: {bool((cache.refs[:left] > 0).all())}")


if __name__ == "__main__":
    main()
