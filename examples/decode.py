"""A small decoder on the framework's decode path: attention over the 4-bit cache, then MoE.

    python examples/decode.py [--layers 4] [--prompts 3] [--beams 2] [--steps 32]
                              [--rotary-base 10000] [--repetition 1.2] [--temperature 0.8]

Each block adds what the one before it made to the residual and norms the sum (``rms_norm``), projects it to queries,
keys and values, appends the keys and values to the paged MXFP4 cache (with ``--rotary-base`` turned by their
positions, ``append_rotated``), attends, norms again, routes (``route``) and sends the result through an MXFP8 MoE
layer (``MoEDecodeLayer``).  Prompts go in as one ragged chunk, then every prompt is forked into beams (whole pages
shared), the beams are decoded token by token, with penalties for tokens that came before if asked for
(``adjust_logits``), the losing beams are freed and the pool is compacted.  Weights are random: what comes out are token
numbers that mean nothing.
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import synth  # noqa: E402
from moe_decode_gate_gb300 import (  # noqa: E402
    KVCache,
    MoEDecodeLayer,
    adjust_logits,
    rms_norm,
    rotation_table,
    route,
)


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

    def __call__(self, delta, x, cache, seqs, q_start=None, max_q=0, cos_sin=None):
        """x bf16 [tokens, H]: the residual of the new tokens of the sequences in slots `seqs`, delta: what the block
        before this one adds to it (None: nothing).  Returns this block's delta, and the residual."""
        hq, hkv, D = self.q_heads, self.kv_heads, self.head_dim
        if delta is None:
            h = rms_norm(x)
        else:
            h, x = rms_norm(delta, None, x)
        qkv = h @ self.qkv.t()
        q = qkv[:, :hq * D].unflatten(1, (hq, D))
        k = qkv[:, hq * D:(hq + hkv) * D].unflatten(1, (hkv, D))
        v = qkv[:, (hq + hkv) * D:].unflatten(1, (hkv, D))
        if cos_sin is None:
            cache.append(self.layer, k, v, seqs, q_start)
        else:
            q = cache.append_rotated(self.layer, q, k, v, cos_sin, seqs, q_start)
        y = cache.attention(self.layer, q, seqs, q_start, max_q=max_q)
        h, x = rms_norm(y.flatten(1) @ self.out.t(), None, x)
        ids, weights = route(h @ self.router.t(), self.K)
        return self.moe(h, ids, weights), x


class Decoder:
    def __init__(self, layers=4, q_heads=8, kv_heads=2, head_dim=64, vocabulary=512, max_tokens=1024,
                 workload="tiny", device="cuda", seed=0, rotary_base=None, positions=4096):
        wl = synth.WORKLOADS[workload]
        g = torch.Generator(device=device).manual_seed(seed)
        self.device = torch.device(device, torch.cuda.current_device())
        self.kv_heads, self.head_dim = kv_heads, head_dim
        self.embedding = torch.randn(vocabulary, wl.H, generator=g, device=device).bfloat16()
        self.blocks = [Block(i, wl, q_heads, kv_heads, head_dim, max_tokens, device, g)
                       for i in range(layers)]
        self.cos_sin = None if rotary_base is None else \
            rotation_table(positions, head_dim, rotary_base, device=self.device)

    def cache(self, num_pages, slots, columns, page_size=16):
        return KVCache(num_pages, slots, columns, len(self.blocks), self.kv_heads, self.head_dim,
                       page_size, device=self.device)

    def __call__(self, tokens, cache, seqs, q_start=None, max_q=0):
        """Logits [tokens, vocabulary] of new tokens whose places the cache has reserved."""
        delta, x = None, self.embedding[tokens.long()]
        for block in self.blocks:
            delta, x = block(delta, x, cache, seqs, q_start, max_q, self.cos_sin)
        h = rms_norm(x) if delta is None else rms_norm(delta, None, x)[0]
        return (h @ self.embedding.t()).float() / math.sqrt(x.shape[1])


def ints(values, device):
    return torch.tensor(values, dtype=torch.int32, device=device)


class Penalties:
    """The tokens so far of each slot, and what repeating them costs."""

    def __init__(self, prompts, beams, steps, repetition, temperature, device):
        n = len(prompts) * beams
        longest = max(len(p) for p in prompts)
        self.tokens = torch.zeros(n, longest + steps, dtype=torch.int32, device=device)
        self.prompt_lengths = ints([len(p) for p in prompts for _ in range(beams)], device)
        for i, p in enumerate(prompts):
            self.tokens[i * beams:(i + 1) * beams, :len(p)] = ints(p, device)
        self.lengths = self.prompt_lengths.clone()
        self.repetition = torch.full((n,), repetition, device=device)
        self.temperature = torch.full((n,), temperature, device=device)

    def add(self, token):
        self.tokens.scatter_(1, self.lengths.long()[:, None], token[:, None])
        self.lengths += 1

    def __call__(self, logits, slots):
        at = slots.long()
        return adjust_logits(logits, history=self.tokens, lengths=self.lengths, prompt_lengths=self.prompt_lengths,
                             seqs=slots, repetition=self.repetition[at], temperature=self.temperature[at], out=logits)


def generate(model, prompts, beams, steps, cache, compact_after=None, repetition=None, temperature=1.0):
    """Beams of each prompt, decoded greedily (beam b starts with the b-th best token), with penalties for tokens that
    came before if ``repetition`` is given.

    Returns the tokens [prompts, beams, steps] and the slots of the beams."""
    dev, n = model.device, len(prompts)
    first = ints([i * beams for i in range(n)], dev)  # the slot of each prompt's first beam
    lens = [len(p) for p in prompts]
    start = ints([sum(lens[:i]) for i in range(n + 1)], dev)
    if not cache.reserve(ints(lens, dev), first).all():
        raise RuntimeError("the cache has too few pages for the prompts")
    penalties = None if repetition is None else Penalties(prompts, beams, steps, repetition, temperature, dev)
    logits = model(torch.cat([ints(p, dev) for p in prompts]), cache, first, start, max(lens))
    logits = logits[start[1:].long() - 1]
    if penalties:
        logits = penalties(logits, first)
    token = logits.topk(beams).indices.flatten().int()
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
        logits = model(token, cache, slots)
        if penalties:
            penalties.add(token)
            logits = penalties(logits, slots)
        token = logits.argmax(-1).int()
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
    ap.add_argument("--rotary-base", type=float, help="turn queries and keys by their positions")
    ap.add_argument("--repetition", type=float, help="penalty for tokens that came before")
    ap.add_argument("--temperature", type=float, default=1.0)
    a = ap.parse_args()
    model = Decoder(a.layers, rotary_base=a.rotary_base)
    r = torch.Generator().manual_seed(1)
    prompts = [torch.randint(0, 512, (5 + 37 * i,), generator=r).tolist() for i in range(a.prompts)]
    cache = model.cache(num_pages=64 * a.prompts * a.beams, slots=a.prompts * a.beams, columns=64)
    tokens, slots = generate(model, prompts, a.beams, a.steps, cache, repetition=a.repetition,
                             temperature=a.temperature)
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
