"""Cases for the operators of the 4-bit cache of keys and values.

Three operators that a decode step uses around the MoE layer:

* append     new keys and values are quantised to MXFP4 and written into the pages of their sequences
* attention  queries attend to the pages of their sequences, dequantised on the way
* pages      forking sequences (whole pages shared, the last one copied; what a slot held before is
             freed) and compacting the pool (live pages move down, tables follow)

The cache is one uint8 tensor ``pool`` [pages, layers, kv heads, page size / 16, group], a group being 16
tokens of one head:

    K codes  [slabs][16 tokens][4 t][blocks][4 bytes]               channel = slab*32*blocks + 32c + 8t + n
    V codes  [slabs][2 halves][8 g][4 i][2 j][blocks][2 bytes]      channel = slab*32*blocks + 32c + 4g + n,
                                                                    token = 8*half + 2i + j
    K scales [16 tokens][D / 32]
    V scales [16 tokens][D / 32]

with blocks = min(4, D / 32) blocks of 32 channels to a slab, and nibble n of a run in byte n / 2, the low
half first.  A value is E2M1(code) * 2^(scale - 127); scale 255 stands for NaN.  ``table`` [slots, columns]
names the pages of each slot's sequence, -1 beyond its end; ``lengths`` [slots] counts its tokens, the new
ones included; ``refs`` [pages] counts how many table entries name a page, and 0 is a free page.
"""
import math

import numpy as np
import torch

own = False
DEVICE = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases ---

def listed():
    return [
        # one sequence of a chat, one token at a time: latency is all there is
        dict(name="attn_one_short", op="attention", B=1, lo=517, hi=517, q_lo=1, q_hi=1, hq=32, hkv=4, D=128, P=16,
             layers=2, window=0, dtype="bf16", empty=0),
        # a decode batch of requests of many lengths; one slot of the batch is idle
        dict(name="attn_batch32", op="attention", B=32, lo=300, hi=8192, q_lo=1, q_hi=1, hq=32, hkv=4, D=128, P=64,
             layers=2, window=0, dtype="bf16", empty=1),
        # a few very long documents
        dict(name="attn_long", op="attention", B=4, lo=100001, hi=131072, q_lo=1, q_hi=1, hq=32, hkv=4, D=128, P=64,
             layers=1, window=0, dtype="bf16", empty=0),
        # drafts of 1 to 5 tokens checked at once, small heads, three queries to a key head
        dict(name="attn_drafts", op="attention", B=24, lo=777, hi=3333, q_lo=1, q_hi=5, hq=24, hkv=8, D=64, P=32,
             layers=1, window=0, dtype="fp16", empty=0),
        # one key head for sixteen wide queries, attending to a window of the last 4096 tokens
        dict(name="attn_window", op="attention", B=64, lo=1000, hi=16000, q_lo=1, q_hi=1, hq=16, hkv=1, D=256, P=128,
             layers=1, window=4096, dtype="bf16", empty=0),
        # a chunk of two prompts over what is cached of them
        dict(name="attn_chunk", op="attention", B=2, lo=4100, hi=6001, q_lo=200, q_hi=256, hq=32, hkv=4, D=128, P=64,
             layers=1, window=0, dtype="bf16", empty=0),
        # the new token of each of 32 sequences
        dict(name="append_batch32", op="append", B=32, lo=300, hi=8192, q_lo=1, q_hi=1, hq=32, hkv=4, D=128, P=64,
             layers=2, dtype="bf16"),
        # eight prompts of a few thousand tokens each, out of the fused projection
        dict(name="append_prompts", op="append", B=8, lo=1500, hi=4096, q_lo=1500, q_hi=4096, hq=32, hkv=8, D=128,
             P=64, layers=1, dtype="bf16"),
        # four beams, each continuing one of them
        dict(name="fork_beams4", op="fork", n=4, lo=333, hi=333, hkv=4, D=128, P=16, layers=48, groups=1, spare=64),
        # 64 beams of eight requests
        dict(name="fork_beams64", op="fork", n=64, lo=900, hi=4000, hkv=4, D=128, P=64, layers=48, groups=8, spare=100),
        # a pool of one layer, many small pages, half of them left behind by finished sequences
        dict(name="compact_pages4096", op="compact", pages=4096, slots=64, hkv=8, D=64, P=16, layers=1, live=0.5),
        # a pool of all layers, large pages, three quarters in use
        dict(name="compact_48_layers", op="compact", pages=1200, slots=48, hkv=4, D=128, P=64, layers=48, live=0.72),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "append", "fork", "compact"])
    D, hkv = rng.choice([64, 128, 128, 256]), rng.choice([1, 2, 4, 8])
    P = rng.choice([16, 32, 64, 128])
    layers = rng.choice([1, 2, 3])
    if op == "attention":
        B, hq = _log(rng, 1, 128), hkv * rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
        q_hi = rng.choice([1, 1, 1, _log(rng, 2, 8), _log(rng, 9, 200)])
        if q_hi > 8:
            B = min(B, 4)
        hi = _log(rng, 1, max(2, min(131072, 268435456 // (B * hkv * D))))
        if q_hi > 8:
            hi = min(hi, max(1, 393216000 // (B * hq * q_hi * D)))
        lo = _log(rng, 1, hi)
        return dict(op=op, B=B, lo=lo, hi=hi, q_lo=rng.choice([1, q_hi]), q_hi=q_hi, hq=hq, hkv=hkv, D=D, P=P, layers=layers,
                    window=rng.choice([0, 0, _log(rng, 1, 2 * hi)]), dtype=rng.choice(["bf16", "fp16"]),
                    empty=rng.choice([0, 1]) if B > 1 else 0)
    if op == "append":
        B = _log(rng, 1, 128)
        q_hi = rng.choice([1, _log(rng, 1, max(2, 22000000 // (B * hkv * D)))])
        return dict(op=op, B=B, lo=q_hi, hi=q_hi + _log(rng, 1, 5000), q_lo=_log(rng, 1, q_hi), q_hi=q_hi,
                    hq=hkv * rng.choice([1, 4, 8]), hkv=hkv, D=D, P=P, layers=layers,
                    dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]))
    if op == "fork":
        n = _log(rng, 2, 64)
        return dict(op=op, n=n, lo=_log(rng, 1, 300), hi=_log(rng, 301, 4000), hkv=rng.choice([1, 2, 4]), D=rng.choice([64, 128]),
                    P=rng.choice([16, 32, 64]), layers=_log(rng, 1, 48), groups=rng.randint(1, n), spare=rng.randint(0, 2 * n))
    layers, P = _log(rng, 1, 48), rng.choice([16, 32, 64])
    hkv, D = rng.choice([1, 2, 4]), rng.choice([64, 128])
    most = min(131072, 1800000000 // page_bytes(dict(layers=layers, hkv=hkv, D=D, P=P)))
    return dict(op=op, pages=_log(rng, 64, most), slots=rng.randint(1, 128), hkv=hkv, D=D, P=P, layers=layers,
                live=round(rng.uniform(0.05, 0.8), 3))


def page_bytes(c):
    return c["layers"] * c["hkv"] * c["P"] * (c["D"] + 2 * (c["D"] // 32))


def _spread(lo, hi, n, seed):
    """n whole numbers from lo to hi, even on a logarithm's scale, in a shuffled order."""
    t = np.linspace(0.0, 1.0, n) if n > 1 else np.ones(1)
    v = np.round(np.exp(math.log(lo) + t * (math.log(hi) - math.log(lo)))).astype(np.int64)
    return np.random.RandomState(seed).permutation(v)


def _ragged(c):
    """Lengths and numbers of new tokens of a batch's sequences: they go by the case alone."""
    lens = _spread(c["lo"], c["hi"], c["B"], c["hi"])
    if c["op"] == "append":
        news = np.minimum(_spread(c["q_lo"], c["q_hi"], c["B"], 7), lens)
    else:
        news = np.random.RandomState(11).randint(c["q_lo"], c["q_hi"] + 1, c["B"])
    if c.get("empty"):
        lens[c["B"] // 2] = 0
    return lens, news


def _live_pages(c):
    """Which pages of the pool to compact are in use: by the case alone."""
    r = np.random.RandomState(c["pages"])
    n = max(1, int(round(c["live"] * c["pages"])))
    return r.permutation(c["pages"])[:n]


def work(c):
    per_token = 2 * (c["D"] // 2 + c["D"] // 32)  # bytes of one token and head in the cache
    if c["op"] == "attention":
        lens, news = _ragged(c)
        read, pairs = 0, 0
        for L, n in zip(lens.tolist(), news.tolist()):
            last = np.arange(L - n, L)
            first = np.maximum(0, last - c["window"] + 1) if c["window"] else np.zeros_like(last)
            seen = np.maximum(0, last - first + 1)
            pairs += int(seen.sum())
            read += int(max(0, L - max(0, int(first[0])))) if L else 0
        rows = int(news.sum()) * c["hq"]
        return {"bytes": read * c["hkv"] * per_token + rows * (2 * 2 * c["D"] + 4), "flops": 4.0 * c["D"] * c["hq"] * pairs}
    if c["op"] == "append":
        size = {"fp32": 4}.get(c["dtype"], 2)
        tokens = int(_ragged(c)[1].sum())
        return {"bytes": tokens * c["hkv"] * (2 * 2 * size * c["D"] + per_token), "flops": 4.0 * tokens * c["hkv"] * c["D"]}
    if c["op"] == "fork":
        lens = _spread(c["lo"], c["hi"], c["groups"], 3)
        src, dst, member = _beams(c)
        copied = sum(1 for a, b in zip(src, dst) if a != b and lens[member[a]] % c["P"])
        return {"bytes": 2 * copied * page_bytes(c) + 8 * sum(-(-int(lens[m]) // c["P"]) for m in member), "flops": 0}
    live = _live_pages(c)
    moved = int((live >= live.size).sum())
    return {"bytes": 2 * moved * page_bytes(c) + 12 * c["pages"] + 8 * live.size, "flops": 0}


# ------------------------------------------------------ the format, plainly ---

def _shape(D):
    blocks = min(4, D // 32)
    return D // 32 // blocks, blocks  # slabs, blocks to a slab


def quantise(x):
    """x [..., D] fp32 -> codes uint8 [..., D] (one to a byte), scales uint8 [..., D / 32]."""
    b = x.unflatten(-1, (-1, 32))
    a = b.abs().amax(-1, keepdim=True)
    e = (torch.frexp(a)[1] - 3).clamp(-127, 127)
    e = torch.where(a == 0, 0, e)
    y = torch.ldexp(torch.ldexp(b.abs(), -e // 2), -e - (-e // 2))
    # the values between 0, .5, 1, 1.5, 2, 3, 4, 6: a tie goes to the even code
    code = ((y > 0.25).to(torch.uint8) + (y >= 0.75) + (y > 1.25) + (y >= 1.75) + (y > 2.5) + (y >= 3.5) + (y > 5.0))
    code = code + 8 * torch.signbit(b)
    bad = ~torch.isfinite(a)
    code = torch.where(bad, 0, code).to(torch.uint8).flatten(-2)
    return code, torch.where(bad, 255, e + 127).to(torch.uint8).squeeze(-1)


def value_of(code, scale):
    """codes [..., D], scales [..., D / 32] -> fp32 [..., D]."""
    m = (code & 7).to(torch.float32)
    v = torch.where(m < 4, m * 0.5, torch.where(m < 6, m - 2, 2 * m - 8))
    v = torch.where(code >= 8, -v, v).unflatten(-1, (-1, 32))
    return (v * _power(scale).unsqueeze(-1)).flatten(-2)


def _power(scale):
    e = scale.to(torch.int32) - 127
    p = torch.ldexp(torch.ldexp(torch.ones_like(e, dtype=torch.float32), e // 2), e - e // 2)
    return torch.where(scale == 255, float("nan"), p)


def _bytes(nibbles):
    return nibbles[..., 0::2] | (nibbles[..., 1::2] << 4)


def _nibbles(b):
    return torch.stack((b & 15, b >> 4), -1).flatten(-2)


def pack_k(code):
    """[..., 16, D] -> [..., 8 D] bytes."""
    ns, nb = _shape(code.shape[-1])
    c = code.unflatten(-1, (ns, nb, 4, 8))  # token, slab, c, t, n
    return _bytes(c.movedim(-4, -5).movedim(-2, -3)).flatten(-5)


def pack_v(code):
    ns, nb = _shape(code.shape[-1])
    c = code.unflatten(-1, (ns, nb, 8, 4)).unflatten(-5, (2, 4, 2))  # half, i, j, slab, c, g, n
    order = [*range(c.dim() - 7), *[c.dim() - 7 + k for k in (3, 0, 5, 1, 2, 4, 6)]]
    return _bytes(c.permute(order)).flatten(-7)


def unpack_k(b, D):
    """[..., 8 D] bytes -> codes [..., 16, D]."""
    ns, nb = _shape(D)
    c = _nibbles(b.unflatten(-1, (ns, 16, 4, nb, 4)))  # slab, token, t, c, n
    return c.movedim(-5, -4).movedim(-3, -2).flatten(-4)


def unpack_v(b, D):
    ns, nb = _shape(D)
    c = _nibbles(b.unflatten(-1, (ns, 2, 8, 4, 2, nb, 2)))  # slab, half, g, i, j, c, n
    order = [*range(c.dim() - 7), *[c.dim() - 7 + k for k in (1, 3, 4, 0, 5, 2, 6)]]
    return c.permute(order).flatten(-4).flatten(-4, -2)


# ---------------------------------------------------------------- prepare ---

def _generator(seed):
    return torch.Generator(device=DEVICE).manual_seed(int(seed) * 2 + 1)


def _tables(lens, P, r, columns, pages):
    """A page table for sequences of these lengths over pages in a shuffled order, and the pages' counts."""
    need = -(-lens // P)
    order = r.permutation(pages)
    table = np.full((len(lens), columns), -1, np.int32)
    refs = np.zeros(pages, np.int32)
    at = 0
    for b, n in enumerate(need.tolist()):
        table[b, :n] = order[at:at + n]
        refs[order[at:at + n]] = 1
        at += n
    return table, refs


def _fill(pool, layer, D, P, g):
    """Keys and values as a model has them, quantised: normal, with channels of unlike size among the keys."""
    pages, _, hkv, groups, _ = pool.shape
    gain = torch.exp(0.5 * torch.randn(hkv, 1, 1, D, generator=g, device=DEVICE))
    step = max(1, (1 << 25) // (hkv * P * D))
    for a in range(0, pages, step):
        n = min(step, pages - a)
        shape = (n, hkv, groups, 16, D)
        kc, ks = quantise(torch.randn(shape, generator=g, device=DEVICE) * gain)
        vc, vs = quantise(torch.randn(shape, generator=g, device=DEVICE))
        pool[a:a + n, layer] = torch.cat((pack_k(kc), pack_v(vc), ks.flatten(-2), vs.flatten(-2)), -1)


def _device(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEVICE)


def _handle(c, s):
    """What a user's program holds: the framework's handle of the cache that these tensors are."""
    if own:
        import moe_decode_gate_gb300 as wd

        s["cache"] = wd.KVCache.from_buffers(s["pool"], s["table"], s["lengths"], s["refs"], layers=c["layers"],
                                             kv_heads=c["hkv"], head_dim=c["D"], page_size=c["P"])
    return s


def prepare(c, seed):
    g, r = _generator(seed), np.random.RandomState(int(seed) % (1 << 31))
    D, P, hkv = c["D"], c["P"], c["hkv"]
    if c["op"] in ("attention", "append"):
        lens, news = _ragged(c)
        B = c["B"]
        need = -(-lens // P)
        columns, pages = int(need.max()) + 1, int(need.sum()) + 3
        table, refs = _tables(lens, P, r, columns, pages)
        slots = r.permutation(B)  # entry b of the batch is the sequence in slot slots[b]
        by_slot, lengths = np.empty_like(table), np.empty(B, np.int32)
        by_slot[slots], lengths[slots] = table, lens
        pool = torch.zeros(pages, c["layers"], hkv, P // 16, 16 * (D + 2 * (D // 32)), dtype=torch.uint8, device=DEVICE)
        layer = c["layers"] - 1
        start = np.concatenate(([0], np.cumsum(news))).astype(np.int32)
        s = dict(c=c, pool=pool, table=_device(by_slot), lengths=_device(lengths), refs=_device(refs),
                 seqs=_device(slots.astype(np.int32)), layer=layer, max_q=int(news.max()),
                 q_start=_device(start) if int(news.max()) > 1 else None, longest=int(lens.max()))
        T = int(start[-1])
        if c["op"] == "attention":
            _fill(pool, layer, D, P, g)
            s["q"] = torch.randn(T, c["hq"], D, generator=g, device=DEVICE).to(DTYPES[c["dtype"]])
        else:  # keys and values as parts of the fused projection's rows
            width = (c["hq"] + 2 * hkv) * D
            s["qkv"] = torch.randn(T, width, generator=g, device=DEVICE).to(DTYPES[c["dtype"]])
        return _handle(c, s)
    if c["op"] == "fork":
        n, groups = c["n"], c["groups"]
        src, dst, member = _beams(c)
        lens = _spread(c["lo"], c["hi"], groups, 3)
        full, part = lens // P, (lens % P > 0).astype(np.int64)
        columns = int((full + part).max()) + 2
        pages = int(full.sum()) + int(part[member].sum()) + n + c["spare"]
        order = r.permutation(pages)
        table, refs = np.full((n, columns), -1, np.int32), np.zeros(pages, np.int32)
        begin = np.concatenate(([0], np.cumsum(full)))
        at = int(begin[-1])
        for b in range(n):  # a request's beams share its whole pages and have each its own last one
            m = member[b]
            shared = order[begin[m]:begin[m + 1]]
            table[b, :full[m]] = shared
            refs[shared] += 1
            if part[m]:
                table[b, full[m]] = order[at]
                refs[order[at]] += 1
                at += 1
        s = dict(c=c, src=_device(src.astype(np.int32)), dst=_device(dst.astype(np.int32)),
                 lengths=_device(lens[member].astype(np.int32)))
    else:
        live = _live_pages(c)
        pages, slots = c["pages"], c["slots"]
        cut = np.sort(np.random.RandomState(slots).randint(0, live.size + 1, slots - 1))
        cut = np.concatenate(([0], cut, [live.size]))
        columns = int(np.diff(cut).max()) + 1
        table, refs = np.full((slots, columns), -1, np.int32), np.zeros(pages, np.int32)
        mine = r.permutation(live)
        refs[mine] = 1
        for b in range(slots):
            table[b, :cut[b + 1] - cut[b]] = mine[cut[b]:cut[b + 1]]
        s = dict(c=c, lengths=_device((np.diff(cut) * P).astype(np.int32)))
        s["table_out"], s["refs_out"] = (torch.empty_like(_device(a)) for a in (table, refs))
    shape = (pages, c["layers"], hkv, P // 16, 16 * (D + 2 * (D // 32)))
    s["pool"] = torch.randint(0, 256, shape, generator=g, device=DEVICE, dtype=torch.uint8)
    s["table"], s["refs"] = _device(table), _device(refs)
    return _handle(c, s)


def _beams(c):
    """Which beam each beam goes on from (one of its own request), and each beam's request."""
    r = np.random.RandomState(c["n"] * 131 + c["groups"])
    member = np.sort(np.concatenate((np.arange(c["groups"]), r.randint(0, c["groups"], c["n"] - c["groups"]))))
    src = np.array([r.choice(np.flatnonzero(member == m)) for m in member])
    return src, np.arange(c["n"]), member


# -------------------------------------------------------------------- run ---

def run(s):
    c = s["c"]
    if c["op"] == "append":
        hq, hkv, D = c["hq"], c["hkv"], c["D"]
        k = s["qkv"][:, hq * D:(hq + hkv) * D].unflatten(1, (hkv, D))
        v = s["qkv"][:, (hq + hkv) * D:].unflatten(1, (hkv, D))
        if own:
            k, v = s["cache"].append(s["layer"], k, v, seqs=s["seqs"], q_start=s["q_start"], return_values=True)
        else:
            k, v = _plain_append(s, k, v)
        return {"k": k, "v": v, "pool": s["pool"]}
    if c["op"] == "attention":
        if own:
            out, lse = s["cache"].attention(s["layer"], s["q"], seqs=s["seqs"], q_start=s["q_start"], max_q=s["max_q"],
                                            window=c["window"], return_lse=True)
        else:
            out, lse = _plain_attention(s)
        return {"out": out, "lse": lse}
    if c["op"] == "fork":
        ok = s["cache"].fork(s["src"], s["dst"]) if own else _plain_fork(s)
        return {"ok": ok, "table": s["table"], "lengths": s["lengths"], "refs": s["refs"], "pool": s["pool"]}
    if own:
        page_map = s["cache"].compact(table_out=s["table_out"], refs_out=s["refs_out"])
    else:
        page_map = _plain_compact(s)
    return {"map": page_map, "table": s["table_out"], "refs": s["refs_out"], "pool": s["pool"]}


def _places(s, tokens):
    """For each new token: its entry of the batch, and its position in that entry's sequence."""
    at = torch.arange(tokens, device=s["pool"].device)
    if s["q_start"] is None:
        b, row, n = at, torch.zeros_like(at), torch.ones_like(at)
    else:
        start = s["q_start"].long()
        b = torch.searchsorted(start, at, right=True) - 1
        row, n = at - start[b], start[b + 1] - start[b]
    return b, row, s["lengths"][s["seqs"].long()].long()[b] - n + row


def _plain_append(s, k, v):
    c, pool = s["c"], s["pool"]
    D, P, layer = c["D"], c["P"], s["layer"]
    ns, nb = _shape(D)
    b, _, pos = _places(s, k.shape[0])
    page = s["table"][s["seqs"].long()[b], pos // P].long()
    group, token = pos % P // 16, pos % 16
    kc, ks = quantise(k.float())
    vc, vs = quantise(v.float())
    half = 8 * D
    rows = pool[..., :half].unflatten(-1, (ns, 16, 16 * nb))
    kb = _bytes(kc.unflatten(-1, (ns, nb, 4, 8)).movedim(-2, -3)).flatten(-3)  # [T, hkv, ns, 16 nb]
    rows[page, layer, :, group, :, token] = kb
    rows = pool[..., half:2 * half].unflatten(-1, (ns, 2, 8, 4, 2, 2 * nb))
    vb = _bytes(vc.unflatten(-1, (ns, nb, 8, 4)).movedim(-2, -3)).flatten(-2)  # [T, hkv, ns, 8, 2 nb]
    rows[page, layer, :, group, :, token // 8, :, token % 8 // 2, token % 2] = vb
    rows = pool[..., 2 * half:].unflatten(-1, (2, 16, D // 32))
    rows[page, layer, :, group, 0, token] = ks
    rows[page, layer, :, group, 1, token] = vs
    return value_of(kc, ks).to(k.dtype), value_of(vc, vs).to(v.dtype)


def _plain_attention(s):
    c, q, P, D, hkv = s["c"], s["q"], s["c"]["P"], s["c"]["D"], s["c"]["hkv"]
    T, hq = q.shape[:2]
    B, n, half = s["seqs"].numel(), max(1, -(-s["longest"] // P)), 8 * D
    seqs = s["seqs"].long()
    pages = s["table"][seqs, :n].clamp(min=0).long()
    groups = s["pool"][pages, s["layer"]].transpose(1, 2).flatten(2, 3)  # [B, hkv, n P / 16, group]
    ks, vs = groups[..., 2 * half:].unflatten(-1, (2, 16, D // 32)).unbind(-3)
    k = value_of(unpack_k(groups[..., :half], D), ks).flatten(2, 3)  # [B, hkv, n P, D]
    v = value_of(unpack_v(groups[..., half:2 * half], D), vs).flatten(2, 3)
    j = torch.arange(n * P, device=q.device)
    v = torch.where((j < s["lengths"][seqs][:, None])[:, None, :, None], v, 0.0)
    b, row, pos = _places(s, T)
    rows = torch.zeros(B, s["max_q"], hq, D, device=q.device)
    rows[b, row] = q.float()
    last = torch.full((B, s["max_q"]), -1, device=q.device)
    last[b, row] = pos
    seen = j <= last[..., None]
    if c["window"]:
        seen = seen & (j > last[..., None] - c["window"])
    x = rows.unflatten(2, (hkv, -1)).permute(0, 2, 3, 1, 4).flatten(2, 3)  # [B, hkv, heads of it * rows, D]
    x = (x @ k.transpose(-1, -2)).unflatten(2, (-1, s["max_q"])) * (1.0 / math.sqrt(D))
    x = torch.where(seen[:, None, None], x, -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(x - m)
    total = p.sum(-1, keepdim=True)
    o = (p.flatten(2, 3) @ v).unflatten(2, (-1, s["max_q"])) / torch.where(total == 0, 1.0, total)
    lse = (m + torch.log(total)).squeeze(-1)
    o = o.permute(0, 3, 1, 2, 4).flatten(2, 3)[b, row]
    return o.to(q.dtype), lse.permute(0, 3, 1, 2).flatten(2, 3)[b, row]


def _plain_fork(s):
    P, table, lengths, refs, pool = s["c"]["P"], s["table"], s["lengths"], s["refs"], s["pool"]
    src, dst = s["src"].long(), s["dst"].long()
    column = torch.arange(table.shape[1], device=table.device)
    length = torch.where(src >= 0, lengths[src.clamp(min=0)], 0)
    changed = src != dst
    partial = changed & (length % P > 0)
    order = torch.cumsum(partial, 0)
    free = torch.argsort((refs > 0).to(torch.int8), stable=True)  # the free pages first, lowest first
    ok = ~partial | (order <= (refs == 0).sum())
    copy, write = partial & ok, changed & ok
    page = free[(order - 1).clamp(0, free.numel() - 1)]
    old, new = table[dst], torch.where(src[:, None] >= 0, table[src.clamp(min=0)], -1)
    whole = (column < (length // P)[:, None]) & write[:, None]
    gone = (column < ((lengths[dst] + P - 1) // P)[:, None]) & write[:, None]
    refs.index_add_(0, new.clamp(min=0).long().flatten(), whole.int().flatten())
    refs.index_add_(0, old.clamp(min=0).long().flatten(), -gone.int().flatten())
    refs.index_add_(0, page, copy.int())
    at = copy[:, None] & (column == (length // P)[:, None])
    pairs = torch.nonzero(copy).squeeze(1)
    pool[page[pairs]] = pool[new[pairs, (length // P)[pairs]].long()]
    new = torch.where(whole, new, torch.where(at, page[:, None].int(), -1))
    table[dst] = torch.where(write[:, None], new, old)
    lengths[dst] = torch.where(write, length, lengths[dst])
    return ok.int()


def _plain_compact(s):
    table, refs, pool = s["table"], s["refs"], s["pool"]
    at = torch.arange(refs.numel(), device=refs.device)
    live = refs > 0
    n = live.sum()
    movers, holes = torch.nonzero(live & (at >= n)).squeeze(1), torch.nonzero(~live & (at < n)).squeeze(1)
    pool[holes] = pool[movers]
    page_map = torch.where(live, at, -1).int()
    page_map[movers] = holes.int()
    s["table_out"].copy_(torch.where(table >= 0, page_map[table.clamp(min=0).long()], -1))
    s["refs_out"].zero_()
    s["refs_out"][page_map[live].long()] = refs[live]
    return page_map


# ------------------------------------------------------------------ exact ---

_E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def exact(c, seed):
    if c["op"] == "append":
        return _exact_append(c, prepare(c, seed))
    if c["op"] == "attention":
        return _exact_attention(c, prepare(c, seed))
    return None


def _exact_append(c, s):
    x = s["qkv"].double()[:, c["hq"] * c["D"]:].unflatten(1, (2, c["hkv"], c["D"] // 32, 32))
    top = x.abs().amax(-1, keepdim=True)
    unit = torch.where(top > 0, torch.exp2(torch.floor(torch.log2(top)) - 2), 1.0)
    y = x.abs() / unit
    grid = torch.tensor(_E2M1, device=y.device)
    up = torch.bucketize(y, grid).clamp(1, 7)  # the first value of the grid that is not below y
    above, below = grid[up] - y, y - grid[up - 1]
    code = torch.where((above < below) | ((above == below) & (up % 2 == 0)), up, up - 1)
    code = torch.where(y >= 6, 7, code)
    x = (torch.sign(x) * grid[code] * unit).flatten(-2)
    return {"k": x[:, 0], "v": x[:, 1], "pool": None}


def _exact_attention(c, s):
    D, P, hkv, hq = c["D"], c["P"], c["hkv"], c["hq"]
    lens, news = _ragged(c)
    nb, half = min(4, D // 32), 8 * D
    ch = torch.arange(D, device=DEVICE)
    slab, inside = ch // (32 * nb), ch % (32 * nb)
    block, lane = inside // 32, inside % 32
    two = torch.exp2(torch.arange(-127, 129, device=DEVICE, dtype=torch.float64))
    two[255] = float("nan")
    grid = torch.tensor(np.concatenate((_E2M1, -_E2M1)), device=DEVICE)
    outs, lses, at = [], [], 0
    for b in range(c["B"]):
        L, n = int(lens[b]), int(news[b])
        q = s["q"][at:at + n].double().reshape(n, hkv, hq // hkv, D).permute(1, 2, 0, 3)
        at += n
        if L == 0:
            outs.append(torch.zeros(n, hq, D, device=DEVICE, dtype=torch.float64))
            lses.append(torch.full((n, hq), -math.inf, device=DEVICE, dtype=torch.float64))
            continue
        from_ = max(0, L - n - c["window"] + 1) if c["window"] else 0
        j = torch.arange(from_, L, device=DEVICE)
        page = s["table"][s["seqs"][b].long()].long()[j // P]
        held = s["pool"][:, s["layer"]]
        t = (j % 16)[:, None]
        kat = slab * 256 * nb + t * 16 * nb + lane // 8 * 4 * nb + block * 4 + lane % 8 // 2
        vat = half + slab * 256 * nb + t // 8 * 128 * nb + lane // 4 * 16 * nb + t % 8 // 2 * 4 * nb + t % 2 * 2 * nb + block * 2 + lane % 4 // 2
        sat = 2 * half + t * (D // 32) + ch // 32
        low = 4 * (ch % 2)
        scale = 1.0 / math.sqrt(D)
        last = torch.arange(L - n, L, device=DEVICE)[:, None]
        seen = j <= last
        if c["window"]:
            seen = seen & (j > last - c["window"])
        o, z = [], []
        for h in range(hkv):
            bytes_ = held[page, h, j % P // 16].long()  # [tokens, group]
            k = grid[(bytes_.gather(1, kat) >> low) & 15] * two[bytes_.gather(1, sat)]
            v = grid[(bytes_.gather(1, vat) >> low) & 15] * two[bytes_.gather(1, sat + D // 2)]
            x = torch.where(seen, (q[h] @ k.T) * scale, -math.inf)
            top = torch.logsumexp(x, -1, keepdim=True)
            p = torch.where(seen, torch.exp(x - torch.where(top == -math.inf, 0.0, top)), 0.0)
            o.append(p @ v)
            z.append(top.squeeze(-1))
        outs.append(torch.stack(o).permute(2, 0, 1, 3).reshape(n, hq, D))
        lses.append(torch.stack(z).permute(2, 0, 1).reshape(n, hq))
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}
