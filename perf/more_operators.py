"""Cases for the operators that stand around attention and experts in a decode step.

* norm     the residual is added and the sum normed by its root mean square; the output in the input's type or
           in MXFP8 (E4M3 codes, one E8M0 scale per 32 channels)
* rotate   queries and keys are rotated by their positions; keys and values go into the pages of the 4-bit cache
* route    the router's logits become the experts and weights that the MoE layer takes
* logits   the last layer's logits are penalised for repeated tokens, biased, scaled and masked

The cache's layout is that of the first file of cases beside this one: groups of 16 tokens of one head,

    K codes  [slabs][16 tokens][4 t][blocks][4 bytes]               channel = slab*32*blocks + 32c + 8t + n
    V codes  [slabs][2 halves][8 g][4 i][2 j][blocks][2 bytes]      channel = slab*32*blocks + 32c + 4g + n,
                                                                    token = 8*half + 2i + j
    K scales [16 tokens][D / 32]
    V scales [16 tokens][D / 32]

with blocks = min(4, D / 32), nibble n of a run in byte n / 2, the low half first.
"""
import math

import numpy as np
import torch

own = False
DEVICE = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZES = {"bf16": 2, "fp16": 2, "fp32": 4}
EPS = 1e-6


# ------------------------------------------------------------------ cases ---

def listed():
    return [
        # the norm before a block for one token of one chat: latency is all there is
        dict(name="norm_token", op="norm", T=1, heads=0, H=2048, dtype="bf16", residual=True, mxfp8=False),
        # a decode batch whose next projection takes MXFP8
        dict(name="norm_batch_mxfp8", op="norm", T=200, heads=0, H=4096, dtype="bf16", residual=True, mxfp8=True),
        # prompts of a few thousand tokens each
        dict(name="norm_prompts", op="norm", T=16384, heads=0, H=2048, dtype="bf16", residual=True, mxfp8=False),
        # the new token of each of 32 sequences: 32 query heads, 4 key heads
        dict(name="rotate_batch32", op="rotate", B=32, lo=300, hi=8192, q_lo=1, q_hi=1, hq=32, hkv=4, D=128, R=128, P=64,
             layers=2, paired=False, dtype="bf16"),
        # drafts of 1 to 5 tokens, half of each head rotated, neighbouring channels as pairs
        dict(name="rotate_drafts", op="rotate", B=24, lo=777, hi=3333, q_lo=1, q_hi=5, hq=24, hkv=8, D=64, R=32, P=32,
             layers=1, paired=True, dtype="fp16"),
        # eight prompts of a few thousand tokens each
        dict(name="rotate_prompts", op="rotate", B=8, lo=1500, hi=4096, q_lo=1500, q_hi=4096, hq=32, hkv=4, D=128, R=128,
             P=64, layers=1, paired=False, dtype="bf16"),
        # the decode batch of the MoE layer's benchmark: 128 experts, 8 of them for a token
        dict(name="route_batch32", op="route", T=32, E=128, K=8, scores="softmax", bias=False, groups=1, top=1, best=1,
             renormalise=True, dtype="bf16"),
        # many experts in groups, chosen with a bias that balances them
        dict(name="route_groups", op="route", T=1000, E=256, K=8, scores="sigmoid", bias=True, groups=8, top=4, best=2,
             renormalise=True, dtype="fp32"),
        # the same layer's prompts
        dict(name="route_prompts", op="route", T=16384, E=128, K=8, scores="softmax", bias=False, groups=1, top=1, best=1,
             renormalise=True, dtype="bf16"),
        # one chat of some hundred tokens
        dict(name="logits_one", op="logits", B=1, V=32768, lo=517, hi=517, biases=8, mask=False, dtype="bf16", out="fp32"),
        # a vocabulary of an odd size, one row in a grammar or another
        dict(name="logits_grammar", op="logits", B=7, V=100003, lo=40, hi=32768, biases=300, mask=True, dtype="fp32",
             out="fp32"),
        # a decode batch of requests of many lengths
        dict(name="logits_batch64", op="logits", B=64, V=131072, lo=300, hi=8192, biases=20, mask=True, dtype="bf16",
             out="fp32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "rotate", "route", "logits"])
    if op == "norm":
        mxfp8, dtype = rng.random() < 0.4, rng.choice(["bf16", "bf16", "fp16", "fp32"])
        heads = 0 if mxfp8 else rng.choice([0, 0, 0, rng.randint(1, 32)])
        H = rng.choice([64, 128, 256]) if heads else 32 * _log(rng, 1, 512) if mxfp8 else _log(rng, 8, 16384)
        T = _log(rng, 1, min(65536, 67108864 // (H * max(1, heads) * SIZES[dtype])))
        return dict(op=op, T=T, heads=heads, H=H, dtype=dtype, residual=not heads and rng.random() < 0.7, mxfp8=mxfp8)
    if op == "rotate":
        D, hkv = rng.choice([64, 128, 128, 256]), rng.choice([1, 2, 4, 8])
        hq, dtype = hkv * rng.choice([1, 2, 3, 4, 5, 8]), rng.choice(["bf16", "bf16", "fp16", "fp32"])
        B = _log(rng, 1, 128)
        q_hi = rng.choice([1, 1, _log(rng, 1, max(2, 160000000 // (B * (hq + 2 * hkv) * D * SIZES[dtype])))])
        return dict(op=op, B=B, lo=q_hi, hi=q_hi + _log(rng, 1, 5000), q_lo=_log(rng, 1, q_hi), q_hi=q_hi, hq=hq, hkv=hkv,
                    D=D, R=rng.choice([D, D, D // 2, D // 4]), P=rng.choice([16, 32, 64, 128]), layers=rng.choice([1, 2, 3]),
                    paired=rng.choice([False, False, True]), dtype=dtype)
    if op == "route":
        groups, scores = rng.choice([1, 1, 1, 2, 4, 8]), rng.choice(["softmax", "sigmoid"])
        E = groups * _log(rng, 8, 512 // groups)
        top = rng.randint(1, groups)
        return dict(op=op, T=_log(rng, 1, 16384), E=E, K=rng.randint(1, min(12, top * (E // groups))), scores=scores,
                    bias=rng.random() < 0.4, groups=groups, top=top, best=rng.choice([1, 2]),
                    renormalise=rng.random() < 0.7, dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]))
    V = _log(rng, 1000, 262144)
    B = _log(rng, 1, max(2, min(128, 8388608 // V)))
    hi = _log(rng, 2, 32768)
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    return dict(op=op, B=B, V=V, lo=_log(rng, 1, hi), hi=hi, biases=rng.choice([0, _log(rng, 1, 300)]),
                mask=rng.random() < 0.5, dtype=dtype, out=rng.choice([dtype, "fp32"]))


def _spread(lo, hi, n, seed):
    """n whole numbers from lo to hi, even on a logarithm's scale, in a shuffled order."""
    t = np.linspace(0.0, 1.0, n) if n > 1 else np.ones(1)
    v = np.round(np.exp(math.log(lo) + t * (math.log(hi) - math.log(lo)))).astype(np.int64)
    return np.random.RandomState(seed).permutation(v)


def _ragged(c):
    """Lengths and numbers of new tokens of a batch's sequences: they go by the case alone."""
    lens = _spread(c["lo"], c["hi"], c["B"], c["hi"])
    return lens, np.minimum(_spread(c["q_lo"], c["q_hi"], c["B"], 7), lens)


def work(c):
    size = SIZES[c["dtype"]]
    if c["op"] == "norm":
        n = c["T"] * max(1, c["heads"]) * c["H"]
        out = 1 + 1 / 32 if c["mxfp8"] else size
        return {"bytes": n * (size * (3 if c["residual"] else 1) + out) + size * c["H"], "flops": 5.0 * n}
    if c["op"] == "rotate":
        lens, news = _ragged(c)
        D, hkv, tokens = c["D"], c["hkv"], int(news.sum())
        rows = len(np.unique(np.concatenate([np.arange(a - b, a) for a, b in zip(lens.tolist(), news.tolist())])))
        cache = 2 * (D // 2 + D // 32)
        return {"bytes": tokens * (2 * size * D * c["hq"] + hkv * (4 * size * D + cache)) + 4 * c["R"] * rows,
                "flops": tokens * (3.0 * c["R"] * (c["hq"] + hkv) + 4.0 * D * hkv)}
    if c["op"] == "route":
        return {"bytes": c["T"] * (c["E"] * size + 8 * c["K"]) + 4 * c["E"] * c["bias"], "flops": 4.0 * c["T"] * c["E"]}
    n, lens = c["B"] * c["V"], _spread(c["lo"], c["hi"], c["B"], 3)
    return {"bytes": n * (size + SIZES[c["out"]]) + n // 8 * c["mask"] + 4 * int(lens.sum()) + 8 * c["B"] * c["biases"],
            "flops": 2.0 * n}


# ---------------------------------------------------------------- prepare ---

def _generator(seed):
    return torch.Generator(device=DEVICE).manual_seed(int(seed) * 2 + 1)


def _device(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEVICE)


def prepare(c, seed):
    g, r = _generator(seed), np.random.RandomState(int(seed) % (1 << 31))
    return {"norm": _prepare_norm, "rotate": _prepare_rotate, "route": _prepare_route, "logits": _prepare_logits}[c["op"]](c, g, r)


def _randn(shape, g, dtype=torch.float32):
    return torch.randn(shape, generator=g, device=DEVICE).to(dtype)


def _prepare_norm(c, g, r):
    """What a block adds, a residual with some channels far larger than others, and the norm's weights."""
    T, H, dtype = c["T"], c["H"], DTYPES[c["dtype"]]
    s = dict(c=c, weight=(1 + 0.2 * _randn((H,), g)).to(dtype), residual=None)
    if c["heads"]:  # the queries' part of the fused projection's rows
        width = (c["heads"] + 2) * H
        s["x"] = _randn((T, width), g, dtype)[:, :c["heads"] * H].unflatten(1, (c["heads"], H))
    else:
        s["x"] = _randn((T, H), g, dtype)
    if c["residual"]:
        gain = torch.exp(_randn((H,), g)) * 3
        s["residual"] = (_randn((T, H), g) * gain).to(dtype)
    return s


def _prepare_rotate(c, g, r):
    D, P, hkv = c["D"], c["P"], c["hkv"]
    lens, news = _ragged(c)
    need = -(-lens // P)
    pages = int(need.sum()) + 3
    order, at = r.permutation(pages), 0
    table, refs = np.full((c["B"], int(need.max()) + 1), -1, np.int32), np.zeros(pages, np.int32)
    slots, lengths = r.permutation(c["B"]), np.empty(c["B"], np.int32)  # entry b is the sequence in slot slots[b]
    for b, n in enumerate(need.tolist()):
        table[slots[b], :n] = order[at:at + n]
        refs[order[at:at + n]] = 1
        lengths[slots[b]] = lens[b]
        at += n
    start = np.concatenate(([0], np.cumsum(news))).astype(np.int32)
    pool = torch.zeros(pages, c["layers"], hkv, P // 16, 16 * (D + 2 * (D // 32)), dtype=torch.uint8, device=DEVICE)
    # the angles of all positions that the model was made for, cosines and then sines of a position's channels
    frequency = 10000.0 ** (-torch.arange(0, c["R"], 2, device=DEVICE, dtype=torch.float64) / c["R"])
    angle = torch.arange(int(lens.max()), device=DEVICE, dtype=torch.float64)[:, None] * frequency
    s = dict(c=c, pool=pool, table=_device(table), lengths=_device(lengths), refs=_device(refs),
             seqs=_device(slots.astype(np.int32)), layer=c["layers"] - 1, q_start=_device(start) if int(news.max()) > 1 else None,
             cos_sin=torch.cat((angle.cos(), angle.sin()), 1).float(),
             qkv=_randn((int(start[-1]), (c["hq"] + 2 * hkv) * D), g, DTYPES[c["dtype"]]))
    if own:
        import moe_decode_gate_gb300 as wd

        s["cache"] = wd.KVCache.from_buffers(pool, s["table"], s["lengths"], s["refs"], layers=c["layers"], kv_heads=hkv,
                                             head_dim=D, page_size=P)
    return s


def _prepare_route(c, g, r):
    s = dict(c=c, logits=(1.5 * _randn((c["T"], c["E"]), g)).to(DTYPES[c["dtype"]]), bias=None)
    if c["bias"]:
        s["bias"] = 0.1 * _randn((c["E"],), g)
    return s


def _prepare_logits(c, g, r):
    """Tokens so far (common ones many times), the requests' settings, and which tokens a grammar allows next."""
    B, V = c["B"], c["V"]
    lens = _spread(c["lo"], c["hi"], B, 3)
    columns = int(lens.max()) + 5
    u = torch.rand(B, columns, generator=g, device=DEVICE)
    s = dict(c=c, logits=(3 * _randn((B, V), g)).to(DTYPES[c["dtype"]]), seqs=_device(r.permutation(B).astype(np.int32)),
             history=(u ** 4 * V).int().clamp(max=V - 1))
    slots = s["seqs"].cpu().numpy()
    lengths, prompts = np.empty(B, np.int32), np.empty(B, np.int32)
    lengths[slots] = lens
    prompts[slots] = (lens * r.uniform(0.1, 1.0, B)).astype(np.int32)
    s["lengths"], s["prompts"] = _device(lengths), _device(prompts)
    for name, lo, hi in (("repetition", 1.0, 1.3), ("presence", -0.5, 1.5), ("frequency", 0.0, 0.5), ("temperature", 0.3, 1.5)):
        s[name] = lo + (hi - lo) * torch.rand(B, generator=g, device=DEVICE)
    s["bias"] = s["mask"] = None
    if c["biases"]:
        n = min(c["biases"], V)
        ids = ((torch.arange(n, device=DEVICE) + torch.rand(B, n, generator=g, device=DEVICE).double()) * (V / n)).int()
        s["bias"] = (_device(np.arange(B + 1, dtype=np.int32) * n), ids.clamp(max=V - 1).flatten(), 2 * _randn((B * n,), g))
    if c["mask"]:  # one row of two is in a grammar that allows a token of 16
        words = -(-V // 32)
        bits = torch.full((B, words), -1, dtype=torch.int32, device=DEVICE)
        few = torch.randint(-2 ** 31, 2 ** 31, (4, B, words), generator=g, device=DEVICE).int()
        few = few[0] & few[1] & few[2] & few[3]
        s["mask"] = torch.where((torch.arange(B, device=DEVICE) % 2 == 0)[:, None], few, bits)
    return s


# -------------------------------------------------------------------- run ---

def run(s):
    return {"norm": _run_norm, "rotate": _run_rotate, "route": _run_route, "logits": _run_logits}[s["c"]["op"]](s)


def _run_norm(s):
    c = s["c"]
    if own:
        import moe_decode_gate_gb300 as wd

        got = wd.rms_norm(s["x"], s["weight"], s["residual"], eps=EPS, mxfp8=c["mxfp8"])
        got = got if isinstance(got, tuple) else (got,)
    else:
        got = _plain_norm(s)
    if c["mxfp8"]:
        out = {"codes": got[0].view(torch.float8_e4m3fn), "scales": got[1].view(torch.float8_e8m0fnu)}
    else:
        out = {"y": got[0]}
    if c["residual"]:
        out["residual"] = got[-1]
    return out


def _plain_norm(s):
    c, dtype = s["c"], s["x"].dtype
    r = s["x"].float()
    if c["residual"]:
        r = r + s["residual"].float()
    y = r * torch.rsqrt((r * r).mean(-1, keepdim=True) + EPS) * s["weight"].float()
    tail = (r.to(dtype),) if c["residual"] else ()
    if not c["mxfp8"]:
        return (y.to(dtype), *tail)
    b = y.unflatten(-1, (-1, 32))
    a = b.abs().amax(-1, keepdim=True)
    e = torch.where(a == 0, 0, (torch.frexp(a)[1] - 9).clamp(-127, 127))
    # E4M3 by hand: a step of 2^-3 of the value's power of two, 2^-9 at least, 448 at most
    z = torch.ldexp(torch.ldexp(b, -e // 2), -e - (-e // 2))
    step = (torch.frexp(z)[1] - 4).clamp(min=-9)
    z = torch.ldexp(torch.round(torch.ldexp(z, -step)), step).clamp(-448, 448)
    return (z.to(torch.float8_e4m3fn).flatten(-2).view(torch.uint8), (e + 127).to(torch.uint8).squeeze(-1), *tail)


def _run_rotate(s):
    c = s["c"]
    hq, hkv, D = c["hq"], c["hkv"], c["D"]
    q, k, v = s["qkv"].split((hq * D, hkv * D, hkv * D), 1)
    q, k, v = q.unflatten(1, (hq, D)), k.unflatten(1, (hkv, D)), v.unflatten(1, (hkv, D))
    if own:
        q, k, v = s["cache"].append_rotated(s["layer"], q, k, v, s["cos_sin"], seqs=s["seqs"], q_start=s["q_start"],
                                            paired=c["paired"], return_values=True)
    else:
        q, k, v = _plain_rotate(s, q, k, v)
    return {"q": q, "k": k, "v": v, "pool": s["pool"]}


def _rotated(x, cos, sin, paired):
    """x [T, heads, D] fp32; cos, sin [T, 1, R / 2]."""
    R = 2 * cos.shape[-1]
    a, b = (x[..., 0:R:2], x[..., 1:R:2]) if paired else (x[..., :R // 2], x[..., R // 2:R])
    y, z = a * cos - b * sin, b * cos + a * sin
    y = torch.stack((y, z), -1).flatten(-2) if paired else torch.cat((y, z), -1)
    return torch.cat((y, x[..., R:]), -1)


def _places(s, tokens):
    """For each new token: its entry of the batch, and its position in that entry's sequence."""
    at = torch.arange(tokens, device=s["pool"].device)
    if s["q_start"] is None:
        b, row, n = at, torch.zeros_like(at), torch.ones_like(at)
    else:
        start = s["q_start"].long()
        b = torch.searchsorted(start, at, right=True) - 1
        row, n = at - start[b], start[b + 1] - start[b]
    return b, s["lengths"][s["seqs"].long()].long()[b] - n + row


def _plain_rotate(s, q, k, v):
    c, pool = s["c"], s["pool"]
    D, P, layer, dtype = c["D"], c["P"], s["layer"], q.dtype
    b, pos = _places(s, q.shape[0])
    cos, sin = s["cos_sin"][pos][:, None].chunk(2, -1)
    q, k = _rotated(q.float(), cos, sin, c["paired"]), _rotated(k.float(), cos, sin, c["paired"])
    page = s["table"][s["seqs"].long()[b], pos // P].long()
    group, token = pos % P // 16, pos % 16
    kc, ks = _quantise(k)
    vc, vs = _quantise(v.float())
    nb, half = min(4, D // 32), 8 * D
    ns = D // 32 // nb
    rows = pool[..., :half].unflatten(-1, (ns, 16, 16 * nb))
    kb = _bytes(kc.unflatten(-1, (ns, nb, 4, 8)).movedim(-2, -3)).flatten(-3)  # [T, hkv, ns, 16 nb]
    rows[page, layer, :, group, :, token] = kb
    rows = pool[..., half:2 * half].unflatten(-1, (ns, 2, 8, 4, 2, 2 * nb))
    vb = _bytes(vc.unflatten(-1, (ns, nb, 8, 4)).movedim(-2, -3)).flatten(-2)  # [T, hkv, ns, 8, 2 nb]
    rows[page, layer, :, group, :, token // 8, :, token % 8 // 2, token % 2] = vb
    rows = pool[..., 2 * half:].unflatten(-1, (2, 16, D // 32))
    rows[page, layer, :, group, 0, token] = ks
    rows[page, layer, :, group, 1, token] = vs
    return q.to(dtype), _value_of(kc, ks).to(dtype), _value_of(vc, vs).to(dtype)


def _quantise(x):
    """x [..., D] fp32 -> codes uint8 [..., D] (one to a byte), scales uint8 [..., D / 32]."""
    b = x.unflatten(-1, (-1, 32))
    a = b.abs().amax(-1, keepdim=True)
    e = torch.where(a == 0, 0, (torch.frexp(a)[1] - 3).clamp(-127, 127))
    y = torch.ldexp(torch.ldexp(b.abs(), -e // 2), -e - (-e // 2))
    # the values between 0, .5, 1, 1.5, 2, 3, 4, 6: a tie goes to the even code
    code = ((y > 0.25).to(torch.uint8) + (y >= 0.75) + (y > 1.25) + (y >= 1.75) + (y > 2.5) + (y >= 3.5) + (y > 5.0))
    return (code + 8 * torch.signbit(b)).to(torch.uint8).flatten(-2), (e + 127).to(torch.uint8).squeeze(-1)


def _value_of(code, scale):
    """codes [..., D], scales [..., D / 32] -> fp32 [..., D]."""
    m = (code & 7).to(torch.float32)
    v = torch.where(m < 4, m * 0.5, torch.where(m < 6, m - 2, 2 * m - 8))
    v = torch.where(code >= 8, -v, v).unflatten(-1, (-1, 32))
    e = (scale.to(torch.int32) - 127).unsqueeze(-1)
    return torch.ldexp(torch.ldexp(v, e // 2), e - e // 2).flatten(-2)


def _bytes(nibbles):
    return nibbles[..., 0::2] | (nibbles[..., 1::2] << 4)


def _run_route(s):
    c = s["c"]
    if own:
        import moe_decode_gate_gb300 as wd

        ids, weights = wd.route(s["logits"], c["K"], scores=c["scores"], bias=s["bias"], groups=c["groups"],
                                top_groups=c["top"], group_best=c["best"], renormalise=c["renormalise"], scale=1.0)
    else:
        ids, weights = _plain_route(s)
    return {"ids": ids, "weights": weights}


def _plain_route(s):
    """Keys in 64 bits: two of them may be nearer to each other than 32 bits tell."""
    c, x = s["c"], s["logits"].double()
    score = torch.sigmoid(x) if c["scores"] == "sigmoid" else torch.exp(x - x.amax(-1, keepdim=True))
    if c["scores"] == "softmax":
        score = score / score.sum(-1, keepdim=True)
    key = score + s["bias"].double() if c["bias"] else score
    # where nothing is added the scores stand in the logits' order, ties and all
    order = key if c["bias"] else x
    if c["groups"] > 1:
        size = c["E"] // c["groups"]
        if c["best"] == 2 and size > 1:
            of_group = key.unflatten(-1, (c["groups"], size)).topk(2).values.sum(-1)
        else:
            of_group = order.unflatten(-1, (c["groups"], size)).amax(-1)
        chosen = torch.argsort(of_group, dim=-1, descending=True, stable=True)[:, :c["top"]]
        inside = torch.zeros_like(of_group, dtype=torch.bool).scatter_(1, chosen, True)
        order = torch.where(inside.repeat_interleave(size, 1), order, -math.inf)
    ids = torch.argsort(order, dim=-1, descending=True, stable=True)[:, :c["K"]]
    weights = score.gather(1, ids)
    if c["renormalise"]:
        weights = weights / weights.sum(-1, keepdim=True)
    return ids.int(), weights.float()


def _run_logits(s):
    c = s["c"]
    if own:
        import moe_decode_gate_gb300 as wd

        return wd.adjust_logits(s["logits"], history=s["history"], lengths=s["lengths"], prompt_lengths=s["prompts"],
                                seqs=s["seqs"], repetition=s["repetition"], presence=s["presence"], frequency=s["frequency"],
                                bias=s["bias"], temperature=s["temperature"], mask=s["mask"], dtype=DTYPES[c["out"]])
    return _plain_logits(s)


def _plain_logits(s):
    c, x = s["c"], s["logits"].float()
    B, V = x.shape
    rows = s["seqs"].long()
    tokens = s["history"][rows].long()
    at = torch.arange(tokens.shape[1], device=x.device)
    there, prompt = at < s["lengths"][rows][:, None], at < s["prompts"][rows][:, None]
    seen = torch.zeros(B, V, dtype=torch.int32, device=x.device).scatter_add_(1, tokens, there.int())
    count = torch.zeros(B, V, dtype=torch.int32, device=x.device).scatter_add_(1, tokens, (there & ~prompt).int())
    p = s["repetition"][:, None]
    x = torch.where(seen > 0, torch.where(x > 0, x / p, x * p), x)
    x = x - (count * s["frequency"][:, None] + (count > 0) * s["presence"][:, None])
    if s["bias"] is not None:
        start, ids, values = s["bias"]
        row = torch.searchsorted(start.long(), torch.arange(ids.numel(), device=x.device), right=True) - 1
        x = x.index_put((row, ids.long()), values, accumulate=True)
    x = x / s["temperature"][:, None]
    if s["mask"] is not None:
        bit = torch.arange(32, device=x.device, dtype=torch.int32)
        allowed = ((s["mask"][..., None] >> bit) & 1).flatten(1)[:, :V] != 0
        x = torch.where(allowed, x, -math.inf)
    return x.to(DTYPES[c["out"]])


# ------------------------------------------------------------------ exact ---

def exact(c, seed):
    s = prepare(c, seed)
    return {"norm": _exact_norm, "rotate": _exact_rotate, "route": _exact_route, "logits": _exact_logits}[c["op"]](c, s)


def _exact_norm(c, s):
    total = s["x"].double() + (s["residual"].double() if c["residual"] else 0.0)
    y = total / torch.sqrt(torch.linalg.vector_norm(total, dim=-1, keepdim=True) ** 2 / c["H"] + EPS) * s["weight"].double()
    out = {"residual": total} if c["residual"] else {}
    if not c["mxfp8"]:
        return {"y": y, **out}
    b = y.reshape(c["T"], -1, 32)
    top = b.abs().amax(-1, keepdim=True)
    unit = torch.where(top > 0, torch.exp2(torch.floor(torch.log2(top)) - 8), 1.0)
    # the values that E4M3 has, the one with the even mantissa where two are as near
    grid = torch.tensor([m * 2.0 ** -9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:-1],
                        device=y.device, dtype=torch.float64)
    z = (b / unit).abs().clamp(max=448.0)
    up = torch.bucketize(z, grid).clamp(1, grid.numel() - 1)
    above, below = grid[up] - z, z - grid[up - 1]
    code = torch.where((above < below) | ((above == below) & (up % 2 == 0)), up, up - 1)
    return {"codes": (torch.sign(b) * grid[code]).reshape(c["T"], -1), "scales": unit.squeeze(-1), **out}


def _exact_rotate(c, s):
    hq, hkv, D, R = c["hq"], c["hkv"], c["D"], c["R"]
    lens, news = _ragged(c)
    pos = torch.cat([torch.arange(int(a - b), int(a)) for a, b in zip(lens, news)]).to(DEVICE)
    x = s["qkv"].double().reshape(pos.numel(), hq + 2 * hkv, D)
    ch = torch.arange(R, device=DEVICE)
    i, first, other = (ch // 2, ch % 2 == 0, ch ^ 1) if c["paired"] else (ch % (R // 2), ch < R // 2, (ch + R // 2) % R)
    turn = s["cos_sin"].double()[pos]
    cos, sin = turn[:, i][:, None], turn[:, R // 2 + i][:, None]
    y = x.clone()
    y[..., :R] = x[..., :R] * cos + torch.where(first, -1.0, 1.0) * x[..., other] * sin
    b = torch.cat((y[:, hq:hq + hkv], x[:, hq + hkv:]), 1).unflatten(-1, (-1, 32))
    top = b.abs().amax(-1, keepdim=True)
    unit = torch.where(top > 0, torch.exp2(torch.floor(torch.log2(top)) - 2), 1.0)
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=DEVICE, dtype=torch.float64)
    z = (b / unit).abs().clamp(max=6.0)
    up = torch.bucketize(z, grid).clamp(1, 7)
    above, below = grid[up] - z, z - grid[up - 1]
    code = torch.where((above < below) | ((above == below) & (up % 2 == 0)), up, up - 1)
    held = (torch.sign(b) * grid[code] * unit).flatten(-2)
    return {"q": y[:, :hq], "k": held[:, :hkv], "v": held[:, hkv:], "pool": None}


def _exact_route(c, s):
    x = s["logits"].double().cpu().numpy()
    if c["scores"] == "sigmoid":
        score = 1.0 / (1.0 + np.exp(-x))
    else:
        e = np.exp(x - x.max(1, keepdims=True))
        score = e / e.sum(1, keepdims=True)
    by = score + s["bias"].double().cpu().numpy() if c["bias"] else x
    key = score + s["bias"].double().cpu().numpy() if c["bias"] else score
    size = c["E"] // c["groups"]
    if c["groups"] > 1:
        inside = np.sort((key if c["best"] == 2 and size > 1 else by).reshape(-1, c["groups"], size), 2)
        rank = inside[:, :, -2:].sum(2) if c["best"] == 2 and size > 1 else inside[:, :, -1]
        place = np.argsort(np.argsort(-rank, 1, kind="stable"), 1, kind="stable")
        by = np.where(np.repeat(place < c["top"], size, 1), by, -np.inf)
    ids = np.argsort(-by, 1, kind="stable")[:, :c["K"]]
    w = np.take_along_axis(score, ids, 1)
    if c["renormalise"]:
        w = w / w.sum(1, keepdims=True)
    return {"ids": None, "weights": w}


def _exact_logits(c, s):
    V, out = c["V"], []
    setting = {n: s[n].double().cpu().numpy() for n in ("repetition", "presence", "frequency", "temperature")}
    slots, lens, prompts = (s[n].cpu().numpy() for n in ("seqs", "lengths", "prompts"))
    tokens = s["history"].cpu().numpy()
    bias = None if s["bias"] is None else [t.cpu().numpy() for t in s["bias"]]
    for b in range(c["B"]):
        x = s["logits"][b].double().cpu().numpy()
        t = tokens[slots[b]]
        n, m = int(lens[slots[b]]), int(prompts[slots[b]])
        seen = np.unique(t[:n])
        x[seen] = np.where(x[seen] > 0, x[seen] / setting["repetition"][b], x[seen] * setting["repetition"][b])
        given, times = np.unique(t[m:n], return_counts=True)
        x[given] -= setting["frequency"][b] * times + setting["presence"][b]
        if bias is not None:
            part = slice(bias[0][b], bias[0][b + 1])
            x[bias[1][part]] += bias[2][part].astype(np.float64)
        x = x / setting["temperature"][b]
        if s["mask"] is not None:
            words = s["mask"][b].cpu().numpy().view(np.uint32)
            bits = np.unpackbits(words.view(np.uint8), bitorder="little")[:V]
            x = np.where(bits == 1, x, -np.inf)
        out.append(x)
    return np.stack(out)
