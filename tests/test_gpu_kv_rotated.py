"""KVCache.append_rotated on the GPU against the plain reference (tests/step_reference.py, tests/kv_reference.py).

The rotation's products and sums are rounded to FP32 one by one, so everything is compared bit by bit: queries, the
values that the cache holds, and the bytes of its pages.
"""
import numpy as np
import pytest
import torch

import kv_reference as ref
import moe_decode_gate_gb300 as wd
import step_reference as step

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
FLAG = wd.KV_FLAG_BAD_INDEX


class Batch:
    def __init__(self, dev, lens, news, hq, hkv, D, P, R, dtype, layers=1, seed=0, paired=False, positions=None):
        r = np.random.RandomState(seed)
        B, need = len(lens), -(-np.asarray(lens) // P)
        pages = int(need.sum()) + 2
        order, at = r.permutation(pages), 0
        self.table = np.full((B + 1, max(1, int(need.max())) + 1), -1, np.int32)
        self.lengths, self.slots = np.zeros(B + 1, np.int32), r.permutation(B + 1)[:B]
        for b in range(B):
            self.table[self.slots[b], :need[b]] = order[at:at + need[b]]
            self.lengths[self.slots[b]] = lens[b]
            at += need[b]
        self.start = np.concatenate(([0], np.cumsum(news)))
        self.pos = np.concatenate([np.arange(L - n, L) for L, n in zip(lens, news)]).astype(int)
        self.of = np.repeat(np.arange(B), news)
        T = int(self.start[-1])
        self.pool = r.randint(0, 256, (pages, layers, hkv, P // 16, ref.group_bytes(D))).astype(np.uint8)
        self.qkv = torch.from_numpy(r.standard_normal((T, (hq + 2 * hkv) * D)) * np.exp(r.standard_normal((T, 1)))).to(dtype)
        self.cos_sin = wd.rotation_table(positions or max(1, max(lens)), R, device="cpu").numpy()
        self.dev, self.hq, self.hkv, self.D, self.P, self.paired, self.layer = dev, hq, hkv, D, P, paired, layers - 1
        refs = np.zeros(pages, np.int32)
        refs[order[:at]] = 1
        d = self.device
        self.cache = wd.KVCache.from_buffers(d(self.pool), d(self.table), d(self.lengths), d(refs), layers=layers, kv_heads=hkv,
                                             head_dim=D, page_size=P)

    def device(self, a):
        return torch.from_numpy(np.ascontiguousarray(a)).to(self.dev)

    def parts(self):
        q, k, v = self.qkv.to(self.dev).split((self.hq * self.D, self.hkv * self.D, self.hkv * self.D), 1)
        return (q.unflatten(1, (self.hq, self.D)), k.unflatten(1, (self.hkv, self.D)), v.unflatten(1, (self.hkv, self.D)))

    def single(self):
        return bool((np.diff(self.start) == 1).all())

    def run(self, q, k, v, **kw):
        return self.cache.append_rotated(
            self.layer, q, k, v, self.device(self.cos_sin), self.device(self.slots.astype(np.int32)),
            None if self.single() else self.device(self.start.astype(np.int32)), paired=self.paired, return_values=True, **kw)

    def check(self, got, skipped=(), flag=0):
        hq, hkv, D, P = self.hq, self.hkv, self.D, self.P
        x = self.qkv.float().numpy().reshape(-1, hq + 2 * hkv, D)
        keep = [t for t in range(x.shape[0]) if t not in set(skipped)]
        q = np.zeros((x.shape[0], hq, D), np.float32)
        k = np.zeros((x.shape[0], hkv, D), np.float32)
        q[keep] = step.rotate(x[keep, :hq], self.cos_sin, self.pos[keep], self.paired)
        k[keep] = step.rotate(x[keep, hq:hq + hkv], self.cos_sin, self.pos[keep], self.paired)
        (kc, ks), (vc, vs) = ref.quantise(k.astype(np.float64)), ref.quantise(x[:, hq + hkv:].astype(np.float64))
        want = self.pool.copy()
        for t in keep:
            page = self.table[self.slots[self.of[t]], self.pos[t] // P]
            for h in range(hkv):
                ref.store(want, page, self.layer, h, self.pos[t] % P, D, kc[t, h], ks[t, h], vc[t, h], vs[t, h])
        assert np.array_equal(self.cache.pool.cpu().numpy(), want)
        dtype = self.qkv.dtype
        for g, w in zip(got, (torch.from_numpy(q), torch.from_numpy(ref.values(kc, ks)), torch.from_numpy(ref.values(vc, vs)))):
            if g is not None:
                g, w = g[keep].cpu(), w.to(dtype)[keep]
                assert torch.equal(g.isnan(), w.isnan()) and torch.equal(g[~g.isnan()], w[~w.isnan()])
        assert self.cache.read_error_flag() == flag


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("paired", [False, True])
@pytest.mark.parametrize("D,R", [(64, 64), (64, 16), (64, 48), (128, 128), (128, 64), (128, 32), (128, 112), (256, 256), (256, 64)])
def test_forms(D, R, paired, dtype, cuda_device):
    b = Batch(cuda_device, [1, 40, 33, 17], [1, 3, 20, 17], 6, 2, D, 16, R, dtype, layers=2, paired=paired)
    b.check(b.run(*b.parts()))


@pytest.mark.parametrize("hq,hkv", [(1, 1), (8, 8), (32, 4), (5, 5), (70, 7), (48, 48), (24, 3)])
@pytest.mark.parametrize("D", [64, 256])
def test_heads(hq, hkv, D, cuda_device):
    b = Batch(cuda_device, [70, 5, 64], [1, 1, 1], hq, hkv, D, 32, D, BF16)
    b.check(b.run(*b.parts()))
    b = Batch(cuda_device, [70, 5, 64], [33, 2, 64], hq, hkv, D, 32, D // 2, FP16, seed=1)
    b.check(b.run(*b.parts()))


@pytest.mark.parametrize("shift", [0, 1, 4])
def test_rows_that_are_not_aligned(shift, cuda_device):
    b = Batch(cuda_device, [9, 30], [9, 4], 4, 2, 64, 16, 64, BF16)
    wide = torch.zeros(13, b.qkv.shape[1] + 5, dtype=BF16)
    wide[:, shift:shift + b.qkv.shape[1]] = b.qkv
    x = wide.to(cuda_device)[:, shift:shift + b.qkv.shape[1]]
    q, k, v = x.split((256, 128, 128), 1)
    b.check(b.run(q.unflatten(1, (4, 64)), k.unflatten(1, (2, 64)), v.unflatten(1, (2, 64))))


def test_heads_first(cuda_device):
    """Tensors whose heads are the slower dimension."""
    b = Batch(cuda_device, [9, 30], [9, 4], 4, 2, 128, 16, 128, BF16)
    q, k, v = (t.transpose(0, 1).contiguous().transpose(0, 1) for t in b.parts())
    b.check(b.run(q, k, v))


def test_many_tokens(cuda_device):
    b = Batch(cuda_device, [700, 1300, 64], [650, 1300, 1], 8, 2, 64, 64, 32, BF16)
    b.check(b.run(*b.parts()))


def test_queries_in_place_and_left_out(cuda_device):
    b = Batch(cuda_device, [20, 4], [7, 1], 4, 2, 64, 16, 64, BF16)
    q, k, v = b.parts()
    q = q.contiguous()
    got = b.run(q, k, v, q_out=q)
    assert got[0] is q
    b.check(got)
    b = Batch(cuda_device, [20, 4], [7, 1], 4, 2, 64, 16, 64, BF16)
    _, k, v = b.parts()
    got = b.run(None, k, v)
    assert got[0] is None
    b.check(got)


def test_no_rotation_is_append(cuda_device):
    """Cosines of 1 and sines of 0: the pages of wd_kv_append, and the queries as they are."""
    b = Batch(cuda_device, [50, 9, 31], [50, 1, 8], 4, 2, 128, 16, 128, BF16)
    b.cos_sin[:, :64], b.cos_sin[:, 64:] = 1.0, 0.0
    q, k, v = b.parts()
    got = b.run(q, k, v)
    b.check(got)
    pool = b.cache.pool.clone()
    b.cache.append(0, k, v, b.device(b.slots.astype(np.int32)), b.device(b.start.astype(np.int32)))
    assert torch.equal(b.cache.pool, pool) and torch.equal(got[0], q)


def test_positions_that_the_table_does_not_have(cuda_device):
    b = Batch(cuda_device, [40, 10], [6, 10], 4, 2, 64, 16, 64, BF16, positions=37)
    late = [t for t in range(16) if b.pos[t] >= 37]
    assert late == [3, 4, 5]
    b.check(b.run(*b.parts()), skipped=late, flag=FLAG)


def test_pages_and_slots_out_of_range(cuda_device):
    b = Batch(cuda_device, [40, 10, 20], [6, 10, 2], 4, 2, 64, 16, 64, BF16)
    b.cache.table[int(b.slots[0]), 2] = 10 ** 6
    parts = b.parts()
    before = b.cache.pool.clone()
    q = b.run(*parts)[0]
    torch.cuda.synchronize()
    want = step.rotate(b.qkv.float().numpy().reshape(-1, 8, 64)[:, :4], b.cos_sin, b.pos, False)
    assert torch.equal(q.cpu(), torch.from_numpy(want).to(BF16))  # the positions are there, only pages are not
    assert b.cache.read_error_flag() == FLAG
    page = int(b.table[int(b.slots[0]), 2])
    assert torch.equal(b.cache.pool[page], before[page])
    b.slots[1] = 99
    b.run(*parts)
    assert b.cache.read_error_flag() == FLAG


def test_values_that_are_not_finite(cuda_device):
    b = Batch(cuda_device, [20], [20], 2, 1, 64, 32, 64, FP32)
    b.qkv[3, 130], b.qkv[4, 140], b.qkv[5, 200], b.qkv[6, 2] = float("nan"), float("inf"), -float("inf"), float("nan")
    b.check(b.run(*b.parts()))


def test_tokens_of_no_entry_are_left_alone(cuda_device):
    b = Batch(cuda_device, [20, 30], [5, 6], 4, 2, 64, 16, 64, BF16)
    q, k, v = b.parts()
    more = torch.full((3, *q.shape[1:]), 9.0, dtype=BF16, device=cuda_device)
    out = torch.full((14, 4, 64), 5.0, dtype=BF16, device=cuda_device)
    got = b.run(torch.cat((q, more)), torch.cat((k, more[:, :2])), torch.cat((v, more[:, :2])), q_out=out)
    assert bool((out[11:] == 5).all())
    b.check([t[:11] for t in got])


def test_attention_after_rotation(cuda_device):
    """Two sequences whose tokens stand one position apart have the same differences of positions, and so, but for the
    quantising of their keys, the same attention."""
    dev, D = cuda_device, 128
    r = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn(24, h, D, generator=r).to(dev).bfloat16() for h in (4, 2, 2))
    table = wd.rotation_table(64, D, device=dev)
    outs = []
    for ahead in (0, 1):
        cache = wd.KVCache(8, 1, 4, 1, 2, D, 16, device=dev)
        n = torch.tensor([24], dtype=torch.int32, device=dev)
        start = torch.tensor([0, 24], dtype=torch.int32, device=dev)
        cache.reserve(n)
        turned = cache.append_rotated(0, q, k, v, table[ahead:].contiguous(), None, start)
        outs.append(cache.attention(0, turned, None, start, max_q=24).float())
    # E2M1 keeps a key's channel to a quarter of it at worst, so logits move by some tenths: the outputs stay alike
    assert float((outs[0] - outs[1]).norm() / outs[0].norm()) < 0.3


@pytest.mark.parametrize("rot", [16, 64, 128])
def test_rotation_table(rot, cuda_device):
    t = wd.rotation_table(70000, rot, base=500000.0, device=cuda_device, scale=1.25)
    p = np.array([0, 1, 65535, 65536, 69999])
    f = 500000.0 ** (-np.arange(0, rot, 2) / rot)
    want = 1.25 * np.concatenate((np.cos(p[:, None] * f), np.sin(p[:, None] * f)), 1)
    # angles of 70,000 in 64 bits: 2^-36; the table's rounding 2^-24 of at most 1.25
    assert np.abs(t[torch.from_numpy(p).to(cuda_device)].double().cpu().numpy() - want).max() < 2.0 ** -23
