"""The 4-bit cache on the GPU against the plain 64-bit reference (tests/kv_reference.py).

Tolerances.  Quantising is exact: bytes are compared.  Attention: FP32 sums, probabilities rounded
once to FP16 (unit roundoff 2^-11), the output rounded once to its type (2^-8 for BF16, 2^-11 for
FP16).  So per element |error| <= u_out |want| + (2^-11 + 2^-15) sum_j p_j |v_j| + 2^-20 max|v|,
where 2^-15 covers the FP32 sums (tens of sequential additions, each within 2^-22 of the
magnitudes summed) and the last term probabilities that FP16 flushes.  lse: each logit is within
2^-20 of scale * sum |q||k| (128 to 256 FP32 products and sums), its exponential within 2^-21, the
sum within 2^-18: 1e-5 + 2^-20 max_j scale |q||k_j|.
"""
import numpy as np
import pytest
import torch

import kv_reference as ref
import moe_decode_gate_gb300 as wd

pytestmark = pytest.mark.gpu

ROUNDOFF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def rounded(x, dtype):
    """Host float64 -> tensor of dtype, and the values it stands for."""
    t = torch.from_numpy(np.ascontiguousarray(x)).to(dtype)
    return t, t.double().numpy()


def quantised_pool(r, pages, layers, hkv, P, D, spread=0.5, junk=0xFF):
    """A pool whose groups hold quantised normals; unset groups are `junk` (NaN scales)."""
    shape = (pages, layers, hkv, P // 16, 16, D)
    pool = np.full((pages, layers, hkv, P // 16, ref.group_bytes(D)), junk, np.uint8)
    gain = np.exp(spread * r.standard_normal((hkv, 1, 1, D)))
    k, v, _ = ref._places(D)
    for layer in range(layers):
        for place, x, at in ((k, r.standard_normal(shape[:1] + shape[2:]) * gain, 16 * D),
                             (v, r.standard_normal(shape[:1] + shape[2:]), 16 * D + D // 2)):
            code, scale = ref.quantise(x)
            pool[:, layer][..., place[:, ::2]] = code[..., ::2] | (code[..., 1::2] << 4)
            pool[:, layer][..., at:at + D // 2] = scale.reshape(*scale.shape[:3], -1)
    return pool


def device(a, dev):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dev)


class Case:
    """A batch over a random cache; pages beyond each sequence's end and the tokens after its last
    one hold NaN scales."""

    def __init__(self, dev, lens, news, hq, hkv, D, P, layers=1, dtype=torch.bfloat16, seed=0,
                 spread=0.5, pool=None, q_scale=1.0):
        r = np.random.RandomState(seed)
        B = len(lens)
        self.dev, self.D, self.P, self.layer, self.dtype = dev, D, P, layers - 1, dtype
        lens = np.asarray(lens)
        need = -(-lens // P)
        pages = int(need.sum()) + 2
        order = r.permutation(pages)
        self.slots = r.permutation(B + 1)[:B]
        self.table = np.full((B + 1, max(1, int(need.max()) + 1)), -1, np.int32)
        self.lengths = np.zeros(B + 1, np.int32)
        at = 0
        for b in range(B):
            self.table[self.slots[b], :need[b]] = order[at:at + need[b]]
            self.lengths[self.slots[b]] = lens[b]
            at += need[b]
        self.pool = quantised_pool(r, pages, layers, hkv, P, D, spread) if pool is None else \
            pool(r, pages, layers, hkv, P, D)
        for b in range(B):  # what lies behind a sequence's end is not to be seen
            if lens[b] % P:
                page = self.table[self.slots[b], need[b] - 1]
                for t in range(lens[b] % P, P):
                    n, g = D // 32, t // 16
                    s = 16 * D + (t % 16) * n
                    self.pool[page, :, :, g, s:s + n] = 255
                    self.pool[page, :, :, g, s + 16 * n:s + 17 * n] = 255
        for p in order[at:]:
            self.pool[p] = 0xFF
        self.q_start = np.concatenate(([0], np.cumsum(news))).astype(np.int32)
        self.single = max(news) == 1 and min(news) == 1
        self.q, self.q_values = rounded(
            q_scale * r.standard_normal((int(self.q_start[-1]), hq, D)), dtype)
        refs = np.zeros(pages, np.int32)
        refs[order[:at]] = 1
        self.cache = wd.KVCache.from_buffers(
            device(self.pool, dev), device(self.table, dev), device(self.lengths, dev),
            device(refs, dev), layers=layers, kv_heads=hkv, head_dim=D, page_size=P)
        self.seqs = device(self.slots.astype(np.int32), dev)

    def run(self, q=None, window=0, scale=None, stream=None, **kw):
        return self.cache.attention(
            self.layer, self.q.to(self.dev) if q is None else q, self.seqs,
            None if self.single else device(self.q_start, self.dev), window=window, scale=scale,
            return_lse=True, stream=stream, **kw)

    def check(self, got, window=0, scale=None, flag=0):
        out, lse = got
        torch.cuda.synchronize()
        scale = 1 / np.sqrt(self.D) if scale is None else scale
        want, want_lse, mag = ref.attention(self.pool, self.table, self.lengths, self.layer,
                                            self.q_values, self.slots, self.q_start, self.D, self.P,
                                            scale, window)
        out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        assert np.array_equal(np.isnan(out), np.isnan(want))
        k, v = ref.decode(self.pool[:, self.layer], self.D)
        fine = np.isfinite(want)
        top = float(np.nanmax(np.abs(v))) if np.isfinite(v).any() else 0.0
        tol = ROUNDOFF[self.dtype] * np.abs(want) + (2.0 ** -11 + 2.0 ** -15) * mag + 2.0 ** -20 * top
        err = np.abs(out - want)
        assert (err <= tol)[fine].all(), f"worst {np.nanmax((err / tol)[fine])} of the tolerance"
        assert np.array_equal(np.isneginf(lse), np.isneginf(want_lse))
        seen = np.isfinite(want_lse)
        reach = scale * np.abs(self.q_values).sum(-1).max() * float(np.nanmax(np.abs(k))) \
            if np.isfinite(k).any() else 0
        if seen.any():
            assert np.abs(lse[seen] - want_lse[seen]).max() <= 1e-5 + 2.0 ** -20 * reach
        assert np.array_equal(np.isnan(lse), np.isnan(want_lse))
        assert self.cache.read_error_flag() == flag


LENGTHS = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 100, 255, 256, 257, 300, 511, 513, 777]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (4, 4), (8, 2), (6, 2), (8, 1), (16, 1), (10, 2), (40, 1)])
def test_single_tokens(cuda_device, D, hq, hkv):
    c = Case(cuda_device, LENGTHS, [1] * len(LENGTHS), hq, hkv, D, 16, seed=hq * D)
    c.check(c.run())


@pytest.mark.parametrize("P", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_page_sizes_layers_and_types(cuda_device, P, dtype):
    c = Case(cuda_device, LENGTHS, [1] * len(LENGTHS), 8, 2, 128, P, layers=3, dtype=dtype, seed=P)
    c.check(c.run())


@pytest.mark.parametrize("D,hq,hkv", [(64, 3, 3), (128, 8, 1), (128, 32, 4), (256, 4, 2)])
@pytest.mark.parametrize("window", [0, 1, 5, 32, 50])
def test_several_tokens_and_windows(cuda_device, D, hq, hkv, window):
    # more new tokens than the sequence is long: the first ones see nothing
    lens = [0, 1, 3, 17, 40, 64, 100, 130, 203]
    news = [2, 3, 5, 1, 8, 0, 33, 7, 70]
    c = Case(cuda_device, lens, news, hq, hkv, D, 32, seed=window + D)
    c.check(c.run(window=window), window=window)
    c.check(c.run(window=window, max_q=70), window=window)
    c.check(c.run(window=window, max_q=1), window=window)  # a hint, nothing hangs on it


@pytest.mark.parametrize("window", [1, 31, 32, 33, 200])
def test_windows_of_single_tokens(cuda_device, window):
    c = Case(cuda_device, LENGTHS, [1] * len(LENGTHS), 4, 2, 128, 64, seed=window)
    c.check(c.run(window=window), window=window)


@pytest.mark.parametrize("B,L,D", [(1, 40001, 128), (3, 9000, 64), (2, 5003, 256), (70, 300, 128)])
def test_sequences_split_over_many_ctas(cuda_device, B, L, D):
    lens = [max(1, L - 7 * b) for b in range(B)]
    c = Case(cuda_device, lens, [1] * B, 4, 1, D, 64, seed=L)
    c.check(c.run())
    first = c.run()
    for _ in range(3):  # and bit for bit the same every time
        again = c.run()
        assert all(torch.equal(x, y) for x, y in zip(first, again))


def test_strided_and_unaligned_queries(cuda_device):
    c = Case(cuda_device, [100, 33, 1, 250], [1] * 4, 6, 2, 128, 32, seed=5)
    want = c.run()
    T, hq, D = c.q.shape
    wide = torch.zeros(T, hq + 4, D, dtype=c.dtype, device=cuda_device)
    wide[:, 2:2 + hq] = c.q.to(cuda_device)
    heads_first = c.q.to(cuda_device).transpose(0, 1).contiguous().transpose(0, 1)
    odd = torch.zeros(T * hq * D + 1, dtype=c.dtype, device=cuda_device)[1:].view(T, hq, D)
    odd.copy_(c.q)
    for q in (wide[:, 2:2 + hq], heads_first, odd):
        got = c.run(q=q)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    c.check(want)


def test_scale_and_sharp_softmax(cuda_device):
    c = Case(cuda_device, [300, 1000], [1, 1], 8, 2, 128, 16, seed=6, q_scale=20.0, spread=1.0)
    c.check(c.run(scale=0.5), scale=0.5)


def test_another_stream(cuda_device):
    c = Case(cuda_device, [700, 20], [1, 1], 8, 2, 128, 16, seed=7)
    want = c.run()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    q = c.q.to(cuda_device)
    torch.cuda.synchronize()
    got = c.run(q=q, stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def wide_scales(r, pages, layers, hkv, P, D):
    """Blocks of wildly different size, so that no one 16-bit range holds them all."""
    pool = quantised_pool(r, pages, layers, hkv, P, D)
    at = 16 * D
    pool[..., at + D // 2:at + D] = r.randint(97, 158, pool[..., at + D // 2:at + D].shape)
    return pool


def rising_scales(r, pages, layers, hkv, P, D):
    pool = quantised_pool(r, pages, layers, hkv, P, D)
    n, at = D // 32, 16 * D + D // 2
    for p in range(pages):
        for g in range(P // 16):
            for t in range(16):
                pool[p, :, :, g, at + t * n:at + (t + 1) * n] = 60 + (t + 16 * g + 5 * p) % 130
    return pool


def with_zero_blocks(r, pages, layers, hkv, P, D):
    pool = quantised_pool(r, pages, layers, hkv, P, D)
    pool[r.rand(*pool.shape[:-1]) < 0.4] = 0  # codes and scale bytes 0: 0 * 2^-127
    return pool


@pytest.mark.parametrize("make", [wide_scales, rising_scales, with_zero_blocks])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_any_scale_byte(cuda_device, make, D):
    lens = [1, 5, 40, 333, 64]
    c = Case(cuda_device, lens, [1, 3, 2, 1, 5], 8, 2, D, 32, seed=D, pool=make)
    # one far larger block hides the others from an absolute tolerance: look at each block alone
    out, lse = c.run()
    torch.cuda.synchronize()
    want, want_lse, mag = ref.attention(c.pool, c.table, c.lengths, c.layer, c.q_values, c.slots,
                                        c.q_start, D, 32, 1 / np.sqrt(D))
    err = np.abs(out.double().cpu().numpy() - want)
    tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2.0 ** -15) * mag + 1e-37
    assert (err <= tol).all(), np.max(err / tol)
    seen = np.isfinite(want_lse)
    assert np.abs(lse.double().cpu().numpy()[seen] - want_lse[seen]).max() <= 1e-4


@pytest.mark.parametrize("side", ["k", "v"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_nan_blocks_show_where_they_are_seen_and_only_there(cuda_device, side, D):
    lens, news = [100, 70, 40], [4, 1, 3]
    c = Case(cuda_device, lens, news, 4, 2, D, 32, seed=3)
    n = D // 32
    at = 16 * D + (16 * n if side == "v" else 0)
    # position 97 of entry 0 (seen by its last three rows), block 1; position 10 of entry 1, last block
    for b, pos, block in ((0, 97, 1), (1, 10, n - 1)):
        page = c.table[c.slots[b], pos // 32]
        c.pool[page, :, 0, pos % 32 // 16, at + (pos % 16) * n + block] = 255
    c.cache.pool.copy_(device(c.pool, cuda_device))
    out, lse = c.run()
    c.check((out, lse))
    out = out.float().cpu().numpy()
    assert np.isfinite(out[0]).all() and np.isnan(out[1:4, 0]).any(-1).all()
    if side == "v":
        assert np.isfinite(out[1:4, 0, :32]).all() and np.isnan(out[1:4, 0, 32:64]).all()


def test_infinite_and_nan_queries_stay_in_their_rows(cuda_device):
    c = Case(cuda_device, [50, 60], [3, 2], 4, 2, 128, 16, seed=9)
    q = c.q.clone()
    q[1, 2, 5] = float("nan")
    q[4, 0, 0] = float("inf")
    got, lse = c.run(q=q.to(cuda_device))
    want, want_lse = c.run()
    same = torch.ones(5, 4, dtype=torch.bool)
    same[1, 2] = same[4, 0] = False
    assert torch.equal(got[same], want[same]) and torch.equal(lse[same], want_lse[same])
    assert got[1, 2].isnan().all() and got[4, 0].isnan().all()


def test_offsets_past_32_bits(cuda_device):
    """A pool of over 4 GiB, the sequence in its last pages."""
    D, P, hkv, layers = 128, 256, 4, 8
    page = wd.wd_kv_page_bytes(layers, hkv, D, P)
    pages = (1 << 32) // page + 40
    r = np.random.RandomState(1)
    host = quantised_pool(r, 3, 1, hkv, P, D)
    cache = wd.KVCache(pages, 2, 4, layers, hkv, D, P, device=cuda_device)
    layer = layers - 1
    table = np.full((2, 4), -1, np.int32)
    table[1, :3] = [pages - 1, pages - 3, pages - 2]
    cache.table.copy_(device(table, cuda_device))
    cache.lengths.copy_(device(np.array([0, 700], np.int32), cuda_device))
    cache.refs[pages - 3:] = 1
    for j in range(3):
        cache.pool[int(table[1, j]), layer] = device(host[j, 0], cuda_device)
    q, q_values = rounded(r.standard_normal((1, 4, D)), torch.bfloat16)
    out, _ = cache.attention(layer, q.to(cuda_device), device(np.array([1], np.int32), cuda_device),
                             return_lse=True)
    want, _, mag = ref.attention(host, np.array([[0, 1, 2]]), [700], 0, q_values, [0], [0, 1], D, P,
                                 1 / np.sqrt(D))
    err = np.abs(out.double().cpu().numpy() - want)
    assert (err <= 2.0 ** -8 * np.abs(want) + 2.0 ** -10 * mag).all()
    x = torch.randn(1, hkv, D, device=cuda_device, dtype=torch.bfloat16)
    cache.append(layer, x, x, device(np.array([1], np.int32), cuda_device))
    got, _ = ref.decode(cache.pool[pages - 2, layer].cpu().numpy(), D)
    code, scale = ref.quantise(x[0].double().cpu().numpy())
    assert np.array_equal(got.reshape(hkv, -1, D)[:, 699 - 512], ref.values(code, scale))
    # and compaction brings the last pages to the front
    cache.compact()
    assert cache.table[1].tolist() == [2, 0, 1, -1]
    again = cache.attention(layer, q.to(cuda_device), device(np.array([1], np.int32), cuda_device))
    assert torch.isfinite(again.float()).all()
    assert cache.read_error_flag() == 0


def test_bad_indices_are_flagged_and_skipped(cuda_device):
    c = Case(cuda_device, [40, 50], [1, 1], 4, 2, 64, 16, seed=2)
    good, _ = c.run()
    q = c.q.to(cuda_device)
    seqs = torch.tensor([int(c.slots[0]), 99], dtype=torch.int32, device=cuda_device)
    out = c.cache.attention(0, q, seqs)
    assert torch.equal(out[0], good[0]) and not out[1].any()
    assert c.cache.read_error_flag() == wd.KV_FLAG_BAD_INDEX
    before = c.cache.pool.clone()
    x = torch.randn(2, 2, 64, device=cuda_device)
    c.cache.append(0, x, x, torch.tensor([-1, 99], dtype=torch.int32, device=cuda_device))
    assert torch.equal(before, c.cache.pool) and c.cache.read_error_flag() == wd.KV_FLAG_BAD_INDEX
    for bad in ([0, 3, 2], [0, -1, 2], [0, 1, 7]):  # not ascending, negative, past the tokens
        c.cache.attention(0, q, c.seqs, torch.tensor(bad, dtype=torch.int32, device=cuda_device))
        assert c.cache.read_error_flag() == wd.KV_FLAG_BAD_INDEX
    c.cache.table[int(c.slots[0]), 1] = 1 << 20  # a page id past the pool
    c.cache.attention(0, q, c.seqs)
    assert c.cache.read_error_flag() == wd.KV_FLAG_BAD_INDEX
    c.cache.lengths[int(c.slots[1])] = 1 << 24  # longer than its row of the table
    c.cache.attention(0, q, c.seqs)
    assert c.cache.read_error_flag() == wd.KV_FLAG_BAD_INDEX


def test_tokens_of_no_entry_are_not_written(cuda_device):
    c = Case(cuda_device, [40, 50], [1, 1], 4, 2, 64, 16, seed=2)
    q = torch.randn(7, 4, 64, device=cuda_device).bfloat16()
    out = torch.full_like(q, 5.0)
    start = torch.tensor([1, 3, 4], dtype=torch.int32, device=cuda_device)
    c.cache.attention(0, q, c.seqs, start, out=out)
    assert (out[[0, 4, 5, 6]] == 5.0).all() and (out[1:4] != 5.0).any(-1).all()
    assert c.cache.read_error_flag() == 0


def test_wrong_tensors_are_refused(cuda_device):
    c = Case(cuda_device, [40, 50], [1, 1], 4, 2, 64, 16, seed=2)
    q = c.q.to(cuda_device)
    for bad in (q.float(), q.cpu(), q[..., :32], q[:, :3], q[:, :, ::2], q[0]):
        with pytest.raises(ValueError):
            c.cache.attention(0, bad, c.seqs)
    with pytest.raises(ValueError):
        c.cache.attention(0, q, c.seqs.long())
    with pytest.raises(ValueError):
        c.cache.attention(0, q, c.seqs, out=torch.empty_like(q).float())
    with pytest.raises(wd.WdError):
        c.cache.attention(1, q, c.seqs)
    k = torch.randn(2, 2, 64, device=cuda_device)
    for k_, v_ in ((k, k.half()), (k.double(), k.double()), (k[:, :1], k[:, :1]), (k, k[:1])):
        with pytest.raises(ValueError):
            c.cache.append(0, k_, v_, c.seqs)
    with pytest.raises(ValueError):
        c.cache.append(0, torch.cat((k, k)), torch.cat((k, k)), c.seqs)
    with pytest.raises(ValueError):
        c.cache.reserve(torch.ones(2, device=cuda_device))
    with pytest.raises(ValueError):
        c.cache.compact(table_out=torch.empty(3, 3, dtype=torch.int32, device=cuda_device))


# -------------------------------------------------------------------- append ---

def special_values(r, shape):
    """Normals of many sizes, ties, zeros, subnormals, and blocks with infinities and NaN."""
    x = r.standard_normal(shape) * np.exp2(r.randint(-20, 15, shape[:-1] + (1,)))
    flat = x.reshape(-1, 32)
    n = len(flat)
    flat[0] = 0.0
    flat[1 % n] = -0.0
    flat[2 % n, 3] = np.inf
    flat[3 % n, 31] = np.nan
    flat[4 % n] = [4.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -5.0, 7.9, -0.25, 6.9, 7.0, 7.1, -0.0,
                   1e-3] * 2
    flat[5 % n] = 2.0 ** -30 * flat[4 % n]
    return x


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("news", [[1, 1, 1], [5, 0, 40, 17], [1, 90]])
def test_append(cuda_device, dtype, D, news):
    r = np.random.RandomState(D + len(news))
    hkv, P, layers, T = 3, 32, 2, sum(news)
    lens = [n + 11 * b for b, n in enumerate(news)]
    B = len(news)
    k, kf = rounded(special_values(r, (T, hkv, D)), dtype)
    v, vf = rounded(special_values(r, (T, hkv, D)), dtype)
    cache = wd.KVCache(20, B + 1, 6, layers, hkv, D, P, device=cuda_device)
    slots = r.permutation(B + 1)[:B].astype(np.int32)
    cache.reserve(device(np.array(lens, np.int32), cuda_device), device(slots, cuda_device))
    cache.pool.fill_(0xAB)
    start = np.concatenate(([0], np.cumsum(news))).astype(np.int32)
    single = max(news) == min(news) == 1
    args = (device(slots, cuda_device), None if single else device(start, cuda_device))
    want = np.full(cache.pool.shape, 0xAB, np.uint8)
    table = cache.table.cpu().numpy()
    (kc, ks), (vc, vs) = ref.quantise(kf), ref.quantise(vf)
    for b in range(B):
        for i in range(news[b]):
            pos, t = lens[b] - news[b] + i, start[b] + i
            for h in range(hkv):
                ref.store(want, table[slots[b], pos // P], 1, h, pos % P, D, kc[t, h], ks[t, h],
                          vc[t, h], vs[t, h])
    got_k, got_v = cache.append(1, k.to(cuda_device), v.to(cuda_device), *args, return_values=True)
    assert np.array_equal(cache.pool.cpu().numpy(), want)
    for got, code, scale in ((got_k, kc, ks), (got_v, vc, vs)):
        values = rounded(ref.values(code, scale), dtype)[0]
        assert torch.equal(got.cpu().isnan(), values.isnan())
        assert torch.equal(got.cpu().nan_to_num(7.0), values.nan_to_num(7.0))
    # out of a fused projection, and from an address that is not a multiple of 16 bytes
    fused = torch.zeros(T, (2 * hkv + 1) * D, dtype=dtype, device=cuda_device)
    fused[:, D:(hkv + 1) * D] = k.to(cuda_device).flatten(1)
    fused[:, (hkv + 1) * D:] = v.to(cuda_device).flatten(1)
    odd = torch.zeros(fused.numel() + 1, dtype=dtype, device=cuda_device)[1:].view(fused.shape)
    odd.copy_(fused)
    for f in (fused, odd):
        cache.pool.fill_(0xAB)
        cache.append(1, f[:, D:(hkv + 1) * D].unflatten(1, (hkv, D)),
                     f[:, (hkv + 1) * D:].unflatten(1, (hkv, D)), *args)
        assert np.array_equal(cache.pool.cpu().numpy(), want)
    assert cache.read_error_flag() == 0


def test_append_of_the_smallest_and_largest_values(cuda_device):
    D, hkv = 64, 1
    x = np.zeros((6, hkv, D))
    x[0] = 2.0 ** -149
    x[1] = 2.0 ** -127 * 1.5
    x[2] = 2.0 ** -126
    x[3] = 3.4e38
    x[4, :, ::2] = 2.0 ** 127
    x[5, :, 1::3] = 2.0 ** -124 * 1.75
    t, xf = rounded(x, torch.float32)
    cache = wd.KVCache(2, 1, 2, 1, hkv, D, 16, device=cuda_device)
    cache.reserve(torch.tensor([6], dtype=torch.int32, device=cuda_device))
    k, _ = cache.append(0, t.to(cuda_device), t.to(cuda_device),
                        q_start=torch.tensor([0, 6], dtype=torch.int32, device=cuda_device),
                        return_values=True)
    code, scale = ref.quantise(xf)
    assert np.array_equal(k.double().cpu().numpy(), ref.values(code, scale))


# --------------------------------------------------------------------- pages ---

class Both:
    """The library's bookkeeping and the plain one, side by side."""

    def __init__(self, dev, pages, slots, columns, P=16, layers=2, hkv=1, D=64):
        self.cache = wd.KVCache(pages, slots, columns, layers, hkv, D, P, device=dev)
        self.pages, self.columns, self.dev, self.tag = ref.Pages(pages, slots, P), columns, dev, 1

    def ints(self, a):
        return torch.tensor(list(a), dtype=torch.int32, device=self.dev)

    def same(self, ok=None, want_ok=None):
        if ok is not None:
            assert ok.tolist() == list(want_ok)
        c, p = self.cache, self.pages
        assert np.array_equal(c.table.cpu().numpy(), p.table(self.columns))
        assert c.lengths.tolist() == p.lengths and c.refs.tolist() == p.refs
        held = c.pool.flatten(1).cpu().numpy()
        for row in p.rows:
            for page in row:
                if p.data[page] is not None:
                    assert (held[page] == p.data[page]).all()

    def write(self):
        """Give every live page bytes of its own."""
        for page, r in enumerate(self.pages.refs):
            if r:
                self.tag = self.tag % 250 + 1
                self.pages.data[page] = self.tag
                self.cache.pool[page] = self.tag

    def reserve(self, seqs, counts):
        got = self.cache.reserve(self.ints(counts), self.ints(seqs))
        self.same(got, self.pages.reserve(seqs, counts, self.columns))

    def fork(self, src, dst):
        got = self.cache.fork(self.ints(src), self.ints(dst))
        self.same(got, self.pages.fork(src, dst))

    def compact(self):
        got = self.cache.compact()
        assert got.tolist() == self.pages.compact()
        self.same()


def test_pages_step_by_step(cuda_device):
    b = Both(cuda_device, 40, 8, 10)
    b.reserve([0, 3, 5], [33, 0, 16])
    b.write()
    b.reserve([3], [1])
    b.fork([0, 0, 5], [1, 2, 6])
    b.fork([1], [1])
    b.fork([-1, 2], [0, 7])
    b.compact()
    assert b.cache.read_error_flag() == 0
    # refusals: a slot named twice, out of range, too long a sequence, a negative count
    b.reserve([4, 4, 9, -1, 7, 6], [5, 6, 1, 1, 200, -1])
    assert b.cache.read_error_flag() == wd.KV_FLAG_BAD_INDEX
    b.fork([1, 1, 9, -2, 3], [4, 4, 0, 0, 77])
    assert b.cache.read_error_flag() == wd.KV_FLAG_BAD_INDEX
    b.cache.free(b.ints([1, 2, 3, 4, 5, 6, 7]))
    b.pages.fork([-1] * 7, [1, 2, 3, 4, 5, 6, 7])
    b.same()
    b.compact()


def test_out_of_pages(cuda_device):
    b = Both(cuda_device, 10, 6, 10)
    b.reserve([0, 1, 2, 3], [40, 100, 60, 16])  # 3 + 7 pages fit, then nothing, nothing
    assert b.cache.read_error_flag() == wd.KV_FLAG_NO_PAGES
    b.write()
    b.cache.free(b.ints([1]))
    b.pages.fork([-1], [1])
    b.same()
    b.fork([0] * 5, [1, 2, 3, 4, 5])
    b.fork([0, 1, 2, 3], [1, 2, 3, 4])
    assert b.cache.read_error_flag() == wd.KV_FLAG_NO_PAGES
    b.compact()


def test_freed_pages_are_not_used_by_the_same_fork(cuda_device):
    # all beams from the last: the old last pages are read while the new ones are written
    b = Both(cuda_device, 13, 4, 10)
    b.reserve([0, 1, 2, 3], [40, 40, 20, 20])
    b.write()
    b.fork([3, 0, 1, 0], [0, 1, 2, 3])
    b.fork([1, 2, 3, 0], [0, 1, 2, 3])


@pytest.mark.parametrize("seed", range(6))
def test_random_page_operations(cuda_device, seed):
    r = np.random.RandomState(seed)
    slots, pages = int(r.randint(1, 40)), int(r.randint(5, 400))
    b = Both(cuda_device, pages, slots, 12, P=int(r.choice([16, 32])), layers=int(r.randint(1, 4)))
    for _ in range(25):
        n = int(r.randint(1, slots + 1))
        which = r.permutation(slots)[:n]
        op = r.randint(4)
        if op == 0:
            b.reserve(which.tolist(), r.randint(0, 90, n).tolist())
            b.write()
        elif op == 1:
            b.fork(r.randint(-1, slots, n).tolist(), which.tolist())
        elif op == 2:
            b.cache.free(b.ints(which))
            b.pages.fork([-1] * n, which.tolist())
            b.same()
        else:
            b.compact()


@pytest.mark.parametrize("pages,live", [(4095, 0.3), (4097, 0.9), (20000, 0.5), (70001, 0.02),
                                        (16384, 1.0), (5000, 0.0)])
def test_compact_of_many_pages(cuda_device, pages, live):
    r = np.random.RandomState(pages)
    on = r.permutation(pages)[:int(live * pages)].astype(np.int32)
    slots = 7
    columns = max(1, -(-len(on) // slots))
    table = np.full((slots, columns), -1, np.int32)
    table.reshape(-1)[:len(on)] = on
    refs = np.zeros(pages, np.int32)
    refs[on] = 1 + on % 3
    pool = r.randint(0, 256, (pages, 16 * 68)).astype(np.uint8)
    lengths = (table >= 0).sum(1).astype(np.int32) * 16
    cache = wd.KVCache.from_buffers(*(device(a, cuda_device) for a in (pool, table, lengths, refs)),
                                    layers=1, kv_heads=1, head_dim=64, page_size=16)
    model = ref.Pages(pages, 1, 16)
    model.refs, model.rows = refs.tolist(), [[int(p) for p in on]]
    table_out, refs_out = torch.empty_like(cache.table), torch.empty_like(cache.refs)
    got = cache.compact(table_out=table_out, refs_out=refs_out)
    want = np.array(model.compact(), np.int32)
    assert np.array_equal(got.cpu().numpy(), want)
    assert refs_out.tolist() == model.refs
    assert np.array_equal(table_out.cpu().numpy(), np.where(table >= 0, want[table], -1))
    assert np.array_equal(cache.table.cpu().numpy(), table)  # the old bookkeeping stands
    assert np.array_equal(cache.refs.cpu().numpy(), refs)
    moved = cache.pool.cpu().numpy()
    assert np.array_equal(moved[want[on]], pool[on]) and np.array_equal(moved[on], pool[on])
    again = cache.compact()  # in place
    assert torch.equal(again, got) and torch.equal(cache.table, table_out)
    assert torch.equal(cache.refs, refs_out) and cache.read_error_flag() == 0


def test_reserve_many_pages_at_once(cuda_device):
    b = Both(cuda_device, 40000, 3, 20000)
    b.reserve([2, 0], [300000, 1000])
    b.reserve([1, 2], [17, 16])
    assert b.cache.read_error_flag() == 0


@pytest.mark.parametrize("seed", range(2))
def test_random_page_operations_in_a_large_pool(cuda_device, seed):
    """A pool whose plans are made once for all CTAs, by kernels of their own."""
    r = np.random.RandomState(100 + seed)
    slots = 300
    b = Both(cuda_device, 16385 + 5000 * seed, slots, 30, layers=1)
    b.reserve(list(range(0, slots, 2)), r.randint(0, 450, slots // 2).tolist())
    for _ in range(6):
        n = int(r.choice([5, 100, 290]))
        which = r.permutation(slots)[:n]
        op = r.randint(3)
        if op == 0:
            b.reserve(which.tolist(), r.randint(0, 40, n).tolist())
            b.write()
        elif op == 1:
            b.fork(r.randint(-1, slots, n).tolist(), which.tolist())
        else:
            b.compact()


def test_more_requests_than_one_kernel_takes(cuda_device):
    r = np.random.RandomState(5)
    b = Both(cuda_device, 3000, 400, 8)
    b.reserve(list(range(400)), r.randint(0, 100, 400).tolist())
    b.write()
    b.fork(r.randint(-1, 400, 400).tolist(), r.permutation(400).tolist())
    b.fork([3] * 300 + [900], list(range(100, 400)) + [1])  # too few pages for all, one bad slot
    b.compact()
    assert b.cache.read_error_flag() & wd.KV_FLAG_BAD_INDEX
