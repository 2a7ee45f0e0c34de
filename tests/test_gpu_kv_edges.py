"""Attention over the 4-bit cache at the edges of what its types hold, on the GPU, against the definition
in 64 bits: scales far apart, values and logits near the ends of FP32, rows that see nothing, keys
that are there and not seen, pages that do not exist.

Tolerances as in test_gpu_kv.py, but from what each row sees: |error| <= u_out |want| + (2^-11 + 2^-15)
sum_j p_j |v_j| + 2^-20 max_j |v_j| over the keys j that the row sees.  lse: 1e-5 + 2^-20 max_j scale
sum_c |q_c| |k_jc| over these keys, which FP32 sums of the products stay within.
"""
import numpy as np
import pytest
import torch

import kv_reference as ref
import moe_decode_gate_gb300 as wd
from test_gpu_kv import ROUNDOFF, Case, device, quantised_pool

pytestmark = pytest.mark.gpu

# few new tokens, and so many that they take the kernel for chunks (8 query heads to a key head)
FEW, MANY = [1, 3], [40, 64]


def definition(c, window=0, scale=None, gone=()):
    """out, lse, and per row sum p |v|, max |v| and max_j sum |q||k| over what it sees; tokens of the pages
    `gone` are seen by nobody."""
    scale = 1 / np.sqrt(c.D) if scale is None else scale
    T, hq, D = c.q_values.shape
    hkv = c.pool.shape[2]
    out, lse = np.zeros((T, hq, D)), np.full((T, hq), -np.inf)
    mag, top, reach = np.zeros((T, hq, D)), np.zeros((T, hq, 1)), np.zeros((T, hq))
    for b, s in enumerate(c.slots):
        L, first, n = int(c.lengths[s]), c.q_start[b], c.q_start[b + 1] - c.q_start[b]
        row = c.table[s][:-(-L // c.P)]
        there = np.repeat([p not in gone for p in row], c.P)[:L]
        for h in range(hkv):
            if not L:
                continue
            k, v = ref.sequence(c.pool, np.where([p in gone for p in row], 0, row), L, c.layer, h, D,
                                c.P)
            for i in range(n):
                p = L - n + i
                lo = max(0, p - window + 1) if window else 0
                at = np.flatnonzero(there[:p + 1][lo:]) + lo if p >= 0 else []
                if not len(at):
                    continue
                for qh in range(h * hq // hkv, (h + 1) * hq // hkv):
                    q = c.q_values[first + i, qh]
                    x = scale * (k[at] @ q)
                    e = np.exp(x - x.max())
                    out[first + i, qh] = e @ v[at] / e.sum()
                    mag[first + i, qh] = e @ np.abs(v[at]) / e.sum()
                    lse[first + i, qh] = x.max() + np.log(e.sum())
                    top[first + i, qh] = np.abs(v[at]).max()
                    reach[first + i, qh] = scale * (np.abs(k[at]) @ np.abs(q)).max()
    return out, lse, mag, top, reach


def check(c, got, window=0, flag=0, gone=()):
    out, lse = (x.double().cpu().numpy() for x in got)
    want, want_lse, mag, top, reach = definition(c, window, gone=gone)
    tol = ROUNDOFF[c.dtype] * np.abs(want) + (2.0 ** -11 + 2.0 ** -15) * mag + 2.0 ** -20 * top
    assert (np.abs(out - want) <= tol).all(), np.argwhere(~(np.abs(out - want) <= tol))[:4]
    nothing = np.isneginf(want_lse)
    assert np.array_equal(np.isneginf(lse), nothing)
    assert (np.abs(lse[~nothing] - want_lse[~nothing]) <= 1e-5 + 2.0 ** -20 * reach[~nothing]).all()
    assert c.cache.read_error_flag() == flag


def shift_scales(side, by):
    """A pool whose keys' (or values') blocks are 2^by times as large."""
    def make(r, pages, layers, hkv, P, D):
        pool = quantised_pool(r, pages, layers, hkv, P, D)
        at = 16 * D + (D // 2 if side == "v" else 0)
        s = pool[..., at:at + D // 2].astype(int)
        pool[..., at:at + D // 2] = np.clip(s + by, 0, 254)
        return pool
    return make


def set_scales(c, side, b, positions, byte, blocks=slice(None)):
    """The scale byte of these tokens of entry b, of all heads, on the host and the GPU."""
    n = c.D // 32
    at = 16 * c.D + (16 * n if side == "v" else 0)
    for pos in positions:
        page = c.table[c.slots[b], pos // c.P]
        g = c.pool[page, :, :, pos % c.P // 16]
        g[..., at + (pos % 16) * n:at + (pos % 16 + 1) * n][..., blocks] = byte
    c.cache.pool.copy_(device(c.pool, c.dev))


# ------------------------------------------------------------ large values ---

@pytest.mark.parametrize("D,lens,news", [
    (64, [1, 40, 300, 3000], [1, 1, 1, 1]), (128, [1, 40, 300, 20000], [1, 1, 1, 1]),
    (256, [50, 4000], [1, 1]), (128, [300, 2000], [3, 2]), (64, [300, 5000], MANY),
    (128, [300, 5000], MANY)])
def test_values_near_the_largest(cuda_device, D, lens, news):
    # values of up to 6 x 2^119: a mean of them is finite, the sum of a few hundred, weighted, is not
    c = Case(cuda_device, lens, news, 8, 1, D, 32, seed=D, pool=shift_scales("v", 118))
    check(c, c.run())


# ---------------------------------------------- values that a row does not see ---

def small_values(r, pages, layers, hkv, P, D):
    pool = quantised_pool(r, pages, layers, hkv, P, D)
    at = 16 * D + D // 2
    pool[..., at:at + D // 2] = r.randint(90, 111, pool[..., at:at + D // 2].shape)
    return pool


@pytest.mark.parametrize("D", [64, 128, 256])
def test_values_before_the_window_do_not_count(cuda_device, D):
    # the window starts inside a step of 32 keys: the keys before it there are copied, and far larger
    c = Case(cuda_device, [100, 300], [1, 1], 8, 2, D, 32, seed=D, pool=small_values)
    set_scales(c, "v", 0, range(0, 80), 254)
    set_scales(c, "v", 1, range(256, 280), 254)
    check(c, c.run(window=20), window=20)


@pytest.mark.parametrize("D", [64, 128])
def test_values_before_the_window_of_a_chunk_do_not_count(cuda_device, D):
    # tiles of 32 tokens: the first one's rows see from 97 on, and its first tile of keys starts at 64
    c = Case(cuda_device, [200], [64], 8, 1, D, 32, seed=D, pool=small_values)
    set_scales(c, "v", 0, range(64, 97), 254)
    check(c, c.run(window=40), window=40)


@pytest.mark.parametrize("news", [[3, 2], [32, 64]])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("window", [0, 20])
def test_values_that_some_rows_see(cuda_device, news, D, window):
    # the last token's values, which the others of the chunk do not see, and those at the start of the
    # first row's window, which the later rows do not see
    c = Case(cuda_device, [100, 300], news, 8, 1, D, 32, seed=D + window, pool=small_values)
    set_scales(c, "v", 0, [99], 250)
    set_scales(c, "v", 1, [299, 300 - news[1] - (window or 300) + 1] if window else [299], 247)
    check(c, c.run(window=window), window=window)


# --------------------------------------------------- key blocks of unlike size ---

@pytest.mark.parametrize("news", [FEW, MANY])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("apart", [22, 23, 24, 25, 40, 60])
def test_small_key_blocks_count_where_the_query_is_zero_in_the_large_one(cuda_device, news, D, apart):
    c = Case(cuda_device, [100, 300], news, 8, 1, D, 32, seed=D + apart)
    q = c.q_values.copy()
    q[..., :32] = 0.0
    c.q = torch.from_numpy(q).to(c.dtype)
    c.q_values = c.q.double().numpy()
    for b, L in enumerate((100, 300)):  # block 0 of every other key
        set_scales(c, "k", b, range(0, L, 2), 126 + apart, slice(0, 1))
    check(c, c.run())


@pytest.mark.parametrize("news", [FEW, MANY])
@pytest.mark.parametrize("D", [64, 128])
def test_key_blocks_apart_of_which_both_count(cuda_device, news, D):
    # the query is as much smaller in the large block as that is larger (and holds it exactly in FP16
    # beside its other channels)
    c = Case(cuda_device, [100, 300], news, 8, 1, D, 32, seed=D)
    q = c.q_values.copy()
    q[..., 32:64] = np.where(q[..., 32:64] < 0, -(2.0 ** -28), 2.0 ** -28)
    c.q = torch.from_numpy(q).to(c.dtype)
    c.q_values = c.q.double().numpy()
    for b, L in enumerate((100, 300)):
        set_scales(c, "k", b, range(L), 126 + 28, slice(1, 2))
    check(c, c.run())


# ------------------------------------------------------------ logits near the ends ---

@pytest.mark.parametrize("news", [FEW, MANY])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("by", [90, 105, 122, -100])
def test_large_keys_and_small_queries(cuda_device, news, D, by):
    # (and the other way round): the logits are those of a plain case
    c = Case(cuda_device, [100, 300], news, 8, 1, D, 32, seed=D, q_scale=2.0 ** -by,
             pool=shift_scales("k", by))
    check(c, c.run())


@pytest.mark.parametrize("news", [FEW, MANY])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("byte", [150, 170, 200, 235])
def test_a_few_far_larger_keys(cuda_device, news, D, byte):
    # logits of up to 2^110: a row's softmax is one of these keys, or none of them
    c = Case(cuda_device, [100, 300], news, 8, 1, D, 32, seed=D + byte)
    for b, L in enumerate((100, 300)):
        set_scales(c, "k", b, [3, 17, 61, L - 2], byte)
    check(c, c.run())


@pytest.mark.parametrize("news", [FEW, MANY])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_all_logits_far_from_zero(cuda_device, news, D):
    c = Case(cuda_device, [100, 300], news, 8, 1, D, 32, seed=D, q_scale=2.0 ** 40)
    check(c, c.run())


# ------------------------------------------------------------- rows that see nothing ---

@pytest.mark.parametrize("lens,news", [([2], [4]), ([20], [40])])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_query_of_nan_that_sees_nothing(cuda_device, lens, news, bad):
    c = Case(cuda_device, lens, news, 8, 1, 128, 32, seed=1)
    want, want_lse = c.run()
    q = c.q.clone()
    q[0, 3, 7] = q[1] = bad
    got, lse = c.run(q=q.to(cuda_device))
    assert torch.equal(got, want) and torch.equal(lse, want_lse)
    assert not got[:2].any() and torch.isneginf(lse[:2]).all()


# ------------------------------------------------------------- pages that do not exist ---

@pytest.mark.parametrize("news", [FEW, MANY])
@pytest.mark.parametrize("D,P", [(64, 16), (64, 64), (128, 16), (128, 32), (256, 16), (256, 64)])
@pytest.mark.parametrize("window", [0, 50])
def test_keys_of_a_page_out_of_range_are_skipped(cuda_device, news, D, P, window):
    c = Case(cuda_device, [200, 2500], news, 8, 2, D, P, seed=D + P)
    for b, column, page in ((0, 160 // P, -1), (0, 64 // P, 1 << 20), (1, 2400 // P, len(c.pool)),
                            (1, 32 // P, -5)):
        c.table[c.slots[b], column] = page
    c.cache.table.copy_(device(c.table, cuda_device))
    gone = {-1, 1 << 20, len(c.pool), -5}
    check(c, c.run(window=window), window=window, flag=wd.KV_FLAG_BAD_INDEX, gone=gone)


@pytest.mark.parametrize("pages", [50, 20000])
def test_a_fork_whose_last_page_is_out_of_range_is_refused(cuda_device, pages):
    cache = wd.KVCache(pages, 6, 8, 1, 1, 64, 16, device=cuda_device)

    def ints(*v):
        return torch.tensor(v, dtype=torch.int32, device=cuda_device)

    assert cache.reserve(ints(20, 40, 33), ints(0, 1, 2)).tolist() == [1, 1, 1]
    cache.pool.copy_(torch.randint(0, 256, cache.pool.shape, device=cuda_device).to(torch.uint8))
    cache.table[1, 2] = pages + 7
    table, refs, lengths = cache.table.clone(), cache.refs.clone(), cache.lengths.clone()
    assert cache.fork(ints(1), ints(2)).tolist() == [0]
    assert cache.read_error_flag() == wd.KV_FLAG_BAD_INDEX
    for now, before in ((cache.table, table), (cache.refs, refs), (cache.lengths, lengths)):
        assert torch.equal(now, before)
    # the others of the call are served, and the refused one takes no page
    assert cache.fork(ints(1, 0, 2), ints(3, 4, 5)).tolist() == [0, 1, 1]
    assert cache.read_error_flag() == wd.KV_FLAG_BAD_INDEX
    assert cache.table[4].tolist() == [0, 8] + [-1] * 6 and cache.table[5, :3].tolist() == [5, 6, 9]
    assert cache.lengths.tolist() == [20, 40, 33, 0, 20, 33]
