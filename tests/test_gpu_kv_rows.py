"""Attention over the 4-bit cache with many query rows to a key head (chunks of a prompt), on the GPU
against the plain 64-bit reference (tests/kv_reference.py).

Tolerances as in test_gpu_kv.py: probabilities are rounded once to FP16, sums are FP32.  A key's
blocks are taken to FP16 beside its largest block and lose what is below 2^-24 of that, which the
2^-20 of scale * sum |q||k| covers.
"""
import numpy as np
import pytest
import torch

import kv_reference as ref
import moe_decode_gate_gb300 as wd
from test_gpu_kv import Case, device, quantised_pool, rising_scales, wide_scales, with_zero_blocks

pytestmark = pytest.mark.gpu

# 8 query heads to a key head: tiles of rows that are empty, part of a half, just a half, one row
# more, just full, one token more, several; more tokens than the sequence has
LENS = [0, 1, 63, 64, 65, 200, 130, 777, 40, 300]
NEWS = [0, 1, 5, 16, 17, 32, 33, 100, 70, 8]


@pytest.mark.parametrize("D,hq,hkv", [(64, 8, 1), (64, 24, 3), (128, 8, 1), (128, 14, 2), (128, 32, 4)])
@pytest.mark.parametrize("window", [0, 1, 40, 64, 129])
def test_chunks_and_windows(cuda_device, D, hq, hkv, window):
    c = Case(cuda_device, LENS, NEWS, hq, hkv, D, 32, seed=window + D + hq)
    c.check(c.run(window=window), window=window)


@pytest.mark.parametrize("P", [16, 64, 256])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_chunks_in_pages_layers_and_types(cuda_device, P, dtype):
    c = Case(cuda_device, LENS, NEWS, 16, 2, 128, P, layers=2, dtype=dtype, seed=P)
    c.check(c.run())


@pytest.mark.parametrize("n", [33, 127, 128, 129, 255, 256, 257, 600])
@pytest.mark.parametrize("D", [64, 128])
def test_a_prompt_alone(cuda_device, n, D):
    c = Case(cuda_device, [n], [n], 2, 2, D, 64, seed=n)
    c.check(c.run())


@pytest.mark.parametrize("B,L,n,D", [(1, 20000, 40, 128), (2, 7001, 130, 64), (3, 5003, 64, 128)])
def test_chunks_split_over_many_ctas(cuda_device, B, L, n, D):
    c = Case(cuda_device, [L - 100 * b for b in range(B)], [n] * B, 4, 1, D, 64, seed=L)
    first = c.run()
    c.check(first)
    for _ in range(3):  # and bit for bit the same every time
        again = c.run()
        assert all(torch.equal(x, y) for x, y in zip(first, again))


def test_many_items(cuda_device):
    # more tiles of rows than CTAs, whole and in several passes
    c = Case(cuda_device, [150] * 24, [140] * 24, 16, 8, 64, 32, seed=1)
    c.check(c.run())


def test_more_entries_than_are_kept(cuda_device):
    c = Case(cuda_device, [20] * 1030, [5] * 1030, 8, 1, 64, 16, seed=2)
    c.check(c.run())


def test_one_chunk_among_single_tokens(cuda_device):
    c = Case(cuda_device, [500] * 30 + [700], [1] * 30 + [300], 8, 2, 128, 32, seed=3)
    c.check(c.run())


def wide_key_scales(r, pages, layers, hkv, P, D):
    """Key blocks of unlike size: no tile has one factor."""
    pool = quantised_pool(r, pages, layers, hkv, P, D)
    at = 16 * D
    pool[..., at:at + D // 2] = r.randint(97, 126, pool[..., at:at + D // 2].shape)
    return pool


def empty_blocks_of_large_scale(r, pages, layers, hkv, P, D):
    """Blocks of zeros whose scale byte is far above their key's other blocks."""
    pool = quantised_pool(r, pages, layers, hkv, P, D)
    n = D // 32
    k, _, _ = ref._places(D)
    for t in range(0, 16, 3):
        block = t % n
        pool[..., np.unique(k[t, 32 * block:32 * block + 32])] = 0
        pool[..., 16 * D + t * n + block] = 200
    return pool


@pytest.mark.parametrize("make", [wide_key_scales, empty_blocks_of_large_scale])
@pytest.mark.parametrize("D", [64, 128])
def test_key_scales(cuda_device, make, D):
    c = Case(cuda_device, LENS, NEWS, 8, 1, D, 32, seed=D, pool=make)
    c.check(c.run())


@pytest.mark.parametrize("make", [wide_scales, rising_scales, with_zero_blocks])
@pytest.mark.parametrize("D", [64, 128])
def test_any_scale_byte(cuda_device, make, D):
    lens, news = [1, 5, 40, 333, 64], [1, 3, 20, 31, 25]
    c = Case(cuda_device, lens, news, 8, 2, D, 32, seed=D, pool=make)
    out, lse = c.run(max_q=31)
    torch.cuda.synchronize()
    want, want_lse, mag = ref.attention(c.pool, c.table, c.lengths, c.layer, c.q_values, c.slots,
                                        c.q_start, D, 32, 1 / np.sqrt(D))
    err = np.abs(out.double().cpu().numpy() - want)
    # (a V block of less than 2^-126 beside its channel's largest is below what FP32 keeps)
    tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2.0 ** -15) * mag + 1e-37
    assert (err <= tol).all(), np.max(err / tol)
    seen = np.isfinite(want_lse)
    assert np.abs(lse.double().cpu().numpy()[seen] - want_lse[seen]).max() <= 1e-4


@pytest.mark.parametrize("side", ["k", "v"])
@pytest.mark.parametrize("D", [64, 128])
def test_nan_blocks_show_where_they_are_seen_and_only_there(cuda_device, side, D):
    lens, news = [150, 70, 90], [40, 33, 34]
    c = Case(cuda_device, lens, news, 4, 2, D, 32, seed=3)
    n = D // 32
    at = 16 * D + (16 * n if side == "v" else 0)
    for b, pos, block in ((0, 130, 1), (1, 10, n - 1)):
        page = c.table[c.slots[b], pos // 32]
        c.pool[page, :, 0, pos % 32 // 16, at + (pos % 16) * n + block] = 255
    c.cache.pool.copy_(device(c.pool, cuda_device))
    out, lse = c.run(max_q=40)
    c.check((out, lse))
    out = out.float().cpu().numpy()
    assert np.isfinite(out[:20]).all() and np.isnan(out[20:40, 0]).any(-1).all()
    if side == "v":
        assert np.isfinite(out[20:40, 0, :32]).all() and np.isnan(out[20:40, 0, 32:64]).all()


def test_infinite_and_nan_queries_stay_in_their_rows(cuda_device):
    c = Case(cuda_device, [150, 160], [40, 70], 8, 2, 128, 16, seed=9)
    q = c.q.clone()
    q[1, 2, 5] = float("nan")
    q[44, 0, 0] = float("inf")
    got, lse = c.run(q=q.to(cuda_device))
    want, want_lse = c.run()
    same = torch.ones(110, 8, dtype=torch.bool)
    same[1, 2] = same[44, 0] = False
    assert torch.equal(got[same], want[same]) and torch.equal(lse[same], want_lse[same])
    assert got[1, 2].isnan().all() and got[44, 0].isnan().all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_strided_and_unaligned(cuda_device, dtype):
    c = Case(cuda_device, [100, 33, 250], [60, 20, 100], 6, 2, 128, 32, seed=5, dtype=dtype)
    want = c.run()
    T, hq, D = c.q.shape
    wide = torch.zeros(T, hq + 4, D, dtype=c.dtype, device=cuda_device)
    wide[:, 2:2 + hq] = c.q.to(cuda_device)
    heads_first = c.q.to(cuda_device).transpose(0, 1).contiguous().transpose(0, 1)
    odd = torch.zeros(T * hq * D + 1, dtype=c.dtype, device=cuda_device)[1:].view(T, hq, D)
    odd.copy_(c.q)
    out = torch.zeros(T * hq * D + 1, dtype=c.dtype, device=cuda_device)[1:].view(T, hq, D)
    for q, kw in ((wide[:, 2:2 + hq], {}), (heads_first, {}), (odd, {}), (odd, dict(out=out))):
        got = c.run(q=q, **kw)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    c.check(want)


def test_large_and_small_queries(cuda_device):
    c = Case(cuda_device, [300, 1000], [50, 64], 8, 2, 128, 16, seed=6, q_scale=20.0, spread=1.0)
    c.check(c.run(scale=0.5), scale=0.5)
    c = Case(cuda_device, [300, 1000], [50, 64], 8, 2, 128, 16, seed=7, q_scale=2.0 ** -60)
    c.check(c.run(scale=2.0 ** 58), scale=2.0 ** 58)


def test_chunk_then_single_tokens_on_another_stream(cuda_device):
    c = Case(cuda_device, [700, 90], [100, 40], 8, 2, 128, 16, seed=8)
    want = c.run()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    q = c.q.to(cuda_device)
    torch.cuda.synchronize()
    got = [c.run(q=q, stream=s) for _ in range(4)]  # back to back: the launches overlap
    s.synchronize()
    for x in got:
        assert torch.equal(x[0], want[0]) and torch.equal(x[1], want[1])
    assert isinstance(c.cache, wd.KVCache)
