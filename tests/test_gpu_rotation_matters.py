"""Rotated append and attention together against the plain 64-bit references, where the rotation decides the result.

Tolerances: the queries and the cache's bytes are exact (tests/test_gpu_kv_rotated.py); attention's is that of
tests/test_gpu_kv.py, |error| <= 2^-8 |want| + (2^-11 + 2^-15) sum_j p_j |v_j| + 2^-20 max |v|.
"""
import numpy as np
import pytest
import torch

import kv_reference as ref
import moe_decode_gate_gb300 as wd
import step_reference as step
from test_gpu_kv_rotated import Batch

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
T, HQ, HKV, D, P = 24, 4, 2, 128, 16


def make(dev, order=None, rotated=True, paired=False, seed=0):
    """One sequence of T tokens, keys and values in another order if given; a table that turns nothing without `rotated`."""
    b = Batch(dev, [T], [T], HQ, HKV, D, P, D, BF16, seed=seed, paired=paired)
    r = np.random.RandomState(seed + 100)
    x = r.standard_normal((T, HQ + 2 * HKV, D))
    x[:, :HQ] *= 3  # so that attention is sharp
    if order is not None:
        x[:, HQ:] = x[order, HQ:]
    b.qkv = torch.from_numpy(x.reshape(T, -1)).to(BF16)
    if not rotated:
        b.cos_sin[:, :D // 2], b.cos_sin[:, D // 2:] = 1.0, 0.0
    return b


def run(b):
    q = b.run(*b.parts())[0]
    return b.cache.attention(0, q, b.device(b.slots.astype(np.int32)), b.device(b.start.astype(np.int32)), max_q=T)


def expected(b):
    """Attention's output, and what its error may be, from the tokens alone."""
    x = b.qkv.float().numpy().reshape(T, HQ + 2 * HKV, D)
    q = torch.from_numpy(step.rotate(x[:, :HQ], b.cos_sin, b.pos, b.paired)).to(BF16).double().numpy()
    k = step.rotate(x[:, HQ:HQ + HKV], b.cos_sin, b.pos, b.paired).astype(np.float64)
    v = x[:, HQ + HKV:].astype(np.float64)
    (kc, ks), (vc, vs) = ref.quantise(k), ref.quantise(v)
    pool = b.pool.copy()
    for t in range(T):
        for h in range(HKV):
            ref.store(pool, b.table[b.slots[0], t // P], 0, h, t % P, D, kc[t, h], ks[t, h], vc[t, h], vs[t, h])
    want, _, mag = ref.attention(pool, b.table, b.lengths, 0, q, b.slots, b.start, D, P, 1 / np.sqrt(D))
    top = np.abs(ref.values(vc, vs)).max()
    return want, 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2.0 ** -15) * mag + 2.0 ** -20 * top


@pytest.mark.parametrize("paired", [False, True])
@pytest.mark.parametrize("seed", [0, 1])
def test_attention_of_turned_queries_and_keys(seed, paired, cuda_device):
    turned, plain = make(cuda_device, seed=seed, paired=paired), make(cuda_device, rotated=False, seed=seed, paired=paired)
    want, tol = expected(turned)
    without, its = expected(plain)
    got = run(turned).double().cpu().numpy()
    assert (np.abs(got - want) <= tol).all()
    assert (np.abs(run(plain).double().cpu().numpy() - without) <= its).all()
    # what turning changes is many times what may be off (the first token sees itself alone)
    assert np.linalg.norm(want[1:] - without[1:]) > 20 * np.linalg.norm(tol[1:])
    assert np.array_equal(want[0], without[0])


def test_the_order_of_tokens_matters_where_keys_are_turned(cuda_device):
    """Two earlier tokens change places: the last one's attention stays without rotation and goes elsewhere with it."""
    order = np.arange(T)
    order[[2, 11]] = [11, 2]
    for rotated in (False, True):
        first, second = make(cuda_device, rotated=rotated), make(cuda_device, order, rotated)
        (a, tol), (b, its) = expected(first), expected(second)
        moved = run(first)[-1].double().cpu().numpy() - run(second)[-1].double().cpu().numpy()
        assert (np.abs(moved - (a[-1] - b[-1])) <= tol[-1] + its[-1]).all()
        if rotated:
            assert np.linalg.norm(a[-1] - b[-1]) > 20 * np.linalg.norm(tol[-1])
        else:
            assert np.abs(a[-1] - b[-1]).max() < 1e-12


@pytest.mark.parametrize("ahead", [1, 7])
def test_queries_turn_by_the_distance_of_their_positions(ahead, cuda_device):
    """A query at two positions `ahead` apart: each pair is moved by 2 sin(ahead f / 2) of its length."""
    b = make(cuda_device)
    q, k, v = b.parts()
    table = wd.rotation_table(T + ahead, D, device=cuda_device)
    start, slots = b.device(b.start.astype(np.int32)), b.device(b.slots.astype(np.int32))
    turned = [b.cache.append_rotated(0, q, k, v, table[at:at + T].contiguous(), slots, start) for at in (0, ahead)]
    moved = (turned[1].double() - turned[0].double()).cpu().numpy()
    x = q.double().cpu().numpy()
    length = np.sqrt(x[..., :D // 2] ** 2 + x[..., D // 2:] ** 2)
    want = 2 * np.abs(np.sin(ahead * 10000.0 ** (-np.arange(0, D, 2) / D) / 2)) * length
    got = np.sqrt(moved[..., :D // 2] ** 2 + moved[..., D // 2:] ** 2)
    # each of the two is rounded to BF16 (2^-8 of a channel, and so of the pair's length), cosines, products and sums to FP32
    assert (np.abs(got - want) <= 2 * (2.0 ** -8 + 2.0 ** -21) * length).all()
