"""wd_route on the GPU against the plain 64-bit reference (tests/step_reference.py).

Ids have to be those of the definition, near keys and all.  Weights: expf is within 2 units (2^-23), its argument within half a
unit of |x - top|, below 2^-19 for the 64 that matter, the sum of up to 1024 of them within 40 2^-24, and the quotient and
products another 4 2^-24: 2^-18 of the weight in all, and what FP32 does not hold (2^-126).
"""
import numpy as np
import pytest
import torch

import moe_decode_gate_gb300 as wd
import step_reference as ref

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


def check(x, K, dev, bias=None, **kw):
    args = dict(scores="softmax", groups=1, top_groups=1, group_best=2, renormalise=True, scale=1.0)
    args.update(kw)
    b = None if bias is None else torch.from_numpy(bias.astype(np.float32)).to(dev)
    ids, w = wd.route(x, K, bias=b, **args)
    want, want_w = ref.route(x.double().cpu().numpy(), K, bias=None if bias is None else b.double().cpu().numpy(), **args)
    assert ids.dtype == torch.int32 and w.dtype == FP32 and ids.shape == w.shape == (x.shape[0], K)
    assert np.array_equal(ids.cpu().numpy(), want)
    got = w.double().cpu().numpy()
    assert (np.abs(got - want_w) <= 2.0 ** -18 * np.abs(want_w) + 2.0 ** -126).all()
    return ids, w


def make(T, E, dtype, dev, seed=0, scale=1.5):
    r = np.random.RandomState(seed)
    return torch.from_numpy(scale * r.standard_normal((T, E))).to(dtype).to(dev)


# experts, K, groups, open groups, best of a group
FORMS = [(1, 1, 1, 1, 2), (7, 7, 1, 1, 2), (8, 2, 1, 1, 2), (33, 5, 1, 1, 2), (64, 6, 1, 1, 2), (128, 8, 1, 1, 2),
         (160, 6, 8, 3, 1), (256, 8, 8, 4, 2), (300, 33, 1, 1, 2), (512, 64, 1, 1, 2), (1024, 64, 1, 1, 2),
         (768, 40, 3, 2, 2), (64, 1, 32, 5, 2), (32, 3, 32, 7, 2), (96, 4, 6, 5, 1), (128, 16, 4, 4, 2), (1000, 9, 2, 1, 2)]


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
def test_forms(form, scores, dtype, cuda_device):
    E, K, groups, top, best = form
    x = make(37, E, dtype, cuda_device, E + K)
    kw = dict(scores=scores, groups=groups, top_groups=top, group_best=best)
    check(x, K, cuda_device, **kw)
    check(x, K, cuda_device, renormalise=False, scale=2.5, **kw)
    bias = 0.2 * np.random.RandomState(3).standard_normal(E)
    check(x, K, cuda_device, bias, **kw)
    check(x, K, cuda_device, bias, renormalise=False, **kw)


@pytest.mark.parametrize("T", [1, 2, 3, 5, 4097])
def test_tokens(T, cuda_device):
    check(make(T, 128, BF16, cuda_device, T), 8, cuda_device)


@pytest.mark.parametrize("E", [128, 40])
def test_strides(E, cuda_device):
    wide = make(9, E + 7, BF16, cuda_device, 1)
    check(wide[:, 3:E + 3], 4, cuda_device)
    check(wide[1::2, :E], 4, cuda_device)


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,top,best", [(1, 1, 2), (8, 3, 2), (8, 3, 1)])
@pytest.mark.parametrize("biased", [False, True])
def test_ties_go_to_the_lowest(scores, groups, top, best, biased, cuda_device):
    r = np.random.RandomState(5)
    x = torch.from_numpy(r.randint(-2, 3, (50, 128)).astype(np.float32)).to(cuda_device)
    x[3] = 0.0
    x[4, ::2] = -0.0
    x[4, 1::2] = 0.0
    bias = r.randint(0, 2, 128) * 0.25 if biased else None
    check(x, 12, cuda_device, bias, scores=scores, groups=groups, top_groups=top, group_best=best)


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,top,best", [(1, 1, 2), (8, 3, 2), (8, 3, 1), (32, 9, 2)])
@pytest.mark.parametrize("E", [64, 256, 992])
def test_keys_nearer_than_32_bits_tell(scores, groups, top, best, E, cuda_device):
    """A bias that brings all of one token's keys together: they differ from the 25th bit on."""
    r = np.random.RandomState(E)
    l = (2 * r.standard_normal(E)).astype(np.float32)
    s = 1 / (1 + np.exp(-l.astype(np.float64)))
    if scores == "softmax":
        s = np.exp(l.astype(np.float64) - l.max())
        s /= s.sum()
    bias = (0.75 - s).astype(np.float32)
    x = torch.from_numpy(np.stack([l, l + np.float32(0.01), l[::-1].copy()])).to(cuda_device)
    check(x, 10, cuda_device, bias, scores=scores, groups=groups, top_groups=top, group_best=best)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("groups,top,best,E", [(1, 1, 2, 256), (8, 3, 2, 256), (8, 3, 1, 256), (4, 2, 2, 1000), (32, 9, 2, 64)])
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
def test_all_alike(scores, groups, top, best, E, dtype, cuda_device):
    """All logits the same, or of two values, with no bias, the same for all, or one in doubt: more ties than are looked at
    one by one."""
    r = np.random.RandomState(11)
    x = torch.from_numpy(np.stack([np.full(E, 0.5), np.where(r.rand(E) < 0.5, 0.5, 0.25), np.full(E, -60.0),
                                   np.where(np.arange(E) % 7 == 3, 1.0, 0.5)])).to(dtype).to(cuda_device)
    kw = dict(scores=scores, groups=groups, top_groups=top, group_best=best)
    for K in (1, 9):
        if K <= top * (E // groups):
            check(x, K, cuda_device, **kw)
            check(x, K, cuda_device, np.zeros(E), **kw)
            check(x, K, cuda_device, np.full(E, 0.125), **kw)
            check(x, K, cuda_device, np.where(np.arange(E) % 50 == 49, 0.125 + 2.0 ** -24, 0.125), **kw)


@pytest.mark.parametrize("E,K", [(256, 8), (1000, 12), (64, 60)])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_logits_of_neighbouring_bits(E, K, dtype, cuda_device):
    """FP32 logits that differ in their last bits alone, and such pairs among others."""
    r = np.random.RandomState(12)
    one = np.float32(1.0) + np.float32(2.0 ** -23) * r.permutation(E).astype(np.float32)
    pairs = np.repeat(r.standard_normal(E // 2).astype(np.float32), 2)
    pairs[1::2] = np.nextafter(pairs[1::2], np.float32(10))
    x = torch.from_numpy(np.stack([one, -one, pairs, pairs[r.permutation(E)]])).to(dtype).to(cuda_device)
    for scores in ("softmax", "sigmoid"):
        check(x, K, cuda_device, scores=scores)


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("renormalise", [False, True])
@pytest.mark.parametrize("groups,top,best", [(1, 1, 2), (4, 2, 2), (4, 2, 1)])
def test_masked_and_infinite(scores, biased, renormalise, groups, top, best, cuda_device):
    x = make(12, 64, FP32, cuda_device, 6)
    inf, nan = float("inf"), float("nan")
    x[0] = -inf
    x[1] = nan
    x[2, 5:] = -inf           # fewer than K are left
    x[3, 10:20] = nan
    x[4, 7] = x[4, 40] = inf
    x[5] = inf
    x[6] = -inf
    x[6, 50] = -3.0           # one alone, in the last group
    x[7] = -200.0             # far below what a sigmoid of 32 bits holds
    x[7, 9] = -190.0
    x[8] = 100.0
    x[9, :32] = -inf
    x[10] = -3e38
    x[10, 3] = 3e38
    bias = np.random.RandomState(7).standard_normal(64) if biased else None
    ids, w = check(x, 8, cuda_device, bias, scores=scores, renormalise=renormalise, groups=groups, top_groups=top,
                   group_best=best)
    assert bool(torch.isfinite(w).all()) and not bool(w[:2].any())


def test_bias_that_is_infinite(cuda_device):
    x = make(5, 64, BF16, cuda_device, 8)
    bias = np.zeros(64)
    bias[10], bias[20], bias[30] = np.inf, -np.inf, np.nan
    ids, _ = check(x, 8, cuda_device, bias, scores="sigmoid")
    assert bool((ids[:, 0] == 10).all()) and not bool(((ids == 20) | (ids == 30)).any())


def test_results_in_given_tensors(cuda_device):
    x = make(6, 128, BF16, cuda_device, 9)
    ids = torch.empty(6, 8, dtype=torch.int32, device=cuda_device)
    w = torch.empty(6, 8, device=cuda_device)
    a, b = wd.route(x, 8, ids=ids, weights=w)
    assert a is ids and b is w
    fresh = wd.route(x, 8)
    assert torch.equal(fresh[0], ids) and torch.equal(fresh[1], w)
    assert wd.route(x[:0], 8)[0].shape == (0, 8)
