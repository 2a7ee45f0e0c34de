"""wd_adjust_logits on the GPU against the plain 64-bit reference (tests/step_reference.py).

Tolerance: each of the steps is one or two FP32 roundings of what is summed up to then (quotient, product and sum of
the penalties, their difference, the bias' sum, the temperature's reciprocal and product), 8 2^-24 of the magnitudes in
all, one more for each further bias of the same token, and one rounding to the output's type.
"""
import numpy as np
import pytest
import torch

import moe_decode_gate_gb300 as wd
import step_reference as ref

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
LEAST = {BF16: 2.0 ** -134, FP16: 2.0 ** -25, FP32: 2.0 ** -150}


def ints(a, dev):
    return torch.from_numpy(np.asarray(a, np.int32)).to(dev)


def floats(a, dev):
    return None if a is None else torch.from_numpy(np.asarray(a, np.float32)).to(dev)


def check(x, dev, dtype=None, out=None, bias=None, **kw):
    """x: the logits on the device; the rest numpy, as the reference takes them."""
    tensors = {n: (ints if n in ("history", "lengths", "prompt_lengths", "seqs", "mask") else floats)(v, dev)
               for n, v in kw.items()}
    b = None if bias is None else (ints(bias[0], dev), ints(bias[1], dev), floats(bias[2], dev))
    values = {n: v if n in ("history", "lengths", "prompt_lengths", "seqs") else v.astype(np.uint32) if n == "mask"
              else np.asarray(v, np.float32).astype(np.float64) for n, v in kw.items()}
    ref_bias = None if bias is None else (bias[0], bias[1], np.asarray(bias[2], np.float32))
    want, mag = ref.adjust_logits(x.double().cpu().numpy(), bias=ref_bias, **values)
    got = wd.adjust_logits(x, bias=b, dtype=dtype, out=out, **tensors)
    to = dtype or (out.dtype if out is not None else x.dtype)
    assert got.dtype == to and got.shape == x.shape
    g = got.double().cpu().numpy()
    assert np.array_equal(np.isnan(g), np.isnan(want))
    assert np.array_equal(np.isinf(g), np.isinf(want)) and np.array_equal(g[np.isinf(g)], want[np.isinf(g)])
    fine = np.isfinite(want)
    g, want, mag = g[fine], want[fine], mag[fine]
    further = 0
    if bias is not None:
        start, ids = np.asarray(bias[0]), np.asarray(bias[1])
        rows = [ids[max(0, lo):max(0, hi)] for lo, hi in zip(start[:-1], start[1:])]
        further = max([int(np.unique(i, return_counts=True)[1].max()) - 1 for i in rows if i.size], default=0)
    tol = (8 + further) * 2.0 ** -24 * mag + torch.finfo(to).eps / 2 * np.abs(want) * (1 + 2.0 ** -10) + LEAST[to]
    assert (np.abs(g - want) <= tol).all()
    return got


def request(B, V, columns, seed=0, slots=None):
    """A batch with everything: settings, histories with repeats, biases, masks."""
    r = np.random.RandomState(seed)
    slots = slots or B + 2
    kw = dict(history=np.minimum((r.rand(slots, columns) ** 3 * V).astype(np.int32), V - 1),
              lengths=r.randint(0, columns + 1, slots), prompt_lengths=r.randint(0, columns + 1, slots),
              seqs=r.permutation(slots)[:B], repetition=r.uniform(0.7, 1.5, B), presence=r.uniform(-1, 1, B),
              frequency=r.uniform(-0.5, 1, B), temperature=r.uniform(0.3, 2, B),
              mask=r.randint(-2 ** 31, 2 ** 31, (B, (V + 31) // 32)))
    n = r.randint(0, min(V, 20) + 1, B)
    start = np.concatenate(([0], np.cumsum(n)))
    kw["bias"] = (start, r.randint(0, V, start[-1]), r.standard_normal(start[-1]))
    return kw


def make(B, V, dtype, dev, seed=0):
    return torch.from_numpy(3 * np.random.RandomState(seed).standard_normal((B, V))).to(dtype).to(dev)


@pytest.mark.parametrize("V", [1, 2, 3, 5, 31, 32, 33, 1000, 1023, 1024, 1025, 1027, 4096, 4099, 32768, 100003])
@pytest.mark.parametrize("B", [1, 3])
@pytest.mark.parametrize("dtype,to", [(BF16, FP32), (BF16, BF16), (FP16, FP16), (FP16, FP32), (FP32, FP32)])
def test_sizes(B, V, dtype, to, cuda_device):
    check(make(B, V, dtype, cuda_device, V), cuda_device, dtype=to, **request(B, V, 300, V))


def test_many_rows(cuda_device):
    check(make(150, 20011, BF16, cuda_device, 1), cuda_device, dtype=FP32, **request(150, 20011, 2000, 1))


@pytest.mark.parametrize("left_out", [
    ("history", "lengths", "prompt_lengths", "seqs", "repetition", "presence", "frequency"), ("prompt_lengths",), ("seqs",),
    ("repetition",), ("presence",), ("frequency",), ("repetition", "frequency"), ("bias",), ("temperature",), ("mask",),
    ("bias", "temperature", "mask"), ("repetition", "presence", "frequency"),
    ("history", "lengths", "prompt_lengths", "seqs", "repetition", "presence", "frequency", "bias", "temperature", "mask")])
def test_what_is_left_out_changes_nothing(left_out, cuda_device):
    kw = {n: v for n, v in request(4, 5003, 100, 2).items() if n not in left_out}
    x = make(4, 5003, BF16, cuda_device, 2)
    got = check(x, cuda_device, dtype=FP32, **kw)
    if not kw:
        assert torch.equal(got, x.float())


@pytest.mark.parametrize("V", [4096, 4099])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_strides_and_places(V, dtype, cuda_device):
    """Rows apart, rows that start anywhere, results in place and in part of a larger tensor."""
    kw = request(5, V, 64, 3)
    wide = make(5, V + 9, dtype, cuda_device, 3)
    for at in (0, 1, 2, 5, 8):
        check(wide[:, at:at + V], cuda_device, dtype=FP32, **kw)
        out = torch.full((5, V + 9), 7.0, dtype=dtype, device=cuda_device)
        check(wide[:, at:at + V], cuda_device, out=out[:, 1:V + 1], **kw)
        assert bool((out[:, :1] == 7).all()) and bool((out[:, V + 1:] == 7).all())
    x = make(5, V, dtype, cuda_device, 4)
    fresh = check(x, cuda_device, **kw)
    tensors = {n: (ints if n in ("history", "lengths", "prompt_lengths", "seqs", "mask") else floats)(v, cuda_device)
               for n, v in kw.items() if n != "bias"}
    b = kw["bias"]
    tensors["bias"] = (ints(b[0], cuda_device), ints(b[1], cuda_device), floats(b[2], cuda_device))
    assert wd.adjust_logits(x, out=x, **tensors) is x
    assert torch.equal(x, fresh)
    part = torch.zeros(5, V + 3, dtype=dtype, device=cuda_device)
    x = make(5, V, dtype, cuda_device, 4)
    part[:, 2:V + 2] = x
    wd.adjust_logits(part[:, 2:V + 2], out=part[:, 2:V + 2], **tensors)
    assert torch.equal(part[:, 2:V + 2], fresh) and not bool(part[:, :2].any()) and not bool(part[:, V + 2:].any())


def test_what_is_out_of_range_counts_for_nothing(cuda_device):
    V = 3001
    kw = request(6, V, 50, 5)
    kw["history"][:, ::3] = np.array([-1, V, V + 5, 2 ** 31 - 1, -2 ** 31, 7, V - 1] * 3)[:17]
    kw["lengths"] = np.array([10 ** 6, -5, 50, 0, 13, 2 ** 31 - 1, 50, -2 ** 31])
    kw["prompt_lengths"] = np.array([-7, 3, 10 ** 9, 5, 13, 4, 0, 0])
    kw["seqs"] = np.array([0, 8, -1, 2, 5, 2 ** 31 - 1])
    start, ids, values = np.array([0, 4, 4, 2, 6, 900, 8]), np.array([5, 5, -1, V, 9, 2 ** 31 - 1, 0, 3]), np.arange(8.0) + 1
    check(make(6, V, BF16, cuda_device, 5), cuda_device, dtype=FP32, **{**kw, "bias": (start, ids, values)})


@pytest.mark.parametrize("columns", [10, 40000])
@pytest.mark.parametrize("B,V", [(1, 203), (3, 9001), (80, 16411)])
@pytest.mark.parametrize("times", [2, 3, 50])
def test_biases_of_a_token_add_up(times, B, V, columns, cuda_device):
    """In their order, the same from run to run; for histories of both kinds and slices of all sizes."""
    r = np.random.RandomState(times)
    rows = []
    for b in range(B):
        ids = np.concatenate((np.full(times, 77 + b), np.full(3, V - 1), np.zeros(2), r.randint(0, V, 40), [-1, -1, V]))
        rows.append(r.permutation(ids).astype(np.int32))
    start, ids = rows[0].size * np.arange(B + 1), np.concatenate(rows)
    kw = request(B, V, columns, 6)
    kw["bias"] = (start, ids, 100 * r.standard_normal(ids.size))
    x = make(B, V, FP32, cuda_device, 6)
    got = check(x, cuda_device, **kw)
    for _ in range(3):
        assert torch.equal(check(x, cuda_device, **kw), got)
    wide = torch.empty((B, V + 3), device=cuda_device)[:, 1:V + 1]  # rows that reach an alignment elsewhere than the input's
    assert torch.equal(check(x, cuda_device, out=wide, **kw), got)


@pytest.mark.parametrize("columns", [10, 40000])
def test_many_tokens_of_several_biases(columns, cuda_device):
    """More than a CTA keeps the sums of, in large slices and with small ones."""
    r = np.random.RandomState(15)
    for B, V, tokens in ((608, 8192, 1300), (1, 1024, 1024), (2, 1500, 1100)):
        ids = r.permutation(np.concatenate((r.permutation(V)[:tokens], r.permutation(V)[:tokens], r.permutation(V)[:tokens])))
        kw = request(B, V, columns, 16)
        kw["bias"] = (ids.size * (np.arange(B + 1) > B // 2), ids, 10 * r.standard_normal(ids.size))
        x = make(B, V, FP32, cuda_device, 17)
        got = check(x, cuda_device, **kw)
        assert torch.equal(check(x, cuda_device, **kw), got)


def test_a_token_a_million_times(cuda_device):
    """The longest history, all of it one token but the last."""
    n = 1 << 20
    h = np.full((1, n), 1234, np.int32)
    h[0, -1] = 5
    kw = dict(history=h, lengths=np.array([n]), frequency=np.array([1e-3]), presence=np.array([0.5]))
    got = check(make(1, 5000, FP32, cuda_device, 7), cuda_device, **kw)
    assert float(got[0, 1234]) < -1000


@pytest.mark.parametrize("columns", [32767, 32768, 32770])
@pytest.mark.parametrize("prompt", [0, 5, 32767])
def test_as_many_tokens_as_a_word_counts(columns, prompt, cuda_device):
    """Histories up to the longest that a count of 15 bits beside the prompt's bit holds, and just beyond, with a bias of
    each token in the same words."""
    V = 1500
    h = np.full((2, columns), 1234, np.int32)
    h[1] = np.arange(columns) % 3
    kw = dict(history=h, lengths=np.array([columns, columns - 1]), prompt_lengths=np.array([prompt, prompt]),
              repetition=np.array([1.25, 0.5]), frequency=np.array([1e-3, 2e-3]), presence=np.array([0.5, -0.25]),
              bias=(np.array([0, V, 2 * V]), np.tile(np.arange(V), 2), np.linspace(-1, 1, 2 * V)))
    check(make(2, V, FP32, cuda_device, 11), cuda_device, **kw)


@pytest.mark.parametrize("n", [32767, 32768, 70001])
def test_as_many_biases_as_a_word_counts(n, cuda_device):
    r = np.random.RandomState(n)
    V = 80000
    ids = r.permutation(V)[:n]
    ids[-3:] = ids[0]  # and one token four times
    kw = request(1, V, 100, 12)
    kw["bias"] = (np.array([0, n]), ids, r.standard_normal(n))
    check(make(1, V, FP32, cuda_device, 12), cuda_device, **kw)


def test_temperatures(cuda_device):
    x = make(6, 1000, BF16, cuda_device, 8)
    t = np.array([0.0, -1.0, np.nan, 1.0, 1e-3, np.inf])
    got = wd.adjust_logits(x, temperature=floats(t, cuda_device), dtype=FP32)
    assert torch.equal(got[:4], x[:4].float()) and not bool(got[5].any())
    want = x[4].double() * 1000
    assert float(((got[4].double() - want).abs() / want.abs().clamp(min=1e-30)).max()) < 2.0 ** -22


def test_infinite_and_missing_logits(cuda_device):
    V = 2050
    x = make(3, V, BF16, cuda_device, 9)
    x[0, ::7] = -float("inf")
    x[1, ::5] = float("nan")
    x[2, 3] = float("inf")
    kw = request(3, V, 200, 9)
    kw["mask"][1] = 0          # NaN where nothing is allowed
    kw["mask"][0] = -1
    got = check(x, cuda_device, dtype=FP32, **kw)
    assert bool((got[1] == -float("inf")).all())


def test_same_from_run_to_run(cuda_device):
    kw = request(40, 30011, 5000, 10)
    x = make(40, 30011, BF16, cuda_device, 10)
    first = check(x, cuda_device, dtype=FP32, **kw)
    for _ in range(3):
        assert torch.equal(check(x, cuda_device, dtype=FP32, **kw), first)


def test_no_rows(cuda_device):
    assert wd.adjust_logits(make(2, 100, BF16, cuda_device)[:0]).shape == (0, 100)
