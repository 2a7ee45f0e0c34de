"""wd_rms_norm on the GPU against the plain 64-bit reference (tests/step_reference.py).

Tolerances.  r: one FP32 addition (2^-24 of r) and one rounding to the type.  y: the sum of squares is at most 32
additions in a thread, 5 shuffles and 16 warps, each within 2^-24 of the sum, so the root is within 27 2^-24 of itself;
rsqrtf 2 units, the division, the addition of eps and two products with r's own rounding another 7: below 2^-18 in
all, and one rounding to the type; FP16 keeps values below 2^-14 to 2^-25.  MXFP8: half a step of E4M3 at the value in units of its block (2^-4
of it, 2^-10 for the smallest), and 2^-18 of the value.
"""
import numpy as np
import pytest
import torch

import moe_decode_gate_gb300 as wd
import step_reference as ref

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
HALF_STEP = {t: torch.finfo(t).eps / 2 for t in (BF16, FP16, FP32)}
LEAST = {BF16: 2.0 ** -134, FP16: 2.0 ** -25, FP32: 2.0 ** -150}


def make(shape, dtype, dev, seed=0, scale=1.0):
    r = np.random.RandomState(seed)
    t = torch.from_numpy(scale * r.standard_normal(shape)).to(dtype)
    return t.to(dev), t.double().numpy()


def check_y(got, want, dtype):
    got = got.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(want))
    fine = np.isfinite(want)
    tol = (HALF_STEP[dtype] + 2.0 ** -18) * np.abs(want) + LEAST[dtype]
    assert (np.abs(got - want)[fine] <= tol[fine]).all(), np.nanmax((np.abs(got - want) / tol)[fine])


def check_sum(got, want, dtype):
    err = np.abs(got.double().cpu().numpy() - want)
    assert (err <= (HALF_STEP[dtype] * (1 + 2.0 ** -10) + 2.0 ** -24) * np.abs(want) + LEAST[dtype]).all()


def check_mxfp8(codes, scales, want):
    codes, scales = codes.cpu().numpy(), scales.cpu().numpy()
    b = want.reshape(*want.shape[:-1], -1, 32)
    top = np.abs(b).max(-1)

    def scale(a):
        return np.where(a > 0, np.clip(np.floor(np.log2(np.where(a > 0, a, 1.0))) - 8, -127, 127) + 127, 127)

    # the scale of a maximum within the tolerance
    assert ((scales == scale(top * (1 - 2.0 ** -18))) | (scales == scale(top * (1 + 2.0 ** -18)))).all()
    unit = ref.e8m0_values(scales)[..., None]
    z = np.clip(b / unit, -448, 448)
    got = ref.e4m3_values(codes).reshape(b.shape)
    half = np.maximum(2.0 ** -10, np.exp2(np.floor(np.log2(np.maximum(np.abs(z), 2.0 ** -20))) - 4))
    assert (np.abs(got - z) <= half * (1 + 2.0 ** -14) + 2.0 ** -18 * np.abs(z)).all()


SIZES = [(1, 1), (3, 7), (5, 32), (2, 250), (4, 256), (3, 264), (2, 511), (3, 512), (2, 520), (5, 1000), (3, 1024),
         (2, 1032), (3, 2048), (2, 2049), (1, 4096), (2, 4104), (3, 5001), (2, 8192), (2, 8200), (1, 16377), (2, 16384)]


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("T,H", SIZES)
def test_sizes(T, H, dtype, cuda_device):
    x, xv = make((T, H), dtype, cuda_device, 1)
    res, rv = make((T, H), dtype, cuda_device, 2, 3.0)
    w, wv = make((H,), dtype, cuda_device, 3)
    want, r = ref.rms_norm(xv, wv, rv, 1e-6)
    y, total = wd.rms_norm(x, w, res)
    assert y.dtype == total.dtype == dtype and y.shape == total.shape == x.shape
    check_y(y, want, dtype)
    check_sum(total, r, dtype)
    check_y(wd.rms_norm(x), ref.rms_norm(xv, None, None, 1e-6)[0], dtype)


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("T,H", [(1, 32), (3, 256), (2, 480), (5, 512), (3, 992), (7, 2048), (2, 4096), (2, 9600), (1, 16384)])
@pytest.mark.parametrize("shift", [0, 1])
def test_mxfp8(T, H, dtype, shift, cuda_device):
    """Also with rows that are not aligned (shift)."""
    x, xv = make((T, H + shift), dtype, cuda_device, 4)
    x, xv = x[:, shift:], xv[:, shift:]
    res, rv = make((T, H), dtype, cuda_device, 5, 10.0)
    w, wv = make((H,), FP32, cuda_device, 6, 20.0)
    want, r = ref.rms_norm(xv, wv, rv, 1e-5)
    y = torch.empty(T, H, dtype=dtype, device=cuda_device)
    codes, scales, total = wd.rms_norm(x, w, res, eps=1e-5, mxfp8=True, out=y)
    assert codes.shape == (T, H) and scales.shape == (T, H // 32) and codes.dtype == scales.dtype == torch.uint8
    check_mxfp8(codes, scales, want)
    check_y(y, want, dtype)
    check_sum(total, r, dtype)
    alone = wd.rms_norm(x, w, res, eps=1e-5, mxfp8=True)
    assert all(torch.equal(a, b) for a, b in zip(alone, (codes, scales, total)))


@pytest.mark.parametrize("shift", [0, 1])
def test_mxfp8_blocks_at_the_ends(shift, cuda_device):
    """Blocks of zeros, of tiny and huge numbers, and one that is not finite for its weights."""
    H = 256
    x, xv = make((2, H + shift), FP32, cuda_device, 7)
    x, xv = x[:, shift:], xv[:, shift:]
    w = np.ones(H, np.float32)
    w[:32], w[32:64], w[64:96], w[100] = 0.0, 1e-38, 1e38, np.inf
    codes, scales = wd.rms_norm(x, torch.from_numpy(w).to(cuda_device), mxfp8=True)
    assert bool((scales[:, 0] == 127).all()) and not bool((codes[:, :32] & 127).any())
    assert bool((scales[:, 3] == 255).all()) and not bool(codes[:, 96:128].any())
    want = ref.rms_norm(xv, w.astype(np.float64), None, 1e-6)[0]
    keep = np.r_[32:96, 128:256]
    check_mxfp8(codes[:, keep].contiguous(), scales[:, [1, 2, 4, 5, 6, 7]].contiguous(), want[:, keep])


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("D", [64, 128, 100])
def test_heads_of_a_projection(D, dtype, cuda_device):
    """Norms of each head, read out of the rows of a fused projection."""
    T, heads = 6, 5
    qkv, v = make((T, (heads + 2) * D + 3), dtype, cuda_device, 8)
    x = qkv[:, D:(heads + 1) * D].unflatten(1, (heads, D))
    w, wv = make((D,), dtype, cuda_device, 9)
    want = ref.rms_norm(v[:, D:(heads + 1) * D].reshape(T, heads, D), wv, None, 1e-6)[0]
    y = wd.rms_norm(x, w)
    assert y.shape == (T, heads, D) and y.is_contiguous()
    check_y(y, want, dtype)
    turned = qkv[:, D:(heads + 1) * D].unflatten(1, (heads, D)).transpose(0, 1)  # heads first
    check_y(wd.rms_norm(turned, w), want.transpose(1, 0, 2), dtype)


def test_in_place(cuda_device):
    x, xv = make((70, 640), BF16, cuda_device, 10)
    res, rv = make((70, 640), BF16, cuda_device, 11)
    fresh = wd.rms_norm(x, None, res)
    y, total = wd.rms_norm(x, None, res, out=x, residual_out=res)
    assert y is x and total is res
    assert torch.equal(x, fresh[0]) and torch.equal(res, fresh[1])


@pytest.mark.parametrize("T,H", [(2, 200), (3, 2048), (2, 16384)])
def test_any_finite_row_has_its_norm(T, H, cuda_device):
    x, xv = make((T, H), FP32, cuda_device, 12)
    for scale in (1e30, 2.0 ** 125, 1e-20):
        big = x / x.abs().max() * scale
        want = ref.rms_norm(big.double().cpu().numpy(), None, None, 1e-6)[0]
        check_y(wd.rms_norm(big), want, FP32)
    zero = torch.zeros(T, H, device=cuda_device, dtype=BF16)
    assert not bool(wd.rms_norm(zero).any())


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("H", [100, 256, 2048])
def test_a_row_that_is_not_finite_is_nan_and_alone(H, bad, cuda_device):
    x, xv = make((9, H), BF16, cuda_device, 13)
    clean = wd.rms_norm(x)
    x[4, H // 2] = bad
    y = wd.rms_norm(x)
    assert bool(y[4].isnan().all())
    rest = [i for i in range(9) if i != 4]
    assert torch.equal(y[rest], clean[rest])


def test_many_rows(cuda_device):
    """More rows than there are CTAs at once, and none."""
    x, xv = make((50001, 64), FP16, cuda_device, 14)
    check_y(wd.rms_norm(x), ref.rms_norm(xv, None, None, 1e-6)[0], FP16)
    assert wd.rms_norm(x[:0]).shape == (0, 64)
    y, r = wd.rms_norm(x[:0], None, x[:0])
    assert y.shape == r.shape == (0, 64)


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("T,H", [(9800, 64), (9800, 72), (9801, 128), (9800, 200), (9803, 256), (9800, 100), (1217, 1040),
                                 (1300, 1500), (1216, 2048), (1217, 2049), (1216, 4104), (1216, 9000)])
def test_many_rows_of(T, H, dtype, cuda_device):
    """Where rows are many a thread has more of each."""
    x, xv = make((T, H), dtype, cuda_device, 16)
    w, wv = make((H,), dtype, cuda_device, 17)
    check_y(wd.rms_norm(x, w), ref.rms_norm(xv, wv, None, 1e-6)[0], dtype)
    res, rv = make((T, H), dtype, cuda_device, 18, 3.0)
    want, r = ref.rms_norm(xv, wv, rv, 1e-6)
    y, total = wd.rms_norm(x, w, res)
    check_y(y, want, dtype)
    check_sum(total, r, dtype)
    if H % 32 == 0:
        check_mxfp8(*wd.rms_norm(x, w, mxfp8=True), ref.rms_norm(xv, wv, None, 1e-6)[0])


@pytest.mark.parametrize("H", [37, 500, 777, 3001])
@pytest.mark.parametrize("shift", range(9))
def test_rows_that_begin_anywhere(H, shift, cuda_device):
    """All tensors alike, and each at a place of its own; nothing around the results changes."""
    T = 5
    for dtype in (BF16, FP32):
        flat, fv = make((T * H + shift,), dtype, cuda_device, 19)
        x, xv = flat[shift:].view(T, H), fv[shift:].reshape(T, H)
        res, rv = make((T, H), dtype, cuda_device, 20)
        want, r = ref.rms_norm(xv, None, rv, 1e-6)
        for at in (shift, 3):
            room = torch.full((2, T * H + 20,), 7.0, dtype=dtype, device=cuda_device)
            y, total = (t[at:at + T * H].view(T, H) for t in room)
            wd.rms_norm(x, None, res, out=y, residual_out=total)
            check_y(y, want, dtype)
            check_sum(total, r, dtype)
            assert bool((room[:, :at] == 7).all()) and bool((room[:, at + T * H:] == 7).all())


def test_offsets_beyond_32_bits(cuda_device):
    """Rows so far apart that their offsets in elements pass 2^32."""
    base = torch.empty(2 ** 33 + 128, dtype=torch.uint8, device=cuda_device).view(BF16)
    x = base.as_strided((3, 64), (2 ** 31, 1))
    x.copy_(make((3, 64), BF16, cuda_device, 15)[0])
    want = ref.rms_norm(x.double().cpu().numpy(), None, None, 1e-6)[0]
    check_y(wd.rms_norm(x), want, BF16)
