"""wd_rms_norm with any eps that it accepts, also where squares or their sum with it leave FP32, on the GPU.

Tolerance as in tests/test_gpu_norm.py: one rounding of the type and 2^-18 of the value.
"""
import numpy as np
import pytest
import torch

import moe_decode_gate_gb300 as wd
import step_reference as ref

pytestmark = pytest.mark.gpu

FP32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("H", [1, 24, 200, 512, 2048, 2049, 16384])
@pytest.mark.parametrize("eps", [1e-37, 1e-6, 1.0, 1e20, 1e30, 1e36, 1e38, 3.4e38])
def test_any_eps(eps, H, dtype, cuda_device):
    base = np.random.RandomState(H).standard_normal((9, H))
    base /= np.abs(base).max(1, keepdims=True)
    x = torch.from_numpy(base * np.array([1e-3, 1.0, 1e10, 1e15, 3e18, 1e19, 1e20, 1e30, 3e38])[:, None]).to(dtype)
    w = torch.from_numpy(np.random.RandomState(1).standard_normal(H)).to(dtype)
    want = ref.rms_norm(x.double().numpy(), w.double().numpy(), None, float(np.float32(eps)))[0]
    got = wd.rms_norm(x.to(cuda_device), w.to(cuda_device), eps=eps).double().cpu().numpy()
    tol = (torch.finfo(dtype).eps / 2 + 2.0 ** -18) * np.abs(want) + (2.0 ** -134 if dtype is BF16 else 2.0 ** -150)
    assert (np.abs(got - want) <= tol).all()
    assert bool(wd.rms_norm(torch.full((2, H), float("inf"), dtype=dtype, device=cuda_device), eps=eps).isnan().all())
