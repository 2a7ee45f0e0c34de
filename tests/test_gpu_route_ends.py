"""wd_route at the ends of what its arguments may be, on the GPU."""
import numpy as np
import pytest
import torch

import moe_decode_gate_gb300 as wd
import step_reference as ref

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,top,K", [(32, 7, 3), (8, 5, 5), (5, 2, 2), (1, 1, 1)])
@pytest.mark.parametrize("best", [1, 2])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_groups_of_one_go_by_their_logits(E, top, K, best, scores, dtype, cuda_device):
    """Without a bias keys order as logits do, also where scores no longer tell them apart: sigmoids beyond 37, and what is
    more than 745 below a softmax' largest."""
    r = np.random.RandomState(E)
    x = torch.from_numpy(np.stack([r.permutation(E) + 40.0, 2.0 * r.permutation(E) + 64.0, 50.0 * r.permutation(E) - 4000.0,
                                   np.where(r.permutation(E) < 2, 5000.0, r.permutation(E) - 300.0),
                                   r.randint(0, 3, E) + 50.0])).to(dtype)
    ids, _ = wd.route(x.to(cuda_device), K, scores=scores, groups=E, top_groups=top, group_best=best)
    want = np.argsort(-x.double().numpy(), 1, kind="stable")[:, :K]
    assert np.array_equal(ids.cpu().numpy(), want)


def compare(x, K, bias, dev, **kw):
    args = dict(scores="sigmoid", groups=1, top_groups=1, group_best=2, renormalise=True, scale=1.0)
    args.update(kw)
    b = torch.from_numpy(np.asarray(bias, np.float32))
    ids, w = wd.route(x.to(dev), K, bias=b.to(dev), **args)
    want, want_w = ref.route(x.double().numpy(), K, bias=b.double().numpy(), **args)
    assert np.array_equal(ids.cpu().numpy(), want)
    assert (np.abs(w.double().cpu().numpy() - want_w) <= 2.0 ** -18 * np.abs(want_w) + 2.0 ** -126).all()


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("best", [1, 2])
@pytest.mark.parametrize("E,groups,top", [(64, 8, 2), (64, 8, 3), (1000, 4, 2), (96, 32, 5)])
def test_infinite_and_huge_biases_in_groups(E, groups, top, best, scores, cuda_device):
    """Several infinite ones in one group, and sums of two that FP32 does not hold, up and down."""
    r, size = np.random.RandomState(E + top), E // groups
    x = torch.from_numpy(r.standard_normal((9, E)).astype(np.float32))
    x[1, 2 * size:3 * size] = -float("inf")
    x[2, :size] = -float("inf")
    kw = dict(scores=scores, groups=groups, top_groups=top, group_best=best)
    infinite = r.standard_normal(E)
    infinite[2 * size:2 * size + 3] = np.inf
    infinite[3 * size] = np.inf
    infinite[0] = -np.inf
    compare(x, 4, infinite, cuda_device, **kw)
    high = np.full(E, 1.0)
    high[0:2], high[size:size + 2], high[2 * size:2 * size + 2], high[3 * size] = 3.0e38, 3.2e38, 3.1e38, 3.3e38
    compare(x, 4, high, cuda_device, **kw)
    compare(x, 4, high[::-1].copy(), cuda_device, **kw)
    low = -np.linspace(2.9e38, 3.3e38, E)
    compare(x, 4, low, cuda_device, **kw)
    compare(x, 4, low[::-1].copy(), cuda_device, **kw)


@pytest.mark.parametrize("scale", [1e30, 3e38, -1e35])
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalise", [False, True])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_any_scale(dtype, renormalise, scores, scale, cuda_device):
    r = np.random.RandomState(5)
    x = torch.from_numpy(np.stack([r.standard_normal(64), r.standard_normal(64) - 37.0, r.uniform(-39, -30, 64)])).to(dtype)
    ids, w = wd.route(x.to(cuda_device), 6, scores=scores, renormalise=renormalise, scale=scale)
    s = float(np.float32(scale))
    want, want_w = ref.route(x.double().numpy(), 6, scores, None, 1, 1, 2, renormalise, s)
    assert np.array_equal(ids.cpu().numpy(), want)
    assert (np.abs(w.double().cpu().numpy() - want_w) <= 2.0 ** -18 * np.abs(want_w) + 2.0 ** -126).all()
