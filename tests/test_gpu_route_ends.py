"""wd_route at the ends of what its arguments may be, on the GPU."""
import numpy as np
import pytest
import torch

import moe_decode_gate_gb300 as wd

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
