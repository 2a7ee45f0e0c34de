"""wd_route where two experts' keys are within an FP32 step of each other, at biases of any level, on the GPU.

Two experts are open (a softmax has a third, far behind, that takes a share of it), and each token's logits bring their keys
together.  The ids have to be those of the keys in 64 bits.
"""
import numpy as np
import pytest
import torch

import moe_decode_gate_gb300 as wd

pytestmark = pytest.mark.gpu

TOKENS = 200_000


def places(E):
    """Pairs of experts at the first and last places of their lanes (a lane has 4 to 32 neighbouring experts)."""
    per_lane = 1
    while 32 * per_lane < E:
        per_lane *= 2
    last = per_lane - 1
    return [(0, last), (last, 0), (0, per_lane), (0, 2 * per_lane + last), (3 * per_lane + last, per_lane)]


def tokens(scores, E, a, b, c, bias, seed):
    """FP32 logits [TOKENS, E] on the CPU of which a and b (and c) are open, and the better of a and b in 64 bits."""
    r = np.random.RandomState(seed)
    apart = float(bias[b]) - float(bias[a])  # score a is ahead of score b by this much
    x = np.full((TOKENS, E), -np.inf, np.float32)
    if scores == "sigmoid":
        s = r.uniform(max(0.0, apart) + 0.02, min(1.0, 1.0 + apart) - 0.02, TOKENS)
        x[:, a] = np.log(s / (1 - s))
        s = 1 / (1 + np.exp(-x[:, a].astype(np.float64))) - apart
        x[:, b] = np.log(s / (1 - s))
    else:
        # shares p, p - apart and the rest
        p = r.uniform(max(0.0, apart) + 0.02, 0.5 + apart / 2 - 0.02, TOKENS)
        x[:, a], x[:, c] = np.log(p), np.log(1 - 2 * p + apart)
        x[:, b] = np.log(p - apart)
    x[:, b] += (r.randint(-2, 3, TOKENS) * 2.0 ** -24).astype(np.float32)
    l = x[:, [a, b, c]].astype(np.float64)
    if scores == "sigmoid":
        s = 1 / (1 + np.exp(-l[:, :2]))
    else:
        s = np.exp(l) / np.exp(l).sum(1, keepdims=True)
    key = s[:, :2] + bias[[a, b]].astype(np.float64)
    first = (key[:, 0] > key[:, 1]) | ((key[:, 0] == key[:, 1]) & (a < b))
    assert np.abs(key[:, 0] - key[:, 1]).max() < 1e-6 * max(1.0, np.abs(key).max())
    return torch.from_numpy(x), np.where(first, a, b)


@pytest.mark.parametrize("scores", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,level", [(128, 15.6), (256, 3.7), (256, 16.0), (512, 0.9), (512, 1.6), (512, 4.0), (1000, 0.6),
                                     (1000, 1.0), (1000, 4.0)])
def test_two_keys_at_any_level(E, level, scores, cuda_device):
    for i, (a, b) in enumerate(places(E)):
        bias = np.full(E, level, np.float32)
        bias[b] += np.float32(0.1)
        c = E - 1
        bias[c] -= 10
        x, want = tokens(scores, E, a, b, c, bias, E + i)
        x, bias = x.to(cuda_device), torch.from_numpy(bias).to(cuda_device)
        ids, _ = wd.route(x, 1, scores=scores, bias=bias)
        wrong = int((ids[:, 0].cpu().numpy() != want).sum())
        assert wrong == 0, f"{wrong} of {TOKENS} tokens, experts {a} and {b}"


@pytest.mark.parametrize("E,level", [(256, 3.7), (512, 1.6), (1000, 0.6)])
@pytest.mark.parametrize("best", [1, 2])
@pytest.mark.parametrize("top", [1, 2])
def test_two_keys_in_groups(E, level, top, best, cuda_device):
    """Both in one group, and one in each of two."""
    groups = 8 if E % 8 == 0 else 2
    size = E // groups
    for i, (a, b) in enumerate([(0, size // 4 - 1), (size // 4 - 1, 0), (1, size), (size - 1, size)]):
        bias = np.full(E, level, np.float32)
        bias[b] += np.float32(0.1)
        x, want = tokens("sigmoid", E, a, b, E - 1, bias, E + i)
        if groups == top:
            continue
        ids, _ = wd.route(x.to(cuda_device), 1, scores="sigmoid", bias=torch.from_numpy(bias).to(cuda_device), groups=groups,
                          top_groups=top, group_best=best)
        wrong = int((ids[:, 0].cpu().numpy() != want).sum())
        assert wrong == 0, f"{wrong} of {TOKENS} tokens, experts {a} and {b}"
