"""wd_adjust_logits where its arguments' numbers are at the ends of their types, on the GPU.

Results are compared bit by bit with those of the same call without what counts for nothing.
"""
import numpy as np
import pytest
import torch

import moe_decode_gate_gb300 as wd

pytestmark = pytest.mark.gpu

MOST = 2 ** 31 - 1


def ints(a, dev):
    return torch.tensor(a, dtype=torch.int32, device=dev)


@pytest.mark.parametrize("columns", [40, 40000])
@pytest.mark.parametrize("V", [100, 5003, 200003])
def test_bias_starts_at_the_ends_of_their_type(V, columns, cuda_device):
    """Rows whose biases' range is none: its ends far out of range, or in the wrong order, with a history and without one.
    A row beside them keeps its biases."""
    starts = [MOST, 0, MOST - 255, MOST - 254, MOST, -MOST - 1, MOST - 100, 5, 2, 2, 7, 10 ** 9, -1, MOST, MOST - 31, 4, 10]
    B, n = len(starts) - 1, 9
    g = torch.Generator(device=cuda_device).manual_seed(V)
    x = torch.randn(B, V, generator=g, device=cuda_device)
    kw = dict(history=(torch.rand(B, columns, generator=g, device=cuda_device) ** 3 * V).int(),
              lengths=torch.full((B,), columns, dtype=torch.int32, device=cuda_device),
              frequency=torch.rand(B, generator=g, device=cuda_device))
    ids = ints([3, 3, 5, 99, 0, 1, 3, 3, 98], cuda_device)
    values = torch.arange(1.0, n + 1, device=cuda_device)
    for more in (kw, {}):
        got = wd.adjust_logits(x, bias=(ints(starts, cuda_device), ids, values), **more)
        want = wd.adjust_logits(x, **more)
        for b, (lo, hi) in enumerate(zip(starts[:-1], starts[1:])):
            if 0 <= lo <= hi <= n and lo < hi:
                row = {k: t[b:b + 1] for k, t in more.items()}
                want[b] = wd.adjust_logits(x[b:b + 1], bias=(ints([0, hi - lo], cuda_device), ids[lo:hi].contiguous(),
                                                             values[lo:hi].contiguous()), **row)[0]
        assert torch.equal(got, want)


def test_as_many_biases_as_their_type_counts(cuda_device):
    """A row's biases are the last of 2^31 - 1: the places that threads of a CTA look at next pass the type's end."""
    V, n = 3001, 40
    r = np.random.RandomState(1)
    last = np.concatenate((r.permutation(V)[:n - 4], [7, 7, 7, V]))
    ids = torch.empty(MOST, dtype=torch.int32, device=cuda_device)
    values = torch.empty(MOST, device=cuda_device)
    ids[-n:], values[-n:] = ints(last, cuda_device), torch.from_numpy(r.standard_normal(n).astype(np.float32)).to(cuda_device)
    x = torch.from_numpy(r.standard_normal((3, V)).astype(np.float32)).to(cuda_device)
    history = dict(history=ints(r.randint(0, V, (3, 300)), cuda_device), lengths=ints([300, 0, 70], cuda_device),
                   presence=torch.ones(3, device=cuda_device))
    for kw in ({}, history):
        got = wd.adjust_logits(x, bias=(ints([MOST - n, MOST - 1, MOST - 1, MOST], cuda_device), ids, values), **kw)
        want = wd.adjust_logits(x, bias=(ints([0, n - 1, n - 1, n], cuda_device), ids[-n:].clone(), values[-n:].clone()), **kw)
        assert torch.equal(got, want)
