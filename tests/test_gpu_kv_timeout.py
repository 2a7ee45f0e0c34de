"""What the calls behind a timeout find, on the GPU.

No wait is made to run out here: the state that one could leave, a raised flag and counters that are not
zero, is written into the workspace from the host, between calls.  (Layout of the workspace: the flag's
256 bytes, then the counters of 8 x 152 units.)
"""
import numpy as np
import pytest
import torch

import moe_decode_gate_gb300 as wd
from test_gpu_kv import Both, Case

pytestmark = pytest.mark.gpu

COUNTERS = 8 * 152


def after_a_timeout(cache):
    words = cache.workspace[:256 + 4 * COUNTERS].view(torch.int32)
    words[0] = wd.KV_FLAG_TIMEOUT | wd.KV_FLAG_BAD_INDEX
    words[64:] = torch.arange(1, COUNTERS + 1, dtype=torch.int32, device=words.device) % 5
    assert cache.read_error_flag() == wd.KV_FLAG_TIMEOUT | wd.KV_FLAG_BAD_INDEX
    assert cache.read_error_flag() == 0
    assert not bool(words.any())


@pytest.mark.parametrize("lens,news,hq", [([20000], [1], 4), ([9000, 30], [3, 2], 8),
                                          ([7001, 6000], [130, 40], 4)])
@pytest.mark.parametrize("D", [64, 128])
def test_attention_behind_a_timeout(cuda_device, lens, news, hq, D):
    # long sequences of few entries: every item has pieces in several CTAs
    c = Case(cuda_device, lens, news, hq, 1, D, 64, seed=D)
    want = c.run()
    after_a_timeout(c.cache)
    for _ in range(2):
        got = c.run()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # and a call leaves the counters as it found them
    assert not bool(c.cache.workspace[256:256 + 4 * COUNTERS].any())
    c.check(want)


@pytest.mark.parametrize("pages", [300, 20000])
def test_page_operations_behind_a_timeout(cuda_device, pages):
    r = np.random.RandomState(pages)
    b = Both(cuda_device, pages, 12, 12, layers=3)
    b.reserve(list(range(8)), r.randint(1, 150, 8).tolist())
    b.write()
    after_a_timeout(b.cache)
    b.fork([0, 1, 2, -1], [8, 9, 10, 3])
    after_a_timeout(b.cache)
    b.compact()
    after_a_timeout(b.cache)
    b.reserve([3, 8], [40, 40])
    assert not bool(b.cache.workspace[256:256 + 4 * COUNTERS].any())
