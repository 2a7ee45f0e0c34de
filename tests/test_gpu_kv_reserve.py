"""Requests for more pages than 32 bits count, in one call of reserve, on the GPU."""
import pytest
import torch

import moe_decode_gate_gb300 as wd

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("first", [1, 0])
def test_requests_that_add_up_past_32_bits(cuda_device, first):
    # 3072 requests of 2^20 pages each (2^32 together, and 2^31 while they are counted), behind one that
    # fits; the table has the most columns that there may be (13 GB)
    slots, columns, page = 3073, 1 << 20, 256
    cache = wd.KVCache(64, slots, columns, 1, 1, 64, page, device=cuda_device)
    counts = torch.full((slots,), columns * page, dtype=torch.int32, device=cuda_device)
    counts[0] = 20 if first else 0
    ok = cache.reserve(counts)
    want = torch.zeros(slots, dtype=torch.int32)
    want[0] = 1
    assert torch.equal(ok.cpu(), want)
    assert cache.read_error_flag() == wd.KV_FLAG_NO_PAGES
    assert cache.refs.tolist() == [first] + [0] * 63
    assert int(cache.lengths.sum()) == int(counts[0])
    assert cache.table[0, :2].tolist() == ([0, -1] if first else [-1, -1])
    assert int(cache.table[1:].max()) == -1
    del cache
    torch.cuda.empty_cache()
