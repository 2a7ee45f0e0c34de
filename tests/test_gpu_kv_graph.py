"""One captured step, replayed while the sequences grow, on the GPU.

The division of attention's work is found on the device from the lengths, and the launches overlap: a graph of
reserve, append and attention has to stay right across pages, steps of 32 keys and pieces.  Every replay
is compared, bit for bit, with the same calls made one by one on a second cache.
"""
import numpy as np
import pytest
import torch

import kv_reference as ref
import moe_decode_gate_gb300 as wd

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,hq,hkv,lens,news,window,replays", [
    (128, 8, 2, [0, 14, 31, 250], [1, 1, 1, 1], 0, 40),
    (64, 16, 1, [5, 4090], [1, 1], 0, 20),
    (256, 4, 2, [60, 0, 500], [1, 1, 1], 48, 40),
    (128, 8, 1, [3, 20, 0], [3, 1, 2], 0, 25),
    (128, 16, 2, [0, 100], [40, 33], 0, 20),
    (64, 8, 1, [0, 700], [64, 40], 100, 15)])
def test_replays_while_sequences_grow(cuda_device, D, hq, hkv, lens, news, window, replays):
    layers, P = 2, 16
    r = np.random.RandomState(D + hq)
    columns = -(-(max(lens) + replays * max(news)) // P) + 1
    pages = columns * len(lens)

    def ints(a):
        return torch.tensor(a, dtype=torch.int32, device=cuda_device)

    def normal(heads):
        return torch.from_numpy(r.standard_normal((sum(news), heads, D))).to(cuda_device).bfloat16()

    caches = [wd.KVCache(pages, len(lens), columns, layers, hkv, D, P, device=cuda_device)
              for _ in range(2)]
    past = torch.from_numpy(r.standard_normal((2, sum(lens), hkv, D))).to(cuda_device).bfloat16()
    for c in caches:
        c.reserve(ints(lens))
        for layer in range(layers):
            c.append(layer, past[0], past[1], q_start=ints(np.cumsum([0] + lens).tolist()))
    q, k, v = normal(hq), normal(hkv), normal(hkv)
    counts, start = ints(news), None if max(news) == 1 else ints(np.cumsum([0] + news).tolist())

    def step(c):
        out = [c.reserve(counts)]
        for layer in range(layers):
            c.append(layer, k, v, q_start=start)
            out += c.attention(layer, q, q_start=start, window=window, return_lse=True)
        return out

    before = [t.clone() for t in (caches[0].pool, caches[0].table, caches[0].lengths, caches[0].refs)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(caches[0])  # loads the kernels
    torch.cuda.current_stream().wait_stream(side)
    for t, x in zip((caches[0].pool, caches[0].table, caches[0].lengths, caches[0].refs), before):
        t.copy_(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(caches[0])
    for i in range(replays):
        for t, heads in ((q, hq), (k, hkv), (v, hkv)):
            t.copy_(normal(heads))
        graph.replay()
        want = step(caches[1])
        assert all(torch.equal(a, b) for a, b in zip(got, want)), f"replay {i}"
        assert bool((got[0] == 1).all())
    assert all(torch.equal(getattr(caches[0], x), getattr(caches[1], x))
               for x in ("pool", "table", "lengths", "refs"))
    assert caches[0].lengths.tolist() == [n + replays * m for n, m in zip(lens, news)]
    assert [c.read_error_flag() for c in caches] == [0, 0]
    # and what the last replay gave is the attention of the cache as it is
    q_start = np.cumsum([0] + news)
    want, _, mag = ref.attention(caches[0].pool.cpu().numpy(), caches[0].table.cpu().numpy(),
                                 caches[0].lengths.tolist(), layers - 1, q.double().cpu().numpy(),
                                 list(range(len(lens))), q_start, D, P, 1 / np.sqrt(D), window)
    # (|v| is below 8 here: what FP16 flushes of the probabilities)
    tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2.0 ** -15) * mag + 2.0 ** -20 * 8
    assert (np.abs(got[-2].double().cpu().numpy() - want) <= tol).all()
