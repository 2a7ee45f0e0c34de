"""The cache's operations together, as examples/decode.py uses them, on the GPU."""
import importlib.util
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PATH = os.path.join(ROOT, "examples", "decode.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("example_decode", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_runs_as_a_program():
    out = subprocess.run([sys.executable, PATH, "--layers", "2", "--steps", "12"], cwd=ROOT,
                         capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, out.stderr[-2000:]
    assert out.stdout.count("prompt") == 6 and "front of the pool: True" in out.stdout


def test_compaction_in_the_middle_changes_nothing(example, cuda_device):
    model = example.Decoder(layers=2)
    prompts = [[1, 2, 3], list(range(40)), [7] * 17]
    caches = [model.cache(200, 12, 20) for _ in range(2)]
    for c in caches:  # leave holes in the pool: sequences that come and go in the slots behind
        c.reserve(example.ints([100, 30], cuda_device), example.ints([10, 11], cuda_device))
        c.free(example.ints([10], cuda_device))
    plain, _ = example.generate(model, prompts, 3, 20, caches[0])
    moved, _ = example.generate(model, prompts, 3, 20, caches[1], compact_after=7)
    assert torch.equal(plain, moved)
    assert all(c.read_error_flag() == 0 for c in caches)


def test_a_chunk_and_its_tokens_one_by_one_agree(example, cuda_device):
    """The logits of a prompt's last token, from the prompt as one chunk and token by token.  The
    two attend to the same cache; they differ by the order of FP32 sums and the BF16 roundings behind
    them (a step of 2^-8 of a value, some tens of them in a row), far below the logits' own size."""
    model = example.Decoder(layers=1)
    tokens = example.ints([3, 1, 4, 1, 5, 9, 2, 6, 5, 3, 5, 8, 9, 7, 9, 3, 2, 3, 8, 4, 6], cuda_device)
    n = tokens.numel()
    slot = example.ints([1], cuda_device)
    whole = model.cache(8, 2, 4)
    whole.reserve(example.ints([n], cuda_device), slot)
    want = model(tokens, whole, slot, example.ints([0, n], cuda_device), n)[-1]
    single = model.cache(8, 2, 4)
    for i in range(n):
        single.reserve(example.ints([1], cuda_device), slot)
        got = model(tokens[i:i + 1], single, slot)[0]
    assert float((got - want).norm() / want.norm()) < 0.05
    assert torch.equal(whole.lengths, single.lengths) and torch.equal(whole.table, single.table)


def test_beams_share_their_prompts_pages(example, cuda_device):
    model = example.Decoder(layers=1)
    cache = model.cache(64, 8, 16)
    prompts = [list(range(35)), list(range(50))]
    example.generate(model, prompts, 4, 2, cache)
    # 35 tokens: 2 whole pages for four beams, and one more each; 50 tokens: 3 whole pages
    refs = cache.refs.tolist()
    assert sorted(r for r in refs if r > 1) == [4] * 5 and refs.count(1) == 8
    cache.free(example.ints([0, 1, 2, 3], cuda_device))
    assert sorted(r for r in cache.refs.tolist() if r) == [1] * 4 + [4] * 3
