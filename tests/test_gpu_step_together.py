"""The step's operators together, as examples/decode.py uses them around attention and experts, on the GPU."""
import importlib.util
import os
import subprocess
import sys

import pytest
import torch

import moe_decode_gate_gb300 as wd

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PATH = os.path.join(ROOT, "examples", "decode.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("example_decode_together", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_runs_as_a_program():
    out = subprocess.run([sys.executable, PATH, "--layers", "2", "--steps", "12", "--rotary-base", "10000", "--repetition",
                          "1.3", "--temperature", "0.7"], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, out.stderr[-2000:]
    assert out.stdout.count("prompt") == 6 and "front of the pool: True" in out.stdout


def plain_norm(x, weight=None, residual=None, **kw):
    r = x.double() + (0 if residual is None else residual.double())
    y = (r / torch.sqrt(r.square().mean(-1, keepdim=True) + 1e-6)).to(x.dtype)
    return y if residual is None else (y, r.to(x.dtype))


def plain_route(logits, K):
    p = torch.softmax(logits.double(), -1)
    order = torch.argsort(logits.double(), dim=-1, descending=True, stable=True)[:, :K]
    w = p.gather(1, order)
    return order.int(), (w / w.sum(-1, keepdim=True)).float()


def plain_append(cache):
    """append_rotated from append: the turned keys, in FP32 as they are quantised."""
    def call(layer, q, k, v, cos_sin, seqs, q_start=None):
        n = q.shape[0]
        at = torch.arange(n, device=q.device)
        if q_start is None:
            pos = cache.lengths[seqs.long()].long() - 1
        else:
            b = torch.searchsorted(q_start.long(), at, right=True) - 1
            pos = cache.lengths[seqs.long()[b]].long() - q_start.long()[b + 1] + at
        c, s = cos_sin[pos][:, None].chunk(2, -1)

        def turn(x):
            a, b = x.float().chunk(2, -1)
            return torch.cat((a * c - b * s, b * c + a * s), -1)

        cache.append(layer, turn(k), v.float(), seqs, q_start)
        return turn(q).to(q.dtype)
    return call


def test_a_decoder_of_them_and_one_of_plain_pieces(example, cuda_device, monkeypatch):
    """Logits of the same decoder with its norms, routing and rotation as plain torch pieces in 64 bits.  The two round the
    same values once each and differ where a value lies at a rounding's border: steps of BF16 (2^-8 of a value) of a few,
    which later layers carry on; a router's pair that is nearer than that changes places, and with it a part of a token."""
    model = example.Decoder(layers=2, rotary_base=1000.0)
    tokens = example.ints(list(range(3, 40)) + [7] * 9, cuda_device)
    start, slots = example.ints([0, 37, 46], cuda_device), example.ints([2, 0], cuda_device)
    logits = []
    for plain in (False, True):
        cache = model.cache(16, 4, 8)
        cache.reserve(example.ints([37, 9], cuda_device), slots)
        if plain:
            monkeypatch.setattr(example, "rms_norm", plain_norm)
            monkeypatch.setattr(example, "route", plain_route)
            monkeypatch.setattr(cache, "append_rotated", plain_append(cache), raising=False)
        logits.append(model(tokens, cache, slots, start, 37))
        assert cache.read_error_flag() == 0
    off = (logits[0] - logits[1]).norm(dim=1) / logits[1].norm(dim=1)
    assert float(off.median()) < 0.02 and float(off.max()) < 0.5


def test_positions_matter_and_beams_share_them(example, cuda_device):
    """With turned keys a chunk and its tokens one by one agree as they do without, and the order of tokens matters."""
    model = example.Decoder(layers=1, rotary_base=10000.0)
    tokens = example.ints([3, 1, 4, 1, 5, 9, 2, 6, 5, 3, 5, 8, 9, 7, 9, 3, 2, 3, 8, 4, 6], cuda_device)
    n, slot = tokens.numel(), example.ints([1], cuda_device)

    def whole(tokens):
        cache = model.cache(8, 2, 4)
        cache.reserve(example.ints([n], cuda_device), slot)
        return model(tokens, cache, slot, example.ints([0, n], cuda_device), n)[-1]

    single = model.cache(8, 2, 4)
    for i in range(n):
        single.reserve(example.ints([1], cuda_device), slot)
        got = model(tokens[i:i + 1], single, slot)[0]
    want = whole(tokens)
    assert float((got - want).norm() / want.norm()) < 0.05
    swapped = tokens.clone()
    swapped[2], swapped[11] = tokens[11], tokens[2]
    assert not torch.equal(whole(swapped), want)


def test_a_captured_step(example, cuda_device):
    """Reserve, the model, the penalties and the choice as one graph: replayed, it gives the tokens of eager steps, while
    sequences and histories grow."""
    model = example.Decoder(layers=2, rotary_base=10000.0)
    prompts, steps = [[5, 6, 7, 8], [9] * 19, [1, 2]], 24
    want, _ = example.generate(model, prompts, 2, steps, model.cache(64, 6, 8), repetition=1.5, temperature=0.7)
    cache = model.cache(64, 6, 8)
    got, slots = example.generate(model, prompts, 2, 4, cache, repetition=1.5, temperature=0.7)
    assert torch.equal(got, want[..., :4])
    penalties = example.Penalties(prompts, 2, steps, 1.5, 0.7, model.device)
    for i in range(3):
        penalties.add(got[..., i].reshape(-1))
    token, one = got[..., 3].reshape(-1).clone(), torch.ones_like(slots)

    def step():
        cache.reserve(one, slots)
        logits = model(token, cache, slots)
        penalties.add(token)
        token.copy_(penalties(logits, slots).argmax(-1).int())

    # what a step changes, for the steps that warm up and capture
    kept = [t.clone() for t in (cache.table, cache.lengths, cache.refs, penalties.tokens, penalties.lengths, token)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t, k in zip((cache.table, cache.lengths, cache.refs, penalties.tokens, penalties.lengths, token), kept):
        t.copy_(k)
    for i in range(4, steps):
        graph.replay()
        assert torch.equal(token.view(3, 2), want[..., i])
    assert cache.read_error_flag() == 0


def test_two_streams_at_once(cuda_device):
    """None of the operators shares anything between streams."""
    x = [torch.randn(400, 2048, device=cuda_device).bfloat16() for _ in range(2)]
    logits = [t[:, :1000].float().contiguous() for t in x]
    history = torch.randint(0, 1000, (400, 300), device=cuda_device).int()
    lengths = torch.randint(0, 300, (400,), device=cuda_device).int()
    f = torch.rand(400, device=cuda_device)

    def work(i):
        return (*wd.rms_norm(x[i], None, x[1 - i], mxfp8=True), *wd.route(x[i][:, :256], 8, scores="sigmoid", groups=8,
                top_groups=3), wd.adjust_logits(logits[i], history=history, lengths=lengths, frequency=f, temperature=f))

    want = [work(i) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        got = []
        for i, s in enumerate(streams):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got.append(work(i))
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(torch.equal(a, b) for a, b in zip(g, w))
