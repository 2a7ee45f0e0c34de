"""What the Python calls of the step's operators refuse, and the memory of calls on a stream that is not the current one.

Without a GPU, through tensors and a library that only take notes; the last test on a GPU.
"""
import contextlib
import types

import pytest

torch = pytest.importorskip("torch")
import moe_decode_gate_gb300 as wd  # noqa: E402
from moe_decode_gate_gb300 import step  # noqa: E402

GPU = torch.device("cuda", 0)
I32, F32, BF16 = torch.int32, torch.float32, torch.bfloat16


class Note:
    """A tensor as the calls look at one."""

    def __init__(self, shape, dtype=BF16, made_on="caller", device=GPU, stride=None):
        self.shape, self.dtype, self.device = torch.Size(shape), dtype, device
        self.made_on, self.used_on, self._stride = made_on, [], stride

    def dim(self):
        return len(self.shape)

    def stride(self, i=None):
        if self._stride is None:
            s, n = [], 1
            for x in reversed(self.shape):
                s.insert(0, n)
                n *= x
            self._stride = tuple(s)
        return self._stride if i is None else self._stride[i]

    def is_contiguous(self):
        return self._stride is None or self._stride == Note(self.shape).stride()

    def data_ptr(self):
        return 4096

    def record_stream(self, stream):
        self.used_on.append(stream)


class Side:
    cuda_stream, device = 7, GPU


@pytest.fixture
def notes(monkeypatch):
    seen, now = types.SimpleNamespace(made=[], launched=[]), ["current"]

    @contextlib.contextmanager
    def on(stream):
        now.append(stream)
        yield
        now.pop()

    def empty(shape, dtype, device):
        seen.made.append(Note(shape, dtype, now[-1], device))
        return seen.made[-1]

    fake = types.SimpleNamespace(
        empty=empty, **{n: getattr(torch, n) for n in ("int32", "float32", "uint8", "bfloat16", "float16")},
        cuda=types.SimpleNamespace(stream=on, current_stream=lambda device=None: now[-1]),
        _C=types.SimpleNamespace(_cuda_getCurrentRawStream=lambda index: 3, _cuda_getDevice=lambda: 0))
    monkeypatch.setattr(step, "torch", fake)
    monkeypatch.setattr(step, "_LIB", types.SimpleNamespace(**{
        n: lambda *a: seen.launched.append(a) or 0 for n in ("wd_rms_norm", "wd_route", "wd_adjust_logits")}))
    return seen


def history(t):
    return dict(history=t((5, 9), I32), lengths=t((5,), I32), prompt_lengths=t((5,), I32), seqs=t((4,), I32))


CALLS = [
    lambda t, s: wd.rms_norm(t((4, 64)), t((64,)), t((4, 64)), stream=s),
    lambda t, s: wd.rms_norm(t((4, 3, 64)), t((64,), F32), mxfp8=True, stream=s),
    lambda t, s: wd.rms_norm(t((4, 64)), None, t((4, 64)), out=t((4, 64)), residual_out=t((4, 64)), mxfp8=True, stream=s),
    lambda t, s: wd.route(t((4, 64)), 8, bias=t((64,), F32), stream=s),
    lambda t, s: wd.route(t((4, 64)), 8, ids=t((4, 8), I32), weights=t((4, 8), F32), stream=s),
    lambda t, s: wd.adjust_logits(t((4, 70)), **history(t), repetition=t((4,), F32), presence=t((4,), F32),
                                  frequency=t((4,), F32), temperature=t((4,), F32), mask=t((4, 3), I32),
                                  bias=(t((5,), I32), t((9,), I32), t((9,), F32)), stream=s),
    lambda t, s: wd.adjust_logits(t((4, 70)), out=t((4, 70), F32), stream=s),
]


@pytest.mark.parametrize("call", CALLS)
def test_memory_of_a_call_on_another_stream(notes, call):
    side, given = Side(), []

    def tensor(*a):
        given.append(Note(*a))
        return given[-1]

    call(tensor, side)
    assert len(notes.launched) == 1 and notes.launched[0][-1] == 7
    for t in notes.made:  # the results: memory of the call's stream, that the current one may read
        assert t.made_on is side and "current" in t.used_on
    for t in (*given, *notes.made):
        assert side in t.used_on


@pytest.mark.parametrize("call", CALLS)
def test_nothing_is_noted_on_the_current_stream(notes, call):
    given = []
    call(lambda *a: given.append(Note(*a)) or given[-1], None)
    assert notes.launched[0][-1] == 3
    assert all(t.made_on == "current" for t in notes.made) and not any(t.used_on for t in (*given, *notes.made))


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("wrong", ["current device", "stream"])
def test_another_device_is_refused(notes, call, wrong):
    side = Side()
    if wrong == "stream":
        side.device = torch.device("cuda", 1)
    else:
        step.torch._C._cuda_getDevice = lambda: 1
    with pytest.raises(ValueError):
        call(Note, side)
    if wrong != "stream":
        with pytest.raises(ValueError):
            call(Note, None)
    assert not notes.launched


T = Note
OTHER = torch.device("cuda", 1)
H = lambda **kw: {**history(T), **kw}  # noqa: E731
REFUSED = [
    lambda: wd.rms_norm(T((4, 64), I32)), lambda: wd.rms_norm(T((64,))), lambda: wd.rms_norm(T((2, 2, 2, 2))),
    lambda: wd.rms_norm(T((4, 64), BF16, "", torch.device("cpu"))), lambda: wd.rms_norm(T((4, 64), stride=(1, 4))),
    lambda: wd.rms_norm(T((4, 64)), T((63,))), lambda: wd.rms_norm(T((4, 64)), T((64,), torch.float16)),
    lambda: wd.rms_norm(T((4, 64)), T((64,), device=OTHER)), lambda: wd.rms_norm(T((4, 64)), T((64,), stride=(2,))),
    lambda: wd.rms_norm(T((4, 64)), None, T((4, 65))), lambda: wd.rms_norm(T((4, 64)), None, T((4, 64), F32)),
    lambda: wd.rms_norm(T((4, 64)), None, T((4, 64), device=OTHER)), lambda: wd.rms_norm(T((4, 60)), mxfp8=True),
    lambda: wd.rms_norm(T((4, 64)), out=T((4, 64), F32)), lambda: wd.rms_norm(T((4, 64)), residual_out=T((4, 64))),
    lambda: wd.rms_norm(T((4, 64)), None, T((4, 64)), residual_out=T((4, 64), stride=(65, 1))),
    lambda: wd.route(T((4, 64), I32), 8), lambda: wd.route(T((64,)), 8), lambda: wd.route(T((4, 64)), 8, scores="tanh"),
    lambda: wd.route(T((4, 64), stride=(1, 4)), 8), lambda: wd.route(T((4, 64)), 8, bias=T((64,))),
    lambda: wd.route(T((4, 64)), 8, bias=T((63,), F32)), lambda: wd.route(T((4, 64)), 8, ids=T((4, 8), torch.int64)),
    lambda: wd.route(T((4, 64)), 8, weights=T((4, 7), F32)), lambda: wd.route(T((4, 64), device=torch.device("cpu")), 8),
    lambda: wd.adjust_logits(T((4, 64), I32)), lambda: wd.adjust_logits(T((64,))),
    lambda: wd.adjust_logits(T((4, 64)), dtype=torch.float16), lambda: wd.adjust_logits(T((4, 64), stride=(1, 4))),
    lambda: wd.adjust_logits(T((4, 64)), out=T((4, 63))), lambda: wd.adjust_logits(T((4, 64)), out=T((4, 64), torch.float16)),
    lambda: wd.adjust_logits(T((4, 64)), out=T((4, 64), device=OTHER)), lambda: wd.adjust_logits(T((4, 64)), repetition=T((4,), F32)),
    lambda: wd.adjust_logits(T((4, 64)), seqs=T((4,), I32)), lambda: wd.adjust_logits(T((4, 64)), **H(lengths=None)),
    lambda: wd.adjust_logits(T((4, 64)), **H(lengths=T((4,), I32))), lambda: wd.adjust_logits(T((4, 64)), **H(seqs=T((5,), I32))),
    lambda: wd.adjust_logits(T((4, 64)), **H(history=T((5, 9), torch.int64))),
    lambda: wd.adjust_logits(T((4, 64)), **H(history=T((5, 9), I32, stride=(1, 5)))),
    lambda: wd.adjust_logits(T((4, 64)), **H(presence=T((5,), F32))), lambda: wd.adjust_logits(T((4, 64)), temperature=T((4,))),
    lambda: wd.adjust_logits(T((4, 64)), mask=T((4, 3), I32)), lambda: wd.adjust_logits(T((4, 64)), mask=T((4, 2))),
    lambda: wd.adjust_logits(T((4, 64)), bias=(T((4,), I32), T((9,), I32), T((9,), F32))),
    lambda: wd.adjust_logits(T((4, 64)), bias=(T((5,), I32), T((9,), I32), T((8,), F32))),
    lambda: wd.adjust_logits(T((4, 64)), bias=(T((5,), I32), T((9,), F32), T((9,), F32))),
]


@pytest.mark.parametrize("call", REFUSED)
def test_refused(notes, call):
    with pytest.raises(ValueError):
        call()
    assert not notes.launched


@pytest.mark.gpu
def test_results_that_are_dropped_at_once(cuda_device):
    """While the other stream is held up, new tensors of the current one must not lie where the results go."""
    x = torch.randn(64, 4096, device=cuda_device).bfloat16()
    side = torch.cuda.Stream()
    calls = [(lambda: wd.rms_norm(x.clone(), None, x.clone(), stream=side), x.shape, BF16),
             (lambda: wd.rms_norm(x.clone(), mxfp8=True, stream=side), x.shape, torch.uint8),
             (lambda: wd.route(x[:, :128], 64, stream=side), (64, 64), I32),
             (lambda: wd.adjust_logits(x.clone(), dtype=F32, stream=side), x.shape, F32)]
    for call, shape, dtype in calls:
        torch.cuda.synchronize()
        wd.wd_bench_hold(100000, stream=side)
        side.wait_stream(torch.cuda.current_stream())
        call()
        mine = [torch.full(shape, 77, dtype=dtype, device=cuda_device) for _ in range(8)]
        torch.cuda.synchronize()
        assert all(bool((t == 77).all()) for t in mine)


# ------------------------------------------------------------ KVCache.append_rotated ---

import test_kv_streams  # noqa: E402
from test_kv_streams import cache  # noqa: E402,F401  (the cache that takes notes)


def kv(shape, dtype=BF16):
    return test_kv_streams.Note(shape, dtype)


def rotated(cache, given=lambda t: t, stream=None, **kw):  # noqa: F811
    cache._lib.wd_kv_append_rotated = lambda *a: cache.launched.append(a) or 0
    d = dict(q=kv((4, 6, 64)), k=kv((4, 2, 64)), v=kv((4, 2, 64)), cos_sin=Note((9, 64), F32, device="gpu"), seqs=kv((4,), I32))
    d.update(kw)
    given(d)
    return cache.append_rotated(0, **d, stream=stream)


def test_rotated_on_another_stream(cache):  # noqa: F811
    side, given = test_kv_streams.Side(), []
    rotated(cache, lambda d: given.extend(d.values()), side, return_values=True, q_start=kv((5,), I32))
    assert len(cache.made) == 3 and len(cache.launched) == 1
    for t in cache.made:
        assert t.made_on is side and "current" in t.used_on
    for t in (*(g for g in given if g is not True), cache.pool, cache.table, cache.lengths, cache.refs, cache.workspace):
        assert side in t.used_on


@pytest.mark.parametrize("kw", [
    dict(q=kv((4, 6, 128))), dict(q=kv((3, 6, 64))), dict(q=kv((4, 6, 64), torch.float16)), dict(q=None, q_out=kv((4, 6, 64))),
    dict(q_out=kv((4, 5, 64))), dict(q_out=kv((4, 6, 64), F32)), dict(k=kv((4, 3, 64))), dict(k=kv((4, 2, 64), I32)),
    dict(v=kv((4, 2, 64), F32)), dict(v=kv((5, 2, 64))), dict(cos_sin=Note((9, 64), BF16, device="gpu")),
    dict(cos_sin=Note((9, 64), F32, device="another gpu")), dict(cos_sin=Note((9, 2, 64), F32, device="gpu")),
    dict(cos_sin=Note((9, 64), F32, device="gpu", stride=(65, 1))), dict(seqs=kv((3,), I32))])
def test_rotated_refuses(cache, kw):  # noqa: F811
    with pytest.raises(ValueError):
        rotated(cache, **kw)
    assert not cache.launched
