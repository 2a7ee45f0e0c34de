"""Memory of KVCache calls on a stream that is not the current one.

What a call allocates has to be that stream's, and what it uses must not be given to another tensor before
it is done: the caller may drop everything as soon as the call returns.  The first tests look at this without
a GPU, through tensors and a library that only take notes; the last one on a GPU.
"""
import contextlib
import types

import pytest

torch = pytest.importorskip("torch")
import moe_decode_gate_gb300 as wd  # noqa: E402
from moe_decode_gate_gb300 import kv_cache  # noqa: E402


class Note:
    """A tensor as the calls look at one."""

    def __init__(self, shape=(4,), dtype=torch.int32, made_on="caller"):
        self.shape = (shape,) if isinstance(shape, int) else tuple(shape)
        self.dtype, self.device, self.made_on, self.used_on = dtype, "gpu", made_on, []
        self.nbytes = 64

    def numel(self):
        n = 1
        for x in self.shape:
            n *= x
        return n

    def dim(self):
        return len(self.shape)

    def stride(self):
        return (self.shape[1] * self.shape[2], self.shape[2], 1)

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 4096

    def record_stream(self, stream):
        self.used_on.append(stream)

    def unbind(self, _):
        return (self, self)


@pytest.fixture
def cache(monkeypatch):
    made, now = [], ["current"]

    @contextlib.contextmanager
    def on(stream):
        now.append(stream)
        yield
        now.pop()

    def empty(shape, dtype, device):
        made.append(Note(shape, dtype, now[-1]))
        return made[-1]

    fake = types.SimpleNamespace(
        empty=empty, int32=torch.int32, float32=torch.float32,
        cuda=types.SimpleNamespace(stream=on, current_stream=lambda device=None: now[-1]),
        _C=types.SimpleNamespace(_cuda_getCurrentRawStream=lambda index: 3,
                                 _cuda_getDevice=lambda: 0))
    monkeypatch.setattr(kv_cache, "torch", fake)
    c = wd.KVCache.__new__(wd.KVCache)
    c.device, c._index, c._ref, c._scale = "gpu", 0, None, 0.1
    c.kv_heads, c.head_dim, c.num_pages, c.slots = 2, 64, 8, 4
    for name in ("pool", "table", "lengths", "refs", "workspace"):
        setattr(c, name, Note())
    c.launched = []
    c._lib = types.SimpleNamespace(**{
        "wd_kv_" + name: lambda *a: c.launched.append(a) or 0
        for name in ("reserve", "append", "attention", "fork", "free", "compact")})
    c.made = made
    return c


class Side:
    cuda_stream = 7
    device = "gpu"


CALLS = [
    lambda c, t, s: c.reserve(t("i"), t("i"), stream=s),
    lambda c, t, s: c.append(0, t("kv"), t("kv"), t("i"), return_values=True, stream=s),
    lambda c, t, s: c.attention(0, t("q"), t("i"), return_lse=True, stream=s),
    lambda c, t, s: c.attention(0, t("q"), t("i"), t("start"), out=t("q"), stream=s),
    lambda c, t, s: c.fork(t("i"), t("i"), stream=s),
    lambda c, t, s: c.fork(t("i"), t("i"), ok=t("i"), stream=s),
    lambda c, t, s: c.free(t("i"), stream=s),
    lambda c, t, s: c.compact(stream=s),
]


@pytest.mark.parametrize("call", CALLS)
def test_memory_of_a_call_on_another_stream(cache, call):
    side, given = Side(), []

    def tensor(kind):
        shape, dtype = {"i": ((4,), torch.int32), "start": ((5,), torch.int32),
                        "kv": ((4, 2, 64), torch.bfloat16), "q": ((4, 6, 64), torch.bfloat16)}[kind]
        given.append(Note(shape, dtype))
        return given[-1]

    call(cache, tensor, side)
    for t in cache.made:  # the results: memory of the call's stream, that the current one may read
        assert t.made_on is side and "current" in t.used_on
    for t in (*given, cache.pool, cache.table, cache.lengths, cache.refs, cache.workspace):
        assert side in t.used_on


def test_nothing_is_noted_on_the_current_stream(cache):
    t = Note()
    cache.reserve(t, t)
    cache.compact()
    assert [x.made_on for x in cache.made] == ["current", "current"]
    assert not any(x.used_on for x in (t, cache.pool, *cache.made))


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("wrong", ["current device", "stream"])
def test_another_device_is_refused(cache, call, wrong):
    # the library launches on the current device, with pointers of the cache's
    side = Side()
    if wrong == "stream":
        side.device = "another gpu"
    else:
        kv_cache.torch._C._cuda_getDevice = lambda: 1

    def tensor(kind):
        shape, dtype = {"i": ((4,), torch.int32), "start": ((5,), torch.int32),
                        "kv": ((4, 2, 64), torch.bfloat16), "q": ((4, 6, 64), torch.bfloat16)}[kind]
        return Note(shape, dtype)

    with pytest.raises(ValueError):
        call(cache, tensor, side)
    if wrong != "stream":
        with pytest.raises(ValueError):
            call(cache, tensor, None)
    assert not cache.launched


@pytest.mark.gpu
def test_results_that_are_dropped_at_once(cuda_device):
    """While the other stream is held up, new tensors of the current one must not lie where the results go."""
    cache = wd.KVCache(50000, 64, 8, 1, 1, 64, 16, device=cuda_device)
    one = torch.ones(64, dtype=torch.int32, device=cuda_device)
    q = torch.randn(64, 8, 64, device=cuda_device).bfloat16()
    k = torch.randn(64, 1, 64, device=cuda_device).bfloat16()
    side = torch.cuda.Stream()
    calls = [(lambda: cache.reserve(one.clone(), stream=side), (64,), torch.int32),
             (lambda: cache.append(0, k.clone(), k.clone(), return_values=True, stream=side),
              (2, 64, 1, 64), torch.bfloat16),
             (lambda: cache.attention(0, q.clone(), stream=side), q.shape, torch.bfloat16),
             (lambda: cache.attention(0, q.clone(), return_lse=True, stream=side), (64, 8),
              torch.float32),
             (lambda: cache.fork(one.clone(), one.clone(), stream=side), (64,), torch.int32),
             (lambda: cache.compact(stream=side), (50000,), torch.int32)]
    for call, shape, dtype in calls:
        torch.cuda.synchronize()
        wd.wd_bench_hold(100000, stream=side)
        side.wait_stream(torch.cuda.current_stream())
        call()
        mine = [torch.full(shape, 77, dtype=dtype, device=cuda_device) for _ in range(8)]
        torch.cuda.synchronize()
        assert all(bool((t == 77).all()) for t in mine)
    cache.read_error_flag()
