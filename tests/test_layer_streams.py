"""Memory of a MoEDecodeLayer call on a stream that is not the current one."""
import contextlib
import types

import pytest

torch = pytest.importorskip("torch")
import moe_decode_gate_gb300 as wd  # noqa: E402
from moe_decode_gate_gb300 import layer as layer_module  # noqa: E402


class Note:
    """A tensor that takes note of where it was made and who uses it."""

    def __init__(self, made_on="caller"):
        self.shape, self.made_on, self.used_on = (2, 64), made_on, []

    def record_stream(self, stream):
        self.used_on.append(stream)


@pytest.mark.parametrize("stream", [None, "side"])
@pytest.mark.parametrize("given", [False, True])
def test_memory_of_a_call(monkeypatch, stream, given):
    now, ran = ["current"], []

    @contextlib.contextmanager
    def on(s):
        now.append(s)
        yield
        now.pop()

    fake = types.SimpleNamespace(
        empty_like=lambda x: Note(now[-1]),
        cuda=types.SimpleNamespace(stream=on, current_stream=lambda device=None: now[-1]))
    monkeypatch.setattr(layer_module, "torch", fake)
    monkeypatch.setattr(layer_module, "wd_moe_decode", lambda *a, stream: ran.append(stream))
    moe = wd.MoEDecodeLayer.__new__(wd.MoEDecodeLayer)
    moe.max_batch, moe.device = 4, "gpu"
    held = ("gate_up", "gate_up_scale", "down", "down_scale", "workspace")
    for name in held:
        setattr(moe, name, Note())
    x, ids, w, mine = Note(), Note(), Note(), Note()
    out = moe(x, ids, w, out=mine if given else None, stream=stream)
    assert ran == [stream]
    used = [x, ids, w, out, *(getattr(moe, name) for name in held)]
    if stream is None:
        assert not any(t.used_on for t in used)
        assert out.made_on == ("caller" if given else "current")
    else:  # nothing is given away before the call is done, nor what it returns before the caller is
        assert all(stream in t.used_on for t in used) and "current" in out.used_on
        assert out.made_on == ("caller" if given else stream)
