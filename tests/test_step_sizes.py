"""Sizes that the C-ABI's 32-bit parameters do not hold are refused by the Python calls, not cut to their low bits.

Without a GPU, through tensors and a library that only take notes.
"""
import pytest

torch = pytest.importorskip("torch")
import moe_decode_gate_gb300 as wd  # noqa: E402
from test_kv_streams import cache  # noqa: E402,F401
from test_step_streams import BF16, F32, I32, Note as T, history, kv, notes, rotated  # noqa: E402,F401

FAR = 2 ** 32 + 64  # its low 32 bits are a size like any other
CALLS = [
    lambda: wd.rms_norm(T((4, FAR))), lambda: wd.rms_norm(T((4, FAR, 64))), lambda: wd.rms_norm(T((4, 2, FAR)), mxfp8=True),
    lambda: wd.rms_norm(T((4, 2 ** 31))),
    lambda: wd.route(T((4, FAR)), 8), lambda: wd.route(T((4, 64)), 2 ** 32 + 8),
    lambda: wd.adjust_logits(T((4, FAR))), lambda: wd.adjust_logits(T((FAR, 64))), lambda: wd.adjust_logits(T((2 ** 31, 64))),
    lambda: wd.adjust_logits(T((4, 64)), **{**history(T), "history": T((5, FAR), I32)}),
    lambda: wd.adjust_logits(T((4, 64)), **{**history(T), "history": T((FAR, 9), I32), "lengths": T((FAR,), I32),
                                            "prompt_lengths": T((FAR,), I32)}),
    lambda: wd.adjust_logits(T((4, 64)), bias=(T((5,), I32), T((FAR,), I32), T((FAR,), F32))),
]


@pytest.mark.parametrize("call", CALLS)
def test_refused(notes, call):  # noqa: F811
    with pytest.raises(ValueError, match="sizes"):
        call()
    assert not notes.launched


@pytest.mark.parametrize("tokens", [FAR, 2 ** 31])
def test_rotated_refuses(cache, tokens):  # noqa: F811
    with pytest.raises(ValueError, match="sizes"):
        rotated(cache, q=None, k=kv((tokens, 2, 64)), v=kv((tokens, 2, 64)), seqs=kv((4,), I32), q_start=kv((5,), I32))
    assert not cache.launched


def test_tokens_of_64_bits_are_passed_whole(notes):  # noqa: F811
    wd.route(T((2 ** 40, 64)), 8)
    wd.rms_norm(T((2 ** 40, 64)))
    assert notes.launched[0][3] == notes.launched[1][4] == 2 ** 40
