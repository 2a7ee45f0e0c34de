"""The C-ABI of wd_step.h and wd_kv_append_rotated without a GPU: symbols, and what the host refuses.

Every call below fails host validation or does nothing, so no kernel is launched.
"""
import ctypes
import os
import re

import pytest

import moe_decode_gate_gb300 as wd
from moe_decode_gate_gb300 import _native
from moe_decode_gate_gb300.kv_cache import _Cache
from moe_decode_gate_gb300.step import _History

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "wd_step.h")
OK, INVALID, SHAPE, SMALL = 0, 1, 2, 3
A = 0x10000  # an aligned fake address: never dereferenced
NAN, INF = float("nan"), float("inf")


def test_library_exports_every_declared_symbol():
    names = re.findall(r"^WD_API\s+[\w\s\*]+?\b(wd_\w+)\s*\(", open(HEADER).read(), flags=re.M)
    assert set(names) == {"wd_rms_norm", "wd_route", "wd_adjust_logits"}
    for name in (*names, "wd_kv_append_rotated"):
        assert hasattr(wd.lib(), name) and name in _native.SIGNATURES, name


def norm(x=A, dtype=0, tokens=4, heads=1, H=256, weight=A, weight_dtype=0, residual=A, residual_out=A, eps=1e-6, y=A,
         codes=None, scales=None):
    return wd.lib().wd_rms_norm(x, dtype, H, H, tokens, heads, H, weight, weight_dtype, residual, H, H, residual_out, eps,
                                y, codes, scales, None)


@pytest.mark.parametrize("kw,want", [
    (dict(tokens=0), OK), (dict(tokens=0, x=None), OK), (dict(x=None), INVALID), (dict(x=A + 1), INVALID),
    (dict(dtype=3), INVALID), (dict(dtype=-1), INVALID), (dict(weight_dtype=1), INVALID), (dict(dtype=2, weight_dtype=0), INVALID),
    (dict(weight_dtype=2, weight=A + 2), INVALID), (dict(tokens=-1), INVALID), (dict(heads=0), INVALID), (dict(H=0), INVALID),
    (dict(H=16385), SHAPE), (dict(tokens=2 ** 31), SHAPE), (dict(tokens=2 ** 20, heads=2 ** 12), SHAPE), (dict(y=None), INVALID),
    (dict(codes=A), INVALID), (dict(scales=A), INVALID), (dict(codes=A, scales=A, H=250), SHAPE), (dict(residual=None), INVALID),
    (dict(residual=A + 1), INVALID), (dict(residual_out=A + 1), INVALID), (dict(y=A + 1), INVALID), (dict(eps=0.0), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=NAN), INVALID), (dict(eps=INF), INVALID), (dict(eps=1e-40), INVALID)])
def test_norm(kw, want):
    assert norm(**kw) == want


def route(logits=A, dtype=0, tokens=4, E=128, K=8, scores=0, bias=None, groups=1, top=1, best=2, scale=1.0, ids=A, weights=A):
    return wd.lib().wd_route(logits, dtype, E, tokens, E, K, scores, bias, groups, top, best, 1, scale, ids, weights, None)


@pytest.mark.parametrize("kw,want", [
    (dict(tokens=0), OK), (dict(tokens=0, logits=None, ids=None), OK), (dict(logits=None), INVALID), (dict(ids=None), INVALID),
    (dict(weights=None), INVALID), (dict(logits=A + 1), INVALID), (dict(ids=A + 2), INVALID), (dict(weights=A + 2), INVALID),
    (dict(bias=A + 2), INVALID), (dict(dtype=5), INVALID), (dict(scores=2), INVALID), (dict(tokens=-1), INVALID),
    (dict(tokens=2 ** 30 + 1), SHAPE), (dict(E=0), INVALID), (dict(E=1025), SHAPE), (dict(K=0), INVALID), (dict(K=129), SHAPE),
    (dict(E=1024, K=65), SHAPE), (dict(groups=0), INVALID), (dict(groups=3), SHAPE), (dict(groups=64), SHAPE),
    (dict(E=1023, groups=3), SHAPE), (dict(groups=8, top=9), INVALID), (dict(groups=8, top=0), INVALID),
    (dict(groups=32, top=1, K=5), SHAPE), (dict(best=0), INVALID), (dict(best=3), INVALID), (dict(scale=NAN), INVALID),
    (dict(scale=INF), INVALID)])
def test_route(kw, want):
    assert route(**kw) == want


def history(**kw):
    d = dict(tokens=A, lengths=A, prompt_lengths=A, seqs=A, stride=64, slots=4, columns=64)
    d.update(kw)
    return _History(**d)


def logits(x=A, dtype=0, B=4, V=1000, h=None, repetition=None, presence=None, frequency=None, start=None, ids=None,
           values=None, biases=0, temperature=None, mask=None, out=2 * A, out_dtype=0, stride=1000, out_stride=1000):
    return wd.lib().wd_adjust_logits(x, dtype, stride, B, V, ctypes.byref(h) if h is not None else None, repetition, presence,
                                     frequency, start, ids, values, biases, temperature, mask, 32, out, out_dtype, out_stride,
                                     None)


@pytest.mark.parametrize("kw,want", [
    (dict(B=0), OK), (dict(B=0, x=None), OK), (dict(x=None), INVALID), (dict(out=None), INVALID), (dict(x=A + 1), INVALID),
    (dict(out=A + 1), INVALID), (dict(out_dtype=2, out=2 * A + 2), INVALID), (dict(dtype=3), INVALID), (dict(out_dtype=1), INVALID),
    (dict(dtype=2, out_dtype=0), INVALID), (dict(B=-1), INVALID), (dict(B=65536), SHAPE), (dict(V=0), INVALID),
    (dict(V=2 ** 24 + 1, out_stride=2 ** 25), SHAPE), (dict(out_stride=999), INVALID), (dict(out_stride=0), INVALID),
    (dict(out=A, out_dtype=2), INVALID), (dict(out=A, out_stride=1001), INVALID), (dict(repetition=A), INVALID),
    (dict(presence=A), INVALID), (dict(frequency=A), INVALID), (dict(repetition=A + 1, h=history()), INVALID),
    (dict(h=history(lengths=None)), INVALID), (dict(h=history(tokens=A + 1)), INVALID), (dict(h=history(seqs=A + 1)), INVALID),
    (dict(h=history(prompt_lengths=A + 1)), INVALID), (dict(h=history(slots=0)), INVALID), (dict(h=history(columns=-1)), INVALID),
    (dict(h=history(columns=2 ** 20 + 1)), SHAPE), (dict(temperature=A + 2), INVALID), (dict(mask=A + 2), INVALID),
    (dict(start=A), INVALID), (dict(start=A, ids=A), INVALID), (dict(ids=A), INVALID), (dict(values=A), INVALID),
    (dict(start=A, ids=A, values=A, biases=-1), INVALID), (dict(start=A, ids=A + 2, values=A), INVALID)])
def test_logits(kw, want):
    assert logits(**kw) == want


def rotated(q=A, k=A, v=A, dtype=0, heads=32, q_out=A, k_out=None, v_out=None, cos_sin=A, positions=100, rot=128, entries=4,
            tokens=4, layer=0, **kw):
    d = dict(pool=A, table=A, lengths=A, refs=A, workspace=A, workspace_bytes=1 << 40, num_pages=64, slots=8, columns=16,
             page_size=64, layers=2, kv_heads=4, head_dim=128)
    d.update(kw)
    return wd.lib().wd_kv_append_rotated(ctypes.byref(_Cache(**d)), layer, q, k, v, dtype, 4096, 128, heads, 512, 128, 512, 128,
                                         q_out, k_out, v_out, cos_sin, positions, rot, 0, None, None, entries, tokens, None)


@pytest.mark.parametrize("kw,want", [
    (dict(tokens=0), OK), (dict(entries=0, tokens=0), OK), (dict(tokens=0, cos_sin=None), OK), (dict(k=None), INVALID),
    (dict(v=None), INVALID), (dict(q=None), INVALID), (dict(q_out=None), INVALID), (dict(q=A + 1), INVALID),
    (dict(q_out=A + 1), INVALID), (dict(heads=0), INVALID), (dict(heads=4097), INVALID), (dict(dtype=3), INVALID),
    (dict(k_out=A), INVALID), (dict(cos_sin=None), INVALID), (dict(cos_sin=A + 8), INVALID), (dict(positions=0), INVALID),
    (dict(rot=0), SHAPE), (dict(rot=8), SHAPE), (dict(rot=24), SHAPE), (dict(rot=144), SHAPE), (dict(rot=-16), SHAPE),
    (dict(layer=2), INVALID), (dict(layer=-1), INVALID), (dict(tokens=5), INVALID), (dict(entries=9, tokens=1), INVALID),
    (dict(head_dim=96), SHAPE), (dict(pool=None), INVALID), (dict(workspace_bytes=1), SMALL)])
def test_append_rotated(kw, want):
    assert rotated(**kw) == want


def test_rotation_table_refuses():
    for bad in (dict(positions=0, rot=16), dict(positions=4, rot=8), dict(positions=4, rot=20), dict(positions=4, rot=0),
                dict(positions=4, rot=16, frequencies=[1.0] * 7)):
        with pytest.raises(ValueError):
            wd.rotation_table(device="cpu", **bad)
    assert wd.rotation_table(4, 16, frequencies=[0.0] * 8, device="cpu").tolist() == [[1.0] * 8 + [0.0] * 8] * 4
