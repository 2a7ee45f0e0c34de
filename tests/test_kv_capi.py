"""The C-ABI of the 4-bit cache without a GPU: symbols, sizes, and what the host refuses.

Every call below fails host validation or does nothing, so no kernel is launched.
"""
import ctypes
import os
import re

import numpy as np
import pytest

import kv_reference as ref
import moe_decode_gate_gb300 as wd
from moe_decode_gate_gb300 import _native
from moe_decode_gate_gb300.kv_cache import _Cache

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include",
                      "wd_kv.h")
OK, INVALID, SHAPE, SMALL = 0, 1, 2, 3
A = 0x10000  # an aligned fake address: never dereferenced


def cache(**kw):
    d = dict(pool=A, table=A, lengths=A, refs=A, workspace=A, workspace_bytes=1 << 40,
             num_pages=64, slots=8, columns=16, page_size=64, layers=2, kv_heads=4, head_dim=128)
    d.update(kw)
    return ctypes.byref(_Cache(**d))


def test_library_exports_every_declared_symbol():
    names = re.findall(r"^WD_API\s+[\w\s\*]+?\b(wd_\w+)\s*\(", open(HEADER).read(), flags=re.M)
    assert {"wd_kv_append", "wd_kv_attention", "wd_kv_fork", "wd_kv_compact"} <= set(names)
    for name in names:
        assert hasattr(wd.lib(), name) and name in _native.SIGNATURES, name


def test_page_bytes():
    assert wd.wd_kv_page_bytes(1, 1, 128, 16) == 16 * 136 == ref.group_bytes(128)
    assert wd.wd_kv_page_bytes(48, 4, 128, 64) == 48 * 4 * 64 * 136
    assert wd.wd_kv_page_bytes(1, 1, 64, 32) == 32 * 68
    assert wd.wd_kv_page_bytes(1, 1, 256, 256) == 256 * 272
    for bad in ((0, 1, 128, 16), (1, 0, 128, 16), (1, 1, 96, 16), (1, 1, 128, 24), (1, 1, 128, 512),
                (1025, 1, 128, 16), (1, 257, 128, 16)):
        assert wd.wd_kv_page_bytes(*bad) == 0


def test_workspace_size():
    size = wd.lib().wd_kv_workspace_size
    n = size(cache())
    assert n > 0 and n % 256 == 0
    assert size(cache(num_pages=1 << 20)) >= n + 3 * 4 * ((1 << 20) - 64)
    assert size(cache(slots=4096)) > n
    for bad in (dict(num_pages=0), dict(num_pages=(1 << 24) + 1), dict(slots=0),
                dict(slots=65537), dict(columns=0), dict(columns=(1 << 20) + 1),
                dict(head_dim=32), dict(page_size=8), dict(kv_heads=0), dict(layers=0)):
        assert size(cache(**bad)) == 0
    assert size(None) == 0


CACHE_FAULTS = [
    (dict(pool=None), INVALID), (dict(table=None), INVALID), (dict(lengths=None), INVALID),
    (dict(refs=None), INVALID), (dict(workspace=None), INVALID), (dict(pool=A + 8), INVALID),
    (dict(table=A + 2), INVALID), (dict(workspace=A + 128), INVALID),
    (dict(workspace_bytes=1000), SMALL), (dict(head_dim=96), SHAPE), (dict(page_size=48), SHAPE),
    (dict(num_pages=0), SHAPE), (dict(slots=0), SHAPE), (dict(columns=0), SHAPE),
]


def append(c, layer=0, k=A, v=A, dtype=0, k_out=None, v_out=None, seqs=None, q_start=None,
           entries=4, tokens=4):
    return wd.lib().wd_kv_append(c, layer, k, v, dtype, 512, 128, 512, 128, k_out, v_out, seqs,
                                 q_start, entries, tokens, None)


def attention(c, layer=0, q=A, dtype=0, heads=32, out=A, lse=None, seqs=None, q_start=None,
              entries=4, tokens=4, max_q=1, scale=0.1, window=0):
    return wd.lib().wd_kv_attention(c, layer, q, dtype, 4096, 128, heads, out, lse, seqs, q_start,
                                    entries, tokens, max_q, scale, window, None)


@pytest.mark.parametrize("kw,status", CACHE_FAULTS)
def test_every_call_looks_at_the_cache(kw, status):
    lib, flag = wd.lib(), ctypes.c_int(9)
    assert append(cache(**kw)) == status
    assert attention(cache(**kw)) == status
    assert lib.wd_kv_reserve(cache(**kw), A, A, 1, A, None) == status
    assert lib.wd_kv_fork(cache(**kw), A, A, 1, A, None) == status
    assert lib.wd_kv_free(cache(**kw), A, 1, None) == status
    assert lib.wd_kv_compact(cache(**kw), None, None, None, None) == status
    assert lib.wd_kv_workspace_init(cache(**kw), None) == status
    assert lib.wd_kv_read_error_flag(cache(**kw), None, ctypes.byref(flag)) == status
    assert flag.value == 9


@pytest.mark.parametrize("kw", [
    dict(layer=-1), dict(layer=2), dict(k=None), dict(v=None), dict(k=A + 1), dict(dtype=3),
    dict(k=A + 2, dtype=2), dict(k_out=A), dict(v_out=A), dict(k_out=A + 1, v_out=A),
    dict(entries=-1), dict(entries=4097, seqs=A), dict(entries=9), dict(tokens=-1),
    dict(tokens=5), dict(tokens=(1 << 20) + 1, q_start=A), dict(seqs=A + 2), dict(q_start=A + 1)])
def test_append_refuses(kw):
    assert append(cache(), **kw) == INVALID


@pytest.mark.parametrize("kw", [
    dict(layer=2), dict(q=None), dict(out=None), dict(q=A + 1), dict(dtype=2), dict(heads=0),
    dict(heads=30), dict(heads=8192), dict(lse=A + 2), dict(max_q=-1), dict(window=-1),
    dict(scale=0.0), dict(scale=-1.0), dict(scale=float("inf")), dict(scale=float("nan")),
    dict(entries=9), dict(tokens=5), dict(tokens=-1)])
def test_attention_refuses(kw):
    assert attention(cache(), **kw) == INVALID


def test_page_calls_refuse():
    lib = wd.lib()
    assert lib.wd_kv_reserve(cache(), A, None, 1, None, None) == INVALID
    assert lib.wd_kv_reserve(cache(), A, A, 9, None, None) == INVALID
    assert lib.wd_kv_reserve(cache(), A, A, -1, None, None) == INVALID
    assert lib.wd_kv_reserve(cache(), A + 1, A, 1, None, None) == INVALID
    assert lib.wd_kv_fork(cache(), A, None, 1, None, None) == INVALID
    assert lib.wd_kv_fork(cache(), A, A, 9, None, None) == INVALID
    assert lib.wd_kv_fork(cache(), A, A, 1, A + 2, None) == INVALID
    assert lib.wd_kv_free(cache(), None, 1, None) == INVALID
    assert lib.wd_kv_compact(cache(), A, None, None, None) == INVALID
    assert lib.wd_kv_compact(cache(), None, A, None, None) == INVALID
    assert lib.wd_kv_compact(cache(), None, None, A + 1, None) == INVALID
    assert lib.wd_kv_read_error_flag(cache(), None, None) == INVALID


def test_empty_calls_do_nothing():
    assert append(cache(), entries=0, tokens=0) == OK
    assert attention(cache(), entries=0, tokens=0) == OK
    assert wd.lib().wd_kv_reserve(cache(), None, None, 0, None, None) == OK
    assert wd.lib().wd_kv_fork(cache(), None, None, 0, None, None) == OK


def test_cache_refuses_tensors_that_are_not_on_a_gpu():
    torch = pytest.importorskip("torch")
    with pytest.raises(ValueError):
        wd.KVCache.from_buffers(torch.zeros(16 * 136, dtype=torch.uint8),
                                torch.zeros(1, 1, dtype=torch.int32),
                                torch.zeros(1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32),
                                layers=1, kv_heads=1, head_dim=128, page_size=16)
    with pytest.raises(ValueError):
        wd.KVCache(4, 1, 4, 1, 1, head_dim=80, device="cpu")


# ------------------------------------------------- the reference itself, pinned ---

def test_reference_rounds_to_the_nearest_code():
    # every value halfway between two codes goes to the even one; past 6 saturates
    x = np.zeros(32)
    x[:16] = [4.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.1, 7.9, -0.25, -0.76, 0.24, 6.0, -0.0,
              -4.0]
    code, scale = ref.quantise(x)
    assert scale.tolist() == [127]
    assert code[:16].tolist() == [6, 0, 2, 2, 4, 4, 6, 6, 7, 7, 8, 10, 0, 7, 8, 14]
    assert ref.values(code, scale)[9] == 6.0
    code, scale = ref.quantise(np.zeros(32))
    assert scale.tolist() == [127] and not code.any()
    for bad in (np.nan, np.inf):
        code, scale = ref.quantise(np.full(32, bad))
        assert scale.tolist() == [255] and np.isnan(ref.values(code, scale)).all()
    assert ref.quantise(np.full(32, 2.0 ** -140))[1].tolist() == [0]


@pytest.mark.parametrize("D", [64, 128, 256])
def test_reference_layout_is_a_bijection(D):
    k, v, shift = ref._places(D)
    where = {(int(b), int(s)) for b, s in zip(np.r_[k.ravel(), v.ravel()],
                                              np.r_[shift.ravel(), shift.ravel()])}
    assert len(where) == 2 * 16 * D and max(b for b, _ in where) == 16 * D - 1


def test_reference_attention_by_hand():
    # two tokens with equal logits: the mean of their values
    D, P = 64, 16
    pool = np.zeros((1, 1, 1, 1, ref.group_bytes(D)), np.uint8)
    for t, x in enumerate((1.0, 3.0)):
        kc, ks = ref.quantise(np.zeros(D))
        vc, vs = ref.quantise(np.full(D, x))
        ref.store(pool, 0, 0, 0, t, D, kc, ks, vc, vs)
    out, lse, _ = ref.attention(pool, np.array([[0]]), np.array([2]), 0, np.ones((1, 2, D)), [0],
                                [0, 1], D, P, 0.5)
    assert np.allclose(out, 2.0) and np.allclose(lse, np.log(2.0))
