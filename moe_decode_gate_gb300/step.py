"""The small operators of a decode step around attention and experts: the C-ABI of include/wd_step.h.

Every call is asynchronous on the current stream (or ``stream``) of its tensors' device, which has to be the
current one.  A call on ``stream`` keeps the memory of what it reads and writes until it is done; that the inputs are
there when it starts, and that it is done before its results are read elsewhere, is the caller's to see to, as with
any two streams.
"""
from __future__ import annotations

import ctypes

import torch

from ._native import _check, lib

_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_SCORES = {"softmax": 0, "sigmoid": 1}
_LIB = None
_MOST = 2 ** 31 - 1  # what the library's int parameters hold: ctypes would cut a larger number to its low bits


class _History(ctypes.Structure):
    """wd_history of include/wd_step.h."""

    _fields_ = [("tokens", ctypes.c_void_p), ("lengths", ctypes.c_void_p),
                ("prompt_lengths", ctypes.c_void_p), ("seqs", ctypes.c_void_p),
                ("stride", ctypes.c_int64), ("slots", ctypes.c_int32), ("columns", ctypes.c_int32)]


def _library():
    global _LIB
    if _LIB is None:
        _LIB = lib()
    return _LIB


def _raw_stream(device, stream):
    """The raw handle of ``stream``, or of the current stream of the tensors' device. The kernels are launched on the
    current device, which has to be that one."""
    index = device.index
    if torch._C._cuda_getDevice() != index:
        raise ValueError(f"the current device must be the tensors', {device}")
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(index)
    if stream.device != device:
        raise ValueError(f"stream must be one of {device}")
    return stream.cuda_stream


def _output(shape, dtype, device, stream):
    """A result of a call on ``stream``: that stream's memory, not given away before the current stream too, on which
    the caller may read it, has done what it was asked until then."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream(device))
    return t


def _keep(stream, *tensors):
    """After a call on ``stream``: the memory of these is not given away before it is done."""
    if stream is not None:
        for t in tensors:
            if t is not None:
                t.record_stream(stream)


def _given(name, t, shape, dtype, device):
    """Pointer of a tensor that the caller gives for a result."""
    if t.shape != shape or t.dtype is not dtype or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous {dtype} {list(shape)} on {device}")
    return t.data_ptr()


def _vector(name, t, n, dtype, device):
    """Pointer of a contiguous vector of n elements (None stays None)."""
    if t is None:
        return None
    if t.dtype is not dtype or t.device != device or t.dim() != 1 or not t.is_contiguous() or \
            (n is not None and t.shape[0] != n):
        raise ValueError(f"{name} must be a contiguous {dtype} vector" +
                         ("" if n is None else f" of {n} elements") + f" on {device}")
    return t.data_ptr()


def _per(name, t, n, dtype, device):
    """_vector of one number to each of n, with few look-ups where it is right."""
    if t is None:
        return None
    if t.dtype is not dtype or t.shape != (n,) or t.device != device or not t.is_contiguous():
        _vector(name, t, n, dtype, device)
    return t.data_ptr()


# As in kv_cache.py each call checks its tensors with as few attribute look-ups as it can (a call costs the host some ten
# microseconds, most of it the results' allocation and the launch), and says what is wrong in the slow path.

def _refuse_rows(name, t, device):
    """Says what is wrong with a tensor that should be [tokens, H] or [tokens, heads, H] with contiguous channels."""
    if t.dtype not in _DTYPES or t.device.type != "cuda":
        raise ValueError(f"{name} must be a BF16, FP16 or FP32 CUDA tensor")
    if t.device != device or t.dim() not in (2, 3):
        raise ValueError(f"{name} must be [tokens, H] or [tokens, heads, H] on {device}")
    raise ValueError(f"{name} must have contiguous channels")


def _refuse_matrix(name, t, columns):
    """Says what is wrong with a tensor that should be [rows, columns] with contiguous rows."""
    if t.dtype not in _DTYPES or t.device.type != "cuda" or t.dim() != 2:
        raise ValueError(f"{name} must be a BF16, FP16 or FP32 CUDA tensor {columns}")
    raise ValueError(f"{name} must have contiguous rows")


def rms_norm(x, weight=None, residual=None, *, eps=1e-6, mxfp8=False, out=None, residual_out=None, stream=None):
    """Root-mean-square norm of each row of x + residual, times ``weight``.

    x: [tokens, H] or [tokens, heads, H] BF16, FP16 or FP32, any strides with contiguous channels; weight [H] of x's
    type or FP32; residual of x's shape and type.  Returns the norm in x's type, or with ``mxfp8`` (codes, scales)
    in MXFP8 as the expert weights have it: uint8 E4M3 [..., H] and E8M0 [..., H / 32]; with a residual the
    sum in x's type comes last.  ``out`` receives the norm in x's type (with ``mxfp8`` in addition to the codes),
    ``residual_out`` the sum; they may be x and residual where those are contiguous."""
    dtype, shape, device = x.dtype, x.shape, x.device
    code, index, strides = _DTYPES.get(dtype), device.index, x.stride()
    n = len(shape)
    if code is None or index is None or not 1 < n < 4 or (strides[-1] != 1 and shape[-1] != 1):
        _refuse_rows("x", x, device)
    tokens, H = shape[0], shape[-1]
    token, head, heads = strides[0], strides[1] if n == 3 else 0, shape[1] if n == 3 else 1
    if H > _MOST or heads > _MOST:
        raise ValueError(f"unsupported sizes: {list(shape)}")
    weight_code, w = code, None
    if weight is not None:
        if weight.dtype is not dtype:
            weight_code = 2
        w = _vector("weight", weight, H, torch.float32 if weight_code == 2 else dtype, device)
    res = res_to = None
    res_token = res_head = 0
    if residual is not None:
        if residual.shape != shape or residual.dtype is not dtype:
            raise ValueError("residual must have x's shape and type")
        strides = residual.stride()
        if residual.device != device or (strides[-1] != 1 and H != 1):
            _refuse_rows("residual", residual, device)
        res_token, res_head = strides[0], strides[1] if n == 3 else 0
        res = residual.data_ptr()
        if residual_out is None:
            residual_out = torch.empty(shape, dtype=dtype, device=device) if stream is None else \
                _output(shape, dtype, device, stream)
            res_to = residual_out.data_ptr()
        else:
            res_to = _given("residual_out", residual_out, shape, dtype, device)
    elif residual_out is not None:
        raise ValueError("residual_out without residual")
    y = codes = scales = codes_to = scales_to = None
    if out is not None:
        y = _given("out", out, shape, dtype, device)
    if mxfp8:
        if H % 32:
            raise ValueError(f"MXFP8 wants a multiple of 32 channels, not {H}")
        u8, per_block = torch.uint8, (*shape[:-1], H // 32)
        codes = torch.empty(shape, dtype=u8, device=device) if stream is None else _output(shape, u8, device, stream)
        scales = torch.empty(per_block, dtype=u8, device=device) if stream is None else \
            _output(per_block, u8, device, stream)
        codes_to, scales_to = codes.data_ptr(), scales.data_ptr()
    elif out is None:
        out = torch.empty(shape, dtype=dtype, device=device) if stream is None else \
            _output(shape, dtype, device, stream)
        y = out.data_ptr()
    if tokens and heads:
        st = (_LIB or _library()).wd_rms_norm(x.data_ptr(), code, token, head, tokens, heads, H, w, weight_code, res,
                                              res_token, res_head, res_to, eps, y, codes_to, scales_to,
                                              _raw_stream(device, stream))
        if st:
            _check("wd_rms_norm", st)
        if stream is not None:
            _keep(stream, x, weight, residual, residual_out, out, codes, scales)
    if mxfp8:
        return (codes, scales) if residual is None else (codes, scales, residual_out)
    return out if residual is None else (out, residual_out)


def route(logits, K, *, scores="softmax", bias=None, groups=1, top_groups=None, group_best=2, renormalise=True,
          scale=1.0, ids=None, weights=None, stream=None):
    """The K experts of each token and their weights, as ``MoEDecodeLayer`` takes them.

    logits: [tokens, E] BF16, FP16 or FP32, rows any stride apart.  ``scores``: "softmax" or "sigmoid" of them; ``bias``
    FP32 [E] is added for the choice and left out of the weights.  Of ``groups`` equal groups the ``top_groups``
    (default: all) with the largest sums of their ``group_best`` (1 or 2) best are open.  Weights are divided by
    their sum if ``renormalise``, and multiplied by ``scale``.  A logit of -inf or NaN masks its expert.  Returns (ids
    int32, weights FP32) [tokens, K], largest key first, the lowest index first of equal ones."""
    shape, device = logits.shape, logits.device
    code, kind = _DTYPES.get(logits.dtype), _SCORES.get(scores)
    if code is None or device.index is None or len(shape) != 2:
        _refuse_matrix("logits", logits, "[tokens, E]")
    if kind is None:
        raise ValueError(f"scores must be one of {', '.join(_SCORES)}")
    tokens, E = shape
    if E > _MOST or K > _MOST:
        raise ValueError(f"unsupported sizes: {K} of {E} experts")
    stride, last = logits.stride()
    if last != 1 and E != 1:
        _refuse_matrix("logits", logits, "[tokens, E]")
    b = None if bias is None else _vector("bias", bias, E, torch.float32, device)
    shape = (tokens, K)
    if ids is None:
        ids = torch.empty(shape, dtype=torch.int32, device=device) if stream is None else \
            _output(shape, torch.int32, device, stream)
        ids_to = ids.data_ptr()
    else:
        ids_to = _given("ids", ids, shape, torch.int32, device)
    if weights is None:
        weights = torch.empty(shape, dtype=torch.float32, device=device) if stream is None else \
            _output(shape, torch.float32, device, stream)
        weights_to = weights.data_ptr()
    else:
        weights_to = _given("weights", weights, shape, torch.float32, device)
    st = (_LIB or _library()).wd_route(logits.data_ptr(), code, stride, tokens, E, K, kind, b, groups,
                                       groups if top_groups is None else top_groups, group_best, renormalise, scale,
                                       ids_to, weights_to, _raw_stream(device, stream))
    if st:
        _check("wd_route", st)
    if stream is not None:
        _keep(stream, logits, bias, ids, weights)
    return ids, weights


def adjust_logits(logits, *, history=None, lengths=None, prompt_lengths=None, seqs=None, repetition=None, presence=None,
                  frequency=None, bias=None, temperature=None, mask=None, dtype=None, out=None, stream=None):
    """What is done to logits before a token is chosen: penalties for tokens that came before, biases, temperature, mask.

    logits: [B, V] BF16, FP16 or FP32, rows any stride apart.  ``history`` int32 [slots, columns] are the tokens so far,
    ``lengths`` int32 [slots] how many, ``prompt_lengths`` int32 [slots] (None: none) how many of them are the prompt;
    row b's request is in slot seqs[b] (slot b without seqs).  ``repetition``, ``presence``, ``frequency`` and
    ``temperature`` are FP32 [B]; ``bias`` is (start int32 [B + 1], ids int32 [N], values FP32 [N]); ``mask`` int32 words
    [B, ceil(V / 32)], a token to a bit.  Steps and order: include/wd_step.h.  Returns [B, V] of ``dtype`` (logits' own
    type, the default, or FP32), in ``out`` if given, which may be logits."""
    kind, shape, device = logits.dtype, logits.shape, logits.device
    code = _DTYPES.get(kind)
    if code is None or device.index is None or len(shape) != 2:
        _refuse_matrix("logits", logits, "[B, V]")
    B, V = shape
    if B > _MOST or V > _MOST:
        raise ValueError(f"unsupported sizes: {list(shape)}")
    stride, last = logits.stride()
    if last != 1 and V != 1:
        _refuse_matrix("logits", logits, "[B, V]")
    to = kind if dtype is None else dtype
    if out is not None and dtype is None:
        to = out.dtype
    if to is not kind and to is not torch.float32:
        raise ValueError(f"dtype must be {kind} or {torch.float32}")
    if out is None:
        out = torch.empty(shape, dtype=to, device=device) if stream is None else _output(shape, to, device, stream)
        out_stride = V
    else:
        if out.shape != shape or out.dtype is not to or out.device != device or (out.stride(1) != 1 and V != 1):
            raise ValueError(f"out must be {to} {[B, V]} with contiguous rows on {device}")
        out_stride = out.stride(0)
    h = None
    if history is not None:
        if history.dtype is not torch.int32 or history.dim() != 2 or history.device != device or \
                (history.stride(1) != 1 and history.shape[1] != 1):
            raise ValueError(f"history must be int32 [slots, columns] with contiguous rows on {device}")
        if lengths is None:
            raise ValueError("history needs lengths")
        slots, columns = history.shape
        if slots > _MOST or columns > _MOST:
            raise ValueError(f"unsupported sizes: a history of {list(history.shape)}")
        i32 = torch.int32
        h = _History(history.data_ptr(), _per("lengths", lengths, slots, i32, device),
                     _per("prompt_lengths", prompt_lengths, slots, i32, device), _per("seqs", seqs, B, i32, device),
                     history.stride(0), slots, columns)
        if not columns:  # nothing came before
            h = repetition = presence = frequency = None
    elif repetition is not None or presence is not None or frequency is not None:
        raise ValueError("penalties need a history")
    elif lengths is not None or prompt_lengths is not None or seqs is not None:
        raise ValueError("lengths, prompt_lengths and seqs go with a history")
    start = ids = values = None
    n = 0
    if bias is not None:
        starts, tokens, amounts = bias
        n = tokens.shape[0]
        if n > _MOST:
            raise ValueError(f"unsupported sizes: {n} biases")
        start = _per("bias start", starts, B + 1, torch.int32, device)
        ids = _per("bias ids", tokens, n, torch.int32, device)
        values = _per("bias values", amounts, n, torch.float32, device)
        if not n:
            start = ids = values = None
    m, mask_stride = None, 0
    if mask is not None:
        if mask.dtype is not torch.int32 or mask.shape != (B, (V + 31) // 32) or mask.device != device or \
                (mask.stride(1) != 1 and mask.shape[1] != 1):
            raise ValueError(f"mask must be int32 {[B, (V + 31) // 32]} with contiguous rows on {device}")
        m, mask_stride = mask.data_ptr(), mask.stride(0)
    f32 = torch.float32
    st = (_LIB or _library()).wd_adjust_logits(
        logits.data_ptr(), code, stride, B, V, None if h is None else ctypes.byref(h),
        _per("repetition", repetition, B, f32, device), _per("presence", presence, B, f32, device),
        _per("frequency", frequency, B, f32, device), start, ids, values, n,
        _per("temperature", temperature, B, f32, device), m, mask_stride, out.data_ptr(), _DTYPES[to], out_stride,
        _raw_stream(device, stream))
    if st:
        _check("wd_adjust_logits", st)
    if stream is not None:
        _keep(stream, logits, history, lengths, prompt_lengths, seqs, repetition, presence, frequency, temperature, mask,
              out, *(bias or ()))
    return out
