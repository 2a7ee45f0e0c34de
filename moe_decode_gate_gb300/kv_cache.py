"""A paged cache of keys and values held in 4 bits (MXFP4): the C-ABI of include/wd_kv.h."""
from __future__ import annotations

import ctypes
import math

import torch

from ._native import _check, lib

KV_FLAG_BAD_INDEX = 1
KV_FLAG_TIMEOUT = 2
KV_FLAG_NO_PAGES = 4

_Q_DTYPES = {torch.bfloat16: 0, torch.float16: 1}
_DTYPES = {**_Q_DTYPES, torch.float32: 2}


class _Cache(ctypes.Structure):
    """wd_kv_cache of include/wd_kv.h."""

    _fields_ = [("pool", ctypes.c_void_p), ("table", ctypes.c_void_p),
                ("lengths", ctypes.c_void_p), ("refs", ctypes.c_void_p),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
                *((name, ctypes.c_int32) for name in ("num_pages", "slots", "columns", "page_size",
                                                      "layers", "kv_heads", "head_dim"))]


def wd_kv_page_bytes(layers: int, kv_heads: int, head_dim: int, page_size: int) -> int:
    """Bytes of one page of all layers; 0 for dimensions that the cache does not take."""
    return int(lib().wd_kv_page_bytes(layers, kv_heads, head_dim, page_size))


def rotation_table(positions: int, rot: int, base: float = 10000.0, frequencies=None, scale: float = 1.0,
                   device="cuda"):
    """cos_sin of ``KVCache.append_rotated``: FP32 [positions, rot], row p the cosines and then the sines of the
    angles p * frequencies[i], i < rot / 2, times ``scale``.

    ``frequencies`` (a sequence or tensor of rot / 2 angles per position) defaults to base ** (-2 i / rot).  Angles
    are taken in 64 bits, so that far positions are as exact as near ones."""
    if rot < 16 or rot % 16 or positions < 1:
        raise ValueError(f"unsupported rotation: {positions} positions, {rot} channels")
    if frequencies is None:
        f = base ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=device) / rot)
    else:
        f = torch.as_tensor(frequencies, dtype=torch.float64, device=device)
        if f.shape != (rot // 2,):
            raise ValueError(f"frequencies must be {rot // 2} numbers")
    table = torch.empty(positions, rot, dtype=torch.float32, device=device)
    for a in range(0, positions, 65536):
        b = min(positions, a + 65536)
        angle = torch.arange(a, b, dtype=torch.float64, device=device)[:, None] * f
        table[a:b, :rot // 2] = scale * angle.cos()
        table[a:b, rot // 2:] = scale * angle.sin()
    return table


class KVCache:
    """Keys and values of ``slots`` sequences in pages of ``page_size`` tokens, MXFP4.

    ``pool`` uint8 [num_pages, layers, kv_heads, page_size / 16, group bytes], ``table`` int32
    [slots, columns] (the pages of each slot's sequence, -1 beyond), ``lengths`` int32 [slots] and
    ``refs`` int32 [num_pages] are the cache, on the device; include/wd_kv.h has their layout.
    The cache's device has to be the current one.
    Every call is asynchronous on the current stream (or ``stream``); calls on different streams
    must be ordered by the caller, as they share the workspace.  A call on ``stream`` keeps the memory of what
    it reads and writes until it is done; that the inputs are there when it starts, and that it is done
    before its results are read elsewhere, is the caller's to see to, as with any two streams.

    A decode step::

        cache.reserve(ones, seqs)                       # a place for each sequence's new token
        for layer in range(cache.layers):
            cache.append(layer, k, v, seqs)
            y = cache.attention(layer, q, seqs)
    """

    def __init__(self, num_pages, slots, columns, layers, kv_heads, head_dim, page_size=64,
                 device="cuda"):
        page = wd_kv_page_bytes(layers, kv_heads, head_dim, page_size)
        if not page:
            raise ValueError(f"unsupported cache: layers={layers}, kv_heads={kv_heads}, "
                             f"head_dim={head_dim}, page_size={page_size}")
        group = page // (layers * kv_heads * (page_size // 16))
        device = torch.device(device)
        self._adopt(torch.zeros(num_pages, layers, kv_heads, page_size // 16, group,
                                dtype=torch.uint8, device=device),
                    torch.full((slots, columns), -1, dtype=torch.int32, device=device),
                    torch.zeros(slots, dtype=torch.int32, device=device),
                    torch.zeros(num_pages, dtype=torch.int32, device=device),
                    layers, kv_heads, head_dim, page_size)

    @classmethod
    def from_buffers(cls, pool, table, lengths, refs, *, layers, kv_heads, head_dim, page_size):
        """A cache over tensors that the caller holds (they are used, not copied)."""
        self = cls.__new__(cls)
        self._adopt(pool, table, lengths, refs, layers, kv_heads, head_dim, page_size)
        return self

    def _adopt(self, pool, table, lengths, refs, layers, kv_heads, head_dim, page_size):
        page = wd_kv_page_bytes(layers, kv_heads, head_dim, page_size)
        if not page:
            raise ValueError(f"unsupported cache: layers={layers}, kv_heads={kv_heads}, "
                             f"head_dim={head_dim}, page_size={page_size}")
        slots, columns = table.shape
        num_pages = refs.numel()
        for name, t, dtype, n in (("pool", pool, torch.uint8, num_pages * page),
                                  ("table", table, torch.int32, slots * columns),
                                  ("lengths", lengths, torch.int32, slots),
                                  ("refs", refs, torch.int32, num_pages)):
            if not t.is_cuda or not t.is_contiguous() or t.dtype != dtype or t.numel() != n:
                raise ValueError(f"{name} must be a contiguous {dtype} CUDA tensor of {n} elements")
            if t.device != pool.device:
                raise ValueError(f"{name} must be on {pool.device}")
        self.pool, self.table, self.lengths, self.refs = pool, table, lengths, refs
        self.device = pool.device
        self.layers, self.kv_heads, self.head_dim = layers, kv_heads, head_dim
        self.page_size, self.num_pages = page_size, num_pages
        self.slots, self.columns = slots, columns
        c = self._c = _Cache(pool.data_ptr(), table.data_ptr(), lengths.data_ptr(), refs.data_ptr(),
                             None, 0, num_pages, slots, columns, page_size, layers, kv_heads,
                             head_dim)
        self._ref = ctypes.byref(c)
        self._lib = lib()
        self._index = self.device.index
        self._scale = 1.0 / math.sqrt(head_dim)
        size = int(self._lib.wd_kv_workspace_size(self._ref))
        if not size:
            raise ValueError(f"unsupported cache: num_pages={num_pages}, slots={slots}, "
                             f"columns={columns}")
        self.workspace = torch.empty(size, dtype=torch.uint8, device=self.device)
        c.workspace, c.workspace_bytes = self.workspace.data_ptr(), size
        _check("wd_kv_workspace_init", self._lib.wd_kv_workspace_init(self._ref, self._stream(None)))

    # ------------------------------------------------------------------ arguments ---

    def _stream(self, stream):
        """The raw handle of ``stream``, or of the current stream of the cache's device (looked up
        without the Stream object that torch.cuda.current_stream() makes: 0.1 against 3 us).  The kernels
        are launched on the current device, which has to be the cache's."""
        if torch._C._cuda_getDevice() != self._index:
            raise ValueError(f"the current device must be the cache's, {self.device}")
        if stream is None:
            return torch._C._cuda_getCurrentRawStream(self._index)
        if stream.device != self.device:
            raise ValueError(f"stream must be one of {self.device}")
        return stream.cuda_stream

    def _output(self, shape, dtype, stream):
        """A result of a call on ``stream``: that stream's memory, so that nothing that still runs on
        another one uses it, and not given away before the current stream too, on which the caller may
        read it, has done what it was asked until then."""
        if stream is None:
            return torch.empty(shape, dtype=dtype, device=self.device)
        with torch.cuda.stream(stream):
            t = torch.empty(shape, dtype=dtype, device=self.device)
        t.record_stream(torch.cuda.current_stream(self.device))
        return t

    def _keep(self, stream, *tensors):
        """After a call on ``stream`` that uses these tensors, and the cache's own: their memory is not
        given away before the call is done, even if the caller drops them at once."""
        if stream is None:
            return
        for t in (*tensors, self.pool, self.table, self.lengths, self.refs, self.workspace):
            if t is not None:
                t.record_stream(stream)

    # Each call checks its tensors with as few attribute look-ups as it can (a call costs the host
    # about ten microseconds, half of it the launch) and says what is wrong in the slow path.

    def _ints(self, name, t, n=None):
        """Pointer of an int32 vector on the cache's device (None stays None)."""
        if t is None:
            return None
        if t.dtype is not torch.int32 or t.dim() != 1 or t.device != self.device or \
                not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous int32 vector on {self.device}")
        if n is not None and t.shape[0] != n:
            raise ValueError(f"{name} must have {n} elements, not {t.shape[0]}")
        return t.data_ptr()

    def _refuse(self, name, t, heads, types):
        """Says what is wrong with a tensor that should be [tokens, heads, head_dim]."""
        if t.dim() != 3 or t.shape[2] != self.head_dim or (heads and t.shape[1] != heads):
            raise ValueError(f"{name} must be [tokens, {heads or 'heads'}, {self.head_dim}], "
                             f"not {list(t.shape)}")
        if t.device != self.device:
            raise ValueError(f"{name} must be on {self.device}")
        if t.dtype not in types:
            raise ValueError(f"{name} must be one of {', '.join(str(d) for d in types)}")
        if t.stride(2) != 1:
            raise ValueError(f"{name} must have contiguous channels")
        raise ValueError(f"{t.shape[1]} query heads over {self.kv_heads} key heads")

    def _entries(self, seqs, q_start, tokens):
        if q_start is not None:
            n = q_start.shape[0] - 1
            if n < 0:
                raise ValueError("q_start must have one element more than there are entries")
            return self._ints("seqs", seqs, n), self._ints("q_start", q_start), n
        if seqs is None:
            return None, None, tokens
        n = seqs.shape[0]
        if tokens > n:
            raise ValueError(f"{tokens} tokens for {n} entries: q_start is needed")
        return self._ints("seqs", seqs), None, n

    # ------------------------------------------------------------------ the calls ---

    def reserve(self, counts, seqs=None, ok=None, stream=None):
        """Room for counts[i] more tokens in slot seqs[i] (slot i without seqs).

        Returns ``ok`` int32 [n]: 0 where a request was refused (see include/wd_kv.h)."""
        n = counts.numel()
        if ok is None:
            ok = self._output(n, torch.int32, stream)
        _check("wd_kv_reserve", self._lib.wd_kv_reserve(
            self._ref, self._ints("seqs", seqs, n), self._ints("counts", counts), n,
            self._ints("ok", ok, n), self._stream(stream)))
        self._keep(stream, counts, seqs, ok)
        return ok

    def append(self, layer, k, v, seqs=None, q_start=None, return_values=False, stream=None):
        """Quantise the new tokens' keys and values and write them into one layer's pages.

        k, v: [tokens, kv_heads, head_dim] BF16, FP16 or FP32, any strides with contiguous channels.
        Entry b of the batch is slot seqs[b] (slot b without seqs) and owns tokens q_start[b] to
        q_start[b + 1] (token b without q_start), the last ones of its sequence.  With
        ``return_values`` returns what the cache now holds for them, (k, v) in their type; tokens
        of no entry are then undefined."""
        dtype, shape = k.dtype, k.shape
        code = _DTYPES.get(dtype)
        if code is None or len(shape) != 3 or shape[1] != self.kv_heads or \
                shape[2] != self.head_dim or k.device != self.device:
            self._refuse("k", k, self.kv_heads, _DTYPES)
        if v.dtype is not dtype or v.shape != shape or v.device != self.device:
            raise ValueError("v must have k's shape and type, on its device")
        k_token, k_head, k_channel = k.stride()
        v_token, v_head, v_channel = v.stride()
        if k_channel != 1 or v_channel != 1:
            raise ValueError("k and v must have contiguous channels")
        tokens = shape[0]
        s, qs, n = self._entries(seqs, q_start, tokens)
        if return_values:
            values = self._output((2, *shape), dtype, stream)
            k_to = values.data_ptr()
            v_to = k_to + values.nbytes // 2
        else:
            values = k_to = v_to = None
        st = self._lib.wd_kv_append(self._ref, layer, k.data_ptr(), v.data_ptr(), code, k_token,
                                    k_head, v_token, v_head, k_to, v_to, s, qs, n, tokens,
                                    self._stream(stream))
        if st:
            _check("wd_kv_append", st)
        self._keep(stream, k, v, seqs, q_start, values)
        return values.unbind(0) if return_values else None

    def append_rotated(self, layer, q, k, v, cos_sin, seqs=None, q_start=None, paired=False, return_values=False,
                       q_out=None, stream=None):
        """``append``, with queries and keys rotated by their positions on the way.

        q: [tokens, q_heads, head_dim] of k's type, any strides with contiguous channels (None: keys and values
        alone); k, v, seqs, q_start as in ``append``.  cos_sin FP32 [positions, rot], as ``rotation_table`` makes
        it: the cosines and then the sines of a position's rot / 2 angles.  The first ``rot`` channels of each
        head are turned, channels i and i + rot / 2 together, or with ``paired`` 2i and 2i + 1.  Returns the turned queries
        (in ``q_out`` if given, which may be q), and with ``return_values`` what the cache now holds, (q, k, v);
        tokens of no entry, and those at positions that cos_sin does not have, are undefined in them."""
        dtype, shape, device, dim = k.dtype, k.shape, self.device, self.head_dim
        code = _DTYPES.get(dtype)
        if code is None or len(shape) != 3 or shape[1] != self.kv_heads or shape[2] != dim or k.device != device:
            self._refuse("k", k, self.kv_heads, _DTYPES)
        if v.dtype is not dtype or v.shape != shape or v.device != device:
            raise ValueError("v must have k's shape and type, on its device")
        k_token, k_head, k_channel = k.stride()
        v_token, v_head, v_channel = v.stride()
        if k_channel != 1 or v_channel != 1:
            raise ValueError("k and v must have contiguous channels")
        tokens, turns = shape[0], cos_sin.shape
        if tokens > 2 ** 31 - 1:  # (ctypes would cut it to its low bits)
            raise ValueError(f"unsupported sizes: {tokens} tokens")
        if cos_sin.dtype is not torch.float32 or len(turns) != 2 or cos_sin.device != device or \
                not cos_sin.is_contiguous():
            raise ValueError(f"cos_sin must be contiguous FP32 [positions, rot] on {device}")
        heads = q_token = q_head = 0
        q_from = q_to = None
        if q is not None:
            q_shape = q.shape
            if q.dtype is not dtype or len(q_shape) != 3 or q_shape[0] != tokens or q_shape[2] != dim or \
                    q.device != device:
                raise ValueError(f"q must be [{tokens}, heads, {dim}] of k's type, on its device")
            q_token, q_head, q_channel = q.stride()
            if q_channel != 1:
                raise ValueError("q must have contiguous channels")
            heads, q_from = q_shape[1], q.data_ptr()
            if q_out is None:
                q_out = torch.empty(q_shape, dtype=dtype, device=device) if stream is None else \
                    self._output(q_shape, dtype, stream)
            elif q_out.shape != q_shape or q_out.dtype is not dtype or not q_out.is_contiguous() or \
                    q_out.device != device:
                raise ValueError("q_out must be contiguous, of q's shape and type")
            q_to = q_out.data_ptr()
        elif q_out is not None:
            raise ValueError("q_out without q")
        s, qs, n = self._entries(seqs, q_start, tokens)
        k_out = v_out = k_to = v_to = None
        if return_values:
            k_out, v_out = self._output(shape, dtype, stream), self._output(shape, dtype, stream)
            k_to, v_to = k_out.data_ptr(), v_out.data_ptr()
        st = self._lib.wd_kv_append_rotated(
            self._ref, layer, q_from, k.data_ptr(), v.data_ptr(), code, q_token, q_head, heads, k_token, k_head,
            v_token, v_head, q_to, k_to, v_to, cos_sin.data_ptr(), turns[0], turns[1], paired, s, qs, n, tokens,
            self._stream(stream))
        if st:
            _check("wd_kv_append_rotated", st)
        if stream is not None:
            self._keep(stream, q, k, v, cos_sin, seqs, q_start, q_out, k_out, v_out)
        return (q_out, k_out, v_out) if return_values else q_out

    def attention(self, layer, q, seqs=None, q_start=None, max_q=0, scale=None, window=0, out=None,
                  return_lse=False, stream=None):
        """Attention of the new tokens' queries over one layer of the cache.

        q: [tokens, q_heads, head_dim] BF16 or FP16; the batch as in ``append``.  A query at
        position p sees keys max(0, p - window + 1) .. p (window 0: all before it).  ``scale``
        defaults to 1 / sqrt(head_dim); ``max_q`` is the most tokens an entry has, if known.
        Returns ``out`` [tokens, q_heads, head_dim], and lse FP32 [tokens, q_heads] with
        ``return_lse``; zeros and -inf where nothing is seen."""
        dtype, shape = q.dtype, q.shape
        code = _Q_DTYPES.get(dtype)
        if code is None or len(shape) != 3 or shape[2] != self.head_dim or \
                q.device != self.device or shape[1] % self.kv_heads or not shape[1]:
            self._refuse("q", q, None, _Q_DTYPES)
        q_token, q_head, q_channel = q.stride()
        if q_channel != 1:
            self._refuse("q", q, None, _Q_DTYPES)
        tokens, heads = shape[0], shape[1]
        if out is None:
            out = self._output(shape, dtype, stream)
        elif out.shape != shape or out.dtype is not dtype or not out.is_contiguous() or \
                out.device != self.device:
            raise ValueError("out must be contiguous, of q's shape and type")
        if return_lse:
            lse = self._output((tokens, heads), torch.float32, stream)
            lse_to = lse.data_ptr()
        else:
            lse = lse_to = None
        s, qs, n = self._entries(seqs, q_start, tokens)
        st = self._lib.wd_kv_attention(self._ref, layer, q.data_ptr(), code, q_token, q_head, heads,
                                       out.data_ptr(), lse_to, s, qs, n, tokens, max_q,
                                       self._scale if scale is None else scale, window,
                                       self._stream(stream))
        if st:
            _check("wd_kv_attention", st)
        self._keep(stream, q, seqs, q_start, out, lse)
        return (out, lse) if return_lse else out

    def fork(self, src, dst, ok=None, stream=None):
        """Slot dst[i] becomes a fork of what slot src[i] held before the call, for all i at once;
        src[i] = -1 frees it.  Returns ``ok`` int32 [n]: 0 where a request was refused."""
        n = dst.numel()
        if ok is None:
            ok = self._output(n, torch.int32, stream)
        _check("wd_kv_fork", self._lib.wd_kv_fork(
            self._ref, self._ints("src", src, n), self._ints("dst", dst), n,
            self._ints("ok", ok, n), self._stream(stream)))
        self._keep(stream, src, dst, ok)
        return ok

    def free(self, seqs, stream=None):
        """Release the sequences in these slots."""
        _check("wd_kv_free", self._lib.wd_kv_free(self._ref, self._ints("seqs", seqs),
                                                  seqs.numel(), self._stream(stream)))
        self._keep(stream, seqs)

    def compact(self, table_out=None, refs_out=None, stream=None):
        """Move the live pages to the front of the pool.  The bookkeeping is rewritten in place, or
        into table_out and refs_out.  Returns int32 [num_pages]: where each page went, -1 if free."""
        page_map = self._output(self.num_pages, torch.int32, stream)
        for name, t, like in (("table_out", table_out, self.table),
                              ("refs_out", refs_out, self.refs)):
            if t is not None and (t.shape != like.shape or t.dtype != torch.int32 or
                                  not t.is_contiguous() or t.device != self.device):
                raise ValueError(f"{name} must be contiguous int32 of shape {list(like.shape)}")
        _check("wd_kv_compact", self._lib.wd_kv_compact(
            self._ref, None if table_out is None else table_out.data_ptr(),
            None if refs_out is None else refs_out.data_ptr(), page_map.data_ptr(),
            self._stream(stream)))
        self._keep(stream, table_out, refs_out, page_map)
        return page_map

    def read_error_flag(self, stream=None):
        """The error flag's bits (KV_FLAG_*) since the last read, then cleared (synchronises)."""
        flag = ctypes.c_int(0)
        st = self._lib.wd_kv_read_error_flag(self._ref, self._stream(stream), ctypes.byref(flag))
        if st not in (0, 6, 7, 8):
            _check("wd_kv_read_error_flag", st)
        return flag.value
