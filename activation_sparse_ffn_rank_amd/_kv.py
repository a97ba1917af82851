"""ctypes binding of the C ABI in include/pi_paged_kv.h: the paged key/value cache, its block tables and
the attention that reads it (argument marshalling only, as in ``_abi``).

What only a tensor knows -- element type, shape, strides -- is checked here and refused with the same
codes that the library uses (``PiError``), and so are numbers that do not fit its 32-bit arguments, which
ctypes would take modulo 2^32; the library checks the rest.  A tensor that is not on the
pages' device has no address there (``PI_ERR_NULL``).  The descriptors keep the tensors that they name
alive.
"""
from __future__ import annotations

import ctypes

import torch

from ._abi import PI_ERR_DTYPE, PI_ERR_NULL, PI_ERR_SHAPE, PI_ERR_WORKSPACE, PI_OK, PiError, _check, lib

_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda device: torch.cuda.current_stream(device).cuda_stream)

PI_KV_F16, PI_KV_BF16 = 1, 2
PI_KV_MAX_REQ, PI_KV_MAX_TABLE, PI_KV_MAX_TOKENS = 4096, 1 << 17, 1 << 19
KV_DTYPES = {torch.float16: PI_KV_F16, torch.bfloat16: PI_KV_BF16}

# Every function the header declares; the CPU tests check that libpi.so exports them all.
KV_EXPORTS = ("pi_kv_step", "pi_kv_append", "pi_kv_attn_workspace_bytes", "pi_kv_attn")

_i32, _i64, _vp, _sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t


class pi_kv_cache(ctypes.Structure):
    _fields_ = [("n_pages", _i32), ("n_kv", _i32), ("page", _i32), ("head_dim", _i32), ("dtype", _i32), ("k_pages", _vp),
                ("v_pages", _vp)]


class pi_kv_batch(ctypes.Structure):
    _fields_ = [("n_req", _i32), ("max_pages", _i32), ("max_q", _i32), ("max_kv", _i32), ("table_stride", _i64),
                ("block_table", _vp), ("q_start", _vp), ("kv_len", _vp)]


class pi_kv_tables(ctypes.Structure):
    _fields_ = [("n_req", _i32), ("page", _i32), ("n_pages", _i32), ("max_pages", _i32), ("max_tokens", _i32),
                ("table_stride", _i64), ("cached", _vp), ("fresh", _vp), ("free_ring", _vp), ("pool", _vp),
                ("block_table", _vp), ("q_start", _vp), ("kv_len", _vp), ("cached_next", _vp), ("slots", _vp),
                ("pool_next", _vp), ("counts", _vp)]


_kv_lib = None


def kv_lib() -> ctypes.CDLL:
    global _kv_lib
    if _kv_lib is None:
        L, P = lib(), ctypes.POINTER
        L.pi_kv_step.restype = ctypes.c_int
        L.pi_kv_step.argtypes = [P(pi_kv_tables), _vp]
        L.pi_kv_append.restype = ctypes.c_int
        L.pi_kv_append.argtypes = [P(pi_kv_cache), _vp, _i64, _i64, _vp, _i64, _i64, _vp, _i32, _vp]
        L.pi_kv_attn_workspace_bytes.restype = _sz
        L.pi_kv_attn_workspace_bytes.argtypes = [P(pi_kv_cache), P(pi_kv_batch), _i32, _i32]
        L.pi_kv_attn.restype = ctypes.c_int
        L.pi_kv_attn.argtypes = [P(pi_kv_cache), P(pi_kv_batch), _vp, _i64, _i64, _vp, _i64, _i64, _i32, _i32,
                                 ctypes.c_float, _i32, _vp, _sz, _vp]
        _kv_lib = L
    return _kv_lib


def _fits(*numbers: int) -> bool:
    """Whether all of them are int32."""
    return all(-2 ** 31 <= x < 2 ** 31 for x in numbers)


def _int32(fn: str, *numbers: int) -> None:
    if not _fits(*numbers):
        raise PiError(fn, PI_ERR_SHAPE)


def _ints(fn: str, t, n: int) -> int:
    """Address of a contiguous int32 tensor [n] (-1: any size)."""
    if t is None:
        raise PiError(fn, PI_ERR_NULL)
    if t.dtype != torch.int32:
        raise PiError(fn, PI_ERR_DTYPE)
    if t.dim() != 1 or (n >= 0 and t.shape[0] != n) or not t.is_contiguous():
        raise PiError(fn, PI_ERR_SHAPE)
    if n < 0:
        _int32(fn, t.shape[0])
    return t.data_ptr()


def _table(fn: str, t, n_req: int) -> tuple[int, int, int]:
    """(address, columns, row stride) of a block table [n_req][columns], rows possibly a slice of wider ones."""
    if t is None:
        raise PiError(fn, PI_ERR_NULL)
    if t.dtype != torch.int32:
        raise PiError(fn, PI_ERR_DTYPE)
    if t.dim() != 2 or t.shape[0] != n_req or t.shape[1] < 1 or t.stride(1) != 1:
        raise PiError(fn, PI_ERR_SHAPE)
    _int32(fn, t.shape[1])
    return t.data_ptr(), t.shape[1], t.stride(0) if n_req > 1 else t.shape[1]


def _rows(fn: str, t, cache: pi_kv_cache) -> tuple[int, int, int, int, int]:
    """(address, token stride, head stride, tokens, heads) of a [tokens][heads][head_dim] tensor."""
    if t is None:
        raise PiError(fn, PI_ERR_NULL)
    if KV_DTYPES.get(t.dtype) != cache.dtype:
        raise PiError(fn, PI_ERR_DTYPE)
    if t.dim() != 3:
        raise PiError(fn, PI_ERR_SHAPE)
    n, heads, hd = t.shape
    ts, hs, one = t.stride()
    if hd != cache.head_dim or one != 1:
        raise PiError(fn, PI_ERR_SHAPE)
    # the stride along an axis of one element is never used
    return t.data_ptr(), ts if n > 1 else heads * hd, hs if heads > 1 else hd, n, heads


def _device(fn: str, *tensors) -> int:
    """Index of the one device that holds all of them (-1: host memory)."""
    d = tensors[0].get_device()
    for t in tensors:
        if t.get_device() != d:
            raise PiError(fn, PI_ERR_NULL)
    return d


def _raw_stream(fn: str, stream, device: int) -> int:
    """As ``_abi._stream``, but the current stream of the device that holds the tensors.  The calls are made with that
    device current: the default stream (address 0) is the current device's."""
    if device < 0:
        raise PiError(fn, PI_ERR_NULL)
    if stream is None:
        return _current_stream(device)
    return stream if isinstance(stream, int) else stream.cuda_stream


def make_kv_cache(k_pages: torch.Tensor, v_pages: torch.Tensor) -> pi_kv_cache:
    """Descriptor of a page pool: k_pages [n_pages][n_kv][page][head_dim], v_pages
    [n_pages][n_kv][head_dim][page], both fp16 or both bf16."""
    if k_pages is None or v_pages is None:
        raise PiError("make_kv_cache", PI_ERR_NULL)
    if k_pages.dtype not in KV_DTYPES or v_pages.dtype != k_pages.dtype:
        raise PiError("make_kv_cache", PI_ERR_DTYPE)
    if k_pages.dim() != 4 or not k_pages.is_contiguous() or not v_pages.is_contiguous():
        raise PiError("make_kv_cache", PI_ERR_SHAPE)
    n_pages, n_kv, page, hd = k_pages.shape
    if tuple(v_pages.shape) != (n_pages, n_kv, hd, page):
        raise PiError("make_kv_cache", PI_ERR_SHAPE)
    _int32("make_kv_cache", n_pages, n_kv, page, hd)
    c = pi_kv_cache(n_pages, n_kv, page, hd, KV_DTYPES[k_pages.dtype], k_pages.data_ptr(), v_pages.data_ptr())
    c._device = _device("make_kv_cache", k_pages, v_pages)
    c._keep = (k_pages, v_pages)
    return c


def make_kv_batch(block_table: torch.Tensor, q_start: torch.Tensor, kv_len: torch.Tensor, *, max_q: int,
                  max_kv: int) -> pi_kv_batch:
    """Descriptor of a step's requests: block_table [n_req][max_pages], q_start [n_req + 1], kv_len [n_req]
    (int32); max_q and max_kv bound the new tokens and the keys of a request."""
    fn = "make_kv_batch"
    length = _ints(fn, kv_len, -1)
    n = kv_len.shape[0]
    table, cols, stride = _table(fn, block_table, n)
    _int32(fn, max_q, max_kv)
    b = pi_kv_batch(n, cols, max_q, max_kv, stride, table, _ints(fn, q_start, n + 1), length)
    b._device = _device(fn, block_table, q_start, kv_len)
    b._keep = (block_table, q_start, kv_len)
    return b


def make_kv_tables(cached: torch.Tensor, fresh: torch.Tensor, free_ring: torch.Tensor, pool: torch.Tensor,
                   block_table: torch.Tensor, page: int, q_start: torch.Tensor, kv_len: torch.Tensor,
                   cached_next: torch.Tensor, slots: torch.Tensor, pool_next: torch.Tensor,
                   counts: torch.Tensor) -> pi_kv_tables:
    """Descriptor of a step of the block tables (int32 tensors, see the header); cached_next may be
    cached and pool_next may be pool, so that the step advances its own state."""
    fn = "make_kv_tables"
    at = _ints(fn, cached, -1)
    n = cached.shape[0]
    table, cols, stride = _table(fn, block_table, n)
    _int32(fn, page)
    ring, rows = _ints(fn, free_ring, -1), _ints(fn, slots, -1)
    t = pi_kv_tables(n, page, free_ring.shape[0], cols, slots.shape[0], stride, at, _ints(fn, fresh, n), ring,
                     _ints(fn, pool, 2), table, _ints(fn, q_start, n + 1), _ints(fn, kv_len, n), _ints(fn, cached_next, n),
                     rows, _ints(fn, pool_next, 2), _ints(fn, counts, 4))
    t._keep = (cached, fresh, free_ring, pool, block_table, q_start, kv_len, cached_next, slots, pool_next, counts)
    t._device = _device(fn, *t._keep)
    return t


def pi_kv_step(tables: pi_kv_tables, stream=None) -> None:
    """One step of the block tables: pages for the new tokens, pages of ended requests back, slot map."""
    stream = _raw_stream("pi_kv_step", stream, tables._device)
    if _current_device() != tables._device:
        with torch.cuda.device(tables._device):
            return pi_kv_step(tables, stream)
    _check("pi_kv_step", kv_lib().pi_kv_step(tables, stream))


def pi_kv_append(cache: pi_kv_cache, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, stream=None) -> None:
    """New keys and values k, v [tokens][n_kv][head_dim] (slices of wider rows are fine) into slots [tokens]."""
    fn = "pi_kv_append"
    kp, kt, kh, n, heads = _rows(fn, k, cache)
    vp, vt, vh, n_v, heads_v = _rows(fn, v, cache)
    if heads != cache.n_kv or heads_v != heads or n_v != n or n >= 2 ** 31:
        raise PiError(fn, PI_ERR_SHAPE)
    at, device = _ints(fn, slots, n), cache._device
    if k.get_device() != device or v.get_device() != device or slots.get_device() != device:
        raise PiError(fn, PI_ERR_NULL)
    stream = _current_stream(device) if stream is None and device >= 0 else _raw_stream(fn, stream, device)
    if _current_device() != device:
        with torch.cuda.device(device):
            return pi_kv_append(cache, k, v, slots, stream)
    rc = (_kv_lib or kv_lib()).pi_kv_append(cache, kp, kt, kh, vp, vt, vh, at, n, stream)
    if rc != PI_OK:
        raise PiError(fn, rc)


def pi_kv_attn_workspace_bytes(cache: pi_kv_cache, batch: pi_kv_batch, total_q: int, n_q: int) -> int:
    """Bytes of workspace pi_kv_attn needs for this batch, packed rows and query heads (0: invalid)."""
    return int(kv_lib().pi_kv_attn_workspace_bytes(cache, batch, total_q, n_q)) if _fits(total_q, n_q) else 0


def pi_kv_attn(cache: pi_kv_cache, batch: pi_kv_batch, q: torch.Tensor, out: torch.Tensor, ws: torch.Tensor, *, scale: float,
               window: int = 0, stream=None) -> None:
    """out [total_q][n_q][head_dim] = attention of the packed new tokens q over their requests' pages."""
    fn = "pi_kv_attn"
    qp, qt, qh, n, heads = _rows(fn, q, cache)
    op, ot, oh, n_o, heads_o = _rows(fn, out, cache)
    if n_o != n or heads_o != heads or n >= 2 ** 31 or heads >= 2 ** 31 or not -2 ** 31 <= window < 2 ** 31:
        raise PiError(fn, PI_ERR_SHAPE)
    device, wp, wn = cache._device, None, 0                  # (the library refuses a missing workspace if it needs one)
    if ws is not None:
        if not ws.is_contiguous():
            raise PiError(fn, PI_ERR_WORKSPACE)
        if ws.get_device() != device:
            raise PiError(fn, PI_ERR_NULL)
        wp, wn = ws.data_ptr(), ws.nbytes
    if q.get_device() != device or out.get_device() != device or batch._device != device:
        raise PiError(fn, PI_ERR_NULL)
    stream = _current_stream(device) if stream is None and device >= 0 else _raw_stream(fn, stream, device)
    if _current_device() != device:
        with torch.cuda.device(device):
            return pi_kv_attn(cache, batch, q, out, ws, scale=scale, window=window, stream=stream)
    rc = (_kv_lib or kv_lib()).pi_kv_attn(cache, batch, qp, qt, qh, op, ot, oh, n, heads, scale, window, wp, wn, stream)
    if rc != PI_OK:
        raise PiError(fn, rc)
