"""ctypes binding of the C ABI in include/pi_paged_kv.h: the paged key/value cache, its block tables, the append with
rotary positions or without, the attention that reads it, drafted tokens, and pages given back, shared and copied
(argument marshalling only, as in ``_abi``).

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
PI_KV_MAX_VOCAB = 1 << 22
PI_ROPE_HALF, PI_ROPE_PAIRS = 0, 1
KV_DTYPES = {torch.float16: PI_KV_F16, torch.bfloat16: PI_KV_BF16}

# Every function the header declares; the CPU tests check that libpi.so exports them all.
KV_EXPORTS = ("pi_kv_step", "pi_kv_append", "pi_kv_attn_workspace_bytes", "pi_kv_attn", "pi_rope_frequencies",
              "pi_kv_rope_append", "pi_kv_attn_sinks_workspace_bytes", "pi_kv_attn_sinks", "pi_kv_verify_workspace_bytes",
              "pi_kv_verify", "pi_kv_pages_workspace_bytes", "pi_kv_release", "pi_kv_fork", "pi_kv_copy")

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


class pi_kv_rope(ctypes.Structure):
    _fields_ = [("rot_dim", _i32), ("layout", _i32), ("norm", _i32), ("scale", ctypes.c_float), ("eps", ctypes.c_float),
                ("freq", _vp), ("q_weight", _vp), ("k_weight", _vp)]


class pi_kv_drafts(ctypes.Structure):
    _fields_ = [("n_req", _i32), ("rows", _i32), ("vocab", _i32), ("q_start", _vp), ("tokens", _vp), ("target", _vp),
                ("target_stride", _i64), ("draft", _vp), ("draft_stride", _i64), ("u_accept", _vp), ("u_next", _vp)]


class pi_kv_pages(ctypes.Structure):
    _fields_ = [("n_req", _i32), ("page", _i32), ("n_pages", _i32), ("max_pages", _i32), ("table_stride", _i64),
                ("cached", _vp), ("free_ring", _vp), ("pool", _vp), ("block_table", _vp), ("shares", _vp), ("cached_next", _vp),
                ("pool_next", _vp), ("counts", _vp), ("ws", _vp), ("ws_bytes", _sz)]


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
        f64 = ctypes.c_double
        L.pi_rope_frequencies.restype = ctypes.c_int
        L.pi_rope_frequencies.argtypes = [_i32, f64, f64, f64, f64, f64, _vp]
        L.pi_kv_rope_append.restype = ctypes.c_int
        L.pi_kv_rope_append.argtypes = [P(pi_kv_cache), P(pi_kv_batch), P(pi_kv_rope), _vp, _i64, _i64, _vp, _i64, _i64, _vp, _i64,
                                        _i64, _vp, _vp, _i64, _i64, _i32, _i32, _vp]
        L.pi_kv_attn_sinks_workspace_bytes.restype = _sz
        L.pi_kv_attn_sinks_workspace_bytes.argtypes = [P(pi_kv_cache), P(pi_kv_batch), _i32, _i32, _i32, _i32]
        L.pi_kv_attn_sinks.restype = ctypes.c_int
        L.pi_kv_attn_sinks.argtypes = [P(pi_kv_cache), P(pi_kv_batch), _vp, _i64, _i64, _vp, _i64, _i64, _i32, _i32,
                                       ctypes.c_float, _i32, _i32, _vp, _sz, _vp]
        L.pi_kv_verify_workspace_bytes.restype = _sz
        L.pi_kv_verify_workspace_bytes.argtypes = [P(pi_kv_drafts)]
        L.pi_kv_verify.restype = ctypes.c_int
        L.pi_kv_verify.argtypes = [P(pi_kv_drafts), _vp, _vp, _vp, _vp, _vp, _sz, _vp]
        L.pi_kv_pages_workspace_bytes.restype = _sz
        L.pi_kv_pages_workspace_bytes.argtypes = [P(pi_kv_pages)]
        L.pi_kv_release.restype = ctypes.c_int
        L.pi_kv_release.argtypes = [P(pi_kv_pages), _vp, _vp, _vp, _vp]
        L.pi_kv_fork.restype = ctypes.c_int
        L.pi_kv_fork.argtypes = [P(pi_kv_pages), _vp, _vp, _i32, _vp, _vp]
        L.pi_kv_copy.restype = ctypes.c_int
        L.pi_kv_copy.argtypes = [P(pi_kv_cache), _vp, _i32, _vp]
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
    shape = t.shape
    if len(shape) != 3:
        raise PiError(fn, PI_ERR_SHAPE)
    n, heads, hd = shape
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


# ------------------------------------------------------------------------------ rotary positions with the append

def pi_rope_frequencies(rot_dim: int, *, base: float = 10000.0, factor: float = 1.0, trained: float = 4096.0, low: float = 0.0,
                        high: float = 0.0) -> torch.Tensor:
    """Radians per position of the rot_dim / 2 pairs (float64, host memory): base^(-2i/rot_dim); with low = high = 0 all
    divided by factor, else those of fewer than `low` turns over `trained` positions divided, those of more than
    `high` kept, a ramp between."""
    fn = "pi_rope_frequencies"
    _int32(fn, rot_dim)
    freq = torch.empty(max(rot_dim // 2, 1), dtype=torch.float64)
    _check(fn, kv_lib().pi_rope_frequencies(rot_dim, base, factor, trained, low, high, freq.data_ptr()))
    return freq


def make_kv_rope(freq: torch.Tensor | None, *, layout: int = PI_ROPE_HALF, scale: float = 1.0, norm: bool | None = None,
                 eps: float = 1e-6, q_weight: torch.Tensor | None = None, k_weight: torch.Tensor | None = None) -> pi_kv_rope:
    """Descriptor of what is done to heads of q and k: RMS norm (norm; by itself where a weight [head_dim] is given), then
    rotation of the first 2 * len(freq) elements (freq: float64 radians per position on the pages' device; None: no
    rotation) in pairs by layout, with cosines and sines times scale."""
    fn = "make_kv_rope"
    kept = [t for t in (freq, q_weight, k_weight) if t is not None]
    if freq is not None and freq.dtype != torch.float64:
        raise PiError(fn, PI_ERR_DTYPE)
    weights = kept if freq is None else kept[1:]
    if any(t.dtype not in KV_DTYPES or t.dtype != weights[0].dtype for t in weights) or (weights and norm is False):
        raise PiError(fn, PI_ERR_DTYPE)
    if any(t.dim() != 1 or not t.is_contiguous() for t in kept) or any(t.shape != weights[0].shape for t in weights):
        raise PiError(fn, PI_ERR_SHAPE)
    rot = 0 if freq is None else 2 * freq.shape[0]
    _int32(fn, rot, layout)
    at = lambda t: None if t is None else t.data_ptr()
    r = pi_kv_rope(rot, layout, int(bool(weights) if norm is None else norm), scale, eps, at(freq), at(q_weight), at(k_weight))
    r._device = _device(fn, *kept) if kept else None
    r._weights = (weights[0].dtype, weights[0].shape[0]) if weights else None
    r._keep = tuple(kept)
    return r


def pi_kv_rope_append(cache: pi_kv_cache, batch: pi_kv_batch, rope: pi_kv_rope, q: torch.Tensor, k: torch.Tensor,
                      v: torch.Tensor, slots: torch.Tensor, q_out: torch.Tensor, stream=None) -> None:
    """k (normed, rotated) and v [total_q][n_kv][head_dim] into slots [total_q], and q [total_q][n_q][head_dim] (normed,
    rotated) to q_out, which may be q.  Positions follow from the batch."""
    fn = "pi_kv_rope_append"
    if q is None or k is None or v is None or q_out is None:
        raise PiError(fn, PI_ERR_NULL)
    dt = q.dtype
    if KV_DTYPES.get(dt) != cache.dtype or k.dtype != dt or v.dtype != dt or q_out.dtype != dt:
        raise PiError(fn, PI_ERR_DTYPE)
    shape, shape_k, width = q.shape, k.shape, cache.head_dim
    if len(shape) != 3 or len(shape_k) != 3 or v.shape != shape_k or q_out.shape != shape:
        raise PiError(fn, PI_ERR_SHAPE)
    n, heads, hd = shape
    if shape_k != (n, cache.n_kv, hd) or hd != width or n >= 2 ** 31 or heads >= 2 ** 31:
        raise PiError(fn, PI_ERR_SHAPE)
    (qt, qh, q1), (kt, kh, k1), (vt, vh, v1), (ot, oh, o1) = q.stride(), k.stride(), v.stride(), q_out.stride()
    if not q1 == k1 == v1 == o1 == 1:
        raise PiError(fn, PI_ERR_SHAPE)
    if n <= 1 or heads <= 1 or shape_k[1] <= 1:              # the stride along an axis of one element is never used
        (_, qt, qh, _, _), (_, kt, kh, _, _), (_, vt, vh, _, _), (_, ot, oh, _, _) = (_rows(fn, t, cache) for t in (q, k, v, q_out))
    weights = rope._weights
    if weights is not None and weights != (dt, width):
        raise PiError(fn, PI_ERR_DTYPE if weights[0] != dt else PI_ERR_SHAPE)
    at, device, on = _ints(fn, slots, n), cache._device, rope._device
    if not (q.get_device() == k.get_device() == v.get_device() == q_out.get_device() == slots.get_device() == batch._device == device
            and (on is None or on == device)):
        raise PiError(fn, PI_ERR_NULL)
    stream = _current_stream(device) if stream is None and device >= 0 else _raw_stream(fn, stream, device)
    if _current_device() != device:
        with torch.cuda.device(device):
            return pi_kv_rope_append(cache, batch, rope, q, k, v, slots, q_out, stream)
    rc = (_kv_lib or kv_lib()).pi_kv_rope_append(cache, batch, rope, q.data_ptr(), qt, qh, k.data_ptr(), kt, kh, v.data_ptr(), vt, vh,
                                                 at, q_out.data_ptr(), ot, oh, n, heads, stream)
    if rc != PI_OK:
        raise PiError(fn, rc)


# ------------------------------------------------------------------------------ a window and the first tokens

def pi_kv_attn_sinks_workspace_bytes(cache: pi_kv_cache, batch: pi_kv_batch, total_q: int, n_q: int, window: int, sinks: int) -> int:
    """Bytes of workspace pi_kv_attn_sinks needs (0: invalid)."""
    if not _fits(total_q, n_q, window, sinks):
        return 0
    return int(kv_lib().pi_kv_attn_sinks_workspace_bytes(cache, batch, total_q, n_q, window, sinks))


def pi_kv_attn_sinks(cache: pi_kv_cache, batch: pi_kv_batch, q: torch.Tensor, out: torch.Tensor, ws: torch.Tensor, *,
                     scale: float, window: int, sinks: int, stream=None) -> None:
    """pi_kv_attn with a window, in which a request's first `sinks` keys stay visible."""
    fn = "pi_kv_attn_sinks"
    qp, qt, qh, n, heads = _rows(fn, q, cache)
    op, ot, oh, n_o, heads_o = _rows(fn, out, cache)
    if n_o != n or heads_o != heads or n >= 2 ** 31 or heads >= 2 ** 31 or not _fits(window, sinks):
        raise PiError(fn, PI_ERR_SHAPE)
    device, wp, wn = cache._device, None, 0
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
            return pi_kv_attn_sinks(cache, batch, q, out, ws, scale=scale, window=window, sinks=sinks, stream=stream)
    rc = (_kv_lib or kv_lib()).pi_kv_attn_sinks(cache, batch, qp, qt, qh, op, ot, oh, n, heads, scale, window, sinks, wp, wn, stream)
    if rc != PI_OK:
        raise PiError(fn, rc)


# ------------------------------------------------------------------------------ drafted tokens

def _floats(fn: str, t, n: int) -> int:
    """Address of a contiguous float32 tensor [n]."""
    if t is None:
        raise PiError(fn, PI_ERR_NULL)
    if t.dtype != torch.float32:
        raise PiError(fn, PI_ERR_DTYPE)
    if t.dim() != 1 or t.shape[0] != n or not t.is_contiguous():
        raise PiError(fn, PI_ERR_SHAPE)
    return t.data_ptr()


def _probs(fn: str, t, rows: int, vocab: int) -> tuple[int, int]:
    """(address, row stride) of float32 rows [rows][vocab], possibly slices of wider ones."""
    if t.dtype != torch.float32:
        raise PiError(fn, PI_ERR_DTYPE)
    if t.dim() != 2 or tuple(t.shape) != (rows, vocab) or (t.stride(1) != 1 and vocab > 1):
        raise PiError(fn, PI_ERR_SHAPE)
    return t.data_ptr(), t.stride(0) if rows > 1 else vocab


def make_kv_drafts(q_start: torch.Tensor, tokens: torch.Tensor, target: torch.Tensor, draft: torch.Tensor | None,
                   u_accept: torch.Tensor, u_next: torch.Tensor) -> pi_kv_drafts:
    """Descriptor of a step's drafted tokens: packed rows by q_start [n_req + 1], tokens [rows] (a request's last one, then its
    drafts), probabilities target and draft [rows][vocab] (draft None: each draft had all of it), random
    numbers u_accept [rows] and u_next [n_req] in [0, 1)."""
    fn = "make_kv_drafts"
    start, toks = _ints(fn, q_start, -1), _ints(fn, tokens, -1)
    n, rows = q_start.shape[0] - 1, tokens.shape[0]
    if target is None:
        raise PiError(fn, PI_ERR_NULL)
    if target.dim() != 2:
        raise PiError(fn, PI_ERR_SHAPE)
    vocab = target.shape[1]
    _int32(fn, vocab)
    p, p_stride = _probs(fn, target, rows, vocab)
    q, q_stride = (None, 0) if draft is None else _probs(fn, draft, rows, vocab)
    d = pi_kv_drafts(n, rows, vocab, start, toks, p, p_stride, q, q_stride, _floats(fn, u_accept, rows), _floats(fn, u_next, n))
    d._keep = tuple(t for t in (q_start, tokens, target, draft, u_accept, u_next) if t is not None)
    d._device = _device(fn, *d._keep)
    return d


def pi_kv_verify_workspace_bytes(drafts: pi_kv_drafts) -> int:
    """Bytes of workspace pi_kv_verify needs (0: invalid)."""
    return int(kv_lib().pi_kv_verify_workspace_bytes(drafts))


def pi_kv_verify(drafts: pi_kv_drafts, accepted: torch.Tensor, next: torch.Tensor, ws: torch.Tensor, *,
                 kv_len: torch.Tensor | None = None, keep: torch.Tensor | None = None, stream=None) -> None:
    """accepted [n_req] drafts of each request, the next token [n_req] behind them, and with kv_len the positions that
    stay, keep [n_req] (int32; of a request that the step refused INT32_MAX, and its last token is the next one again)."""
    fn = "pi_kv_verify"
    n, device = drafts.n_req, drafts._device
    ap, np_ = _ints(fn, accepted, n), _ints(fn, next, n)
    lp, kp = None if kv_len is None else _ints(fn, kv_len, n), None if keep is None else _ints(fn, keep, n)
    wp, wn = None, 0
    if ws is not None:
        if not ws.is_contiguous():
            raise PiError(fn, PI_ERR_WORKSPACE)
        wp, wn = ws.data_ptr(), ws.nbytes
    for t in (accepted, next, ws, kv_len, keep):
        if t is not None and t.get_device() != device:
            raise PiError(fn, PI_ERR_NULL)
    stream = _raw_stream(fn, stream, device)
    if _current_device() != device:
        with torch.cuda.device(device):
            return pi_kv_verify(drafts, accepted, next, ws, kv_len=kv_len, keep=keep, stream=stream)
    rc = (_kv_lib or kv_lib()).pi_kv_verify(drafts, lp, ap, np_, kp, wp, wn, stream)
    if rc != PI_OK:
        raise PiError(fn, rc)


# ------------------------------------------------------------------------------ pages given back, shared and copied

def make_kv_pages(cached: torch.Tensor, free_ring: torch.Tensor, pool: torch.Tensor, block_table: torch.Tensor, page: int,
                  shares: torch.Tensor, cached_next: torch.Tensor, pool_next: torch.Tensor, counts: torch.Tensor,
                  ws: torch.Tensor | None = None) -> pi_kv_pages:
    """Descriptor of the block tables' state for pi_kv_release and pi_kv_fork (int32 tensors, as of make_kv_tables, and shares
    [n_pages], the owners of each page beyond the first); cached_next may be cached and pool_next may be pool.  Without ws
    (at least pi_kv_pages_workspace_bytes of any type) the descriptor has a workspace of its own."""
    fn = "make_kv_pages"
    at = _ints(fn, cached, -1)
    n = cached.shape[0]
    table, cols, stride = _table(fn, block_table, n)
    _int32(fn, page)
    ring = _ints(fn, free_ring, -1)
    n_pages = free_ring.shape[0]
    p = pi_kv_pages(n, page, n_pages, cols, stride, at, ring, _ints(fn, pool, 2), table, _ints(fn, shares, n_pages),
                    _ints(fn, cached_next, n), _ints(fn, pool_next, 2), _ints(fn, counts, 4))
    if ws is None:
        ws = torch.empty(max(16, pi_kv_pages_workspace_bytes(p)), dtype=torch.uint8, device=cached.device)
    if not ws.is_contiguous():
        raise PiError(fn, PI_ERR_WORKSPACE)
    p.ws, p.ws_bytes = ws.data_ptr(), ws.nbytes
    p._keep = (cached, free_ring, pool, block_table, shares, cached_next, pool_next, counts, ws)
    p._device = _device(fn, *p._keep)
    return p


def pi_kv_pages_workspace_bytes(pages: pi_kv_pages) -> int:
    """Bytes of workspace the state's calls need (0: invalid)."""
    return int(kv_lib().pi_kv_pages_workspace_bytes(pages))


def _copies(fn: str, t, n: int) -> int:
    """Address of contiguous int32 pairs [n][2] (n -1: any number)."""
    if t is None:
        raise PiError(fn, PI_ERR_NULL)
    if t.dtype != torch.int32:
        raise PiError(fn, PI_ERR_DTYPE)
    if t.dim() != 2 or t.shape[1] != 2 or (n >= 0 and t.shape[0] != n) or not t.is_contiguous():
        raise PiError(fn, PI_ERR_SHAPE)
    return t.data_ptr()


def _on(fn: str, device: int, *tensors) -> None:
    for t in tensors:
        if t is not None and t.get_device() != device:
            raise PiError(fn, PI_ERR_NULL)


def pi_kv_release(pages: pi_kv_pages, drop_from: torch.Tensor, drop_to: torch.Tensor | None, copies: torch.Tensor, stream=None) -> None:
    """Gives up positions drop_from .. drop_to - 1 [n_req] of every request (drop_to None: to the end); copies [n_req][2]
    receives the page copies that are due (pi_kv_copy)."""
    fn = "pi_kv_release"
    n, device = pages.n_req, pages._device
    fp, tp, cp = _ints(fn, drop_from, n), None if drop_to is None else _ints(fn, drop_to, n), _copies(fn, copies, n)
    _on(fn, device, drop_from, drop_to, copies)
    stream = _raw_stream(fn, stream, device)
    if _current_device() != device:
        with torch.cuda.device(device):
            return pi_kv_release(pages, drop_from, drop_to, copies, stream)
    _check(fn, kv_lib().pi_kv_release(pages, fp, tp, cp, stream))


def pi_kv_fork(pages: pi_kv_pages, src: torch.Tensor, dst: torch.Tensor, copies: torch.Tensor, stream=None) -> None:
    """Makes the empty requests dst [n] copies of the requests src [n], sharing their full pages; copies [n][2] receives the
    page copies that are due (pi_kv_copy)."""
    fn = "pi_kv_fork"
    sp, device = _ints(fn, src, -1), pages._device
    n = src.shape[0]
    dp, cp = _ints(fn, dst, n), _copies(fn, copies, n)
    _on(fn, device, src, dst, copies)
    stream = _raw_stream(fn, stream, device)
    if _current_device() != device:
        with torch.cuda.device(device):
            return pi_kv_fork(pages, src, dst, copies, stream)
    _check(fn, kv_lib().pi_kv_fork(pages, sp, dp, n, cp, stream))


def pi_kv_copy(cache: pi_kv_cache, copies: torch.Tensor, stream=None) -> None:
    """Keys and values of page copies[i][0] to page copies[i][1] (pairs with an entry out of range are skipped)."""
    fn = "pi_kv_copy"
    cp, device = _copies(fn, copies, -1), cache._device
    n = copies.shape[0]
    _int32(fn, n)
    _on(fn, device, copies)
    stream = _raw_stream(fn, stream, device)
    if _current_device() != device:
        with torch.cuda.device(device):
            return pi_kv_copy(cache, copies, stream)
    _check(fn, kv_lib().pi_kv_copy(cache, cp, n, stream))
