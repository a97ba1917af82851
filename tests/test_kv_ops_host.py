"""The operators around paged attention without a GPU: refusals with the documented codes before any HIP call, the
frequencies of rotary positions, and the references' own hand-worked values."""
import ctypes
import math
import random

import pytest
import torch

import kv_ops_util as U
from activation_sparse_ffn_rank_amd import _abi, _kv, build

A, A8, A4 = 0x10000, 0x10008, 0x10004        # fake addresses: 16-, 8- and 4-byte aligned
NULL, SHAPE, DTYPE, ALIGN, WS = _abi.PI_ERR_NULL, _abi.PI_ERR_SHAPE, _abi.PI_ERR_DTYPE, _abi.PI_ERR_ALIGN, _abi.PI_ERR_WORKSPACE


@pytest.fixture(scope="module")
def L():
    if build.is_stale():
        build.build()
    return _kv.kv_lib()


def cache(n_pages=100, n_kv=8, page=16, hd=128, dtype=1, k=A, v=A):
    return _kv.pi_kv_cache(n_pages, n_kv, page, hd, dtype, k, v)


def batch(n_req=4, max_pages=50, max_q=1, max_kv=800, table=A, starts=A, kv=A):
    return _kv.pi_kv_batch(n_req, max_pages, max_q, max_kv, max_pages, table, starts, kv)


def rope(rot=128, layout=0, norm=0, scale=1.0, eps=1e-6, freq=A, qw=None, kw=None):
    return _kv.pi_kv_rope(rot, layout, norm, scale, eps, freq, qw, kw)


def drafts(**kw):
    base = dict(n_req=4, rows=12, vocab=1000, q_start=A, tokens=A, target=A4, target_stride=1000, draft=A4, draft_stride=1000,
                u_accept=A, u_next=A)
    base.update(kw)
    return _kv.pi_kv_drafts(**base)


def pages(**kw):
    base = dict(n_req=4, page=16, n_pages=100, max_pages=50, table_stride=50, ws=A, ws_bytes=1 << 20)
    base.update({f: A for f in ("cached", "free_ring", "pool", "block_table", "shares", "cached_next", "pool_next", "counts")})
    base.update(kw)
    return _kv.pi_kv_pages(**base)


def test_rope_append_rejects(L):
    def call(c=None, b=None, r=None, q=A, qt=4096, qh=128, k=A, kt=1024, kh=128, v=A, vt=1024, vh=128, slots=A, out=A + 4096,
             ot=4096, oh=128, n=4, n_q=32):
        return L.pi_kv_rope_append(c or cache(), b or batch(), r or rope(), q, qt, qh, k, kt, kh, v, vt, vh, slots, out, ot, oh, n, n_q,
                                   None)
    assert call(n=0) == _abi.PI_OK and call(n=0, q=0, k=0, v=0, slots=0, out=0) == _abi.PI_OK
    args = (A, 4096, 128, A, 1024, 128, A, 1024, 128, A, A, 4096, 128, 4, 32, None)
    assert L.pi_kv_rope_append(None, batch(), rope(), *args) == NULL
    assert L.pi_kv_rope_append(cache(), None, rope(), *args) == NULL
    assert L.pi_kv_rope_append(cache(), batch(), None, *args) == NULL
    for kw in (dict(q=0), dict(k=0), dict(v=0), dict(slots=0), dict(out=0), dict(b=batch(starts=0)), dict(b=batch(kv=0)),
               dict(r=rope(freq=0))):
        assert call(**kw) == NULL, kw
    for kw in (dict(n=-1), dict(n=(1 << 19) + 1), dict(n_q=0), dict(n_q=30), dict(n_q=1032), dict(qt=-8), dict(kh=-8), dict(vt=-8),
               dict(ot=-8), dict(r=rope(rot=136)), dict(r=rope(rot=-16)), dict(r=rope(rot=24)), dict(r=rope(rot=8)),
               dict(r=rope(scale=math.inf)), dict(r=rope(scale=math.nan)), dict(r=rope(eps=-1e-6)), dict(r=rope(eps=math.nan)),
               dict(ot=64), dict(oh=64), dict(ot=0), dict(out=A, ot=8192), dict(out=A, oh=256, ot=8192)):
        assert call(**kw) == SHAPE, kw
    for kw in (dict(r=rope(layout=2)), dict(r=rope(layout=-1)), dict(r=rope(qw=A)), dict(r=rope(kw=A)), dict(c=cache(dtype=3))):
        assert call(**kw) == DTYPE, kw
    for kw in (dict(q=A8), dict(k=A8), dict(v=A8), dict(out=A8), dict(qt=4097), dict(kt=1025), dict(vh=4), dict(oh=132),
               dict(r=rope(freq=A4)), dict(r=rope(norm=1, qw=A8)), dict(r=rope(norm=1, kw=A8))):
        assert call(**kw) == ALIGN, kw


def test_sinks_reject(L):
    size = lambda c, b, t, h, w, s: L.pi_kv_attn_sinks_workspace_bytes(c, b, t, h, w, s)
    need = size(cache(), batch(), 4, 32, 100, 4)
    assert need >= 16 and size(cache(), batch(), 4, 32, 100, 0) == L.pi_kv_attn_workspace_bytes(cache(), batch(), 4, 32)
    assert size(None, batch(), 4, 32, 100, 4) == 0 and size(cache(), None, 4, 32, 100, 4) == 0 and size(cache(), batch(), 4, 30, 100, 4) == 0
    assert size(cache(), batch(), 4, 32, 0, 4) == 0 and size(cache(), batch(), 4, 32, -1, 4) == 0 and size(cache(), batch(), 4, 32, 9, -1) == 0
    assert size(cache(), batch(), 4, 32, -1, 0) == 0
    # a short window over long requests is not cut, a long one is
    assert size(cache(), batch(max_kv=60000), 4, 32, 30, 4) == 16 and size(cache(), batch(max_kv=60000), 4, 32, 30000, 4) > 1 << 16

    need = max(need, size(cache(), batch(), 4, 32, 100, 0))

    def call(c=None, b=None, q=A, qt=4096, qh=128, out=A, ot=4096, oh=128, total=4, n_q=32, scale=0.1, window=100, sinks=4, ws=A, n=need):
        return L.pi_kv_attn_sinks(c or cache(), b or batch(), q, qt, qh, out, ot, oh, total, n_q, scale, window, sinks, ws, n, None)
    for s in (0, 4):
        assert call(total=0, sinks=s) == _abi.PI_OK and call(total=0, q=0, out=0, ws=0, sinks=s) == _abi.PI_OK
        for kw in (dict(q=0), dict(out=0), dict(b=batch(table=0)), dict(b=batch(starts=0)), dict(b=batch(kv=0))):
            assert call(sinks=s, **kw) == NULL
        for kw in (dict(n_q=30), dict(n_q=0), dict(total=-1), dict(total=(1 << 19) + 1), dict(scale=0.0), dict(scale=math.nan),
                   dict(scale=math.inf), dict(window=-1), dict(qt=-8), dict(ot=64), dict(b=batch(n_req=0)), dict(b=batch(max_q=0)),
                   dict(b=batch(max_kv=-1))):
            assert call(sinks=s, **kw) == SHAPE, kw
        for kw in (dict(q=A8), dict(out=A8), dict(qt=4097), dict(oh=4), dict(ws=A8)):
            assert call(sinks=s, **kw) == ALIGN, kw
        assert call(ws=0, sinks=s) == WS and call(n=15, sinks=s) == WS
        assert call(c=cache(dtype=0), sinks=s) == DTYPE
    assert call(sinks=-1) == SHAPE and call(window=0) == SHAPE and call(window=0, sinks=1 << 30) == SHAPE


def test_verify_rejects(L):
    need = L.pi_kv_verify_workspace_bytes(drafts())
    assert need >= 16 and L.pi_kv_verify_workspace_bytes(None) == 0 and L.pi_kv_verify_workspace_bytes(drafts(vocab=0)) == 0

    def call(d=None, kv=A, accepted=A, nxt=A, keep=A, ws=A, n=need):
        return L.pi_kv_verify(d or drafts(), kv, accepted, nxt, keep, ws, n, None)
    assert L.pi_kv_verify(None, A, A, A, A, A, need, None) == NULL
    for kw in (dict(kv=0), dict(keep=0), dict(accepted=0), dict(nxt=0), *(dict(d=drafts(**{f: 0})) for f in
               ("q_start", "tokens", "target", "u_accept", "u_next"))):
        assert call(**kw) == NULL, kw
    for kw in (dict(n_req=0), dict(n_req=4097), dict(rows=0), dict(rows=(1 << 19) + 1), dict(vocab=0), dict(vocab=(1 << 22) + 1),
               dict(target_stride=999), dict(draft_stride=999), dict(target_stride=-1000)):
        assert call(d=drafts(**kw)) == SHAPE, kw
    for kw in (dict(target=0x10002), dict(draft=0x10001)):
        assert call(d=drafts(**kw)) == ALIGN, kw
    assert call(ws=0) == WS and call(n=need - 1) == WS and call(ws=A8) == ALIGN


def test_pages_reject(L):
    release = lambda p=None, f=A, t=A, c=A: L.pi_kv_release(p or pages(), f, t, c, None)
    fork = lambda p=None, s=A, d=A, n=2, c=A: L.pi_kv_fork(p or pages(), s, d, n, c, None)
    assert L.pi_kv_release(None, A, A, A, None) == NULL and L.pi_kv_fork(None, A, A, 2, A, None) == NULL
    for f in ("cached", "free_ring", "pool", "block_table", "shares", "cached_next", "pool_next", "counts"):
        assert release(pages(**{f: 0})) == NULL and fork(pages(**{f: 0})) == NULL
    assert release(f=0) == NULL and release(c=0) == NULL and fork(s=0) == NULL and fork(d=0) == NULL and fork(c=0) == NULL
    for kw in (dict(n_req=0), dict(n_req=4097), dict(page=24), dict(n_pages=0), dict(max_pages=0), dict(max_pages=(1 << 17) + 1),
               dict(table_stride=49), dict(n_pages=1 << 27)):
        assert release(pages(**kw)) == SHAPE and fork(pages(**kw)) == SHAPE, kw
    size = L.pi_kv_pages_workspace_bytes
    assert size(None) == 0 and size(pages(page=24)) == 0 and size(pages()) == 16 and size(pages(n_req=1000, max_pages=1000, table_stride=1000)) > 4000
    assert release(pages(ws=0)) == WS and release(pages(ws_bytes=15)) == WS and release(pages(ws=A8)) == ALIGN
    assert release(pages(n_req=1000, max_pages=1000, table_stride=1000, ws_bytes=4000)) == WS
    assert fork(n=-1) == SHAPE and fork(n=4097) == SHAPE
    copy = lambda c=None, p=A, n=3: L.pi_kv_copy(c or cache(), p, n, None)
    assert copy(n=0) == _abi.PI_OK and copy(n=0, p=0) == _abi.PI_OK and L.pi_kv_copy(None, A, 3, None) == NULL and copy(p=0) == NULL
    assert copy(n=-1) == SHAPE and copy(n=(1 << 19) + 1) == SHAPE and copy(c=cache(page=7)) == SHAPE
    assert copy(c=cache(dtype=9)) == DTYPE and copy(c=cache(v=A8)) == ALIGN


def code(fn):
    with pytest.raises(_abi.PiError) as e:
        fn()
    return e.value.code


def test_tensors_are_checked():
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    half, f32 = torch.float16, lambda *s: torch.zeros(s)
    k, v = torch.zeros(4, 2, 16, 64, dtype=half), torch.zeros(4, 2, 64, 16, dtype=half)
    c, b = _kv.make_kv_cache(k, v), _kv.make_kv_batch(i32(3, 5), i32(4), i32(3), max_q=1, max_kv=80)
    freq, w = torch.zeros(32, dtype=torch.float64), torch.ones(64, dtype=half)
    # rotary descriptors
    assert code(lambda: _kv.make_kv_rope(freq.float())) == DTYPE
    assert code(lambda: _kv.make_kv_rope(freq[None])) == SHAPE
    assert code(lambda: _kv.make_kv_rope(freq[::2])) == SHAPE
    assert code(lambda: _kv.make_kv_rope(freq, q_weight=w, k_weight=w.bfloat16())) == DTYPE
    assert code(lambda: _kv.make_kv_rope(freq, q_weight=w.float())) == DTYPE
    assert code(lambda: _kv.make_kv_rope(freq, q_weight=w, k_weight=w[:32])) == SHAPE
    assert code(lambda: _kv.make_kv_rope(freq, q_weight=w, norm=False)) == DTYPE
    assert code(lambda: _kv.make_kv_rope(freq, layout=2 ** 31)) == SHAPE
    r = _kv.make_kv_rope(freq, layout=_kv.PI_ROPE_PAIRS, scale=1.5, q_weight=w)
    assert (r.rot_dim, r.layout, r.norm, r.scale) == (64, 1, 1, 1.5) and _kv.make_kv_rope(freq).norm == 0
    assert _kv.make_kv_rope(None, norm=True).norm == 1 and _kv.make_kv_rope(None).rot_dim == 0
    x, q, slots = torch.zeros(5, 2, 64, dtype=half), torch.zeros(5, 4, 64, dtype=half), i32(5)
    plain = _kv.make_kv_rope(freq)
    call = lambda r=plain, q=q, k=x, v=x, s=slots, o=q: _kv.pi_kv_rope_append(c, b, r, q, k, v, s, o, 0)
    assert code(lambda: call(k=x[:, :1])) == SHAPE and code(lambda: call(v=x[:4])) == SHAPE and code(lambda: call(s=i32(4))) == SHAPE
    assert code(lambda: call(o=q[:, :2])) == SHAPE and code(lambda: call(q=q.bfloat16())) == DTYPE and code(lambda: call(s=slots.long())) == DTYPE
    assert code(lambda: call(q=torch.zeros(5, 4, 128, dtype=half))) == SHAPE and code(lambda: call(s=None)) == NULL
    assert code(lambda: call(r=_kv.make_kv_rope(freq, q_weight=w.bfloat16()))) == DTYPE
    assert code(lambda: call(r=_kv.make_kv_rope(freq, k_weight=w[:32].contiguous()))) == SHAPE
    assert code(call) == NULL                                                # host memory
    # a window and the first tokens
    ws = torch.zeros(64, dtype=torch.uint8)
    sinks = lambda o=q, w=ws, **kw: _kv.pi_kv_attn_sinks(c, b, q, o, w, scale=1.0, stream=0, **{"window": 3, "sinks": 1, **kw})
    assert code(lambda: sinks(o=q[:4])) == SHAPE and code(lambda: sinks(sinks=2 ** 31)) == SHAPE and code(lambda: sinks(window=2 ** 31)) == SHAPE
    assert code(lambda: sinks(w=ws[::2])) == WS and code(sinks) == NULL
    assert _kv.pi_kv_attn_sinks_workspace_bytes(c, b, 2 ** 32 + 1, 4, 3, 1) == 0
    # drafted tokens
    p = f32(6, 10)
    mk = lambda s=i32(3), t=i32(6), p=p, q=p, u=f32(6), un=f32(2): _kv.make_kv_drafts(s, t, p, q, u, un)
    d = mk(p=f32(6, 12)[:, :10], q=None)
    assert (d.n_req, d.rows, d.vocab, d.target_stride, d.draft) == (2, 6, 10, 12, None)
    assert code(lambda: mk(p=p.half())) == DTYPE and code(lambda: mk(q=p.double())) == DTYPE and code(lambda: mk(s=torch.zeros(3))) == DTYPE
    assert code(lambda: mk(p=p[:5])) == SHAPE and code(lambda: mk(q=p[:, :9])) == SHAPE and code(lambda: mk(p=f32(10, 6).t())) == SHAPE
    assert code(lambda: mk(u=f32(5))) == SHAPE and code(lambda: mk(un=f32(3))) == SHAPE and code(lambda: mk(u=f32(6).double())) == DTYPE
    assert code(lambda: mk(p=None)) == NULL and code(lambda: mk(un=None)) == NULL and code(lambda: mk(p=f32(60))) == SHAPE
    big = torch.zeros(64, dtype=torch.uint8)
    ver = lambda a=i32(2), n=i32(2), w=big, **kw: _kv.pi_kv_verify(d, a, n, w, stream=0, **kw)
    assert code(lambda: ver(a=i32(3))) == SHAPE and code(lambda: ver(n=torch.zeros(2))) == DTYPE and code(lambda: ver(w=big[::2])) == WS
    assert code(lambda: ver(kv_len=i32(1))) == SHAPE and code(ver) == NULL
    # pages
    mk = lambda **kw: _kv.make_kv_pages(**{**dict(cached=i32(3), free_ring=i32(9), pool=i32(2), block_table=i32(3, 4), page=16, shares=i32(9),
                                               cached_next=i32(3), pool_next=i32(2), counts=i32(4)), **kw})
    st = mk(block_table=i32(3, 7)[:, :4])
    assert (st.n_req, st.n_pages, st.max_pages, st.table_stride, st.ws_bytes) == (3, 9, 4, 7, 16)
    assert mk(ws=torch.zeros(99, dtype=torch.uint8)).ws_bytes == 99 and code(lambda: mk(ws=i32(8)[::2])) == WS
    assert code(lambda: mk(shares=i32(8))) == SHAPE and code(lambda: mk(counts=i32(3))) == SHAPE and code(lambda: mk(pool=None)) == NULL
    assert code(lambda: mk(cached_next=i32(2))) == SHAPE and code(lambda: mk(shares=f32(9))) == DTYPE and code(lambda: mk(page=2 ** 31)) == SHAPE
    assert code(lambda: _kv.pi_kv_release(st, i32(2), None, i32(3, 2), 0)) == SHAPE
    assert code(lambda: _kv.pi_kv_release(st, i32(3), None, i32(3), 0)) == SHAPE
    assert code(lambda: _kv.pi_kv_release(st, i32(3), None, None, 0)) == NULL
    assert code(lambda: _kv.pi_kv_release(st, i32(3), None, i32(3, 2).long(), 0)) == DTYPE
    assert code(lambda: _kv.pi_kv_release(st, i32(3), None, i32(3, 2), 0)) == NULL                     # host memory
    assert code(lambda: _kv.pi_kv_fork(st, i32(2), i32(1), i32(2, 2), 0)) == SHAPE
    assert code(lambda: _kv.pi_kv_fork(st, i32(2), i32(2), i32(1, 2), 0)) == SHAPE
    assert code(lambda: _kv.pi_kv_copy(c, i32(2, 3), 0)) == SHAPE and code(lambda: _kv.pi_kv_copy(c, i32(4, 2).t(), 0)) == SHAPE
    assert code(lambda: _kv.pi_kv_copy(c, i32(2, 2), 0)) == NULL


def test_frequencies(L):
    f = _kv.pi_rope_frequencies(8, base=10000.0)
    assert f.dtype == torch.float64 and torch.allclose(f, torch.tensor([1.0, 0.1, 0.01, 0.001], dtype=torch.float64), rtol=1e-15, atol=0)
    assert torch.allclose(_kv.pi_rope_frequencies(8, factor=4.0), f / 4, rtol=1e-15, atol=0)
    # by parts: 4096 / (2 pi) = 651.9, 65.2, 6.52 and 0.652 turns; between 1 and 32 turns a ramp
    g = _kv.pi_rope_frequencies(8, factor=4.0, trained=4096.0, low=1.0, high=32.0)
    keep = (4096 * 0.01 / (2 * math.pi) - 1) / 31
    want = torch.tensor([1.0, 0.1, 0.01 * (keep + (1 - keep) / 4), 0.001 / 4], dtype=torch.float64)
    assert torch.allclose(g, want, rtol=1e-14, atol=0)
    bad = [dict(rot=7), dict(rot=0), dict(rot=258), dict(rot=-2), dict(base=0.0), dict(base=math.inf), dict(factor=-1.0), dict(trained=0.0),
           dict(low=2.0, high=1.0), dict(low=1.0, high=1.0), dict(low=-1.0, high=1.0), dict(low=math.nan), dict(high=math.inf)]
    for kw in bad:
        kw = dict(kw)
        assert code(lambda: _kv.pi_rope_frequencies(kw.pop("rot", 8), **kw)) == SHAPE
    assert L.pi_rope_frequencies(8, 1e4, 1.0, 4096.0, 0.0, 0.0, None) == NULL
    assert code(lambda: _kv.pi_rope_frequencies(2 ** 32 + 8)) == SHAPE


# ------------------------------------------------------------------------------ the references

def test_rope_reference_by_hand():
    x = torch.tensor([[[1.0, 2.0, 3.0, 4.0]]])
    freq = torch.tensor([math.pi / 2], dtype=torch.float64)
    y, _ = U.rope_head(x, torch.tensor([1]), freq, 1, 1.0, False, 0.0, None)
    assert torch.allclose(y, torch.tensor([[[-2.0, 1.0, 3.0, 4.0]]], dtype=torch.float64), atol=1e-12)
    freq = torch.tensor([math.pi / 2, math.pi], dtype=torch.float64)
    y, _ = U.rope_head(x, torch.tensor([1]), freq, 0, 2.0, False, 0.0, None)
    assert torch.allclose(y, torch.tensor([[[-6.0, -4.0, 2.0, -8.0]]], dtype=torch.float64), atol=1e-12)
    y, _ = U.rope_head(2 * x, torch.tensor([5]), None, 0, 1.0, True, 0.0, torch.tensor([1.0, 1.0, 1.0, 2.0]))
    assert torch.allclose(y, x.double() / math.sqrt(7.5) * torch.tensor([1.0, 1.0, 1.0, 2.0]), atol=1e-12)


def test_verify_reference_by_hand():
    p = torch.tensor([[0.5, 0.25, 0.25], [0.2, 0.2, 0.6], [0.0, 1.0, 0.0]])
    q = torch.tensor([[0.25, 0.5, 0.25], [0.5, 0.25, 0.25], [0.0, 0.0, 0.0]])
    run = lambda tokens, u, un, q=q: U.verify_reference([0, 3], tokens, p, q, u, [un], [10])
    assert run([9, 0, 2], [0.9, 0.9, 0.0], 0.5) == ([2], [1], [10])                       # both accepted
    assert run([9, 1, 2], [0.4, 0.9, 0.0], 0.5) == ([2], [1], [10])                       # 0.4 * 0.5 < 0.25
    assert run([9, 1, 2], [0.5, 0.9, 0.0], 0.5) == ([0], [0], [8])                        # 0.25 is not below 0.25: the rest is on 0
    assert run([9, 0, 0], [0.9, 0.9, 0.0], 0.99) == ([1], [2], [9])                       # 0.9 * 0.5 against 0.2
    assert run([9, 0, 7], [0.9, 0.0, 0.0], 0.0) == ([1], [2], [9])                        # no such token
    assert run([9, 0, 2], [0.6, 0.0, 0.0], 0.6, None) == ([0], [2], [8])                  # without draft: 0.25, 0.25 left
    assert U.verify_reference([0, 0, 1], [9], p[:1], None, [0.0], [0.1, 0.7], [4, 5]) == ([0, 0], [-1, 1], [4, 5])


def test_page_references_keep_count_of_owners():
    for seed in range(30):
        page = random.Random(seed).choice((16, 32))
        st = U.pages_state(seed, 9, page, 6)
        U.check_owned(st)
        at, to = U.release_ranges(seed, st)
        got = U.release_reference(st, at, to)
        after = dict(cached=got["cached_next"], table=got["block_table"], ring=got["free_ring"], pool=got["pool_next"], shares=got["shares"], page=page)
        U.check_owned(after)
        empty = [r for r, c in enumerate(after["cached"]) if c == 0]
        held = [r for r, c in enumerate(after["cached"]) if c > 0]
        if empty and held:
            rng = random.Random(seed)
            src, dst = [rng.choice(held) for _ in empty], empty
            got = U.fork_reference(after, src, dst)
            U.check_owned(dict(cached=got["cached_next"], table=got["block_table"], ring=got["free_ring"], pool=got["pool_next"],
                               shares=got["shares"], page=page))


def test_release_reference_by_hand():
    st = dict(cached=[40, 40, 33], table=[[4, 5, 6], [4, 5, 7], [8, 9, 1]], ring=[2, 3, -1, -1, -1, -1, -1, -1, -1, -1], pool=[0, 2],
              shares=[0, 0, 0, 0, 1, 1, 0, 0, 0, 0], page=16)
    # the first is cut inside page 5, which the second has too; the third loses its middle page
    got = U.release_reference(st, [20, 40, 16], [U.ALL, U.ALL, 32])
    assert got["copies"] == [[5, 2], [-1, -1], [-1, -1]] and got["block_table"] == [[4, 2, 6], [4, 5, 7], [8, -1, 1]]
    assert got["shares"][5] == 0 and got["shares"][4] == 1 and got["cached_next"] == [20, 40, 33]
    assert got["free_ring"][2:4] == [6, 9] and got["pool_next"] == [1, 3] and got["counts"] == [3, 2, 1, 0]
