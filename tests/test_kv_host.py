"""The paged-cache entry points without a GPU: exports, refusals with the documented codes before any HIP call,
and the references' own hand-worked values."""
import ctypes
import math
import os
import re
import subprocess

import pytest
import torch

import kv_util
from activation_sparse_ffn_rank_amd import _abi, _kv, build

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "pi_paged_kv.h")
A, U = 0x10000, 0x10008        # fake addresses: 16-byte aligned, 8-byte aligned


@pytest.fixture(scope="module")
def L():
    if build.is_stale():
        build.build()
    return _kv.kv_lib()


def test_exports_every_declared_function(L):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(pi_[a-z_]+)\s*\(", text))
    assert names == set(_kv.KV_EXPORTS)
    for n in names:
        assert hasattr(L, n), n


def cache(n_pages=100, n_kv=8, page=16, hd=128, dtype=1, k=A, v=A):
    return _kv.pi_kv_cache(n_pages, n_kv, page, hd, dtype, k, v)


def batch(n_req=4, max_pages=50, max_q=1, max_kv=800, stride=None, table=A, starts=A, kv=A):
    return _kv.pi_kv_batch(n_req, max_pages, max_q, max_kv, max_pages if stride is None else stride, table, starts, kv)


def tables(**kw):
    base = dict(n_req=4, page=16, n_pages=100, max_pages=50, max_tokens=64, table_stride=50)
    base.update({f: A for f in ("cached", "fresh", "free_ring", "pool", "block_table", "q_start", "kv_len", "cached_next",
                                "slots", "pool_next", "counts")})
    base.update(kw)
    return _kv.pi_kv_tables(**base)


def test_cache_rejects(L):
    call = lambda c, n=4: L.pi_kv_append(c, A, 1024, 128, A, 1024, 128, A, n, None)
    assert call(None) == _abi.PI_ERR_NULL
    for c, code in ((cache(k=0), _abi.PI_ERR_NULL), (cache(v=0), _abi.PI_ERR_NULL), (cache(dtype=3), _abi.PI_ERR_DTYPE),
                    (cache(page=8), _abi.PI_ERR_SHAPE), (cache(page=48), _abi.PI_ERR_SHAPE), (cache(page=512), _abi.PI_ERR_SHAPE),
                    (cache(hd=96), _abi.PI_ERR_SHAPE), (cache(hd=512), _abi.PI_ERR_SHAPE), (cache(n_kv=0), _abi.PI_ERR_SHAPE),
                    (cache(n_kv=1025), _abi.PI_ERR_SHAPE), (cache(n_pages=0), _abi.PI_ERR_SHAPE),
                    (cache(n_pages=1 << 27), _abi.PI_ERR_SHAPE), (cache(k=U), _abi.PI_ERR_ALIGN), (cache(v=U), _abi.PI_ERR_ALIGN)):
        assert call(c) == code


def test_append_rejects(L):
    c = cache()
    call = lambda k=A, kt=1024, kh=128, v=A, vt=1024, vh=128, slots=A, n=4: L.pi_kv_append(c, k, kt, kh, v, vt, vh, slots, n, None)
    assert call(n=0) == _abi.PI_OK and call(n=0, k=0, v=0, slots=0) == _abi.PI_OK
    for kw in (dict(k=0), dict(v=0), dict(slots=0)):
        assert call(**kw) == _abi.PI_ERR_NULL
    for kw in (dict(n=-1), dict(n=(1 << 19) + 1), dict(kt=-1024), dict(vh=-128)):
        assert call(**kw) == _abi.PI_ERR_SHAPE
    for kw in (dict(k=U), dict(v=U), dict(kt=1020), dict(kh=130), dict(vt=1), dict(vh=4)):
        assert call(**kw) == _abi.PI_ERR_ALIGN


def test_step_rejects(L):
    assert L.pi_kv_step(None, None) == _abi.PI_ERR_NULL
    for f in ("cached", "fresh", "free_ring", "pool", "block_table", "q_start", "kv_len", "cached_next", "slots", "pool_next",
              "counts"):
        assert L.pi_kv_step(tables(**{f: 0}), None) == _abi.PI_ERR_NULL
    for kw in (dict(n_req=0), dict(n_req=4097), dict(page=24), dict(n_pages=0), dict(max_pages=0), dict(max_pages=(1 << 17) + 1),
               dict(max_tokens=0), dict(max_tokens=(1 << 19) + 1), dict(table_stride=49), dict(n_pages=1 << 27)):
        assert L.pi_kv_step(tables(**kw), None) == _abi.PI_ERR_SHAPE


def test_attn_rejects(L):
    need = L.pi_kv_attn_workspace_bytes(cache(), batch(), 4, 32)
    assert need >= 16

    def call(c=None, b=None, q=A, qt=4096, qh=128, out=A, ot=4096, oh=128, total=4, n_q=32, scale=0.1, window=0, ws=A, n=need):
        return L.pi_kv_attn(c or cache(), b or batch(), q, qt, qh, out, ot, oh, total, n_q, scale, window, ws, n, None)
    assert call(total=0) == _abi.PI_OK and call(total=0, q=0, out=0, ws=0) == _abi.PI_OK
    assert L.pi_kv_attn(None, batch(), A, 4096, 128, A, 4096, 128, 4, 32, 0.1, 0, A, need, None) == _abi.PI_ERR_NULL
    assert L.pi_kv_attn(cache(), None, A, 4096, 128, A, 4096, 128, 4, 32, 0.1, 0, A, need, None) == _abi.PI_ERR_NULL
    for kw in (dict(q=0), dict(out=0), dict(b=batch(table=0)), dict(b=batch(starts=0)), dict(b=batch(kv=0))):
        assert call(**kw) == _abi.PI_ERR_NULL
    for kw in (dict(n_q=30), dict(n_q=0), dict(n_q=1032), dict(total=-1), dict(total=(1 << 19) + 1), dict(scale=0.0),
               dict(scale=-1.0), dict(scale=math.nan), dict(scale=math.inf), dict(window=-1), dict(qt=-8), dict(b=batch(n_req=0)),
               dict(b=batch(n_req=4097)), dict(b=batch(max_pages=0)), dict(b=batch(stride=49)), dict(b=batch(max_q=0)),
               dict(b=batch(max_kv=-1))):
        assert call(**kw) == _abi.PI_ERR_SHAPE, kw
    for kw in (dict(q=U), dict(out=U), dict(qt=4097), dict(oh=4), dict(ws=U)):
        assert call(**kw) == _abi.PI_ERR_ALIGN, kw
    assert call(ws=0) == _abi.PI_ERR_WORKSPACE and call(n=need - 1) == _abi.PI_ERR_WORKSPACE
    assert call(c=cache(dtype=0)) == _abi.PI_ERR_DTYPE


def test_workspace_sizes(L):
    size = lambda c, b, t, h: L.pi_kv_attn_workspace_bytes(c, b, t, h)
    # long key ranges of few rows are cut and need partial sums; short ones and many rows do not
    assert size(cache(), batch(max_kv=60000), 4, 32) > 1 << 16
    assert size(cache(), batch(max_kv=64), 4, 32) == 16
    assert size(cache(n_kv=32), batch(max_q=4096, max_kv=60000), 16384, 32) == 16
    assert size(None, batch(), 4, 32) == 0 and size(cache(), None, 4, 32) == 0
    assert size(cache(), batch(), 4, 31) == 0 and size(cache(page=7), batch(), 4, 32) == 0


def code(fn):
    with pytest.raises(_abi.PiError) as e:
        fn()
    return e.value.code


def test_descriptors_reject():
    k, v = torch.zeros(4, 2, 16, 64, dtype=torch.float16), torch.zeros(4, 2, 64, 16, dtype=torch.float16)
    c = _kv.make_kv_cache(k, v)
    assert (c.n_pages, c.n_kv, c.page, c.head_dim, c.dtype) == (4, 2, 16, 64, _kv.PI_KV_F16)
    assert code(lambda: _kv.make_kv_cache(k, None)) == _abi.PI_ERR_NULL
    assert code(lambda: _kv.make_kv_cache(k.float(), v.float())) == _abi.PI_ERR_DTYPE
    assert code(lambda: _kv.make_kv_cache(k, v.bfloat16())) == _abi.PI_ERR_DTYPE
    assert code(lambda: _kv.make_kv_cache(k, k)) == _abi.PI_ERR_SHAPE
    assert code(lambda: _kv.make_kv_cache(k[:, :1], v[:, :1])) == _abi.PI_ERR_SHAPE
    table, starts, kv = torch.zeros(3, 9, dtype=torch.int32), torch.zeros(4, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    b = _kv.make_kv_batch(table[:, :5], starts, kv, max_q=1, max_kv=80)
    assert (b.n_req, b.max_pages, b.table_stride) == (3, 5, 9)
    assert code(lambda: _kv.make_kv_batch(table.long(), starts, kv, max_q=1, max_kv=80)) == _abi.PI_ERR_DTYPE
    assert code(lambda: _kv.make_kv_batch(table.t(), starts, kv, max_q=1, max_kv=80)) == _abi.PI_ERR_SHAPE
    assert code(lambda: _kv.make_kv_batch(table, kv, kv, max_q=1, max_kv=80)) == _abi.PI_ERR_SHAPE
    assert code(lambda: _kv.make_kv_batch(table, None, kv, max_q=1, max_kv=80)) == _abi.PI_ERR_NULL
    x, slots = torch.zeros(5, 2, 64, dtype=torch.float16), torch.zeros(5, dtype=torch.int32)
    assert code(lambda: _kv.pi_kv_append(c, x, x[:, :1], slots, 0)) == _abi.PI_ERR_SHAPE
    assert code(lambda: _kv.pi_kv_append(c, x, x[:4], slots, 0)) == _abi.PI_ERR_SHAPE
    assert code(lambda: _kv.pi_kv_append(c, x, x.bfloat16(), slots, 0)) == _abi.PI_ERR_DTYPE
    assert code(lambda: _kv.pi_kv_append(c, x, x, slots[:4], 0)) == _abi.PI_ERR_SHAPE
    assert code(lambda: _kv.pi_kv_append(c, x, x, slots.long(), 0)) == _abi.PI_ERR_DTYPE
    assert code(lambda: _kv.pi_kv_attn(c, b, x, x[:, :, ::2], None, scale=1.0, stream=0)) == _abi.PI_ERR_SHAPE
    assert code(lambda: _kv.pi_kv_attn(c, b, None, x, None, scale=1.0, stream=0)) == _abi.PI_ERR_NULL
    ints = lambda n: torch.zeros(n, dtype=torch.int32)
    good = [ints(3), ints(3), ints(7), ints(2), table, 16, ints(4), ints(3), ints(3), ints(20), ints(2), ints(4)]
    assert _kv.make_kv_tables(*good).max_tokens == 20
    for i in (1, 3, 6, 7, 8, 10, 11):
        bad = list(good)
        bad[i] = ints(9)
        assert code(lambda: _kv.make_kv_tables(*bad)) == _abi.PI_ERR_SHAPE
        bad[i] = bad[i].long()
        assert code(lambda: _kv.make_kv_tables(*bad)) == _abi.PI_ERR_DTYPE


def test_host_tensors_are_refused():
    """Tensors in host memory, and workspaces whose bytes do not lie together."""
    k, v = torch.zeros(4, 2, 16, 64, dtype=torch.float16), torch.zeros(4, 2, 64, 16, dtype=torch.float16)
    ints = lambda n: torch.zeros(n, dtype=torch.int32)
    c = _kv.make_kv_cache(k, v)
    b = _kv.make_kv_batch(torch.zeros(3, 5, dtype=torch.int32), ints(4), ints(3), max_q=1, max_kv=80)
    t = _kv.make_kv_tables(ints(3), ints(3), ints(7), ints(2), torch.zeros(3, 5, dtype=torch.int32), 16, ints(4), ints(3), ints(3),
                           ints(20), ints(2), ints(4))
    x, ws = torch.zeros(3, 2, 64, dtype=torch.float16), torch.zeros(1 << 16, dtype=torch.uint8)
    for stream in (None, 0):
        assert code(lambda: _kv.pi_kv_step(t, stream)) == _abi.PI_ERR_NULL
        assert code(lambda: _kv.pi_kv_append(c, x, x, ints(3), stream)) == _abi.PI_ERR_NULL
        assert code(lambda: _kv.pi_kv_attn(c, b, x, x, ws, scale=1.0, stream=stream)) == _abi.PI_ERR_NULL
    assert code(lambda: _kv.pi_kv_attn(c, b, x, x, ws[:1].expand(1 << 20), scale=1.0, stream=0)) == _abi.PI_ERR_WORKSPACE


def test_step_reference_by_hand():
    # page 4; request 0 grows into a second page, 1 ends, 2 is a prompt of 6, 3 finds no page left
    got = kv_util.step_reference([4, 5, 0, 8], [1, -1, 6, 1], [9, 8, 7, -1, -1, -1, -1, -1, -1, -1], [0, 3],
                                 [[0, -1, -1], [1, 2, -1], [-1, -1, -1], [3, 4, -1]], 4, 10)
    assert got["block_table"] == [[0, 9, -1], [1, 2, -1], [8, 7, -1], [3, 4, -1]]
    assert got["free_ring"][:5] == [9, 8, 7, 1, 2] and got["pool_next"] == [3, 2]
    assert got["q_start"] == [0, 1, 1, 7, 8] and got["kv_len"] == [5, 0, 6, 0] and got["cached_next"] == [5, 0, 6, 8]
    assert got["slots"] == [36, 32, 33, 34, 35, 28, 29, -1, -1, -1] and got["counts"] == [8, 3, 2, 1]


def test_attn_reference_by_hand():
    # one head, keys with scores 0 and ln 3 for the last token: weights 1/4 and 3/4; a window of one sees itself only
    k, v = torch.zeros(1, 1, 16, 64), torch.zeros(1, 1, 64, 16)
    k[0, 0, 1, 0] = math.log(3)
    v[0, 0, :, 0], v[0, 0, :, 1] = 1.0, 5.0
    q = torch.zeros(2, 1, 64)
    q[:, 0, 0] = 1.0
    out, mag = kv_util.attn_reference(q, k, v, [[0]], [0, 2], [2], 1.0, 0)
    assert torch.allclose(out[0], torch.ones(1, 64).double()) and torch.allclose(out[1], torch.full((1, 64), 4.0).double())
    out, _ = kv_util.attn_reference(q, k, v, [[0]], [0, 2], [2], 1.0, 1)
    assert torch.allclose(out[1], torch.full((1, 64), 5.0).double())
    out, _ = kv_util.attn_reference(q, k, v, [[0]], [0, 2], [1], 1.0, 0)       # the first token has no position
    assert out[0].abs().max() == 0 and torch.allclose(out[1], torch.ones(1, 64).double())


@pytest.mark.parametrize("big", (2 ** 31, 2 ** 32, 2 ** 32 + 5, 2 ** 40, -2 ** 31 - 1, -2 ** 32 + 5))
def test_numbers_past_32_bits_are_refused(big):
    """What does not fit the library's 32-bit arguments is refused, and not taken modulo 2^32."""
    k, v = torch.zeros(4, 2, 16, 64, dtype=torch.float16), torch.zeros(4, 2, 64, 16, dtype=torch.float16)
    ints = lambda n: torch.zeros(n, dtype=torch.int32)
    c, table = _kv.make_kv_cache(k, v), torch.zeros(3, 5, dtype=torch.int32)
    b = _kv.make_kv_batch(table, ints(4), ints(3), max_q=1, max_kv=80)
    x, ws = torch.zeros(3, 2, 64, dtype=torch.float16), torch.zeros(1 << 16, dtype=torch.uint8)
    assert code(lambda: _kv.make_kv_batch(table, ints(4), ints(3), max_q=big, max_kv=80)) == _abi.PI_ERR_SHAPE
    assert code(lambda: _kv.make_kv_batch(table, ints(4), ints(3), max_q=1, max_kv=big)) == _abi.PI_ERR_SHAPE
    assert code(lambda: _kv.make_kv_tables(ints(3), ints(3), ints(7), ints(2), table, big, ints(4), ints(3), ints(3), ints(20),
                                           ints(2), ints(4))) == _abi.PI_ERR_SHAPE
    assert code(lambda: _kv.pi_kv_attn(c, b, x, x, ws, scale=1.0, window=big, stream=0)) == _abi.PI_ERR_SHAPE
    assert _kv.pi_kv_attn_workspace_bytes(c, b, big, 2) == 0 and _kv.pi_kv_attn_workspace_bytes(c, b, 3, big) == 0
    if big < 0:
        return
    # lengths of tensors (no memory behind them)
    many, rows = torch.empty(big, dtype=torch.int32, device="meta"), x[:1].expand(big, 2, 64)
    assert code(lambda: _kv.pi_kv_append(c, rows, rows, many, 0)) == _abi.PI_ERR_SHAPE
    assert code(lambda: _kv.pi_kv_attn(c, b, rows, rows, ws, scale=1.0, stream=0)) == _abi.PI_ERR_SHAPE
    assert code(lambda: _kv.make_kv_batch(table[:, :1].expand(3, 1), ints(4), many, max_q=1, max_kv=80)) == _abi.PI_ERR_SHAPE
    pages = lambda *shape: torch.empty(shape, dtype=torch.float16, device="meta")
    assert code(lambda: _kv.make_kv_cache(pages(big, 2, 16, 64), pages(big, 2, 64, 16))) == _abi.PI_ERR_SHAPE
    wide = torch.empty((3, big), dtype=torch.int32, device="meta")
    assert code(lambda: _kv.make_kv_batch(wide, ints(4), ints(3), max_q=1, max_kv=80)) == _abi.PI_ERR_SHAPE
    for at in (2, 9):
        args = [ints(3), ints(3), ints(7), ints(2), table, 16, ints(4), ints(3), ints(3), ints(20), ints(2), ints(4)]
        args[at] = many
        assert code(lambda: _kv.make_kv_tables(*args)) == _abi.PI_ERR_SHAPE


class _OnDevice1(torch.Tensor):
    """Host memory that says it is on device 1."""
    def get_device(self):
        return 1


@pytest.mark.parametrize("current", (0, 1))
def test_calls_run_on_the_device_of_the_tensors(monkeypatch, current):
    """With another device current, a call is made with the tensors' device current, and it is set back."""
    at, calls = [current], []

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.before, at[0] = at[0], self.index

        def __exit__(self, *exc):
            at[0] = self.before

    class Lib:
        def __getattr__(self, name):
            def call(*args):
                calls.append((name, at[0]))
                return _abi.PI_OK if len(calls) % 2 else _abi.PI_ERR_HIP      # the second call of each fails
            return call

    monkeypatch.setattr(_kv, "_current_device", lambda: at[0], raising=False)
    monkeypatch.setattr(_kv, "_current_stream", lambda device: 0)
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(_kv, "_kv_lib", Lib())
    here = lambda t: t.as_subclass(_OnDevice1)
    ints = lambda *n: here(torch.zeros(n, dtype=torch.int32))
    half = lambda *n: here(torch.zeros(n, dtype=torch.float16))
    cache = _kv.make_kv_cache(half(4, 2, 16, 64), half(4, 2, 64, 16))
    batch = _kv.make_kv_batch(ints(3, 5), ints(4), ints(3), max_q=1, max_kv=80)
    tables = _kv.make_kv_tables(ints(3), ints(3), ints(7), ints(2), ints(3, 5), 16, ints(4), ints(3), ints(3), ints(20), ints(2),
                                ints(4))
    for name, fn in (("pi_kv_step", lambda: _kv.pi_kv_step(tables)),
                     ("pi_kv_append", lambda: _kv.pi_kv_append(cache, half(3, 2, 64), half(3, 2, 64), ints(3))),
                     ("pi_kv_attn", lambda: _kv.pi_kv_attn(cache, batch, half(3, 2, 64), half(3, 2, 64), ints(64), scale=1.0))):
        del calls[:]
        fn()
        assert at == [current]
        assert code(fn) == _abi.PI_ERR_HIP
        assert calls == [(name, 1), (name, 1)] and at == [current]


@pytest.mark.parametrize("text,ok", [('asm volatile("s_mov_b32 m0, %0" ::"s"(x) : "m0");', False),
                                     ('asm volatile("s_nop 0" ::"{m0}"(x));', True)])
def test_build_refuses_clobbers_of_reserved_registers(tmp_path, text, ok):
    """The flags that the kernels are built with end the build at an asm statement that clobbers m0."""
    src = tmp_path / "t.hip"
    src.write_text('#include <hip/hip_runtime.h>\n__global__ void k(int x) { ' + text + ' }\n')
    res = subprocess.run([build.HIPCC, *build.FLAGS, "--cuda-device-only", "-S", str(src), "-o", str(tmp_path / "t.s")],
                         capture_output=True, text=True)
    assert (res.returncode == 0) == ok, res.stderr


def test_outputs_whose_rows_overlap_are_refused(L):
    """Rows of the output that share elements would be written by several workgroups, in any order."""
    def call(ot, oh, total=4, n_q=32, qt=0, qh=0):
        return L.pi_kv_attn(cache(), batch(), A, qt, qh, A, ot, oh, total, n_q, 0.1, 0, 0, 0, None)
    fine = _abi.PI_ERR_WORKSPACE                   # refused later, for the missing workspace
    # (rows of queries may be shared: only reads)
    assert call(4096, 128) == fine and call(4096, 128, qt=8, qh=0) == fine
    assert call(128, 512) == fine and call(128, 520) == fine                  # heads outermost
    assert call(0, 128, total=1) == fine and call(136, 0, n_q=8, total=1) == _abi.PI_ERR_SHAPE
    for ot, oh in ((0, 128), (4096, 0), (120, 4096), (4096, 120), (0, 0), (128, 128), (4088, 128), (128, 504), (2048, 128),
                   (1 << 62, 0)):
        assert call(ot, oh) == _abi.PI_ERR_SHAPE, (ot, oh)
    assert call(1 << 62, 128) == fine and call(128, 1 << 62) == fine
    # interleaved: distinct as long as no multiple of one stride meets one of the other
    assert call(3 * 128, 2 * 128, total=2, n_q=8) == fine
    assert call(3 * 128, 2 * 128, total=3, n_q=8) == _abi.PI_ERR_SHAPE        # 2 x 3 = 3 x 2
    assert call(17 * 128, 2 * 128, total=2, n_q=8) == fine and call(15 * 128, 2 * 128, total=2, n_q=8) == fine
    # against every pair of rows
    for ot in range(64, 900, 64):
        for oh in range(64, 900, 64):
            at = sorted(t * ot + h * oh for t in range(3) for h in range(8))
            want = _abi.PI_ERR_SHAPE if min(b - a for a, b in zip(at, at[1:])) < 128 else fine
            assert call(ot, oh, total=3, n_q=8) == want, (ot, oh)
