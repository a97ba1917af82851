"""The operators around paged attention on the GPU against plain 64-bit references: rotary positions and head norms
with the append, attention over a window and the first tokens, drafted tokens, pages given back, shared and copied, and all of
them together in a replayed graph."""
import importlib.util
import math
import os
import random

import pytest
import torch

import activation_sparse_ffn_rank_amd as pi
from activation_sparse_ffn_rank_amd import _abi, _kv
import kv_ops_util as U
import kv_util
import synth
from gpu_util import announce

pytestmark = pytest.mark.gpu


def dev(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device="cuda")


def code(fn):
    with pytest.raises(_abi.PiError) as e:
        fn()
    return e.value.code


# ------------------------------------------------------------------------------ rotary positions with the append

def rope_case(seed, lens, n_q, n_kv, hd, page, dtype, rot, layout, norm, *, pad=3, weights=True, scale=1.0, base=10000.0):
    """Packed rows of requests (new tokens, keys), slots in random pages, some rows without a slot; CPU tensors."""
    gen = torch.Generator().manual_seed(seed)
    rng = random.Random(seed)
    dt = kv_util.DT[dtype]
    starts = [0]
    for n, _ in lens:
        starts.append(starts[-1] + n)
    rows = starts[-1] + pad
    n_pages = rows // page + 3
    slots = list(range(n_pages * page))
    rng.shuffle(slots)
    slots = slots[:rows]
    for t in range(rows):
        if rng.random() < 0.1:
            slots[t] = rng.choice((-1, n_pages * page, 2 ** 31 - 1, -2 ** 31))
    normal = lambda *s: torch.randn(s, generator=gen)
    freq = _kv.pi_rope_frequencies(rot, base=base) if rot else None
    weight = lambda: (1 + 0.3 * normal(hd)).to(dt) if norm and weights else None
    return dict(starts=starts, kv=[m for _, m in lens], rows=rows, slots=slots, qkv=(3 * normal(rows, n_q + 2 * n_kv, hd)).to(dt),
                k=normal(n_pages, n_kv, page, hd).to(dt), v=normal(n_pages, n_kv, hd, page).to(dt), freq=freq, layout=layout, norm=norm,
                scale=scale, eps=1e-5, qw=weight(), kw=weight(), n_q=n_q, n_kv=n_kv, page=page, dt=dt)


def run_rope(c, *, in_place=False, fused=True, stream=None, starts=None):
    """(queries, K pages, V pages, the projection's output) after the call."""
    n_q, n_kv, hd = c["n_q"], c["n_kv"], c["k"].shape[3]
    kg, vg = c["k"].cuda(), c["v"].cuda()
    put = lambda t: None if t is None else t.cuda()
    rope = pi.make_kv_rope(put(c["freq"]), layout=c["layout"], scale=c["scale"], norm=c["norm"], eps=c["eps"], q_weight=put(c["qw"]),
                           k_weight=put(c["kw"]))
    starts = dev(c["starts"] if starts is None else starts)
    batch = pi.make_kv_batch(torch.zeros((len(c["kv"]), 1), dtype=torch.int32, device="cuda"), starts, dev(c["kv"]), max_q=1, max_kv=0)
    qkv = c["qkv"].cuda()
    q, k, v = qkv.split((n_q, n_kv, n_kv), dim=1)
    if not fused:
        q, k, v = q.contiguous(), k.transpose(0, 1).contiguous().transpose(0, 1), v.contiguous()
    wide = torch.full((c["rows"], n_q + 1, hd + 8), 7.0, dtype=c["dt"], device="cuda")
    out = q if in_place else wide[:, :n_q, :hd]
    pi.pi_kv_rope_append(pi.make_kv_cache(kg, vg), batch, rope, q, k, v, dev(c["slots"]), out, stream)
    torch.cuda.synchronize()
    got = out.cpu()
    if not in_place:
        out.fill_(7.0)
        assert bool((wide == 7.0).all()), "written outside the output's rows"
    return got, kg.cpu(), vg.cpu(), qkv.cpu()


def check_rope(c, got, untouched, far=1 << 20):
    q_out, k_out, v_out = got[:3]
    starts, page, n_q, n_kv = c["starts"], c["page"], c["n_q"], c["n_kv"]
    n_pages = c["k"].shape[0]
    q, k, v = c["qkv"].split((n_q, n_kv, n_kv), dim=1)
    k_want, v_want = c["k"].double(), c["v"].clone()
    k_tol, q_want, q_tol = torch.zeros_like(k_want), untouched.double(), torch.zeros(q.shape, dtype=torch.float64)
    for r, m in enumerate(c["kv"]):
        a, b = starts[r], starts[r + 1]
        pos = torch.arange(m - (b - a), m)
        y, mag = U.rope_head(q[a:b], pos, c["freq"], c["layout"], c["scale"], c["norm"], c["eps"], c["qw"])
        q_want[a:b], q_tol[a:b] = y, U.rope_tolerance(y, mag, c["dt"], c["norm"], far)
        y, mag = U.rope_head(k[a:b], pos, c["freq"], c["layout"], c["scale"], c["norm"], c["eps"], c["kw"])
        tol = U.rope_tolerance(y, mag, c["dt"], c["norm"], far)
        for i, t in enumerate(range(a, b)):
            s = c["slots"][t]
            if 0 <= s < n_pages * page:
                k_want[s // page, :, s % page], k_tol[s // page, :, s % page] = y[i], tol[i]
                v_want[s // page, :, :, s % page] = v[t]
    assert bool(((q_out.double() - q_want).abs() <= q_tol).all()), "queries"
    assert bool(((k_out.double() - k_want).abs() <= k_tol).all()), "keys"
    assert torch.equal(v_out.view(torch.int16), v_want.view(torch.int16)), "values"


ROPE_LENS = [(1, 1), (1, 77), (5, 5), (0, 9), (37, 1000), (1, 100000), (20, 1 << 20), (2, 2)]


@pytest.mark.parametrize("dtype", ("f16", "bf16"))
@pytest.mark.parametrize("norm", (False, True))
@pytest.mark.parametrize("layout", (0, 1))
@pytest.mark.parametrize("n_q,n_kv,hd,rot,page", [(4, 4, 64, 64, 16), (16, 1, 64, 32, 64), (10, 2, 128, 128, 32), (3, 3, 128, 16, 16),
                                                  (8, 1, 256, 256, 128), (2, 2, 256, 64, 256), (5, 5, 128, 0, 16)])
def test_rope_append(n_q, n_kv, hd, rot, page, layout, norm, dtype):
    announce(f"rope append heads={n_q}/{n_kv} hd={hd} rot={rot} page={page} layout={layout} norm={norm} {dtype}")
    c = rope_case(hd + rot, ROPE_LENS, n_q, n_kv, hd, page, dtype, rot, layout, norm, scale=1.25)
    check_rope(c, run_rope(c), torch.full(c["qkv"][:, :n_q].shape, 7.0))


@pytest.mark.parametrize("n_q,n_kv,hd,dtype", [(4, 2, 64, "f16"), (12, 4, 128, "bf16"), (2, 1, 256, "f16")])
def test_rope_append_in_place(n_q, n_kv, hd, dtype):
    announce(f"rope append in place heads={n_q}/{n_kv} hd={hd} {dtype}")
    for layout in (0, 1):
        c = rope_case(3, ROPE_LENS, n_q, n_kv, hd, 16, dtype, hd, layout, True)
        got = run_rope(c, in_place=True)
        check_rope(c, got, c["qkv"][:, :n_q])
        assert torch.equal(got[3][:, n_q:].view(torch.int16), c["qkv"][:, n_q:].view(torch.int16))        # k and v as they were


def test_rope_append_strided_rows_and_one_token():
    announce("rope append strided rows")
    for lens in ([(1, 1)], [(1, 40)], [(3, 3)], [(2, 900), (1, 4)]):
        for pad in (0, 2):
            c = rope_case(5, lens, 6, 3, 128, 16, "f16", 64, 0, True, pad=pad, weights=False)
            check_rope(c, run_rope(c, fused=False), torch.full(c["qkv"][:, :6].shape, 7.0))


@pytest.mark.parametrize("n_req", (1, 63, 64, 65, 500, 4096))
def test_rope_append_of_many_requests(n_req):
    announce(f"rope append n_req={n_req}")
    rng = random.Random(n_req)
    lens = [(n, n + rng.randint(0, 5000)) for n in (rng.choice((0, 1, 1, 1, 2, 5)) for _ in range(n_req))]
    lens[0] = (1, 8)
    c = rope_case(n_req, lens, 2, 1, 64, 16, "bf16", 64, 0, False)
    check_rope(c, run_rope(c), torch.full(c["qkv"][:, :2].shape, 7.0))


def test_rope_append_of_many_tokens():
    """Enough rows for every way of sharing them out."""
    announce("rope append many tokens")
    for n_q, n_kv, hd, rot, lens in ((16, 16, 64, 64, [(1500, 1500), (700, 5000)]), (32, 4, 128, 128, [(2100, 9000)]), (9, 3, 256, 128, [(1000, 1000)])):
        c = rope_case(11, lens, n_q, n_kv, hd, 64, "f16", rot, 0, True)
        check_rope(c, run_rope(c), torch.full(c["qkv"][:, :n_q].shape, 7.0))


def test_rope_append_at_the_farthest_positions():
    announce("rope append far positions")
    top = 2 ** 31 - 1
    c = rope_case(8, [(4, top), (1, top), (3, top - 12345), (6, 2)], 4, 2, 128, 16, "f16", 128, 1, False)
    check_rope(c, run_rope(c), torch.full(c["qkv"][:, :4].shape, 7.0), far=2 ** 31)


def test_rope_append_row_ranges_out_of_bounds():
    """Rows of ranges that are negative, past the rows or decreasing are left out; nothing outside the arrays is touched."""
    announce("rope append ranges out of bounds")
    c = rope_case(2, [(4, 9), (4, 9), (4, 30)], 4, 2, 64, 16, "f16", 64, 0, False, pad=4)
    want = c["qkv"][:, :4].clone()
    for starts in ([-4, 0, 4, 8], [0, 4, 8, 99], [0, 4, 2, 6], [2 ** 31 - 1] * 4, [-2 ** 31] * 4, [5, 5, 5, 5]):
        got = run_rope(c, starts=starts)
        rows = [any(0 <= a <= t < b <= c["rows"] for a, b in zip(starts, starts[1:])) for t in range(c["rows"])]
        for t, ok in enumerate(rows):
            if not ok:
                assert bool((got[0][t] == 7.0).all()), (starts, t)
    assert torch.equal(c["qkv"][:, :4], want)


@pytest.mark.parametrize("heads,hd", [((4, 2), 64), ((80, 80), 128)])      # values in tiles of 16 tokens and of 64
def test_rope_append_leaves_keys_and_values_of_cut_ranges_alone(heads, hd):
    """A range that leaves the rows belongs to no request: neither keys nor values of its rows are appended."""
    announce(f"rope append cut ranges {heads}")
    n = 120
    c = rope_case(4, [(n, n), (n, 2 * n), (n, 300)], *heads, hd, 64, "f16", hd, 0, False, pad=4 if hd == 64 else 64)
    n_q, n_kv = heads
    for starts in ([-4, n, 2 * n, 3 * n], [-9, -4, n, 2 * n], [0, n, 2 * n, 3 * n + 99], [0, n, 3 * n + 99, 3 * n + 99], [-1, 2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1],
                   [-2 ** 31, n, n, n], [0, 7, 7, 9]):
        got = run_rope(c, starts=starts)
        k_kept, v_kept = torch.ones(c["k"].shape[0], c["page"], dtype=torch.bool), c["v"].clone()
        for t, slot in enumerate(c["slots"]):
            if any(0 <= a <= t < b <= c["rows"] for a, b in zip(starts, starts[1:])) and 0 <= slot < k_kept.numel():
                k_kept[slot // c["page"], slot % c["page"]] = False
                v_kept[slot // c["page"], :, :, slot % c["page"]] = c["qkv"][t, n_q + n_kv:]
        assert torch.equal(got[2].view(torch.int16), v_kept.view(torch.int16)), ("values", starts)
        same = (got[1].view(torch.int16) == c["k"].view(torch.int16)).all(-1).all(1)
        assert torch.equal(same, k_kept), ("keys", starts)


@pytest.mark.parametrize("bad", (math.nan, math.inf, -math.inf))
def test_rope_append_keeps_bad_numbers_in_their_head(bad):
    announce(f"rope append {bad}")
    c = rope_case(4, [(6, 20)], 4, 2, 128, 16, "f16", 64, 0, True, pad=0)
    c["slots"] = list(range(6))
    clean = run_rope(c)
    c["qkv"][2, 1, 100] = bad                # an element of query head 1 that is not rotated
    c["qkv"][3, 4, 3] = bad                  # of key head 0
    c["qkv"][4, 7, 9] = bad                  # of value head 1
    got = run_rope(c)
    keep = torch.ones(6, 4, dtype=torch.bool)
    keep[2, 1] = False
    assert torch.equal(got[0][keep], clean[0][keep]) and not torch.isfinite(got[0][2, 1, 100])
    assert torch.equal(got[1][0, 0, [0, 1, 2, 4, 5]], clean[1][0, 0, [0, 1, 2, 4, 5]]) and torch.equal(got[1][:, 1], clean[1][:, 1])
    got[2][0, 1, 9, 4] = 0.0
    clean[2][0, 1, 9, 4] = 0.0
    assert torch.equal(got[2], clean[2])


def test_rope_append_without_rotation_and_norm_is_append():
    announce("rope append as append")
    c = rope_case(6, [(30, 30), (7, 9)], 4, 2, 64, 32, "bf16", 0, 0, False, pad=0)
    got = run_rope(c)
    kg, vg = c["k"].cuda(), c["v"].cuda()
    qkv = c["qkv"].cuda()
    pi.pi_kv_append(pi.make_kv_cache(kg, vg), qkv[:, 4:6], qkv[:, 6:], dev(c["slots"]))
    torch.cuda.synchronize()
    same = lambda a, b: torch.equal(a.view(torch.int16), b.view(torch.int16))
    assert same(got[1], kg.cpu()) and same(got[2], vg.cpu()) and same(got[0].contiguous(), c["qkv"][:, :4].contiguous())


# ------------------------------------------------------------------------------ a window and the first tokens

def run_sinks(c, window, sinks, *, max_q=None, max_kv=None, stream=None):
    n = [b - a for a, b in zip(c["starts"], c["starts"][1:])]
    rows, n_q, hd = c["q"].shape
    out = torch.full((rows, n_q, hd), 7.0, dtype=c["q"].dtype, device="cuda")
    q = c["q"].cuda()
    cache = pi.make_kv_cache(c["k"].cuda(), c["v"].cuda())
    batch = pi.make_kv_batch(dev(c["table"]), dev(c["starts"]), dev(c["kv"]), max_q=max_q or max(1, max(n)),
                             max_kv=max(c["kv"]) if max_kv is None else max_kv)
    size = pi.pi_kv_attn_sinks_workspace_bytes(cache, batch, rows, n_q, window, sinks)
    assert size >= 16
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    pi.pi_kv_attn_sinks(cache, batch, q, out, ws, scale=c["scale"], window=window, sinks=sinks, stream=stream)
    torch.cuda.synchronize()
    return out.cpu()


def evict(c, window, sinks):
    """Takes the pages between the first tokens and every window out of the tables."""
    page = c["page"]
    for r, m in enumerate(c["kv"]):
        n = c["starts"][r + 1] - c["starts"][r]
        for col in range(kv_util.ceil_div(sinks, page), max(m - n - window + 1, 0) // page):
            c["table"][r][col] = -1


def check_sinks(c, window, sinks, got=None, rows=None, **kw):
    got = run_sinks(c, window, sinks, **kw) if got is None else got
    want, mag = U.sinks_reference(c, window, sinks, rows)
    tol = kv_util.attn_tolerance(want, mag, c["q"].dtype, c["q"].shape[2])
    assert torch.isfinite(got).all()
    err = (got.double() - want).abs()
    if rows is not None:
        pick = sorted(rows)
        err, tol = err[pick], tol[pick]
    assert bool((err <= tol).all()), f"worst {float((err / tol).max()):.3f} of the tolerance"
    return got


HEADS = ((4, 4, 64), (2, 2, 128), (16, 1, 64), (10, 2, 128), (8, 1, 256))
FIRST = (1, 4, 63, 64, 65, 130, 700)


@pytest.mark.parametrize("dtype", ("f16", "bf16"))
@pytest.mark.parametrize("page", (16, 64, 256))
@pytest.mark.parametrize("n_q,n_kv,hd", HEADS)
def test_sinks_single_tokens(n_q, n_kv, hd, page, dtype):
    lens = [(1, m) for m in (1, 2, 16, 33, 64, 65, 127, 129, 300, 517, 800)]
    for i, sinks in enumerate(FIRST):
        window = (1, 2, 20, 64, 150, 33, 90)[i]
        announce(f"sinks single tokens heads={n_q}/{n_kv} hd={hd} page={page} {dtype} window={window} sinks={sinks}")
        c = kv_util.attn_case(page + hd + i, lens, n_q, n_kv, hd, page, dtype)
        evict(c, window, sinks)
        kv_util.past_end(c, math.nan)
        check_sinks(c, window, sinks)


@pytest.mark.parametrize("window,sinks", [(1, 1), (20, 4), (150, 70), (64, 64), (33, 300)])
@pytest.mark.parametrize("n_q,n_kv,hd,page,dtype", [(4, 4, 64, 16, "f16"), (2, 2, 128, 64, "bf16"), (16, 1, 64, 32, "bf16"),
                                                    (10, 2, 128, 16, "f16"), (8, 1, 256, 256, "f16"), (2, 2, 256, 16, "bf16")])
def test_sinks_ragged_chunks(n_q, n_kv, hd, page, dtype, window, sinks):
    announce(f"sinks ragged chunks heads={n_q}/{n_kv} hd={hd} page={page} {dtype} window={window} sinks={sinks}")
    lens = [(3, 3), (1, 700), (40, 300), (17, 17), (5, 900), (130, 200), (0, 50), (2, 1)]
    c = kv_util.attn_case(hd + page, lens, n_q, n_kv, hd, page, dtype)
    evict(c, window, sinks)
    kv_util.past_end(c, math.nan)
    check_sinks(c, window, sinks)


@pytest.mark.parametrize("n_q,n_kv,hd,page,dtype", [(4, 4, 64, 64, "bf16"), (2, 2, 128, 16, "f16"), (16, 1, 64, 16, "f16"), (4, 1, 256, 32, "bf16")])
def test_sinks_chunk_of_many_tiles(n_q, n_kv, hd, page, dtype):
    """Tiles before, at and past the place where the window leaves the first tokens."""
    for n, m, window, sinks in ((600, 600, 100, 10), (500, 1100, 64, 65), (300, 300, 7, 200)):
        announce(f"sinks chunk {n} on {m} heads={n_q}/{n_kv} hd={hd} page={page} {dtype} window={window} sinks={sinks}")
        c = kv_util.attn_case(7, [(n, m), (1, 40)], n_q, n_kv, hd, page, dtype)
        rng = random.Random(n)
        check_sinks(c, window, sinks, rows={0, n - 1, n, *rng.sample(range(n), 60), *range(window, min(n, window + sinks + 3), 9)})


@pytest.mark.parametrize("n_q,n_kv,hd,page,dtype,window,sinks,lens", [
    (4, 4, 64, 16, "f16", 5000, 4, [(1, 20000)]), (2, 2, 128, 64, "bf16", 3000, 900, [(1, 9000), (1, 100)]),
    (16, 1, 64, 32, "bf16", 4000, 3000, [(5, 9000), (1, 30)]), (8, 1, 256, 16, "f16", 2500, 130, [(1, 6000)]),
    (2, 1, 128, 16, "f16", 1500, 65, [(150, 7000), (1, 6000)]), (2, 2, 64, 16, "bf16", 1000, 5000, [(1, 7000)])])
def test_sinks_long_ranges(n_q, n_kv, hd, page, dtype, window, sinks, lens):
    """Ranges that are cut into pieces, pieces across the step from the first tokens to the window among them."""
    announce(f"sinks long ranges heads={n_q}/{n_kv} hd={hd} page={page} {dtype} window={window} sinks={sinks}")
    c = kv_util.attn_case(hd, lens, n_q, n_kv, hd, page, dtype)
    evict(c, window, sinks)
    rows = c["starts"][-1]
    check_sinks(c, window, sinks, rows=set(random.Random(1).sample(range(rows), min(rows, 12))) | {0, rows - 1})


@pytest.mark.parametrize("n_q,n_kv,hd,page,dtype,n_req", [(56, 56, 128, 16, "f16", 20), (16, 16, 64, 32, "bf16", 60), (16, 16, 64, 16, "f16", 8)])
def test_sinks_many_and_few_short_ranges(n_q, n_kv, hd, page, dtype, n_req):
    announce(f"sinks short ranges heads={n_q}/{n_kv} hd={hd} page={page} {dtype} n_req={n_req}")
    rng = random.Random(n_req)
    c = kv_util.attn_case(n_req, [(1, rng.randint(1, 3000)) for _ in range(n_req)], n_q, n_kv, hd, page, dtype)
    for window, sinks in ((100, 4), (400, 70)):
        check_sinks(c, window, sinks, rows=set(rng.sample(range(n_req), 6)))


@pytest.mark.parametrize("bad", (math.nan, math.inf, -math.inf))
@pytest.mark.parametrize("n_q,n_kv,hd,page,dtype", [(4, 4, 64, 16, "f16"), (8, 1, 128, 64, "bf16"), (2, 1, 256, 32, "f16")])
def test_sinks_masked_places_have_no_effect(n_q, n_kv, hd, page, dtype, bad):
    """What no token of a request sees holds anything; what some tokens see and others do not reaches only those."""
    announce(f"sinks masked places heads={n_q}/{n_kv} hd={hd} page={page} {dtype} {bad}")
    for lens, window, sinks in (([(1, 500), (3, 200)], 40, 5), ([(40, 400), (1, 90)], 30, 20), ([(200, 600)], 50, 3)):
        c = kv_util.attn_case(1, lens, n_q, n_kv, hd, page, dtype)
        clean = run_sinks(c, window, sinks)
        for r, (n, m) in enumerate(lens):
            for j in range(sinks, max(m - n - window + 1, 0)):
                p = c["table"][r][j // page]
                c["k"][p, :, j % page] = bad
                c["v"][p, :, :, j % page] = bad
        kv_util.past_end(c, bad)
        assert torch.equal(run_sinks(c, window, sinks), clean)
        # a value that leaves the window of the last request's tokens one after another
        r, (n, m) = len(lens) - 1, lens[-1]
        j = max(m - n - window + 1, 0) + n // 2
        c["v"][c["table"][r][j // page], :, 3, j % page] = bad
        got = run_sinks(c, window, sinks)
        a = c["starts"][r]
        for i in range(n):
            p = m - n + i
            if j <= p and (j > p - window or j < sinks):
                assert not torch.isfinite(got[a + i, :, 3]).any(), i
            else:
                assert torch.equal(got[a + i], clean[a + i]), i
        rest = torch.ones(got.shape[0], dtype=torch.bool)
        rest[a: a + n] = False
        assert torch.equal(got[rest], clean[rest])


def test_sinks_rows_without_keys():
    """More new tokens than keys, no keys, a first page that is missing: zeros where nothing is seen."""
    announce("sinks rows without keys")
    for n_q, n_kv, hd in ((4, 4, 64), (16, 1, 128)):
        c = kv_util.attn_case(3, [(5, 3), (2, 0), (1, 200), (30, 20)], n_q, n_kv, hd, 16, "f16")
        c["table"][2][0] = -1
        c["table"][2][-1] = 10 ** 6
        c["table"][2][kv_util.ceil_div(200, 16) - 1] = -5
        got = check_sinks(c, 5, 9)
        assert not bool(got[:2].any()) and not bool(got[5:8].any()) and not bool(got[8: 18].any())


def test_sinks_bounds_cut_lengths():
    announce("sinks bounds")
    c = kv_util.attn_case(4, [(1, 900), (6, 700)], 4, 2, 64, 16, "bf16")
    got = run_sinks(c, 50, 70, max_kv=400)
    # keys past max_kv are not read: only the first ones are left
    for r, t in ((0, 0), (1, 6)):
        ref = dict(c, q=c["q"][t: t + 1], starts=[0, 1], table=[c["table"][r]], kv=[70])
        want, mag = U.sinks_reference(ref, 1000, 1)
        err = (got[t].double() - want[0]).abs()
        assert bool((err <= kv_util.attn_tolerance(want[0], mag[0], torch.bfloat16, 64)).all())
    assert bool((run_sinks(c, 50, 70, max_q=4)[5:] == 7.0).all())           # rows past max_q are left as they were


def test_sinks_of_none_and_of_all():
    announce("sinks of none and of all")
    for n_q, n_kv, hd, dtype in ((4, 2, 64, "f16"), (6, 2, 128, "bf16")):
        c = kv_util.attn_case(9, [(1, 300), (20, 310), (150, 150)], n_q, n_kv, hd, 32, dtype)
        window = pi.make_kv_cache(c["k"].cuda(), c["v"].cuda())
        batch = pi.make_kv_batch(dev(c["table"]), dev(c["starts"]), dev(c["kv"]), max_q=150, max_kv=310)
        for w, s in ((40, 0), (0, 0), (2 ** 31 - 1, 5), (40, 2 ** 31 - 1), (1, 310)):
            out = torch.empty_like(c["q"], device="cuda")
            ws = torch.empty(max(pi.pi_kv_attn_sinks_workspace_bytes(window, batch, 171, n_q, w, s),
                                 pi.pi_kv_attn_workspace_bytes(window, batch, 171, n_q)), dtype=torch.uint8, device="cuda")
            pi.pi_kv_attn_sinks(window, batch, c["q"].cuda(), out, ws, scale=c["scale"], window=w, sinks=s)
            torch.cuda.synchronize()
            if s == 0:
                want = torch.empty_like(out)
                pi.pi_kv_attn(window, batch, c["q"].cuda(), want, ws, scale=c["scale"], window=w)
                torch.cuda.synchronize()
                assert torch.equal(out, want)
            else:
                check_sinks(c, min(w, 1000), min(s, 1000), out.cpu(), rows={0, 1, 20, 21, 100, 170})


# ------------------------------------------------------------------------------ drafted tokens

def run_verify(starts, tokens, target, draft, u, un, kv_len=None, *, offset=0, slack=0, stream=None):
    """Rows at `offset` elements past 16 bytes, `slack` elements apart."""
    def put(x):
        if x is None:
            return None
        rows, vocab = x.shape
        buf = torch.full((rows * (vocab + slack) + offset,), math.nan, device="cuda")
        view = buf[offset: offset + rows * (vocab + slack)].view(rows, vocab + slack)[:, :vocab]
        view.copy_(x)
        return view
    n = len(starts) - 1
    d = pi.make_kv_drafts(dev(starts), dev(tokens), put(target), put(draft), dev(u, torch.float32), dev(un, torch.float32))
    ws = torch.full((pi.pi_kv_verify_workspace_bytes(d),), 255, dtype=torch.uint8, device="cuda")
    ws[: 4 * 4096] = 0                       # (what else it holds does not matter)
    new = lambda: torch.full((n,), -77, dtype=torch.int32, device="cuda")
    accepted, nxt = new(), new()
    keep = None if kv_len is None else dev(kv_len)                          # in place
    pi.pi_kv_verify(d, accepted, nxt, ws, kv_len=keep, keep=keep, stream=stream)
    torch.cuda.synchronize()
    assert not bool(ws[: 4 * 4096].any()), "not ready for the next call"
    return accepted.tolist(), nxt.tolist(), [None] * n if keep is None else keep.tolist()


def verify_case(seed, counts, vocab, likeness=2.0, sharp=3.0):
    """Probabilities of a draft and a target near it, drafts drawn from the draft's."""
    gen = torch.Generator().manual_seed(seed)
    starts = [0]
    for n in counts:
        starts.append(starts[-1] + n)
    rows = max(starts[-1], 1)
    base = sharp * torch.randn((rows, vocab), generator=gen)
    draft = torch.softmax(base, -1)
    target = torch.softmax(base + torch.randn((rows, vocab), generator=gen) / likeness, -1)
    tokens = torch.multinomial(draft.double(), 1, generator=gen)[:, 0].roll(1).tolist()
    u, un = torch.rand(rows, generator=gen).tolist(), torch.rand(len(counts), generator=gen).tolist()
    return starts, tokens, target, draft, u, un


@pytest.mark.parametrize("with_draft", (True, False))
@pytest.mark.parametrize("vocab", (1, 2, 3, 255, 1023, 1024, 1025, 4097, 50001))
def test_verify(vocab, with_draft):
    announce(f"verify vocab={vocab} draft={with_draft}")
    rng = random.Random(vocab)
    counts = [rng.choice((0, 1, 2, 3, 5, 9)) for _ in range(40)]
    starts, tokens, target, draft, u, un = verify_case(vocab, counts, vocab)
    if not with_draft:
        draft = None
        u = [x * 0.3 for x in u]
    kv = [n + 50 for n in counts]
    for offset, slack in ((0, 0), (1, 3), (0, 4 - vocab % 4)):
        got = run_verify(starts, tokens, target, draft, u, un, kv, offset=offset, slack=slack)
        assert got == U.verify_reference(starts, tokens, target, draft, u, un, kv)
    assert run_verify(starts, tokens, target, draft, u, un)[:2] == got[:2]


def test_verify_many_drafts():
    """More drafts than lanes; all of them accepted in some requests."""
    announce("verify many drafts")
    counts = [64, 65, 66, 130, 200, 129, 1]
    starts, tokens, target, _, u, un = verify_case(5, counts, 300)
    u = [0.999 * x for x in u]
    for stop in (None, 0, 62, 63, 64, 65, 127, 128, 198):
        p = target.clone()
        q = target.clone()                   # the same: every draft is accepted
        if stop is not None:
            for a, b in zip(starts, starts[1:]):
                if a + stop + 1 < b:
                    p[a + stop, tokens[a + stop + 1]] = 0.0
        got = run_verify(starts, tokens, p, q, u, un)
        assert got == U.verify_reference(starts, tokens, p, q, u, un)
        want = [min(n - 1, n - 1 if stop is None else stop) for n in counts]
        assert got[0] == want


def test_verify_random_numbers_at_their_ends():
    announce("verify ends")
    for vocab in (5, 1030, 3000):
        starts, tokens, target, draft, u, _ = verify_case(vocab, [2] * 8, vocab)
        target[:, 0] = 0.0
        target[:, -1] = 0.0
        for un in (0.0, 1.0 - 2.0 ** -24, 1.0, 2.0, math.inf, math.nan, -1.0):
            got = run_verify(starts, tokens, target, draft, u, [un] * 8)
            want = U.verify_reference(starts, tokens, target, draft, u, [un] * 8)
            assert got == want, un
            w = [target[t + a] for t, a in zip(starts, got[0])]
            assert all(float(x[j]) > 0 for x, j in zip(w, got[1]))


def test_verify_odd_rows():
    """One-hot rows, rows without probability, infinities and NaN, tokens out of range, and row ranges out of bounds."""
    announce("verify odd rows")
    vocab = 2050
    starts, tokens, target, draft, u, un = verify_case(1, [3] * 12 + [1, 1], vocab)
    target[0:2] = 0.0
    target[0, tokens[1]] = 1.0               # a certain target that agrees, and one that does not
    target[1, (tokens[2] + 1) % vocab] = 1.0
    target[3] = draft[3]
    target[3, tokens[4]] = 0.0               # rejected, and nothing of the rest is above zero: the target's own
    target[6] = 0.0                          # no probability at all
    target[9, 5] = math.nan
    draft[12, 7] = math.nan
    target[15, tokens[16]] = math.nan
    draft[18, tokens[19]] = math.inf
    target[21, 3] = math.inf
    tokens[25], tokens[28] = vocab, -1
    u[30] = math.nan
    target[36] = -1.0
    target[36, 9] = 1.0
    draft[3, :] = draft[3] + 0.0
    for q in (draft, None):
        got = run_verify(starts, tokens, target, q, u, un)
        assert got == U.verify_reference(starts, tokens, target, q, u, un)
    assert got[1][12] == 9
    for s in ([0, 4, 2, 6], [-3, 0, 3, 6], [30, 33, 36, 99], [2 ** 31 - 1] * 4, [-2 ** 31, 2 ** 31 - 1, 0, 1]):
        got = run_verify(s, tokens, target, draft, u, un[:3], [7, 8, 9])
        assert got == U.verify_reference(s, tokens, target, draft, u, un[:3], [7, 8, 9]), s


def test_verify_leaves_the_targets_distribution():
    """With drafts drawn from q, the first token out is distributed as p: frequencies of 5 x 4096 requests against p,
    within five standard deviations."""
    announce("verify distribution")
    n, vocab, trials = 4096, 7, 5
    gen = torch.Generator().manual_seed(3)
    p = torch.softmax(torch.randn(vocab, generator=gen), 0)
    q = torch.softmax(torch.randn(vocab, generator=gen), 0)
    seen = torch.zeros(vocab)
    for _ in range(trials):
        x = torch.multinomial(q.double(), n, replacement=True, generator=gen)
        tokens = torch.stack([torch.zeros(n, dtype=torch.int64), x], 1).view(-1).tolist()
        starts = list(range(0, 2 * n + 1, 2))
        u, un = torch.rand(2 * n, generator=gen).tolist(), torch.rand(n, generator=gen).tolist()
        accepted, nxt, _ = run_verify(starts, tokens, p.expand(2 * n, vocab), q.expand(2 * n, vocab), u, un)
        first = torch.where(torch.tensor(accepted) > 0, x, torch.tensor(nxt))
        seen += torch.bincount(first, minlength=vocab)
    total = n * trials
    sigma = torch.sqrt(total * p * (1 - p))
    assert bool(((seen - total * p).abs() <= 5 * sigma).all())


def test_verify_calls_of_any_size_share_a_workspace():
    announce("verify shared workspace")
    cases = [verify_case(s, counts, vocab) for s, (counts, vocab) in enumerate((([3, 2, 5], 40000), ([2] * 300, 700), ([4], 9000), ([1, 3] * 20, 3000)))]
    sets = []
    for starts, tokens, target, draft, u, un in cases:
        sets.append(pi.make_kv_drafts(dev(starts), dev(tokens), target.cuda(), draft.cuda(), dev(u, torch.float32), dev(un, torch.float32)))
    ws = torch.zeros(max(pi.pi_kv_verify_workspace_bytes(d) for d in sets), dtype=torch.uint8, device="cuda")
    outs = [torch.full((2, d.n_req), -77, dtype=torch.int32, device="cuda") for _ in range(3) for d in sets]
    for out, d in zip(outs, sets * 3):
        pi.pi_kv_verify(d, out[0], out[1], ws)
    torch.cuda.synchronize()
    for i, out in enumerate(outs):
        want = U.verify_reference(*cases[i % len(cases)])
        assert (out[0].tolist(), out[1].tolist()) == want[:2], i


def test_verify_large():
    """The largest vocabulary, and the most requests."""
    announce("verify large")
    top = 1 << 22
    gen = torch.Generator().manual_seed(2)
    for vocab, counts in ((top, [3, 1]), (top - 1, [2])):
        rows = sum(counts)
        target, draft = (torch.rand((rows, vocab), generator=gen) for _ in range(2))
        starts = [sum(counts[:r]) for r in range(len(counts) + 1)]
        tokens = [vocab - 1] * rows
        u, un = [0.9] * rows, [0.7, 0.99][: len(counts)]
        assert run_verify(starts, tokens, target, draft, u, un) == U.verify_reference(starts, tokens, target, draft, u, un)
    args = verify_case(6, [1, 2, 0, 2] * 1024, 33)
    assert run_verify(*args) == U.verify_reference(*args)


# ------------------------------------------------------------------------------ pages

def device_state(st, in_place, slack=3):
    n, cols = len(st["table"]), len(st["table"][0])
    wide = torch.full((n, cols + slack), -7, dtype=torch.int32, device="cuda")
    wide[:, :cols] = dev(st["table"])
    new = lambda *s: torch.full(s, -77, dtype=torch.int32, device="cuda")
    d = dict(cached=dev(st["cached"]), free_ring=dev(st["ring"]), pool=dev(st["pool"]), block_table=wide[:, :cols], shares=dev(st["shares"]),
             counts=new(4), wide=wide, slack=slack)
    d["cached_next"] = d["cached"] if in_place else new(n)
    d["pool_next"] = d["pool"] if in_place else new(2)
    d["pages"] = pi.make_kv_pages(d["cached"], d["free_ring"], d["pool"], d["block_table"], st["page"], d["shares"], d["cached_next"],
                                  d["pool_next"], d["counts"])
    return d


def check_state(d, want):
    torch.cuda.synchronize()
    for name, value in want.items():
        assert d[name].cpu().tolist() == value, name
    assert bool((d["wide"][:, d["wide"].shape[1] - d["slack"]:] == -7).all())


PAGE_CASES = [(1, 16, 1), (1, 256, 5), (9, 16, 6), (64, 32, 40), (200, 16, 9), (1025, 64, 4), (1500, 16, 30), (2000, 32, 64), (4096, 16, 5), (4096, 16, 9), (3000, 16, 100)]


@pytest.mark.parametrize("in_place", (False, True))
@pytest.mark.parametrize("n_req,page,max_pages", PAGE_CASES)
def test_release(n_req, page, max_pages, in_place):
    for seed, free, bad in ((0, None, 0.0), (1, 2, 0.0), (2, None, 0.1), (3, 0, 0.0)):
        announce(f"release n_req={n_req} page={page} max_pages={max_pages} in_place={in_place} seed={seed}")
        st = U.pages_state(seed + n_req, n_req, page, max_pages, free=free, bad=bad)
        at, to = U.release_ranges(seed, st)
        if seed == 3:
            to = None
        want = U.release_reference(st, at, to)
        d = device_state(st, in_place)
        copies = torch.full((n_req, 2), -77, dtype=torch.int32, device="cuda")
        d["copies"] = copies
        pi.pi_kv_release(d["pages"], dev(at), None if to is None else dev(to), copies)
        check_state(d, want)


def test_release_of_pages_named_twice():
    """Tables that contradict their owners' counts: a page goes back once, nothing is touched out of bounds."""
    announce("release pages named twice")
    st = dict(cached=[64, 64, 64], table=[[3, 3, 4, 5], [3, 5, 99, -4], [6, 6, 6, 6]], ring=[0, 1, 2, 7, 8, 9, -1, -1, -1, -1], pool=[0, 6],
              shares=[0, 0, 0, 1, 0, 5, 0, 0, 0, 0], page=16)
    for at in ([0, 0, 0], [20, 20, 20], [64, 5, 33]):
        want = U.release_reference(st, at, None)
        d = device_state(st, False)
        d["copies"] = torch.zeros((3, 2), dtype=torch.int32, device="cuda")
        pi.pi_kv_release(d["pages"], dev(at), None, d["copies"])
        check_state(d, want)


@pytest.mark.parametrize("in_place", (False, True))
@pytest.mark.parametrize("n_req,page,max_pages", PAGE_CASES)
def test_fork(n_req, page, max_pages, in_place):
    for seed, free, bad in ((0, None, 0.0), (1, 2, 0.0), (2, None, 0.1), (3, 0, 0.0)):
        announce(f"fork n_req={n_req} page={page} max_pages={max_pages} in_place={in_place} seed={seed}")
        rng = random.Random(seed)
        st = U.pages_state(seed + n_req, n_req, page, max_pages, free=free, bad=bad, empty=0.5)
        n = rng.choice((0, 1, n_req, min(4096, 2 * n_req)))
        wild = (-1, n_req, 2 ** 31 - 1, -2 ** 31) if bad else (0,)
        src = [rng.choice((rng.randrange(n_req),) * 9 + wild) for _ in range(n)]
        dst = [rng.choice((rng.randrange(n_req),) * 9 + wild) for _ in range(n)]
        if not bad:
            dst = random.Random(seed).sample(range(n_req), min(n, n_req))
            src = src[: len(dst)]
        want = U.fork_reference(st, src, dst)
        d = device_state(st, in_place)
        d["copies"] = torch.full((len(src), 2), -77, dtype=torch.int32, device="cuda")
        pi.pi_kv_fork(d["pages"], dev(src), dev(dst), d["copies"])
        if not len(src):
            del want["copies"]
        check_state(d, want)


@pytest.mark.parametrize("n_kv,page,hd,dtype", [(1, 16, 64, "f16"), (3, 32, 128, "bf16"), (2, 256, 256, "f16"), (40, 64, 128, "f16")])
def test_copy(n_kv, page, hd, dtype):
    announce(f"copy n_kv={n_kv} page={page} hd={hd} {dtype}")
    gen = torch.Generator().manual_seed(page)
    n_pages = 23
    k = torch.randint(-2 ** 15, 2 ** 15, (n_pages, n_kv, page, hd), generator=gen, dtype=torch.int16)
    v = torch.randint(-2 ** 15, 2 ** 15, (n_pages, n_kv, hd, page), generator=gen, dtype=torch.int16)
    ids = torch.randperm(n_pages, generator=gen).tolist()
    for pairs in ([[ids[0], ids[1]]], [[ids[2 * i], ids[2 * i + 1]] for i in range(11)],
                  [[-1, -1], [ids[0], ids[5]], [ids[0], ids[6]], [n_pages, ids[7]], [ids[8], n_pages], [-5, ids[9]], [2 ** 31 - 1, 2 ** 31 - 1], [ids[3], ids[3]]],
                  [[-1, -1]] * 3000 + [[ids[1], ids[2]]]):
        kg, vg = k.cuda(), v.cuda()
        pi.pi_kv_copy(pi.make_kv_cache(kg.view(kv_util.DT[dtype]), vg.view(kv_util.DT[dtype])), dev(pairs))
        torch.cuda.synchronize()
        kw, vw = k.clone(), v.clone()
        for a, b in pairs:
            if 0 <= a < n_pages and 0 <= b < n_pages:
                kw[b], vw[b] = k[a], v[a]
        assert torch.equal(kg.cpu(), kw) and torch.equal(vg.cpu(), vw)


# ------------------------------------------------------------------------------ together

class Drafting:
    """Requests that draft, verify and fork over one pool of pages: step -> rotary append -> attention over a window and the
    first tokens -> probabilities -> verification -> rejected pages back -> copies.  Each request's drafts are fixed
    functions of its last token."""

    def __init__(self, n, drafts, page, max_pages, n_pages, n_q=4, n_kv=2, hd=64, vocab=61, window=40, sinks=5):
        self.n, self.rows, self.per, self.page, self.n_q, self.n_kv, self.hd, self.vocab = n, n * (1 + drafts), 1 + drafts, page, n_q, n_kv, hd, vocab
        self.window, self.sinks = window, sinks
        gen = torch.Generator().manual_seed(17)
        half = lambda *s: torch.zeros(s, dtype=torch.float16, device="cuda")
        ints = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
        self.embed = torch.randn((vocab, n_q + 2 * n_kv, hd), generator=gen).half().cuda()
        self.head = (torch.randn((n_q * hd, vocab), generator=gen) / 4).cuda()
        self.like = torch.softmax(torch.randn((vocab, vocab), generator=gen), -1).cuda()
        self.k, self.v = half(n_pages, n_kv, page, hd), half(n_pages, n_kv, hd, page)
        self.cached, self.fresh, self.ring, self.pool = ints(n), ints(n), torch.arange(n_pages, dtype=torch.int32, device="cuda"), dev([0, n_pages])
        self.table, self.shares = torch.full((n, max_pages), -1, dtype=torch.int32, device="cuda"), ints(n_pages)
        self.q_start, self.kv_len, self.slots, self.counts, self.dropped = ints(n + 1), ints(n), ints(self.rows), ints(4), ints(4)
        self.tokens, self.accepted, self.next, self.keep, self.copies = ints(self.rows), ints(n), ints(n), ints(n), ints(n, 2)
        self.q, self.out = half(self.rows, n_q, hd), half(self.rows, n_q, hd)
        self.target, self.draft = (torch.zeros((self.rows, vocab), device="cuda") for _ in range(2))
        self.u, self.un = torch.zeros(self.rows, device="cuda"), torch.zeros(n, device="cuda")
        self.tables = pi.make_kv_tables(self.cached, self.fresh, self.ring, self.pool, self.table, page, self.q_start, self.kv_len, self.cached,
                                        self.slots, self.pool, self.counts)
        self.pages = pi.make_kv_pages(self.cached, self.ring, self.pool, self.table, page, self.shares, self.cached, self.pool, self.dropped)
        self.cache = pi.make_kv_cache(self.k, self.v)
        self.batch = pi.make_kv_batch(self.table, self.q_start, self.kv_len, max_q=self.per, max_kv=max_pages * page)
        self.rope = pi.make_kv_rope(pi.pi_rope_frequencies(hd).cuda(), norm=True)
        self.ws = torch.empty(pi.pi_kv_attn_sinks_workspace_bytes(self.cache, self.batch, self.rows, n_q, window, sinks), dtype=torch.uint8, device="cuda")
        self.drafts = pi.make_kv_drafts(self.q_start, self.tokens, self.target, self.draft, self.u, self.un)
        self.vws = torch.zeros(pi.pi_kv_verify_workspace_bytes(self.drafts), dtype=torch.uint8, device="cuda")

    def step(self):
        """One step of all requests, each with its last token and its drafts."""
        last = self.next.long()
        rows = [last]
        for i in range(1, self.per):
            rows.append((rows[-1] * 5 + 3 * i) % self.vocab)
        self.tokens.copy_(torch.stack(rows, 1).view(-1))
        self.draft.copy_(self.like[self.tokens.long()])
        x = self.embed[self.tokens.long()]
        q, k, v = x.split((self.n_q, self.n_kv, self.n_kv), dim=1)
        pi.pi_kv_step(self.tables)
        pi.pi_kv_rope_append(self.cache, self.batch, self.rope, q, k, v, self.slots, self.q)
        pi.pi_kv_attn_sinks(self.cache, self.batch, self.q, self.out, self.ws, scale=1 / math.sqrt(self.hd), window=self.window, sinks=self.sinks)
        self.target.copy_(torch.softmax(self.out.view(self.rows, -1).float() @ self.head + 2 * torch.log(self.draft + 1e-6), -1))
        pi.pi_kv_verify(self.drafts, self.accepted, self.next, self.vws, kv_len=self.kv_len, keep=self.keep)
        pi.pi_kv_release(self.pages, self.keep, None, self.copies)
        pi.pi_kv_copy(self.cache, self.copies)

    def fork(self, src, dst):
        copies = torch.zeros((len(src), 2), dtype=torch.int32, device="cuda")
        pi.pi_kv_fork(self.pages, dev(src), dev(dst), copies)
        pi.pi_kv_copy(self.cache, copies)

    def cut(self, which, back):
        """Takes the last `back` positions of a request away; the page that it is cut inside of may have other owners."""
        at = self.cached.clone()
        at[which] -= back
        pi.pi_kv_release(self.pages, at, None, self.copies)
        pi.pi_kv_copy(self.cache, self.copies)

    def state(self):
        return {k: getattr(self, k).clone() for k in ("cached", "ring", "pool", "table", "shares", "tokens", "accepted", "next", "keep", "copies", "k",
                                                      "v", "q", "out", "target", "slots", "kv_len", "q_start", "dropped")}


@pytest.mark.parametrize("page", (16, 32))
def test_drafting_forking_steps_in_a_replayed_graph(page):
    """Replayed steps equal eager ones and follow the references; forks share pages, cuts copy them, and no page is lost."""
    announce(f"drafting steps page={page}")
    n, drafts, max_pages = 7, 4, 30
    rng = random.Random(page)
    gen = torch.Generator().manual_seed(page)
    a, b = (Drafting(n, drafts, page, max_pages, n * max_pages + 3) for _ in range(2))
    for st in (a, b):
        st.fresh.fill_(1 + drafts)
    # the captured call needs a warm library and handle; requests start from nothing either way
    saved = a.state()
    a.step()
    torch.cuda.synchronize()
    for name, value in saved.items():
        getattr(a, name).copy_(value)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.step()
    copied = cut = 0
    for it in range(60):
        u, un = torch.rand(a.rows, generator=gen).cuda() * 0.6, torch.rand(n, generator=gen).cuda()
        for st in (a, b):
            st.u.copy_(u)
            st.un.copy_(un)
        torch.cuda.synchronize()
        graph.replay()
        b.step()
        torch.cuda.synchronize()
        x, y = a.state(), b.state()
        for name in x:
            assert torch.equal(x[name], y[name]), (it, name)
        starts, kv = x["q_start"].tolist(), x["kv_len"].tolist()
        assert all(m > 0 for m in kv) and starts[-1] == a.rows
        want = U.verify_reference(starts, x["tokens"].tolist(), a.target.cpu(), a.draft.cpu(), u.cpu().tolist(), un.cpu().tolist(), kv)
        assert (x["accepted"].tolist(), x["next"].tolist(), x["keep"].tolist()) == want
        assert x["cached"].tolist() == want[2]
        cut += sum(k < m for k, m in zip(want[2], kv))
        U.check_owned(dict(cached=x["cached"].tolist(), table=x["table"].tolist(), ring=x["ring"].tolist(), pool=x["pool"].tolist(),
                           shares=x["shares"].tolist(), page=page))
        # attention of this step's rows that stay (the pages of the rejected ones may have been given away)
        case = dict(table=x["table"].tolist(), starts=starts, kv=kv, k=x["k"].cpu(), v=x["v"].cpu(), q=x["q"].cpu(), scale=1 / math.sqrt(a.hd))
        rows = {starts[r] for r in range(n)}
        ref, mag = U.sinks_reference(case, a.window, a.sinks, rows)
        tol = kv_util.attn_tolerance(ref, mag, torch.float16, a.hd)
        for t in rows:
            assert bool(((x["out"][t].cpu().double() - ref[t]).abs() <= tol[t]).all()), (it, t)
        if it % 5 == 4 or max(want[2]) > max_pages * page - 3 * (1 + drafts):
            # the longest ends, another one is continued in its place
            long = max(range(n), key=lambda r: want[2][r])
            src = rng.choice([r for r in range(n) if r != long])
            for st in (a, b):
                st.cut(long, int(st.cached[long]))
                st.fork([src], [long])
                st.next[long] = int(st.next[src])
            torch.cuda.synchronize()
            held = int(a.cached[src])
            assert int(a.cached[long]) == held and torch.equal(a.table, b.table)
            back = held % page + 5
            if held > back:                    # into the last page that both have
                for st in (a, b):
                    st.cut(long, back)
                torch.cuda.synchronize()
                old, new = a.copies[long].tolist()
                assert old >= 0 and int(a.table[long, (held - back) // page]) == new and torch.equal(a.k[old], a.k[new])
                copied += 1
    assert cut > 20 and copied > 0


def test_example_streams_past_its_window():
    """The example with rotary positions, a window and first tokens: replayed steps equal eager ones, attention equals the
    reference on the pages of the last step, and no page is lost."""
    announce("paged decode example, streaming")
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "paged_decode.py")
    spec = importlib.util.spec_from_file_location("paged_decode_streaming", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    cfg = synth.custom_config(1024, 2048, 64, layers=2, seed=3)
    opts = dict(head_dim=64, kv_heads=4, rope=True, window=20, sinks=3)
    graph, eager, _ = example.generate(cfg, 2, [5, 70, 33], 30, **opts)
    assert torch.isfinite(eager).all() and torch.equal(graph, eager)
    st = example.PagedStack(cfg, 2, 3, 120, **opts)
    gen = torch.Generator(device="cuda").manual_seed(1)
    free = []
    for fresh in ([5, 70, 33], *[[1, 1, 1]] * 25):
        st.fresh.copy_(dev(fresh))
        p = st.plan(sum(fresh), max(fresh), 120)
        real, seen = example.pi.pi_kv_attn_sinks, []

        def attn(cache, batch, q, out, ws, **kw):
            real(cache, batch, q, out, ws, **kw)
            seen.append((st.caches.index(cache), q.cpu(), out.cpu(), st.table.tolist(), st.q_start.tolist(), st.kv_len.tolist()))

        example.pi.pi_kv_attn_sinks = attn
        try:
            st.step(p, torch.randn((sum(fresh), cfg.d), generator=gen, device="cuda"))
        finally:
            example.pi.pi_kv_attn_sinks = real
        assert st.counts.tolist()[3] == 0
        l, q, out, table, starts, kv = seen[-1]
        k, v = (t.cpu() for t in st.caches[l]._keep)
        want, mag = U.sinks_reference(dict(table=table, starts=starts, kv=kv, k=k, v=v, q=q, scale=1 / 8), 20, 3)
        assert bool(((out.double() - want).abs() <= kv_util.attn_tolerance(want, mag, torch.float16, 64, partial=16.0)).all())
        U.check_owned(dict(cached=st.cached.tolist(), table=st.table.tolist(), ring=st.ring.tolist(), pool=st.pool.tolist(),
                           shares=st.pages._keep[4].tolist(), page=st.page))
        free.append(st.pool.tolist()[1])
    assert free[-1] >= free[1] - 3            # longer requests hold no more pages: the first one's, the window's, one in between


def test_on_another_stream():
    """Calls on a stream of their own, ordered behind work there, while the current stream is another one."""
    announce("other streams")
    side = torch.cuda.Stream()
    c = rope_case(1, ROPE_LENS, 4, 2, 64, 16, "f16", 64, 0, True)
    check_rope(c, run_rope(c, stream=side), torch.full(c["qkv"][:, :4].shape, 7.0))
    c = kv_util.attn_case(1, [(1, 300), (9, 70)], 4, 2, 64, 16, "f16")
    check_sinks(c, 30, 5, stream=side)
    args = verify_case(2, [3, 5, 1], 3000)
    assert run_verify(*args, stream=side.cuda_stream) == U.verify_reference(*args)
    st = U.pages_state(4, 30, 16, 9)
    at, to = U.release_ranges(4, st)
    d = device_state(st, True)
    d["copies"] = torch.zeros((30, 2), dtype=torch.int32, device="cuda")
    with torch.cuda.stream(side):
        pi.pi_kv_release(d["pages"], dev(at), dev(to), d["copies"])
    check_state(d, U.release_reference(st, at, to))


def test_calls_of_no_rows():
    announce("calls of no rows")
    k, v = torch.ones((4, 2, 16, 64), dtype=torch.float16, device="cuda"), torch.ones((4, 2, 64, 16), dtype=torch.float16, device="cuda")
    cache, none = pi.make_kv_cache(k, v), torch.empty((0, 2, 64), dtype=torch.float16, device="cuda")
    batch = pi.make_kv_batch(dev([[0], [1]]), dev([0, 0, 0]), dev([5, 0]), max_q=1, max_kv=16)
    rope = pi.make_kv_rope(pi.pi_rope_frequencies(64).cuda(), norm=True)
    q = torch.empty((0, 4, 64), dtype=torch.float16, device="cuda")
    pi.pi_kv_rope_append(cache, batch, rope, q, none, none, dev([]), q.clone())
    pi.pi_kv_attn_sinks(cache, batch, q, q.clone(), torch.empty(16, dtype=torch.uint8, device="cuda"), scale=1.0, window=3, sinks=2)
    pi.pi_kv_copy(cache, torch.empty((0, 2), dtype=torch.int32, device="cuda"))
    # rows that belong to no request, and requests without rows
    x, out = torch.ones((3, 2, 64), dtype=torch.float16, device="cuda"), torch.full((3, 4, 64), 7.0, dtype=torch.float16, device="cuda")
    pi.pi_kv_rope_append(cache, batch, rope, torch.ones_like(out), x + 1, x + 1, dev([0, 1, 2]), out)
    torch.cuda.synchronize()
    assert bool((k == 1).all()) and bool((v == 1).all()) and bool((out == 7).all())


def test_two_graphs_share_a_workspace():
    """Verification and attention captured twice over the same workspaces, replayed in turn with eager calls between."""
    announce("two graphs, one workspace")
    cases = [verify_case(s, [3, 2, 1, 4] * 5, vocab) for s, vocab in ((1, 9000), (2, 40001))]
    drafts = [pi.make_kv_drafts(dev(c[0]), dev(c[1]), c[2].cuda(), c[3].cuda(), dev(c[4], torch.float32), dev(c[5], torch.float32)) for c in cases]
    vws = torch.zeros(max(pi.pi_kv_verify_workspace_bytes(d) for d in drafts), dtype=torch.uint8, device="cuda")
    outs = [torch.zeros((2, 20), dtype=torch.int32, device="cuda") for _ in cases]
    attn = []
    for seed, lens in ((1, [(5, 9000), (1, 4000)]), (2, [(1, 20000), (2, 9000)])):
        c = kv_util.attn_case(seed, lens, 16, 2, 64, 16, "f16")
        batch = pi.make_kv_batch(dev(c["table"]), dev(c["starts"]), dev(c["kv"]), max_q=5, max_kv=20000)
        attn.append((pi.make_kv_cache(c["k"].cuda(), c["v"].cuda()), batch, c["q"].cuda(), torch.zeros_like(c["q"], device="cuda")))
    args = dict(window=5000, sinks=70)
    ws = torch.empty(max(pi.pi_kv_attn_sinks_workspace_bytes(a[0], a[1], len(a[2]), 16, *args.values()) for a in attn), dtype=torch.uint8, device="cuda")
    assert ws.numel() > 1 << 16               # key ranges are cut: partial sums pass through it

    def call(i):
        pi.pi_kv_verify(drafts[i], outs[i][0], outs[i][1], vws)
        pi.pi_kv_attn_sinks(*attn[i], ws, scale=0.125, **args)
    want = []
    for i in (0, 1):
        call(i)
        torch.cuda.synchronize()
        want.append((outs[i].clone(), attn[i][3].clone()))
        assert want[i][0].tolist() == [list(x) for x in U.verify_reference(*cases[i])[:2]]
    graphs = [torch.cuda.CUDAGraph() for _ in (0, 1)]
    for i, g in enumerate(graphs):
        with torch.cuda.graph(g):
            call(i)
    for it in range(6):
        for i in (it % 2, 1 - it % 2):
            outs[i].zero_()
            attn[i][3].zero_()
            graphs[i].replay()
            call(1 - i)
        torch.cuda.synchronize()
        for i in (0, 1):
            assert torch.equal(outs[i], want[i][0]) and torch.equal(attn[i][3], want[i][1]), (it, i)


@pytest.mark.parametrize("n", (700, 4000))          # in one launch, and in several
def test_release_of_long_lists_in_a_replayed_graph(n):
    announce(f"release in a graph, n={n}")
    states = [U.pages_state(s, n, 16, 70, forks=0.0 if s == 2 else 0.4) for s in range(4)]
    n_pages = max(len(s["ring"]) for s in states) + 5
    for s in states:                          # one size of pool for all
        extra = list(range(len(s["ring"]), n_pages))
        head, count = s["pool"]
        old = s["ring"]
        s["ring"] = [old[(head + i) % len(old)] for i in range(count)] + extra + [-1] * (len(old) - count)
        s["pool"], s["shares"] = [0, count + len(extra)], s["shares"] + [0] * len(extra)
    d = device_state(states[0], True)
    at, to, copies = (torch.zeros(x, dtype=torch.int32, device="cuda") for x in ((n,), (n,), (n, 2)))
    d["copies"] = copies

    def put(s, r):
        for name, value in (("cached", s["cached"]), ("free_ring", s["ring"]), ("pool", s["pool"]), ("block_table", s["table"]), ("shares", s["shares"])):
            d[name].copy_(dev(value))
        at.copy_(dev(r[0]))
        to.copy_(dev(r[1]))
    put(states[0], U.release_ranges(0, states[0]))
    pi.pi_kv_release(d["pages"], at, to, copies)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pi.pi_kv_release(d["pages"], at, to, copies)
    for it in range(8):
        s = states[it % 4]
        # lists of all lengths: everything at once, the usual ranges, and a token each
        r = (U.release_ranges(it, s), ([0] * n, [U.ALL] * n), ([max(c - 1, 0) for c in s["cached"]], [U.ALL] * n))[it % 3]
        put(s, r)
        graph.replay()
        check_state(d, U.release_reference(s, *r))


def test_host_tensors_are_refused():
    host, gpu = torch.zeros(3, dtype=torch.int32), torch.zeros(3, dtype=torch.int32, device="cuda")
    st = U.pages_state(1, 3, 16, 4)
    d = device_state(st, False)
    pairs = torch.zeros((3, 2), dtype=torch.int32, device="cuda")
    assert code(lambda: pi.pi_kv_release(d["pages"], host, None, pairs)) == _abi.PI_ERR_NULL
    assert code(lambda: pi.pi_kv_release(d["pages"], gpu, host, pairs)) == _abi.PI_ERR_NULL
    assert code(lambda: pi.pi_kv_release(d["pages"], gpu, None, pairs.cpu())) == _abi.PI_ERR_NULL
    assert code(lambda: pi.pi_kv_fork(d["pages"], gpu, host, pairs)) == _abi.PI_ERR_NULL
    k, v = torch.zeros((4, 1, 16, 64), dtype=torch.float16, device="cuda"), torch.zeros((4, 1, 64, 16), dtype=torch.float16, device="cuda")
    cache = pi.make_kv_cache(k, v)
    assert code(lambda: pi.pi_kv_copy(cache, pairs.cpu())) == _abi.PI_ERR_NULL
    freq = pi.pi_rope_frequencies(64)
    batch = pi.make_kv_batch(torch.zeros((3, 1), dtype=torch.int32, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda"), gpu, max_q=1, max_kv=1)
    x, s = torch.zeros((2, 1, 64), dtype=torch.float16, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    assert code(lambda: pi.pi_kv_rope_append(cache, batch, pi.make_kv_rope(freq), x, x, x, s, x.clone())) == _abi.PI_ERR_NULL
    assert code(lambda: pi.pi_kv_rope_append(cache, batch, pi.make_kv_rope(freq.cuda()), x, x.cpu(), x, s, x.clone())) == _abi.PI_ERR_NULL
    assert code(lambda: pi.make_kv_drafts(gpu, s, torch.zeros((2, 5), device="cuda"), None, torch.zeros(2), torch.zeros(2, device="cuda"))) == _abi.PI_ERR_NULL


# ------------------------------------------------------------------------------ requests that a step refused

@pytest.mark.parametrize("vocab", (61, 1024, 5000))          # in one workgroup of a request and in several
@pytest.mark.parametrize("with_draft", (True, False))
def test_verify_of_refused_requests(vocab, with_draft):
    """Fewer keys than rows, or none: nothing is accepted, the last token is the next one again, and all positions stay."""
    announce(f"verify refused vocab={vocab} draft={with_draft}")
    counts = [3, 1, 0, 5, 2, 1, 0, 70, 4, 5]
    kv = [0, 0, 0, 4, 2, -1, 9, 0, -2 ** 31, 5]
    starts, tokens, target, draft, u, un = verify_case(vocab, counts, vocab)
    u = [0.3 * x for x in u]
    tokens[starts[1]] = -9                   # whatever token it was
    got = run_verify(starts, tokens, target, draft if with_draft else None, u, un, kv)
    assert got == U.verify_reference(starts, tokens, target, draft if with_draft else None, u, un, kv)
    for r in (0, 1, 3, 5, 7, 8):
        assert (got[0][r], got[1][r], got[2][r]) == (0, tokens[starts[r]], U.ALL), r
    assert got[2][2] == U.ALL and got[1][2] == -1 and got[2][6] == 9 and got[2][9] == 5 - 4 + got[0][9]
    # without lengths a refused request is one as any other
    got = run_verify(starts, tokens, target, draft if with_draft else None, u, un)
    assert got == U.verify_reference(starts, tokens, target, draft if with_draft else None, u, un)


@pytest.mark.parametrize("page", (16, 32))
def test_refused_requests_keep_their_cache_in_a_replayed_graph(page):
    """Steps over a pool that runs out, eager and replayed: a request without pages for its tokens keeps its positions and
    pages and asks again, and goes on once another one has ended."""
    announce(f"refused requests page={page}")
    n, drafts, max_pages = 6, 4, 12
    rng = random.Random(page)
    gen = torch.Generator().manual_seed(page)
    a, b = (Drafting(n, drafts, page, max_pages, 19) for _ in range(2))
    for st in (a, b):
        st.fresh.fill_(1 + drafts)
    saved = a.state()
    a.step()
    torch.cuda.synchronize()
    for name, value in saved.items():
        getattr(a, name).copy_(value)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.step()
    waits, refused, again = [0] * n, 0, 0
    for it in range(80):
        u, un = torch.rand(a.rows, generator=gen).cuda() * 0.3, torch.rand(n, generator=gen).cuda()
        for st in (a, b):
            st.u.copy_(u)
            st.un.copy_(un)
        torch.cuda.synchronize()
        before = a.state()
        graph.replay()
        b.step()
        torch.cuda.synchronize()
        x, y = a.state(), b.state()
        for name in x:
            assert torch.equal(x[name], y[name]), (it, name)
        listed = lambda s, name: s[name].cpu().tolist()
        # the chain by its references
        step = kv_util.step_reference(listed(before, "cached"), [1 + drafts] * n, listed(before, "ring"), listed(before, "pool"),
                                      listed(before, "table"), page, a.rows)
        assert (listed(x, "kv_len"), listed(x, "q_start"), listed(x, "slots")) == (step["kv_len"], step["q_start"], step["slots"])
        tokens = listed(x, "tokens")
        want = U.verify_reference(step["q_start"], tokens, a.target.cpu(), a.draft.cpu(), u.cpu().tolist(), un.cpu().tolist(), step["kv_len"])
        assert (listed(x, "accepted"), listed(x, "next"), listed(x, "keep")) == want
        state = dict(cached=step["cached_next"], table=step["block_table"], ring=step["free_ring"], pool=step["pool_next"],
                     shares=listed(before, "shares"), page=page)
        after = U.release_reference(state, want[2], None)
        for name, key in (("cached", "cached_next"), ("table", "block_table"), ("ring", "free_ring"), ("pool", "pool_next"), ("shares", "shares")):
            assert listed(x, name) == after[key], (it, name)
        U.check_owned(dict(cached=after["cached_next"], table=after["block_table"], ring=after["free_ring"], pool=after["pool_next"],
                           shares=after["shares"], page=page))
        for r in range(n):
            if step["kv_len"][r]:
                again += waits[r] > 0
                waits[r] = 0
                assert after["cached_next"][r] == int(before["cached"][r]) + 1 + want[0][r]
                continue
            refused += 1
            waits[r] += 1
            held = kv_util.ceil_div(int(before["cached"][r]), page)
            assert after["cached_next"][r] == int(before["cached"][r]) and int(x["next"][r]) == int(before["next"][r])
            assert torch.equal(x["table"][r, :held], before["table"][r, :held])
            for t in ("k", "v"):
                ids = before["table"][r, :held].long()
                assert torch.equal(x[t][ids], before[t][ids])
        if max(waits) > 2 or max(after["cached_next"]) > (max_pages - 2) * page:
            # the longest of those that were served ends
            long = max((r for r in range(n) if not waits[r]), key=lambda r: after["cached_next"][r], default=0)
            for st in (a, b):
                st.cut(long, int(st.cached[long]))
                st.next[long] = rng.randrange(a.vocab) if st is a else a.next[long]
            torch.cuda.synchronize()
    assert refused >= 10 and again > 3       # (the pool ran out, and requests went on)


@pytest.mark.parametrize("window", (1, 2))
def test_example_streams_with_the_smallest_windows(window):
    """A token that sees itself and the first tokens only, or one token more: requests keep their lengths, and
    attention equals the reference."""
    announce(f"paged decode example, window {window}")
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "paged_decode.py")
    spec = importlib.util.spec_from_file_location("paged_decode_small_windows", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    cfg = synth.custom_config(1024, 2048, 64, layers=1, seed=3)
    opts = dict(head_dim=64, kv_heads=4, rope=True, window=window, sinks=3)
    lengths = [5, 70, 32, 1]
    graph, eager, _ = example.generate(cfg, 1, lengths, 20, **opts)
    assert torch.isfinite(eager).all() and torch.equal(graph, eager)
    st = example.PagedStack(cfg, 1, len(lengths), 120, **opts)
    gen = torch.Generator(device="cuda").manual_seed(1)
    real, seen = example.pi.pi_kv_attn_sinks, []

    def attn(cache, batch, q, out, ws, **kw):
        real(cache, batch, q, out, ws, **kw)
        seen.append((q.cpu(), out.cpu(), st.table.tolist(), st.q_start.tolist(), st.kv_len.tolist()))

    example.pi.pi_kv_attn_sinks = attn
    try:
        for it in range(20):
            fresh = lengths if it == 0 else [1] * len(lengths)
            st.fresh.copy_(dev(fresh))
            st.step(st.plan(sum(fresh), max(fresh), 120), torch.randn((sum(fresh), cfg.d), generator=gen, device="cuda"))
            q, out, table, starts, kv = seen[-1]
            assert kv == [m + it for m in lengths] and st.cached.tolist() == kv
            k, v = (t.cpu() for t in st.caches[0]._keep)
            want, mag = U.sinks_reference(dict(table=table, starts=starts, kv=kv, k=k, v=v, q=q, scale=1 / 8), window, 3)
            assert bool(((out.double() - want).abs() <= kv_util.attn_tolerance(want, mag, torch.float16, 64, partial=16.0)).all())
            U.check_owned(dict(cached=st.cached.tolist(), table=st.table.tolist(), ring=st.ring.tolist(), pool=st.pool.tolist(),
                               shares=st.pages._keep[4].tolist(), page=st.page))
    finally:
        example.pi.pi_kv_attn_sinks = real


@pytest.mark.parametrize("heads,hd", [((4, 2), 64), ((80, 80), 128)])      # values in tiles of 16 tokens and of 64
@pytest.mark.parametrize("n_req", (3, 64, 65, 500, 4096))
def test_rope_append_writes_all_of_a_row_or_nothing(heads, hd, n_req):
    """Row starts that decrease: a row's query, key and value are written together or not at all, and those of no
    range's rows are not."""
    announce(f"rope append of decreasing starts {heads} n_req={n_req}")
    rng = random.Random(n_req)
    rows = 480 if hd == 128 else 200
    c = rope_case(9, [(rows - 4, 900)], *heads, hd, 64, "f16", hd, 0, False)
    n_q, n_kv = heads
    c["kv"] = [rng.randint(1, 5000) for _ in range(n_req)]
    kinds = [[rng.randint(-3, rows + 3) for _ in range(n_req + 1)], [r * rows // n_req for r in range(n_req, -1, -1)],
             [(r * 2 % n_req) * rows // n_req for r in range(n_req + 1)], [0, *(rng.randint(0, rows) for _ in range(n_req))]]
    if n_req == 3:
        kinds += [[0, 4, 2, 6], [5, 100, 60, rows], [0, rows, 0, rows], [100, 0, rows, 50]]
    total = c["rows"]
    for starts in kinds:
        got = run_rope(c, starts=starts)
        ranges = [(x, y) for x, y in zip(starts, starts[1:]) if 0 <= x < y <= total]
        query = (got[0] != 7.0).flatten(1).any(1)
        for t, slot in enumerate(c["slots"]):
            if not any(x <= t < y for x, y in ranges):
                assert not bool(query[t]), (starts[:9], t)
            if not 0 <= slot < c["k"].shape[0] * c["page"]:
                continue
            p, i = divmod(slot, c["page"])
            key = bool((got[1][p, :, i] != c["k"][p, :, i]).any())
            value = bool((got[2][p, :, :, i] != c["v"][p, :, :, i]).any())
            assert key == value == bool(query[t]), (starts[:9], t, key, value)


# ------------------------------------------------------------------------------ masks at every place of a block

def plant(c, window, sinks):
    """Keys that the single token of a request does not see score far above those that it sees, and their values are large;
    such places lie at every offset of the blocks at the window's and the keys' ends."""
    page, n_kv = c["page"], c["k"].shape[1]
    for r, m in enumerate(c["kv"]):
        t = c["starts"][r]
        if c["starts"][r + 1] - t != 1:
            continue
        q = c["q"][t].view(n_kv, -1, c["q"].shape[2]).float().sum(1).to(c["q"].dtype)
        low = max(m - window, 0)
        held = kv_util.ceil_div(m, page) * page
        for j in [*range(min(sinks, low), low), *range(m, held)]:
            p = c["table"][r][j // page]
            c["k"][p, :, j % page] = q
            c["v"][p, :, :, j % page] = 1000.0


@pytest.mark.parametrize("dtype", ("f16", "bf16"))
@pytest.mark.parametrize("sinks", (0, 5, 39))
@pytest.mark.parametrize("n_q,n_kv,hd,page", [(4, 4, 64, 16), (4, 2, 128, 32), (2, 2, 256, 64)])
def test_no_score_outside_the_masks_counts(n_q, n_kv, hd, page, sinks, dtype):
    """For the kernels of every number of waves and the one of chunks: lengths that put both ends of the window at
    every offset of a block of 32 keys."""
    few, many = [200 + i for i in range(33)], [90 + i % 33 for i in range(300)]
    cases = [("four waves", [(1, m) for m in few], None), ("more waves", [(1, m + 100) for m in few], 400), ("one wave", [(1, m) for m in many], 256),
             ("cut", [(1, m + 2500) for m in few], 9000), ("beside a chunk", [(300, 300)] + [(1, m) for m in few], None)]
    for name, lens, max_kv in cases:
        for window in {"cut": (2200,), "more waves": (7, 250)}.get(name, (7, 45)):
            announce(f"masks {name} heads={n_q}/{n_kv} hd={hd} page={page} {dtype} window={window} sinks={sinks}")
            c = kv_util.attn_case(hd + sinks, lens, n_q, n_kv, hd, page, dtype)
            plant(c, window, sinks)
            rows = {c["starts"][r] for r, (n, _) in enumerate(lens) if n == 1}
            pick = rows if name != "cut" else set(sorted(rows)[::4])
            got = run_sinks(c, window, sinks, max_kv=max_kv)
            assert torch.isfinite(got).all() and float(got[sorted(rows)].abs().max()) < 100, "a masked key counts"
            check_sinks(c, window, sinks, got, rows=pick)


@pytest.mark.parametrize("dtype", ("f16", "bf16"))
@pytest.mark.parametrize("n_q,n_kv,hd,page,lens,window,sinks", [
    (16, 16, 64, 16, [(1, m) for m in range(2, 70, 2)], 20, 5),                  # few short ranges
    (24, 12, 128, 32, [(1, 2 + r % 150) for r in range(90)], 60, 33),            # many short ranges
    (8, 2, 64, 16, [(1, 9000), (1, 3), (1, 5200), (2, 700)], 3000, 130),         # cut and joined
    (4, 2, 256, 64, [(1, 12), (2, 500), (1, 300), (3, 40)], 90, 4),
    (4, 4, 128, 16, [(150, 150)] + [(1, 2 + 9 * r) for r in range(30)], 50, 4)])  # beside a chunk
def test_sinks_single_tokens_lose_no_bits_of_their_weights(n_q, n_kv, hd, page, lens, window, sinks, dtype):
    """Off by no more than the output's own rounding and what 32-bit scores leave."""
    announce(f"sinks precision heads={n_q}/{n_kv} hd={hd} page={page} {dtype} window={window} sinks={sinks}")
    c = kv_util.attn_case(hd + len(lens), lens, n_q, n_kv, hd, page, dtype)
    kv_util.past_end(c, math.nan)
    got = run_sinks(c, window, sinks)
    rows = [c["starts"][r] + i for r, (n, _) in enumerate(lens) if n <= 3 for i in range(n)]
    want, mag = U.sinks_reference(c, window, sinks, set(rows))
    tol = kv_util.attn_tolerance_of_few_rows(want, mag, c["q"].dtype, hd)[rows]
    err = (got.double() - want).abs()[rows]
    assert bool((err <= tol).all()), f"worst {float((err / tol).max()):.3f} of the tolerance"
