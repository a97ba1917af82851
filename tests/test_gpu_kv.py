"""The paged-cache operators on the GPU against plain 64-bit references: block tables, append, attention, and
the three together in a replayed graph."""
import math
import random

import pytest
import torch

import activation_sparse_ffn_rank_amd as pi
from activation_sparse_ffn_rank_amd import _kv
import kv_util
from gpu_util import announce

pytestmark = pytest.mark.gpu


def dev(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device="cuda")


# ------------------------------------------------------------------------------ tables

def run_step(cached, fresh, ring, pool, table, page, max_tokens, in_place=False, slack=0):
    n = len(cached)
    wide = torch.full((n, len(table[0]) + slack), -7, dtype=torch.int32, device="cuda")
    st = dict(cached=dev(cached), fresh=dev(fresh), free_ring=dev(ring), pool=dev(pool))
    st["block_table"] = wide[:, : len(table[0])]
    st["block_table"].copy_(dev(table))
    new = lambda m: torch.full((m,), -77, dtype=torch.int32, device="cuda")
    st.update(q_start=new(n + 1), kv_len=new(n), slots=new(max_tokens), counts=new(4))
    st["cached_next"] = st["cached"] if in_place else new(n)
    st["pool_next"] = st["pool"] if in_place else new(2)
    tables = pi.make_kv_tables(st["cached"], st["fresh"], st["free_ring"], st["pool"], st["block_table"], page, st["q_start"],
                               st["kv_len"], st["cached_next"], st["slots"], st["pool_next"], st["counts"])
    pi.pi_kv_step(tables)
    torch.cuda.synchronize()
    assert slack == 0 or bool((wide[:, len(table[0]):] == -7).all())
    return st, tables


def check_step(st, want):
    for name, value in want.items():
        assert st[name].cpu().tolist() == value, name


@pytest.mark.parametrize("in_place", (False, True))
@pytest.mark.parametrize("n_req,page,max_pages,max_tokens,free", [
    (1, 16, 1, 1, None), (1, 256, 3, 700, None), (7, 16, 5, 100, None), (64, 32, 9, 300, None), (64, 16, 40, 257, 20),
    (333, 128, 4, 4000, 100), (1025, 64, 3, 5000, None), (1500, 16, 70, 40000, None), (4096, 16, 6, 70000, 3000), (200, 16, 9, 30, 0)])
def test_step(n_req, page, max_pages, max_tokens, free, in_place):
    announce(f"kv step n_req={n_req} page={page} max_pages={max_pages} max_tokens={max_tokens} free={free} in_place={in_place}")
    for seed in range(2):
        args = kv_util.step_inputs(seed, n_req, page, max_pages, max_tokens, free=free)
        want = kv_util.step_reference(*args, page, max_tokens)
        st, _ = run_step(*args, page, max_tokens, in_place, slack=seed * 3)
        check_step(st, want)


def test_step_no_tokens_and_all_ended():
    for kinds in ((0,), (-1,), (-9,)):
        announce(f"kv step kinds={kinds}")
        args = kv_util.step_inputs(3, 50, 16, 8, 10, kinds=kinds)
        st, _ = run_step(*args, 16, 10)
        check_step(st, kv_util.step_reference(*args, 16, 10))


def test_step_lengths_out_of_bounds():
    announce("kv step lengths out of bounds")
    args = kv_util.step_inputs(4, 300, 32, 6, 2000, in_bounds=False)
    st, _ = run_step(*args, 32, 2000)
    check_step(st, kv_util.step_reference(*args, 32, 2000))


def test_steps_in_place_follow_the_rules():
    """Forty steps on their own state (in place, replayed as a graph): every page stays in one place."""
    page, max_pages, n, max_tokens = 16, 12, 24, 400
    rng = random.Random(5)
    n_pages = 150
    cached, table, ring, pool = [0] * n, [[-1] * max_pages for _ in range(n)], list(range(n_pages)), [0, n_pages]
    announce("kv step in place, 40 steps")
    st, tables = run_step(cached, [0] * n, ring, pool, table, page, max_tokens, in_place=True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pi.pi_kv_step(tables)
    for _ in range(40):
        fresh = [rng.choice((1, 1, 1, 0, rng.randint(1, 40), -1)) for _ in range(n)]
        st["fresh"].copy_(dev(fresh))
        want = kv_util.step_reference(st["cached"].tolist(), fresh, st["free_ring"].tolist(), st["pool"].tolist(),
                                      st["block_table"].tolist(), page, max_tokens)
        graph.replay()
        torch.cuda.synchronize()
        check_step(st, want)
        head, count = st["pool"].tolist()
        free = [st["free_ring"].tolist()[(head + j) % n_pages] for j in range(count)]
        held = [p for row, c in zip(st["block_table"].tolist(), st["cached"].tolist()) for p in row[: kv_util.ceil_div(c, page)]]
        assert sorted(free + held) == list(range(n_pages))


# ------------------------------------------------------------------------------ append

@pytest.mark.parametrize("tokens,n_kv,hd,page,dtype,fused", [
    (1, 1, 64, 16, "f16", False), (3, 2, 128, 16, "bf16", True), (16, 32, 128, 16, "f16", True), (63, 3, 256, 32, "bf16", False),
    (64, 2, 64, 256, "f16", True), (65, 8, 64, 64, "bf16", True), (500, 4, 128, 128, "f16", False), (1031, 2, 256, 64, "f16", True),
    (777, 5, 64, 32, "bf16", False)])
def test_append(tokens, n_kv, hd, page, dtype, fused):
    announce(f"kv append tokens={tokens} n_kv={n_kv} hd={hd} page={page} {dtype} fused={fused}")
    gen = torch.Generator().manual_seed(tokens)
    rng = random.Random(tokens)
    n_pages = kv_util.ceil_div(tokens, page) * 2 + 3
    for scattered in (False, True):
        # runs of neighbouring slots from odd places on, or slots in any order; some rows without one
        perm = torch.randperm(n_pages * page, generator=gen)[:tokens] if scattered else torch.arange(tokens) + rng.randrange(page)
        slots = perm.to(torch.int32)
        for t in range(0, tokens, 11):
            if tokens > 1:
                slots[t] = (-1, n_pages * page, -2 ** 31, 2 ** 31 - 1)[t // 11 % 4]
        k0 = torch.randn((n_pages, n_kv, page, hd), generator=gen).to(kv_util.DT[dtype])
        v0 = torch.randn((n_pages, n_kv, hd, page), generator=gen).to(kv_util.DT[dtype])
        if fused:
            qkv = torch.randn((tokens, 3 * n_kv + 1, hd), generator=gen).to(kv_util.DT[dtype]).cuda()
            k, v = qkv[:, 1: 2 * n_kv: 2] if n_kv > 1 else qkv[:, 1:2], qkv[:, 2 * n_kv: 3 * n_kv]
        else:
            k, v = (torch.randn((tokens, n_kv, hd), generator=gen).to(kv_util.DT[dtype]).cuda() for _ in range(2))
        kg, vg = k0.cuda(), v0.cuda()
        pi.pi_kv_append(pi.make_kv_cache(kg, vg), k[:, :n_kv], v, slots.cuda())
        torch.cuda.synchronize()
        kc, vc = k.cpu(), v.cpu()
        for t, s in enumerate(slots.tolist()):
            if 0 <= s < n_pages * page:
                k0[s // page, :, s % page] = kc[t]
                v0[s // page, :, :, s % page] = vc[t]
        assert torch.equal(kg.cpu().view(torch.int16), k0.view(torch.int16)), "keys"
        assert torch.equal(vg.cpu().view(torch.int16), v0.view(torch.int16)), "values"


# ------------------------------------------------------------------------------ attention

def run_attn(c, window=0, *, max_q=None, max_kv=None, stream=None, wide=False):
    """The call on a case's tensors; `wide`: queries, outputs and tables are slices of wider rows."""
    n = [b - a for a, b in zip(c["starts"], c["starts"][1:])]
    dt, (rows, n_q, hd) = c["q"].dtype, c["q"].shape
    table = dev(c["table"])
    if wide:
        buf = torch.full((rows, n_q + 3, hd + 8), 7.0, dtype=dt, device="cuda")
        q, o_all = buf[:, 1: n_q + 1, :hd], torch.full((rows + 2, n_q + 5, hd + 16), 7.0, dtype=dt, device="cuda")
        q.copy_(c["q"].cuda())
        out = o_all[1: rows + 1, 2: n_q + 2, 8: hd + 8]
        t_all = torch.full((table.shape[0], table.shape[1] + 5), 1 << 30, dtype=torch.int32, device="cuda")
        t_all[:, : table.shape[1]] = table
        table = t_all[:, : table.shape[1]]
    else:
        q, out = c["q"].cuda(), torch.full((rows, n_q, hd), 7.0, dtype=dt, device="cuda")
    cache = pi.make_kv_cache(c["k"].cuda(), c["v"].cuda())
    batch = pi.make_kv_batch(table, dev(c["starts"]), dev(c["kv"]), max_q=max_q or max(1, max(n)),
                             max_kv=max(c["kv"]) if max_kv is None else max_kv)
    ws = torch.full((pi.pi_kv_attn_workspace_bytes(cache, batch, rows, n_q),), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    pi.pi_kv_attn(cache, batch, q, out, ws, scale=c["scale"], window=window, stream=stream)
    torch.cuda.synchronize()
    if wide:
        got = out.clone()
        out.fill_(7.0)
        assert bool((o_all == 7.0).all()), "written outside the output's rows"
        return got
    return out


def attn(c, window=0, **kw):
    got = run_attn(c, window, **kw)
    return got.cpu()


def check_attn(c, window=0, got=None, **kw):
    got = attn(c, window, **kw) if got is None else got
    want, mag = kv_util.attn_reference(c["q"], c["k"], c["v"], c["table"], c["starts"], c["kv"], c["scale"], window)
    tol = kv_util.attn_tolerance(want, mag, c["q"].dtype, c["q"].shape[2])
    err = (got.double() - want).abs()
    assert torch.isfinite(got).all()
    assert bool((err <= tol).all()), f"worst {float((err / tol).max()):.3f} of the tolerance"
    return got


HEADS = ((4, 4, 64), (2, 2, 128), (16, 1, 64), (10, 2, 128), (8, 1, 256), (3, 1, 128), (40, 2, 64), (2, 2, 256))


@pytest.mark.parametrize("dtype", ("f16", "bf16"))
@pytest.mark.parametrize("page", (16, 32, 64, 128, 256))
@pytest.mark.parametrize("n_q,n_kv,hd", HEADS)
def test_attn_single_tokens(n_q, n_kv, hd, page, dtype):
    lens = [(1, m) for m in (1, 2, 15, 16, 17, 31, 33, 64, 127, 300, 517)]
    announce(f"kv attn single tokens heads={n_q}/{n_kv} hd={hd} page={page} {dtype}")
    c = kv_util.attn_case(page + hd, lens, n_q, n_kv, hd, page, dtype)
    kv_util.past_end(c, math.nan)
    check_attn(c)


@pytest.mark.parametrize("window", (0, 1, 20, 150))
@pytest.mark.parametrize("n_q,n_kv,hd,page,dtype", [(4, 4, 64, 16, "f16"), (2, 2, 128, 64, "bf16"), (16, 1, 64, 32, "bf16"),
                                                    (10, 2, 128, 16, "f16"), (8, 1, 256, 256, "f16"), (2, 2, 256, 16, "bf16")])
def test_attn_ragged_chunks(n_q, n_kv, hd, page, dtype, window):
    """Prompts without a past, chunks behind one, drafts and single tokens in one call."""
    lens = [(1, 70), (5, 5), (0, 40), (33, 90), (2, 259), (130, 130), (1, 1), (47, 300), (0, 0), (64, 64)]
    announce(f"kv attn ragged heads={n_q}/{n_kv} hd={hd} page={page} {dtype} window={window}")
    c = kv_util.attn_case(window + hd, lens, n_q, n_kv, hd, page, dtype)
    kv_util.past_end(c, math.nan)
    check_attn(c, window, wide=True)


@pytest.mark.parametrize("n_q,n_kv,hd,page,dtype", [(4, 4, 64, 64, "bf16"), (2, 2, 128, 128, "f16"), (16, 1, 64, 16, "f16"),
                                                    (8, 1, 256, 32, "bf16"), (10, 2, 128, 16, "bf16")])
def test_attn_chunk_of_many_tiles(n_q, n_kv, hd, page, dtype):
    lens = [(200, 1000), (321, 321), (1, 900), (257, 640)]
    announce(f"kv attn chunk heads={n_q}/{n_kv} hd={hd} page={page} {dtype}")
    c = kv_util.attn_case(hd, lens, n_q, n_kv, hd, page, dtype)
    kv_util.past_end(c, math.inf)
    check_attn(c)
    check_attn(c, 100)


@pytest.mark.parametrize("n_q,n_kv,hd,page,dtype,window", [
    (8, 2, 64, 16, "f16", 0), (4, 1, 128, 32, "bf16", 0), (2, 1, 256, 64, "f16", 0), (16, 1, 64, 256, "bf16", 0),
    (2, 2, 128, 16, "f16", 2500), (5, 1, 128, 16, "bf16", 3000)])
def test_attn_long_ranges(n_q, n_kv, hd, page, dtype, window):
    """Key ranges that are cut and joined, for single tokens and for drafts of several."""
    for lens in ([(1, 4097), (1, 3), (1, 2900)], [(5, 4000), (3, 513), (1, 1)]):
        announce(f"kv attn long heads={n_q}/{n_kv} hd={hd} page={page} {dtype} window={window} lens={lens}")
        c = kv_util.attn_case(hd + page, lens, n_q, n_kv, hd, page, dtype)
        kv_util.past_end(c, math.nan)
        got = check_attn(c, window)
        assert torch.equal(got, attn(c, window)), "the result depends on timing"
        # bounds looser than the lengths change the grid, not the values
        check_attn(c, window, max_q=70, max_kv=9000)


def test_attn_many_requests():
    lens = [(1, 1 + 37 * r % 200) for r in range(300)]
    announce("kv attn 300 requests")
    c = kv_util.attn_case(1, lens, 2, 1, 64, 16, "f16")
    check_attn(c)
    c = kv_util.attn_case(2, [(r % 4, max(r % 4, 7 * r % 90)) for r in range(150)], 4, 2, 64, 16, "bf16")
    check_attn(c)


@pytest.mark.parametrize("bad", (math.nan, math.inf, -math.inf))
@pytest.mark.parametrize("n_q,n_kv,hd,page,dtype", [(4, 4, 64, 16, "f16"), (8, 1, 128, 64, "bf16"), (2, 1, 256, 32, "f16")])
def test_attn_masked_places_have_no_effect(n_q, n_kv, hd, page, dtype, bad):
    """Infinite and NaN keys and values: tokens that do not see them come out as if they were zero."""
    for lens, window in (([(90, 200), (3, 45)], 0), ([(90, 200), (1, 190)], 33), ([(300, 700)], 0), ([(300, 700)], 70)):
        announce(f"kv attn masked {bad} heads={n_q}/{n_kv} hd={hd} page={page} {dtype} lens={lens} window={window}")
        c = kv_util.attn_case(7, lens, n_q, n_kv, hd, page, dtype)
        kv_util.past_end(c, bad)
        m = c["kv"][0]
        spots = (m - 40, m - 41, m - 7, m - lens[0][0] // 2, 100)
        seen_by = torch.zeros(lens[0][0], dtype=torch.bool)
        for j in spots:
            pos = torch.arange(m - lens[0][0], m)
            seen_by |= (pos >= j) & ((pos - j < window) if window else torch.ones_like(pos, dtype=torch.bool))
            for t in ("k", "v"):
                x = c[t][c["table"][0][j // page]]
                (x[:, j % page] if t == "k" else x[:, :, j % page]).zero_()
        want, mag = kv_util.attn_reference(c["q"], c["k"], c["v"], c["table"], c["starts"], c["kv"], c["scale"], window)
        tol = kv_util.attn_tolerance(want, mag, c["q"].dtype, hd)
        for which in ("k", "v"):
            d = dict(c, k=c["k"].clone(), v=c["v"].clone())
            for j in spots:
                x = d[which][c["table"][0][j // page]]
                if which == "k":
                    x[:, j % page] = bad
                else:
                    x[:, ::3, j % page] = bad
            got = attn(d, window)
            for t in range(lens[0][0]):
                if not seen_by[t]:
                    assert bool(((got[t].double() - want[t]).abs() <= tol[t]).all()), (which, t)
            if which == "v":
                clean = torch.arange(hd) % 3 != 0              # columns of V without the bad values
                e = (got[: lens[0][0]].double() - want[: lens[0][0]]).abs()
                assert bool((e[..., clean] <= tol[: lens[0][0]][..., clean]).all())
                # a token that sees such a value passes it on
                assert not torch.isfinite(got[lens[0][0] - 1][:, 0]).any() or not bool(seen_by[-1])


def test_attn_rows_without_keys():
    """No keys at all, fewer keys than new tokens, and table entries out of range."""
    announce("kv attn rows without keys")
    c = kv_util.attn_case(9, [(3, 0), (6, 2), (1, 40), (20, 100), (1, 600)], 4, 2, 64, 16, "bf16")
    kv_util.past_end(c, math.nan)
    c["table"][3][2], c["table"][3][5] = -1, c["k"].shape[0]
    c["table"][4][0], c["table"][4][7], c["table"][4][8] = 2 ** 31 - 1, -2 ** 31, -1
    got = check_attn(c)
    assert got[:7].abs().max() == 0
    c["table"][2] = [-1] * len(c["table"][2])
    got = check_attn(c)
    assert got[9].abs().max() == 0


def test_attn_extreme_scores():
    """Scores far apart: one key carries everything; equal large scores share; the range is not exceeded."""
    for dtype in ("f16", "bf16"):
        announce(f"kv attn extreme {dtype}")
        c = kv_util.attn_case(3, [(1, 300), (40, 300)], 2, 1, 64, 32, dtype)
        c["q"] *= 40
        want, mag = kv_util.attn_reference(c["q"], c["k"], c["v"], c["table"], c["starts"], c["kv"], c["scale"], 0)
        got = attn(c)
        tol = kv_util.attn_tolerance(want, mag, c["q"].dtype, 64, partial=8.0 * 40)
        assert bool(((got.double() - want).abs() <= tol).all())
        c["q"].zero_()
        check_attn(c)


def test_attn_bounds_cut_lengths():
    """New tokens past max_q are not written; keys past max_kv are not read."""
    announce("kv attn bounds")
    c = kv_util.attn_case(4, [(1, 300), (9, 200)], 4, 4, 64, 16, "f16")
    got = attn(c, max_q=4, max_kv=300)
    assert bool((got[5:] == 7.0).all())
    want, mag = kv_util.attn_reference(c["q"], c["k"], c["v"], c["table"], c["starts"], c["kv"], c["scale"], 0)
    tol = kv_util.attn_tolerance(want, mag, torch.float16, 64)
    assert bool(((got.double() - want).abs()[:5] <= tol[:5]).all())
    d = kv_util.attn_case(5, [(1, 300)], 4, 4, 64, 16, "f16")
    got = attn(d, max_kv=150)
    want, mag = kv_util.attn_reference(d["q"], d["k"], d["v"], d["table"], [0, 1], [150], d["scale"], 0)
    assert bool(((got.double() - want).abs() <= kv_util.attn_tolerance(want, mag, torch.float16, 64)).all())


def test_attn_row_ranges_out_of_bounds():
    """A request whose rows lie outside the packed queries is left out; the others are computed."""
    announce("kv attn row ranges")
    c = kv_util.attn_case(6, [(2, 30), (3, 50)], 2, 2, 64, 16, "f16")
    want, mag = kv_util.attn_reference(c["q"], c["k"], c["v"], c["table"], c["starts"], c["kv"], c["scale"], 0)
    tol = kv_util.attn_tolerance(want, mag, torch.float16, 64)
    for starts, ok in (([0, 2, 9], slice(0, 2)), ([-4, 2, 5], slice(2, 5)), ([0, 2, 1], slice(0, 2))):
        d = dict(c, starts=starts)
        got = attn(d, max_q=3)
        assert bool(((got.double() - want).abs()[ok] <= tol[ok]).all())
        rest = torch.ones(5, dtype=torch.bool)
        rest[ok] = False
        assert bool((got[rest] == 7.0).all())


def test_attn_offsets_past_32_bits():
    """A pool of more than 2^32 elements: pages at its end are read and written in their place."""
    page, n_kv, hd = 256, 8, 256
    n_pages = (1 << 32) // (page * n_kv * hd) + 40
    announce(f"kv attn pool of {n_pages} pages")
    c = kv_util.attn_case(8, [(1, 700), (3, 300)], 8, 8, hd, page, "bf16")
    small = c["k"].shape[0]
    k = torch.zeros((n_pages, n_kv, page, hd), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros((n_pages, n_kv, hd, page), dtype=torch.bfloat16, device="cuda")
    at = n_pages - small
    cache = pi.make_kv_cache(k, v)
    rows = small * page
    kt = c["k"].transpose(1, 2).reshape(rows, n_kv, hd).cuda()
    vt = c["v"].permute(0, 3, 1, 2).reshape(rows, n_kv, hd).cuda()
    pi.pi_kv_append(cache, kt, vt, torch.arange(rows, dtype=torch.int32, device="cuda") + at * page)
    table = [[p + at if p >= 0 else p for p in row] for row in c["table"]]
    batch = pi.make_kv_batch(dev(table), dev(c["starts"]), dev(c["kv"]), max_q=3, max_kv=700)
    out = torch.empty(c["q"].shape, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(pi.pi_kv_attn_workspace_bytes(cache, batch, 4, 8), dtype=torch.uint8, device="cuda")
    pi.pi_kv_attn(cache, batch, c["q"].cuda(), out, ws, scale=c["scale"])
    torch.cuda.synchronize()
    assert torch.equal(k[at:].cpu(), c["k"]) and torch.equal(v[at:].cpu(), c["v"]) and not bool(k[:at].any())
    check_attn(c, got=out.cpu())


# ------------------------------------------------------------------------------ together

def test_steps_in_a_replayed_graph_on_another_stream():
    """Tables, append and attention captured once and replayed with new lengths, against eager calls on
    copies of the same state and against the reference."""
    n, page, max_pages, n_q, n_kv, hd, max_tokens, n_pages = 6, 16, 20, 4, 2, 64, 64, 90
    gen = torch.Generator().manual_seed(1)
    rng = random.Random(1)
    announce("kv steps in a graph")

    def state():
        ints = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
        st = dict(cached=ints(n), fresh=ints(n), ring=torch.arange(n_pages, dtype=torch.int32, device="cuda"),
                  pool=dev([3, n_pages]), table=torch.full((n, max_pages), -1, dtype=torch.int32, device="cuda"),
                  q_start=ints(n + 1), kv_len=ints(n), slots=ints(max_tokens), counts=ints(4),
                  k=torch.zeros((n_pages, n_kv, page, hd), dtype=torch.float16, device="cuda"),
                  v=torch.zeros((n_pages, n_kv, hd, page), dtype=torch.float16, device="cuda"),
                  qkv=torch.zeros((max_tokens, n_q + 2 * n_kv, hd), dtype=torch.float16, device="cuda"),
                  out=torch.zeros((max_tokens, n_q, hd), dtype=torch.float16, device="cuda"))
        st["tables"] = pi.make_kv_tables(st["cached"], st["fresh"], st["ring"], st["pool"], st["table"], page, st["q_start"],
                                         st["kv_len"], st["cached"], st["slots"], st["pool"], st["counts"])
        st["cache"] = pi.make_kv_cache(st["k"], st["v"])
        st["batch"] = pi.make_kv_batch(st["table"], st["q_start"], st["kv_len"], max_q=24, max_kv=max_pages * page)
        st["ws"] = torch.empty(pi.pi_kv_attn_workspace_bytes(st["cache"], st["batch"], max_tokens, n_q), dtype=torch.uint8,
                               device="cuda")
        return st

    def step(st, stream=None):
        pi.pi_kv_step(st["tables"], stream)
        pi.pi_kv_append(st["cache"], st["qkv"][:, n_q: n_q + n_kv], st["qkv"][:, n_q + n_kv:], st["slots"], stream)
        pi.pi_kv_attn(st["cache"], st["batch"], st["qkv"][:, :n_q], st["out"], st["ws"], scale=0.125, stream=stream)

    a, b = state(), state()
    side = torch.cuda.Stream()
    step(a)                                   # no tokens: builds nothing, changes nothing
    step(b)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(a)
    for it in range(12):
        fresh = [rng.choice((1, 1, 1, 0, rng.randint(1, 24), -1)) for _ in range(n)] if it else [5, 20, 1, 0, 7, 3]
        while sum(max(f, 0) for f in fresh) > max_tokens:
            fresh = [min(f, 5) for f in fresh]
        qkv = torch.randn((max_tokens, n_q + 2 * n_kv, hd), generator=gen).half().cuda()
        for st in (a, b):
            st["fresh"].copy_(dev(fresh))
            st["qkv"].copy_(qkv)
        torch.cuda.synchronize()
        graph.replay()
        step(b, side)
        torch.cuda.synchronize()
        for name in ("cached", "ring", "pool", "table", "q_start", "kv_len", "slots", "counts", "k", "v", "out"):
            assert torch.equal(a[name], b[name]), (it, name)
        rows = int(a["counts"][0])
        want, mag = kv_util.attn_reference(a["qkv"][:rows, :n_q].cpu(), a["k"].cpu(), a["v"].cpu(), a["table"].tolist(),
                                           a["q_start"].tolist(), a["kv_len"].tolist(), 0.125, 0)
        tol = kv_util.attn_tolerance(want, mag, torch.float16, hd)
        assert bool(((a["out"][:rows].cpu().double() - want).abs() <= tol).all()), it


# ------------------------------------------------------------------------------ the kernels' variants by size

@pytest.mark.parametrize("n_q,n_kv,hd,page,dtype,n_req,most", [
    (13, 13, 64, 16, "f16", 70, 250), (56, 56, 128, 64, "bf16", 20, 18), (24, 12, 128, 16, "f16", 60, 256),
    (8, 4, 256, 32, "bf16", 140, 90)])
def test_attn_many_short_ranges(n_q, n_kv, hd, page, dtype, n_req, most):
    """More workgroups than the chip holds, of at most 256 keys each."""
    announce(f"kv attn many short heads={n_q}/{n_kv} hd={hd} page={page} {dtype} n_req={n_req} most={most}")
    rng = random.Random(most)
    c = kv_util.attn_case(3, [(1, rng.choice((0, 1, most, rng.randint(1, most)))) for _ in range(n_req - 1)] + [(1, most)], n_q, n_kv,
                          hd, page, dtype)
    kv_util.past_end(c, math.nan)
    check_attn(c)
    check_attn(c, 17, max_kv=256)


@pytest.mark.parametrize("n_q,n_kv,hd,page,dtype,lens", [
    (16, 16, 64, 16, "f16", [(1, 513)]), (4, 2, 64, 256, "bf16", [(1, 1024), (1, 0), (1, 31), (1, 700)]),
    (32, 32, 128, 16, "bf16", [(1, 512), (1, 1)]), (35, 7, 128, 32, "f16", [(2, 300), (3, 257), (1, 64), (0, 9)]),
    (64, 64, 128, 64, "f16", [(1, 1000), (1, 5), (1, 999)]), (40, 40, 64, 16, "bf16", [(1, 2000), (1, 1500), (1, 100), (1, 33)])])
def test_attn_few_short_ranges(n_q, n_kv, hd, page, dtype, lens):
    """Short ranges with a compute unit for each: read by one workgroup of more waves."""
    announce(f"kv attn few short heads={n_q}/{n_kv} hd={hd} page={page} {dtype} lens={lens}")
    c = kv_util.attn_case(hd, lens, n_q, n_kv, hd, page, dtype)
    kv_util.past_end(c, math.inf)
    check_attn(c)
    check_attn(c, 40)


@pytest.mark.parametrize("n_q,n_kv,hd,page,dtype,window", [
    (4, 2, 64, 16, "f16", 0), (2, 2, 128, 32, "bf16", 0), (8, 1, 128, 64, "f16", 3000), (4, 1, 256, 16, "bf16", 0),
    (6, 2, 256, 256, "f16", 900)])
def test_attn_long_single_tokens_beside_chunks(n_q, n_kv, hd, page, dtype, window):
    """Prompt chunks, single tokens whose key ranges are cut, and requests without either, in one call."""
    lens = [(1, 4500), (180, 400), (1, 2900), (0, 50), (1, 1), (3, 1700), (1, 0), (1, 3000)]
    announce(f"kv attn long single tokens beside chunks heads={n_q}/{n_kv} hd={hd} page={page} {dtype} window={window}")
    c = kv_util.attn_case(page, lens, n_q, n_kv, hd, page, dtype)
    kv_util.past_end(c, math.nan)
    got = check_attn(c, window, wide=True)
    assert torch.equal(got, attn(c, window, wide=True)), "the result depends on timing"


@pytest.mark.parametrize("bad", (math.nan, math.inf))
def test_attn_masked_values_beside_chunks(bad):
    """A value that is not finite reaches exactly the tokens that see its key, chunks and single tokens alike."""
    lens, window = [(1, 300), (150, 400), (1, 90), (1, 120), (1, 40)], 60
    for hd, page, dtype in ((64, 16, "bf16"), (128, 64, "f16")):
        announce(f"kv attn masked values beside chunks hd={hd} page={page} {dtype} {bad}")
        c = kv_util.attn_case(5, lens, 2, 1, hd, page, dtype)
        kv_util.past_end(c, bad)
        spots = {0: (239, 240, 100), 1: (251, 300, 5, 399), 2: (10,), 3: (119,)}
        for r, js in spots.items():
            for j in js:
                c["v"][c["table"][r][j // page]][:, 7, j % page] = bad
        got = attn(c, window).double()
        clean = dict(c, v=torch.nan_to_num(c["v"], nan=0.0, posinf=0.0))
        want, mag = kv_util.attn_reference(c["q"], c["k"], clean["v"], c["table"], c["starts"], c["kv"], c["scale"], window)
        tol = kv_util.attn_tolerance(want, mag, c["q"].dtype, hd)
        for r, (n, m) in enumerate(lens):
            for i in range(n):
                t, pos = c["starts"][r] + i, m - n + i
                hit = any(pos - window < j <= pos for j in spots.get(r, ()))
                rest = torch.arange(hd) != 7
                assert bool(((got[t] - want[t]).abs() <= tol[t])[:, rest].all()), (r, i)
                assert bool(torch.isfinite(got[t][:, 7]).all()) == (not hit), (r, i)
                assert hit or bool(((got[t] - want[t]).abs() <= tol[t])[:, 7].all()), (r, i)


def test_attn_windows_past_all_positions():
    """The largest window is no window, for tokens before position 0 too."""
    announce("kv attn window 2^31 - 1")
    for lens in ([(6, 2), (1, 40), (9, 0)], [(40, 30), (1, 5)]):
        c = kv_util.attn_case(2, lens, 4, 2, 64, 16, "f16")
        kv_util.past_end(c, math.nan)
        got = check_attn(c, 2 ** 31 - 1)
        assert torch.equal(got, attn(c, 0))


def test_tensors_of_other_devices_are_refused():
    """Host tensors in a call on device pages; and calls without rows, which need no workspace."""
    announce("kv refusals of host tensors")
    c = kv_util.attn_case(1, [(1, 20), (2, 30)], 4, 2, 64, 16, "f16")
    k, v, q = c["k"].cuda(), c["v"].cuda(), c["q"].cuda()
    cache = pi.make_kv_cache(k, v)
    batch = pi.make_kv_batch(dev(c["table"]), dev(c["starts"]), dev(c["kv"]), max_q=2, max_kv=30)
    ws = torch.empty(pi.pi_kv_attn_workspace_bytes(cache, batch, 3, 4), dtype=torch.uint8, device="cuda")
    out, new, slots = torch.empty_like(q), torch.zeros((3, 2, 64), dtype=torch.float16, device="cuda"), dev([0, 1, 2])

    def refused(fn):
        with pytest.raises(pi.PiError) as e:
            fn()
        return e.value.code
    assert refused(lambda: pi.make_kv_cache(k, c["v"])) == -1
    assert refused(lambda: pi.make_kv_batch(dev(c["table"]), dev(c["starts"]), torch.tensor(c["kv"], dtype=torch.int32), max_q=2,
                                            max_kv=30)) == -1
    assert refused(lambda: pi.pi_kv_append(cache, new, new, slots.cpu())) == -1
    assert refused(lambda: pi.pi_kv_append(cache, new.cpu(), new, slots)) == -1
    assert refused(lambda: pi.pi_kv_attn(cache, batch, c["q"], out, ws, scale=0.1)) == -1
    assert refused(lambda: pi.pi_kv_attn(cache, batch, q, out.cpu(), ws, scale=0.1)) == -1
    assert refused(lambda: pi.pi_kv_attn(cache, batch, q, out, ws.cpu(), scale=0.1)) == -1
    assert refused(lambda: pi.pi_kv_attn(cache, batch, q, out, None, scale=0.1)) == -5
    pi.pi_kv_attn(cache, batch, q[:0], out[:0], None, scale=0.1)
    pi.pi_kv_append(cache, new[:0], new[:0], slots[:0])
    torch.cuda.synchronize()
    assert torch.equal(k.cpu(), c["k"]) and torch.equal(v.cpu(), c["v"])


@pytest.mark.parametrize("n_q,n_kv,hd,page,dtype", [(4, 4, 64, 16, "f16"), (2, 1, 128, 16, "bf16"), (2, 2, 256, 16, "bf16"),
                                                    (2, 2, 128, 32, "f16")])
def test_attn_masked_values_far_into_the_table(n_q, n_kv, hd, page, dtype):
    """Values that are not finite at the end of more pages than one read of the table holds: tokens before them are as if
    they were not there."""
    n, m = 300, 5000
    announce(f"kv attn masked values far into the table heads={n_q}/{n_kv} hd={hd} page={page} {dtype}")
    c = kv_util.attn_case(11, [(n, m)], n_q, n_kv, hd, page, dtype)
    kv_util.past_end(c, math.nan)
    want, mag = kv_util.attn_reference(c["q"], c["k"], c["v"], c["table"], c["starts"], c["kv"], c["scale"], 0)
    tol = kv_util.attn_tolerance(want, mag, c["q"].dtype, hd, keys=m)
    spot = m - 100
    c["v"][c["table"][0][spot // page]][:, ::5, spot % page] = math.inf
    got = attn(c)
    before = n - 100
    assert bool(((got[:before].double() - want[:before]).abs() <= tol[:before]).all())
    clean = torch.arange(hd) % 5 != 0
    assert bool(((got.double() - want).abs() <= tol)[..., clean].all())
    assert not torch.isfinite(got[before:][..., ~clean]).any()


# ------------------------------------------------------------------------------ tables longer than one read of 64 entries

def look_at(c, r, i, j):
    """Token i of request r asks for key j: its score there is about 12, and elsewhere of the order of 1."""
    n_kv, page, hd = c["k"].shape[1:]
    key = c["k"][c["table"][r][j // page], :, j % page].float() * (12 / math.sqrt(hd))
    c["q"][c["starts"][r] + i] = key.repeat_interleave(c["q"].shape[1] // n_kv, 0).to(c["q"].dtype)


def shared_pages_case(seed, lens, n_q, n_kv, hd, page, dtype):
    """Requests whose tables name the same pages, each in an order of its own (long caches in little memory)."""
    most = max(m for _, m in lens)
    c = kv_util.attn_case(seed, [(0, most)] + [(n, 0) for n, _ in lens], n_q, n_kv, hd, page, dtype, extra_pages=0)
    rng, cols = random.Random(seed), kv_util.ceil_div(most, page)
    c["table"] = [rng.sample(range(cols), kv_util.ceil_div(m, page)) for _, m in lens]
    c["table"] = [row + [-1] * (cols - len(row)) for row in c["table"]]
    c["starts"], c["kv"] = c["starts"][1:], [m for _, m in lens]
    return c


def attn_uncut(c, window=0):
    """The call, on bounds with which no key range is cut: an item, or a quarter of one, has more pages than one read of
    its table."""
    n, (n_pages, n_kv, page, hd) = [b - a for a, b in zip(c["starts"], c["starts"][1:])], c["k"].shape
    dtype = {"f16": pi.PI_KV_F16, "bf16": pi.PI_KV_BF16}[c["dtype"]]
    cache = _kv.pi_kv_cache(n_pages, n_kv, page, hd, dtype, 16, 16)
    batch = _kv.pi_kv_batch(len(n), len(c["table"][0]), max(n), max(c["kv"]), len(c["table"][0]), 16, 16, 16)
    assert pi.pi_kv_attn_workspace_bytes(cache, batch, *c["q"].shape[:2]) == 16, "key ranges are cut"
    return attn(c, window)


def reference_of(c, picks, heads, window):
    """(rows, query heads, output, tolerance) of tokens `picks` = (request, token), for some kv heads."""
    group = c["q"].shape[1] // c["k"].shape[1]
    # a token is a request of one token, without the keys behind it
    kv = [c["kv"][r] - (c["starts"][r + 1] - c["starts"][r]) + i + 1 for r, i in picks]
    rows, qh = [c["starts"][r] + i for r, i in picks], [h * group + g for h in heads for g in range(group)]
    want, mag = kv_util.attn_reference(c["q"][rows][:, qh], c["k"][:, heads], c["v"][:, heads], [c["table"][r] for r, _ in picks],
                                       list(range(len(picks) + 1)), kv, c["scale"], window)
    return rows, qh, want, kv_util.attn_tolerance(want, mag, c["q"].dtype, c["q"].shape[2], partial=20.0, keys=max(kv))


def check_some(c, got, picks, heads, window=0):
    rows, qh, want, tol = reference_of(c, picks, heads, window)
    err = (got[rows][:, qh].double() - want).abs()
    assert bool((err <= tol).all()), f"worst {float((err / tol).max()):.3f} of the tolerance"


@pytest.mark.parametrize("n_q,n_kv,hd,page,dtype,m", [
    (64, 64, 256, 16, "bf16", 1500), (64, 64, 256, 32, "f16", 2500), (100, 100, 128, 16, "f16", 1500), (100, 100, 128, 32, "bf16", 2500),
    (150, 150, 64, 16, "bf16", 1500), (150, 150, 64, 64, "f16", 4600)])
def test_attn_chunk_on_a_table_of_several_reads(n_q, n_kv, hd, page, dtype, m):
    """A chunk whose tiles walk more than 64 pages, uncut; then with a missing page behind the 64th; then with values
    that are not finite, which take the tiles through their keys a second time."""
    n, heads, cols = 300, [0, n_kv // 2, n_kv - 1], kv_util.ceil_div(m, page)
    announce(f"kv attn chunk, {cols} pages, heads={n_q}/{n_kv} hd={hd} page={page} {dtype}")
    c = kv_util.attn_case(m, [(n, m)], n_q, n_kv, hd, page, dtype)
    kv_util.past_end(c, math.nan)
    picks = [(0, i) for i in (0, 1, 40, 127, 128, 190, 199, 200, 255, 256, 298, 299)]
    for at, (_, i) in enumerate(picks):            # keys of the first read, and of the second one
        look_at(c, 0, i, (3 * at + 1) * page + at if at % 2 else 65 * page + 3 * at)
    for window in (0, 65 * page):
        check_some(c, attn_uncut(c, window), picks, heads, window)

    gone = dict(c, table=[list(c["table"][0])])
    gone["table"][0][66] = -1
    for window in (0, m - 67 * page - 20):         # seen by the first tokens, and not by the last ones
        check_some(gone, attn_uncut(gone, window), picks, heads, window)

    rows, qh, want, tol = reference_of(c, picks, heads, 0)
    spot = m - 100
    bad = dict(c, v=c["v"].clone())
    bad["v"][c["table"][0][spot // page]][:, ::5, spot % page] = math.inf
    got = attn_uncut(bad)[rows][:, qh]
    near = (got.double() - want).abs() <= tol
    clean = torch.arange(hd) % 5 != 0
    before = torch.tensor([m - n + i < spot for _, i in picks])
    assert bool(near[before].all()) and bool(near[..., clean].all())
    assert not torch.isfinite(got[~before][..., ~clean]).any()


@pytest.mark.parametrize("n_q,n_kv,hd,page,dtype,n_req,m", [
    (64, 64, 128, 16, "f16", 64, 4400), (128, 64, 64, 16, "bf16", 96, 4400), (64, 64, 256, 16, "f16", 32, 4400),
    (40, 40, 128, 32, "bf16", 103, 8500)])
@pytest.mark.parametrize("chunk", (1, 200))
def test_attn_single_tokens_on_tables_of_several_reads(n_q, n_kv, hd, page, dtype, n_req, m, chunk):
    """Single tokens, alone or beside a chunk, whose waves walk more than 64 pages each, with a missing page behind the
    64th of a wave."""
    lens = [(chunk, m)] + [(1, m - 7 * r % 90) for r in range(1, n_req)]
    announce(f"kv attn {n_req} requests on {m} keys, chunk={chunk} heads={n_q}/{n_kv} hd={hd} page={page} {dtype}")
    c = shared_pages_case(m, lens, n_q, n_kv, hd, page, dtype)
    picks = [(0, chunk - 1)] + [(r, 0) for r in (1, 2, 3, n_req // 2, n_req - 3, n_req - 2, n_req - 1)]
    for r, i in picks:
        part = (kv_util.ceil_div(lens[r][1], 4) + 31) & ~31             # keys of a wave
        assert part > 65 * page + 8
        look_at(c, r, i, r % 3 * part + 65 * page + 8)
    for r in range(2, n_req, 3):
        c["table"][r][64] = c["table"][r][(m - 90) // 4 // page + 67] = -1
    for window in (0, m - 66 * page):              # (starting behind column 64 too)
        check_some(c, attn_uncut(c, window), picks, [0, n_kv - 1], window)


def test_attn_most_requests():
    """As many requests as a step may have, some of them long enough to be cut, the last one among them."""
    lens = [(1, 1 + 37 * r % 40) for r in range(pi._kv.PI_KV_MAX_REQ)]
    for r in (0, 63, 64, 2000, 4095):
        lens[r] = (1, 5000 - r % 1000)
    lens[77], lens[4000] = (0, 33), (1, 0)
    announce(f"kv attn {len(lens)} requests")
    for n_q, n_kv, hd, dtype in ((2, 1, 64, "f16"), (4, 4, 128, "bf16")):
        c = shared_pages_case(n_q, lens, n_q, n_kv, hd, 16, dtype)
        picks = [(r, 0) for r in (0, 1, 62, 63, 64, 65, 78, 1999, 2000, 2001, 3999, 4000, 4001, 4094, 4095)]
        for r, i in picks:
            if lens[r][1]:
                look_at(c, r, i, lens[r][1] * 5 // 8)
        got = attn(c)
        assert got[c["starts"][4000]].abs().max() == 0
        check_some(c, got, picks, list(range(n_kv)))
        assert torch.equal(got, attn(c)), "the result depends on timing"


# ------------------------------------------------------------------------------ precision of single tokens

@pytest.mark.parametrize("dtype", ("f16", "bf16"))
@pytest.mark.parametrize("n_q,n_kv,hd,page,lens", [
    (16, 16, 64, 16, [(1, m) for m in range(2, 34)]),                           # few short ranges
    (24, 12, 128, 32, [(1, 2 + r % 50) for r in range(90)]),                    # many short ranges
    (8, 2, 64, 16, [(1, 4000), (1, 3), (1, 1200), (2, 700)]),                   # cut and joined
    (4, 2, 256, 64, [(1, 12), (2, 5), (1, 300), (3, 40)]),
    (4, 4, 128, 16, [(150, 150)] + [(1, 2 + r) for r in range(30)])])           # beside a chunk
def test_attn_single_tokens_lose_no_bits_of_their_weights(n_q, n_kv, hd, page, lens, dtype):
    """Off by no more than the output's own rounding and what 32-bit scores leave."""
    announce(f"kv attn precision heads={n_q}/{n_kv} hd={hd} page={page} {dtype}")
    c = kv_util.attn_case(hd + len(lens), lens, n_q, n_kv, hd, page, dtype)
    kv_util.past_end(c, math.nan)
    got = check_attn(c)
    want, mag = kv_util.attn_reference(c["q"], c["k"], c["v"], c["table"], c["starts"], c["kv"], c["scale"], 0)
    tol = kv_util.attn_tolerance_of_few_rows(want, mag, c["q"].dtype, hd)
    rows = [c["starts"][r] + i for r, (n, _) in enumerate(lens) if n <= 3 for i in range(n)]
    err = (got.double() - want).abs()[rows]
    assert bool((err <= tol[rows]).all()), f"worst {float((err / tol[rows]).max()):.3f} of the tolerance"


@pytest.mark.parametrize("dtype", ("f16", "bf16"))
@pytest.mark.parametrize("n_q,n_kv,hd,page,lens", [
    (4, 2, 64, 16, [(1, 40), (1, 300), (1, 3000)]), (2, 2, 128, 64, [(1, 33), (3, 900)]), (2, 1, 256, 32, [(1, 700)]),
    (2, 1, 128, 16, [(150, 500), (1, 200)])])
def test_attn_infinite_values_keep_their_sign(n_q, n_kv, hd, page, lens, dtype):
    """A token that sees an infinite value gets that infinity, as its weight is above zero."""
    announce(f"kv attn infinite values heads={n_q}/{n_kv} hd={hd} page={page} {dtype} lens={lens}")
    c = kv_util.attn_case(hd, lens, n_q, n_kv, hd, page, dtype)
    for r, (n, m) in enumerate(lens):
        for at, d in ((0, 3), ((m - n) // 2, 5), (m - n, 9)):
            c["v"][c["table"][r][at // page]][:, d, at % page] = math.inf
            c["v"][c["table"][r][at // page]][:, d + 1, at % page] = -math.inf
    got = attn(c)
    for d in (3, 5, 9):
        assert bool((got[..., d] == math.inf).all()) and bool((got[..., d + 1] == -math.inf).all()), d
    finite = torch.ones(hd, dtype=torch.bool)
    finite[[3, 4, 5, 6, 9, 10]] = False
    assert torch.isfinite(got[..., finite]).all()


def test_attn_overlapping_row_ranges_take_no_old_partial_sums():
    """Row ranges that overlap ask for more items than a call has: what is left out is not joined from what the
    workspace held before."""
    announce("kv attn overlapping row ranges")
    n_req = 4096
    for group in (1, 4):
        c = kv_util.attn_case(group, [(1, 60000)], group, 1, 64, 64, "f16")
        # every other request has the one row there is; all have few keys, but for the last of them
        c["starts"] = [r % 2 for r in range(n_req + 1)]
        c["kv"] = [1 + r % 30 for r in range(n_req)]
        c["kv"][n_req - 2] = 60000
        c["table"] = c["table"] * n_req
        got = run_attn(c, max_q=1)                 # (on a workspace of NaN)
        assert torch.isfinite(got).all()
