"""Plain 64-bit references of the paged-cache operators and their inputs (no test functions here)."""
from __future__ import annotations

import math
import random

import torch

DT = {"f16": torch.float16, "bf16": torch.bfloat16}


def ceil_div(a, b):
    return -(-a // b)


# ------------------------------------------------------------------------------ tables

def step_reference(cached, fresh, ring, pool, table, page, max_tokens):
    """One step by its rules, one request after the other; lists in, lists out."""
    ring, table = list(ring), [list(row) for row in table]
    n_pages, max_pages = len(ring), len(table[0])
    head, count = pool[0] % n_pages, min(max(pool[1], 0), n_pages)
    slots, starts, kv, nxt = [-1] * max_tokens, [0], [], []
    rows = asked = taken = back = refused = 0
    for r, (c, f) in enumerate(zip(cached, fresh)):
        bad = c < 0 or c > max_pages * page
        if f < 0:
            for p in table[r][: 0 if bad else ceil_div(c, page)]:
                ring[(head + count + back) % n_pages] = p
                back += 1
            kv.append(0)
            nxt.append(0)
            starts.append(min(rows, max_tokens))
            continue
        rows += f
        starts.append(min(rows, max_tokens))
        ok = not bad and c + f <= max_pages * page and rows <= max_tokens
        have, want = ceil_div(c, page), ceil_div(c + f, page)
        if ok:
            asked += want - have
            ok = want == have or asked <= count
        if not ok:
            refused += 1
            kv.append(0)
            nxt.append(c)
            continue
        for col in range(have, want):
            table[r][col] = ring[(head + taken) % n_pages]
            taken += 1
        for i in range(f):
            slots[rows - f + i] = table[r][(c + i) // page] * page + (c + i) % page
        kv.append(c + f)
        nxt.append(c + f)
    return dict(block_table=table, free_ring=ring, q_start=starts, kv_len=kv, cached_next=nxt, slots=slots,
                pool_next=[(head + taken) % n_pages, count - taken + back],
                counts=[min(rows, max_tokens), taken, back, refused])


def step_inputs(seed, n_req, page, max_pages, max_tokens, *, kinds=(0, 1, 1, 1, 5, 40, -1), free=None, in_bounds=True):
    rng = random.Random(seed)
    room = max_pages * page
    cached = [rng.choice((0, 1, page - 1, page, page + 1, rng.randint(0, room))) for _ in range(n_req)]
    cached = [min(max(c, 0), room) for c in cached]
    fresh = [rng.choice(kinds) for _ in range(n_req)]
    if not in_bounds:
        for r in range(0, n_req, 7):
            cached[r] = rng.choice((-5, room + 1, 2 ** 31 - 1, -2 ** 31))
            fresh[r] = rng.choice((2 ** 31 - 1, 1, -1))
    held = [ceil_div(c, page) if 0 <= c <= room else 0 for c in cached]
    n_pages = sum(held) + (sum(min(max(f, 0), 4000) // page + 1 for f in fresh) + 3)
    ids = list(range(n_pages))
    rng.shuffle(ids)
    table, at = [], 0
    for h in held:
        table.append(ids[at: at + h] + [-1] * (max_pages - h))
        at += h
    rest = ids[at:]
    count = len(rest) if free is None else min(free, len(rest))
    head = rng.randrange(n_pages)
    ring = [-1] * n_pages
    for i, p in enumerate(rest[:count]):
        ring[(head + i) % n_pages] = p
    return cached, fresh, ring, [head, count], table


# ------------------------------------------------------------------------------ attention

def attn_reference(q, k_pages, v_pages, table, q_start, kv_len, scale, window):
    """(output, sum of weight x |value|) in float64 on the host, from the formulas: every token sees its keys
    only.  Lists of ints and CPU tensors in.  A table entry out of range has no keys."""
    n_pages, n_kv, page, hd = k_pages.shape
    n_q = q.shape[1]
    out = torch.zeros(q.shape, dtype=torch.float64)
    mag = torch.zeros(q.shape, dtype=torch.float64)
    for r, m in enumerate(kv_len):
        n = q_start[r + 1] - q_start[r]
        ids = table[r][: ceil_div(m, page)]
        live = torch.tensor([0 <= ids[j // page] < n_pages for j in range(m)], dtype=torch.bool)
        pg = torch.tensor([min(max(p, 0), n_pages - 1) for p in ids], dtype=torch.long)
        k = k_pages[pg].double().transpose(1, 2).reshape(-1, n_kv, hd)[:m]
        v = v_pages[pg].double().permute(0, 3, 1, 2).reshape(-1, n_kv, hd)[:m]
        for i in range(n):
            p = m - n + i
            lo = max(0, p - window + 1) if window else 0
            if p < 0:
                continue
            see = torch.arange(lo, p + 1)
            see = see[live[lo: p + 1]]
            if not len(see):
                continue
            kk = k[see].repeat_interleave(n_q // n_kv, 1)
            vv = v[see].repeat_interleave(n_q // n_kv, 1)
            t = q_start[r] + i
            s = (kk * q[t].double()).sum(-1) * scale            # [keys][heads]
            w = torch.softmax(s, 0)[..., None]
            out[t] = (w * vv).sum(0)
            mag[t] = (w * vv.abs()).sum(0)
    return out, mag


def attn_tolerance(out, mag, dtype, head_dim, partial=8.0, keys=4096):
    """Half a step of the type for each weight (they enter the second product rounded; the sum may be of
    the unrounded ones) and half a step for the output; scores in fp32: head_dim additions, each off by
    at most 2^-24 of a partial sum (scaled, below `partial` for these inputs), enter the exponent of
    numerator and sum; fp16 weights below its subnormals: at most 2^-32 of the largest, per key."""
    half = torch.finfo(dtype).eps / 2
    exponent = 2 * head_dim * 2.0 ** -24 * partial
    return half * (mag + out.abs() + half * mag) + exponent * mag + keys * 2.0 ** -30


def attn_tolerance_of_few_rows(out, mag, dtype, head_dim, partial=8.0, keys=4096):
    """As attn_tolerance, where a weight enters the second product as two numbers of the type: all but a share of
    it, rounded, and the rest (the share, and what was rounded), of which half a step is lost."""
    half = torch.finfo(dtype).eps / 2
    share = 2.0 ** -7 if dtype == torch.float16 else 2.0 ** -6
    weights = half * (share + half) * mag + 2 * head_dim * 2.0 ** -24 * partial * mag + keys * 2.0 ** -30
    return half * out.abs() + (1 + half) * weights


def attn_case(seed, lens, n_q, n_kv, hd, page, dtype, extra_pages=3, max_pages=None):
    """Random pages and queries of requests (new tokens, keys): dict of CPU tensors and lists."""
    gen = torch.Generator().manual_seed(seed)
    rng = random.Random(seed)
    held = [ceil_div(m, page) for _, m in lens]
    n_pages = sum(held) + extra_pages
    ids = list(range(n_pages))
    rng.shuffle(ids)
    cols = max_pages or max(1, max(held))
    table, at = [], 0
    for h in held:
        table.append(ids[at: at + h] + [-1] * (cols - h))
        at += h
    starts = [0]
    for n, _ in lens:
        starts.append(starts[-1] + n)
    normal = lambda *shape: torch.randn(shape, generator=gen).to(DT[dtype])
    return dict(k=normal(n_pages, n_kv, page, hd), v=normal(n_pages, n_kv, hd, page), q=(1.5 * torch.randn(
        (starts[-1], n_q, hd), generator=gen)).to(DT[dtype]), table=table, starts=starts, kv=[m for _, m in lens],
        scale=1 / math.sqrt(hd), dtype=dtype, page=page)


def past_end(case, value):
    """Fills the positions past each request's keys, and the pages that no request holds, with `value`."""
    n_pages, page = case["k"].shape[0], case["page"]
    held = {p for row, m in zip(case["table"], case["kv"]) for p in row[: ceil_div(m, page)]}
    for p in set(range(n_pages)) - held:
        case["k"][p] = value
        case["v"][p] = value
    for row, m in zip(case["table"], case["kv"]):
        if m % page:
            case["k"][row[m // page], :, m % page:] = value
            case["v"][row[m // page], :, :, m % page:] = value
