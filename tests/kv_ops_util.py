"""Plain 64-bit references of the operators around paged attention, and their inputs (no test functions here)."""
from __future__ import annotations

import math
import random

import torch

from kv_util import ceil_div

ALL = 2 ** 31 - 1


# ------------------------------------------------------------------------------ rotary positions

def rope_head(x, pos, freq, layout, scale, norm, eps, weight):
    """(heads [n][h][hd] normed and rotated at positions pos [n], in float64; sum of the products' magnitudes per element)."""
    x = x.double()
    if norm:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
        if weight is not None:
            x = x * weight.double()
    y, mag = x.clone(), x.abs().clone()
    half = 0 if freq is None else len(freq)
    if half:
        angle = pos.double()[:, None] * freq.double()
        c, s = (scale * torch.cos(angle))[:, None], (scale * torch.sin(angle))[:, None]
        ia = torch.arange(half) if layout == 0 else torch.arange(0, 2 * half, 2)
        ib = ia + half if layout == 0 else ia + 1
        a, b = x[..., ia], x[..., ib]
        y[..., ia], y[..., ib] = a * c - b * s, a * s + b * c
        mag[..., ia] = mag[..., ib] = abs(scale) * (a.abs() + b.abs())
    return y, mag


def rope_tolerance(y, mag, dtype, norm, far=1 << 20):
    """Half a step of the type for the result.  Before that, in fp32: the angle is off by at most 2^-25 of a turn
    (its fraction rounded) and sine and cosine by 2 units of 2^-24, so each product by (2 pi 2^-25 + 2^-23) of the
    magnitude, then four roundings; with a norm the sum of up to 256 squares (a tree of at most 16 + 4 additions per lane
    and across), root, division and two products: 24 roundings; of the smallest numbers half a subnormal step.  Angles of up
    to `far` radians (frequencies up to 1): four roundings in fp64 here and in the reference, 6 * 2^-53 of them at most."""
    half = torch.finfo(dtype).eps / 2
    before = (far * 6 * 2.0 ** -53 + 2 * math.pi * 2.0 ** -25 + 2.0 ** -23 + (4 + (24 if norm else 0)) * 2.0 ** -24) * mag
    return half * (y.abs() + before) + before + torch.finfo(dtype).smallest_normal * half


# ------------------------------------------------------------------------------ a window and the first tokens

def sinks_reference(c, window, sinks, rows=None):
    """(output, sum of weight x |value|) in float64 on the host for a case of kv_util.attn_case: every token sees its
    keys only.  rows: of these packed rows only."""
    table, starts, k_pages, v_pages = c["table"], c["starts"], c["k"], c["v"]
    n_pages, n_kv, page, hd = k_pages.shape
    n_q = c["q"].shape[1]
    out = torch.zeros(c["q"].shape, dtype=torch.float64)
    mag = torch.zeros(c["q"].shape, dtype=torch.float64)
    for r, m in enumerate(c["kv"]):
        n = starts[r + 1] - starts[r]
        for i in range(n):
            t, p = starts[r] + i, m - n + i
            if p < 0 or (rows is not None and t not in rows):
                continue
            low = max(0, p - window + 1)
            see = [j for j in [*range(min(sinks, low)), *range(low, p + 1)] if 0 <= table[r][j // page] < n_pages]
            if not see:
                continue
            pg = torch.tensor([table[r][j // page] for j in see])
            off = torch.tensor([j % page for j in see])
            kk = k_pages[pg, :, off].double().repeat_interleave(n_q // n_kv, 1)
            vv = v_pages[pg, :, :, off].double().repeat_interleave(n_q // n_kv, 1)
            s = (kk * c["q"][t].double()).sum(-1) * c["scale"]
            w = torch.softmax(s, 0)[..., None]
            out[t] = (w * vv).sum(0)
            mag[t] = (w * vv.abs()).sum(0)
    return out, mag


# ------------------------------------------------------------------------------ drafted tokens

def verify_reference(starts, tokens, target, draft, u_accept, u_next, kv_len=None, rows=None):
    """(accepted, next, keep) by the rules, one request after the other; lists, and CPU tensors [rows][vocab].  A request
    with fewer keys than rows, or none, was refused by its step: it keeps all that it holds (ALL)."""
    rows, vocab = len(tokens) if rows is None else rows, target.shape[1]
    accepted, nxt, keep = [], [], []
    for r in range(len(starts) - 1):
        a, b = starts[r], starts[r + 1]
        n = b - a
        if a < 0 or n <= 0 or b > rows:
            accepted.append(0)
            nxt.append(-1)
            keep.append(None if kv_len is None else kv_len[r] if kv_len[r] > 0 else ALL)
            continue
        if kv_len is not None and kv_len[r] < n:
            accepted.append(0)
            nxt.append(tokens[a])
            keep.append(ALL)
            continue
        i = 0
        while i < n - 1:
            t, x = a + i, tokens[a + i + 1]
            if not 0 <= x < vocab:
                break
            q = 1.0 if draft is None else float(draft[t, x])
            if not float(u_accept[t]) * q < float(target[t, x]):
                break
            i += 1
        row = target[a + i].double()
        clean = lambda w: torch.where(w > 0, w, torch.zeros_like(w))       # (NaN: 0)
        full = clean(row)
        w = full
        if i < n - 1:
            if draft is not None:
                w = clean(row - draft[a + i].double())
            else:
                w = full.clone()
                if 0 <= tokens[a + i + 1] < vocab:
                    w[tokens[a + i + 1]] = 0
            if not float(w.sum()) > 0:
                w = full
        upto = torch.cumsum(w, 0)
        if not float(upto[-1]) > 0:
            pick = -1
        else:
            over = ((upto > float(u_next[r]) * float(upto[-1])) & (w > 0)).nonzero()[:, 0]
            pick = int(over[0]) if len(over) else int((w > 0).nonzero()[-1, 0])
        accepted.append(i)
        nxt.append(pick)
        keep.append(None if kv_len is None else kv_len[r] - (n - 1 - i))
    return accepted, nxt, keep


# ------------------------------------------------------------------------------ pages

def clamp_pool(pool, n_pages):
    return pool[0] % n_pages, min(max(pool[1], 0), n_pages)


def release_reference(st, drop_from, drop_to):
    """By the rules, one request after the other.  st: dict of lists (cached, table, ring, pool, shares) and page."""
    page, table, ring, shares = st["page"], [list(x) for x in st["table"]], list(st["ring"]), list(st["shares"])
    n_pages, max_pages = len(ring), len(table[0])
    head, count = clamp_pool(st["pool"], n_pages)
    valid = lambda p: 0 <= p < n_pages
    nxt, copies, given, free = [], [], [], []
    asked = taken = refused = 0
    for r, c in enumerate(st["cached"]):
        f, t = max(drop_from[r], 0), ALL if drop_to is None else drop_to[r]
        copy = [-1, -1]
        if not 0 <= c <= max_pages * page:
            refused += 1
            nxt.append(c)
            copies.append(copy)
            continue
        cut = t >= c and f < c
        mine = []
        if cut and f % page and valid(table[r][f // page]) and st["shares"][table[r][f // page]] > 0:
            asked += 1
            if asked > count:
                refused += 1
                nxt.append(c)
                copies.append(copy)
                continue
            old = table[r][f // page]
            copy = [old, st["ring"][(head + taken) % n_pages]]
            free.append((r, f // page, copy[1]))
            taken += 1
            mine.append(old)
        last = 0 if f >= c else ceil_div(c, page) if cut else max(t, 0) // page
        for col in range(ceil_div(f, page), last):
            if valid(table[r][col]):
                mine.append(table[r][col])
                if not cut:
                    table[r][col] = -1
        given += mine
        nxt.append(f if cut else c)
        copies.append(copy)
    for p in given:
        shares[p] -= 1
    back = 0
    for p in given:
        if shares[p] < 0:
            ring[(head + count + back) % n_pages] = p
            back += 1
            shares[p] = 0
    for r, col, new in free:
        table[r][col] = new
    return dict(block_table=table, free_ring=ring, shares=shares, cached_next=nxt, copies=copies,
                pool_next=[(head + taken) % n_pages, min(count - taken + back, n_pages)], counts=[len(given), back, taken, refused])


def fork_reference(st, src, dst):
    page, table, ring, shares = st["page"], [list(x) for x in st["table"]], list(st["ring"]), list(st["shares"])
    n_pages, max_pages, n_req = len(ring), len(table[0]), len(table)
    head, count = clamp_pool(st["pool"], n_pages)
    cached, nxt, copies, named = st["cached"], list(st["cached"]), [], set()
    done = more = asked = refused = 0
    for s, d in zip(src, dst):
        first = 0 <= d < n_req and d not in named
        if 0 <= d < n_req:
            named.add(d)
        ok = first and 0 <= s < n_req and s != d and 0 <= cached[s] <= max_pages * page and cached[d] == 0
        copy = [-1, -1]
        if ok:
            full, part = divmod(cached[s], page)
            if part and 0 <= st["table"][s][full] < n_pages:
                asked += 1
                if asked > count:
                    ok = False
                else:
                    copy = [st["table"][s][full], ring[(head + asked - 1) % n_pages]]
        copies.append(copy)
        if not ok:
            refused += 1
            continue
        done += 1
        nxt[d] = cached[s]
        for col in range(full):
            p = table[d][col] = st["table"][s][col]
            if 0 <= p < n_pages:
                shares[p] += 1
        more += full
        if part:
            table[d][full] = copy[1]
    taken = min(asked, count)
    return dict(block_table=table, free_ring=ring, shares=shares, cached_next=nxt, copies=copies,
                pool_next=[(head + taken) % n_pages, count - taken], counts=[done, more, taken, refused])


def pages_state(seed, n_req, page, max_pages, *, forks=0.4, holes=0.2, empty=0.2, free=None, bad=0.0):
    """A state of requests, some sharing full pages, some with pages given back from their middles, some empty."""
    rng = random.Random(seed)
    room = max_pages * page
    cached, rows, used = [], [], 0
    for r in range(n_req):
        row, c = [-1] * max_pages, 0
        if rng.random() >= empty:
            c = rng.choice((1, page - 1, page, page + 1, rng.randint(1, room), room))
            full = 0
            if r and rng.random() < forks:
                s = rng.randrange(r)
                full = cached[s] // page
                c = min(room, full * page + rng.randint(0, page + 3))
                row[:full] = rows[s][:full]
            for col in range(full, ceil_div(c, page)):
                if rng.random() < holes and 0 < col < c // page:
                    continue
                row[col] = used
                used += 1
        cached.append(c)
        rows.append(row)
    n_pages = used + rng.randint(1, n_req + 4)
    ids = list(range(n_pages))
    rng.shuffle(ids)
    table = [[ids[v] if v >= 0 else -1 for v in row] for row in rows]
    shares = [-1] * n_pages
    for row in table:
        for p in row:
            if p >= 0:
                shares[p] += 1
    shares = [max(x, 0) for x in shares]
    spare = ids[used:]
    count = len(spare) if free is None else min(free, len(spare))
    head = rng.randrange(n_pages)
    ring = [-1] * n_pages
    for i, p in enumerate(spare[:count]):
        ring[(head + i) % n_pages] = p
    for r in range(n_req):
        if rng.random() < bad:
            cached[r] = rng.choice((-1, room + 1, ALL, -2 ** 31))
            table[r][rng.randrange(max_pages)] = rng.choice((-7, n_pages, ALL))
    return dict(cached=cached, table=table, ring=ring, pool=[head, count], shares=shares, page=page)


def release_ranges(seed, st):
    rng = random.Random(seed)
    at, to = [], []
    for c in st["cached"]:
        kind = rng.randrange(6)
        c = min(max(c, 0), 10 ** 6)
        if kind == 0:
            at.append(rng.choice((0, -3)))
            to.append(ALL)
        elif kind == 1:
            a = rng.randint(0, c + 2)
            at.append(a)
            to.append(rng.randint(0, c + 2))
        elif kind == 2:
            at.append(c + rng.randint(0, 5))
            to.append(rng.choice((ALL, c, -2 ** 31)))
        else:
            at.append(max(0, c - rng.randint(0, st["page"] + 5)))
            to.append(rng.choice((ALL, c)))
    return at, to


def check_owned(st, extra=()):
    """Every page is either free or held by as many table entries as it has owners."""
    n_pages = len(st["ring"])
    held = [0] * n_pages
    for r, c in enumerate(st["cached"]):
        for col in range(ceil_div(c, st["page"])):
            if st["table"][r][col] >= 0:
                held[st["table"][r][col]] += 1
    head, count = st["pool"]
    free = [st["ring"][(head + i) % n_pages] for i in range(count)]
    assert len(set(free)) == count and all(0 <= p < n_pages for p in free)
    for p in range(n_pages):
        assert (held[p] == 0) == (p in set(free)), p
        assert st["shares"][p] == max(held[p] - 1, 0), p
