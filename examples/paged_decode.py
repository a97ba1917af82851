#!/usr/bin/env python3
"""Prompts and decode steps through a small stack: paged attention, then the predictor-gated sparse FFN.

A step of the stack is
  pi_kv_step                 pages and slots of the step's new tokens, from their numbers per request
  per layer: q, k, v         one library product; pi_kv_append takes k and v as slices of its output
             pi_kv_append    into the pages (every layer has its own pages, all share the tables)
             pi_kv_attn      over the pages, and the output projection
             pi_ffn_layer    predictor, compaction and sparse FFN, 16 tokens at a time
With --rope the append also norms and rotates q and k (pi_kv_rope_append); with --window attention sees a window and
the first --sinks tokens (pi_kv_attn_sinks), and a step ends with pi_kv_release, which gives the pages between them back.
The prompts run in one eager step; then every request gets one token per step, replayed from one HIP graph:
lengths, tables and slots live on the device and the step advances them itself.  Weights are seeded
random ones of the named layer stack's shapes; the hidden state of a token is fed back as the next one.

  python examples/paged_decode.py [--config 2] [--layers 4] [--requests 8] [--prompt 200] [--steps 64]
                                  [--rope] [--window 64 [--sinks 4]]
"""
from __future__ import annotations

import argparse
import dataclasses
import math
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import activation_sparse_ffn_rank_amd as pi  # noqa: E402
import synth  # noqa: E402

FFN_TOKENS = 16


class PagedStack:
    """Layers, pages and tables of `requests` requests of at most `max_len` tokens each."""

    def __init__(self, cfg, layers, requests, max_len, head_dim=128, kv_heads=None, page=16, rope=False, window=0, sinks=0):
        self.cfg, self.n, self.hd, self.window, self.sinks = cfg, requests, head_dim, window, sinks
        self.n_q = cfg.d // head_dim
        self.n_kv = kv_heads or self.n_q
        self.ffn = [pi.DeviceLayer.from_host(synth.make_layer(cfg, l)) for l in range(layers)]
        self.ffn_ws = {}
        gen = torch.Generator(device="cuda").manual_seed(cfg.seed)
        weight = lambda i, o: (torch.randn((i, o), generator=gen, device="cuda") / math.sqrt(i)).half()
        wide = (self.n_q + 2 * self.n_kv) * head_dim
        self.w_qkv = [weight(cfg.d, wide) for _ in range(layers)]
        self.w_out = [weight(self.n_q * head_dim, cfg.d) for _ in range(layers)]
        self.max_pages = -(-max_len // page)
        n_pages = requests * self.max_pages
        half = lambda *shape: torch.zeros(shape, dtype=torch.float16, device="cuda")
        ints = lambda *shape: torch.zeros(shape, dtype=torch.int32, device="cuda")
        self.caches = [pi.make_kv_cache(half(n_pages, self.n_kv, page, head_dim), half(n_pages, self.n_kv, head_dim, page))
                       for _ in range(layers)]
        self.page, self.fresh, self.cached = page, ints(requests), ints(requests)
        self.ring, self.pool = torch.arange(n_pages, dtype=torch.int32, device="cuda"), ints(2)
        self.pool[1] = n_pages
        self.table = torch.full((requests, self.max_pages), -1, dtype=torch.int32, device="cuda")
        self.q_start, self.kv_len, self.counts = ints(requests + 1), ints(requests), ints(4)
        self.rope = pi.make_kv_rope(pi.pi_rope_frequencies(head_dim).cuda(), norm=True) if rope else None
        if window:
            self.drop_from, self.drop_to, self.copies = ints(requests).fill_(sinks), ints(requests), ints(requests, 2)
            self.pages = pi.make_kv_pages(self.cached, self.ring, self.pool, self.table, page, ints(n_pages), self.cached, self.pool,
                                          ints(4))

    def plan(self, rows, max_q, max_kv):
        """What a step of `rows` packed tokens keeps: slots, descriptors, workspaces, buffers."""
        p = dict(rows=rows, slots=torch.zeros(rows, dtype=torch.int32, device="cuda"))
        p["tables"] = pi.make_kv_tables(self.cached, self.fresh, self.ring, self.pool, self.table, self.page, self.q_start,
                                        self.kv_len, self.cached, p["slots"], self.pool, self.counts)
        p["batch"] = pi.make_kv_batch(self.table, self.q_start, self.kv_len, max_q=max_q, max_kv=max_kv)
        args = (self.caches[0], p["batch"], rows, self.n_q)
        size = pi.pi_kv_attn_sinks_workspace_bytes(*args, self.window, self.sinks) if self.window else pi.pi_kv_attn_workspace_bytes(*args)
        p["ws"] = torch.empty(size, dtype=torch.uint8, device="cuda")
        p["heads"] = torch.empty((rows, self.n_q, self.hd), dtype=torch.float16, device="cuda")
        p["y"] = torch.empty((rows, self.cfg.d), dtype=torch.float32, device="cuda")
        for b in {min(FFN_TOKENS, rows - t) for t in range(0, rows, FFN_TOKENS)}:
            self.ffn_ws.setdefault(b, self.ffn[0].workspace(b))
        return p

    @staticmethod
    def norm(x):
        return (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)).half()

    def step(self, p, x):
        """Hidden states x [rows][d] (fp32) of the step's tokens through the stack."""
        pi.pi_kv_step(p["tables"])
        rows = p["rows"]
        for l, ffn in enumerate(self.ffn):
            qkv = (self.norm(x) @ self.w_qkv[l]).view(rows, -1, self.hd)
            q, k, v = qkv.split((self.n_q, self.n_kv, self.n_kv), dim=1)
            if self.rope is None:
                pi.pi_kv_append(self.caches[l], k, v, p["slots"])
            else:
                pi.pi_kv_rope_append(self.caches[l], p["batch"], self.rope, q, k, v, p["slots"], q)
            if self.window:
                pi.pi_kv_attn_sinks(self.caches[l], p["batch"], q, p["heads"], p["ws"], scale=1 / math.sqrt(self.hd),
                                    window=self.window, sinks=self.sinks)
            else:
                pi.pi_kv_attn(self.caches[l], p["batch"], q, p["heads"], p["ws"], scale=1 / math.sqrt(self.hd))
            x = x + (p["heads"].view(rows, -1) @ self.w_out[l]).float()
            h = self.norm(x)
            for t in range(0, rows, FFN_TOKENS):
                b = min(FFN_TOKENS, rows - t)
                pi.pi_ffn_layer(ffn.pred, ffn.ffn, h[t: t + b], b, p["y"][t: t + b], None, None, None, self.ffn_ws[b])
            x = x + p["y"]
        if self.window:                # the next token sees the keys from kv_len - window + 1 on; a drop to kv_len would be a cut
            torch.sub(self.kv_len, max(self.window - 1, 1), out=self.drop_to)
            pi.pi_kv_release(self.pages, self.drop_from, self.drop_to, self.copies)
        return x


def generate(cfg, layers, lengths, steps, **kw):
    """Prompts of the given lengths, then `steps` tokens each.  Returns the last hidden states, the same from
    eager steps, and seconds per replayed step."""
    n = len(lengths)
    gen = torch.Generator(device="cuda").manual_seed(7)
    prompt = torch.randn((sum(lengths), cfg.d), generator=gen, device="cuda")
    last = torch.tensor([sum(lengths[: r + 1]) - 1 for r in range(n)], device="cuda")
    out, seconds = [], 0.0
    for replay in (False, True):
        st = PagedStack(cfg, layers, n, max(lengths) + steps, **kw)
        st.fresh.copy_(torch.tensor(lengths, dtype=torch.int32))
        x = st.step(st.plan(len(prompt), max(lengths), max(lengths)), prompt)[last].contiguous()
        st.fresh.fill_(1)
        p = st.plan(n, 1, max(lengths) + steps)
        if not replay:
            for _ in range(steps):
                x = st.step(p, x)
        else:
            graph = torch.cuda.CUDAGraph()
            torch.cuda.synchronize()
            with torch.cuda.graph(graph):
                x.copy_(st.step(p, x))
            torch.cuda.synchronize()
            begin = time.perf_counter()
            for _ in range(steps):
                graph.replay()
            torch.cuda.synchronize()
            seconds = (time.perf_counter() - begin) / steps
        assert st.counts.tolist()[3] == 0, "a request was refused: too few pages"
        assert st.kv_len.tolist() == [m + steps for m in lengths]
        out.append(x)
    return out[1], out[0], seconds


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--config", type=int, default=2, choices=sorted(synth.CONFIGS), help="layer stack whose shapes are used")
    ap.add_argument("--layers", type=int, default=4)
    ap.add_argument("--requests", type=int, default=8)
    ap.add_argument("--prompt", type=int, default=200, help="longest prompt; the others are shorter")
    ap.add_argument("--steps", type=int, default=64)
    ap.add_argument("--rope", action="store_true", help="norms and rotary positions of queries and keys")
    ap.add_argument("--window", type=int, default=0, help="keys that a token sees, at most (0: all)")
    ap.add_argument("--sinks", type=int, default=4, help="first tokens that stay visible beside the window")
    a = ap.parse_args(argv)
    cfg = dataclasses.replace(synth.CONFIGS[a.config], layers=a.layers)
    lengths = [max(1, a.prompt * (r + 1) // a.requests) for r in range(a.requests)]
    graph, eager, seconds = generate(cfg, a.layers, lengths, a.steps, head_dim=64 if cfg.d == 1024 else 128,
                                    rope=a.rope, window=a.window, sinks=a.sinks if a.window else 0)
    print(f"{cfg.name}, {a.layers} layers, {a.requests} requests, prompts {lengths[0]}..{lengths[-1]}: "
          f"{1e6 * seconds:.1f} us per step, {a.requests / seconds:.0f} tokens/s; "
          f"replayed steps {'equal' if torch.equal(graph, eager) else 'differ from'} the eager ones")


if __name__ == "__main__":
    main()
