"""examples/paged_decode.py: prompts and replayed decode steps through attention and the sparse FFN."""
import importlib.util
import math
import os

import pytest
import torch

import kv_util
import synth
from gpu_util import announce

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "paged_decode.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("paged_decode", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("lengths,kv_heads", [([5, 1, 33], None), ([40, 17, 16, 2, 9], 4)])
def test_replayed_steps_equal_eager_ones(example, lengths, kv_heads):
    announce(f"paged decode example lengths={lengths} kv_heads={kv_heads}")
    cfg = synth.custom_config(1024, 2048, 64, layers=2, seed=3)
    graph, eager, seconds = example.generate(cfg, 2, lengths, 20, head_dim=64, kv_heads=kv_heads)
    assert torch.isfinite(eager).all() and torch.equal(graph, eager) and seconds > 0


@pytest.mark.parametrize("lengths,kv_heads", [([5, 1, 33], None), ([40, 17, 16, 2, 9], 4)])
def test_steps_equal_a_plain_stack(example, monkeypatch, lengths, kv_heads):
    """Every step against the stack written out without a cache: what the kernels are given follows from what they
    returned before, and attention equals the formula over all of a request's keys and values so far."""
    announce(f"paged decode example against a plain stack, lengths={lengths} kv_heads={kv_heads}")
    cfg, layers, n, hd, steps = synth.custom_config(1024, 2048, 64, layers=2, seed=3), 2, len(lengths), 64, 4
    calls, pi = [], example.pi
    real = {name: getattr(pi, name) for name in ("pi_kv_attn", "pi_ffn_layer")}

    def attn(cache, batch, q, out, ws, **kw):
        real["pi_kv_attn"](cache, batch, q, out, ws, **kw)
        calls.append(("attn", q.clone(), out.clone()))

    def ffn(pred, weights, h, b, y, *rest):
        real["pi_ffn_layer"](pred, weights, h, b, y, *rest)
        calls.append(("ffn", h.clone(), y.clone()))

    monkeypatch.setattr(pi, "pi_kv_attn", attn)
    monkeypatch.setattr(pi, "pi_ffn_layer", ffn)
    st = example.PagedStack(cfg, layers, n, max(lengths) + steps, head_dim=hd, kv_heads=kv_heads)
    n_q, n_kv = st.n_q, st.n_kv
    held = [[torch.empty(0, 2, n_kv, hd).half() for _ in range(n)] for _ in range(layers)]     # keys and values so far
    gen = torch.Generator(device="cuda").manual_seed(9)
    for step in range(1 + steps):
        fresh = lengths if step == 0 else [1] * n
        starts = [sum(fresh[:r]) for r in range(n + 1)]
        x = torch.randn((sum(fresh), cfg.d), generator=gen, device="cuda")
        st.fresh.copy_(torch.tensor(fresh, dtype=torch.int32))
        del calls[:]
        out = st.step(st.plan(len(x), max(fresh), max(lengths) + step), x)
        torch.cuda.synchronize()
        assert st.counts.tolist()[3] == 0
        left = list(calls)
        for l in range(layers):
            rms = lambda t: (t * torch.rsqrt(t.square().mean(-1, keepdim=True) + 1e-6)).half()
            qkv = rms(x) @ st.w_qkv[l]
            kind, q, heads = left.pop(0)
            assert kind == "attn" and torch.equal(q.reshape(len(x), -1), qkv[:, : n_q * hd])
            kv = qkv[:, n_q * hd:].reshape(len(x), 2, n_kv, hd).cpu()
            held[l] = [torch.cat((old, kv[starts[r]: starts[r + 1]])) for r, old in enumerate(held[l])]
            lens = [len(h) for h in held[l]]
            pool = torch.zeros(n, 2, n_kv, max(lens), hd).half()
            for r, h in enumerate(held[l]):
                pool[r, :, :, : lens[r]] = h.permute(1, 2, 0, 3)
            want, mag = kv_util.attn_reference(q.cpu(), pool[:, 0], pool[:, 1].transpose(2, 3), [[r] for r in range(n)], starts, lens,
                                               1 / math.sqrt(hd), 0)
            tol = kv_util.attn_tolerance(want, mag, torch.float16, hd, partial=16.0)
            assert bool(((heads.cpu().double() - want).abs() <= tol).all()), (step, l)
            x = x + (heads.reshape(len(x), -1) @ st.w_out[l]).float()
            ys = []
            while left and left[0][0] == "ffn" and sum(map(len, ys)) < len(x):
                _, h, y = left.pop(0)
                at = sum(map(len, ys))
                assert torch.equal(h, rms(x)[at: at + len(h)])
                ys.append(y)
            x = x + torch.cat(ys)
        assert not left and torch.equal(out, x), step
