"""examples/paged_decode.py: prompts and replayed decode steps through attention and the sparse FFN."""
import importlib.util
import os

import pytest
import torch

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
