"""Predictor-gated, neuron-aware sparse FFN for MI355X (gfx950): a C-ABI HIP library plus a thin binding.

PowerInfer (arXiv 2312.12456) observes that a ReLU-family FFN fires only a small,
input-dependent set of neurons per token; a low-rank predictor picks them and a neuron-aware
sparse operator computes only those, with a GPU index naming the neurons resident on the
device.  This package exposes that decode-step hot path:

* ``pi_predict``    predictor GEMVs -> firing mask (batch union)
* ``pi_compact``    placement restriction + ascending active-neuron list
* ``pi_sparse_ffn`` gathered up/gate rows with fused ReLU/ReGLU, then the active rows of W_down^T
* ``pi_ffn_layer``  all three, stream-ordered (also as ``pi_predict_hidden`` + ``pi_ffn_layer_from_hidden``)

The attention side of the same step works on a paged key/value cache:

* ``pi_kv_step``    request lengths -> block tables and slot map, on the device
* ``pi_kv_append``  new keys and values into the pages
* ``pi_kv_attn``    attention of the new tokens (decode, drafts, prompt chunks) over the pages

and around it, for steps that rotate, stream, draft or fork:

* ``pi_kv_rope_append``  head norms and rotary positions of queries and keys, with the append
* ``pi_kv_attn_sinks``   attention over a window and the first tokens
* ``pi_kv_verify``       which drafted tokens stay, and the token behind them
* ``pi_kv_release``, ``pi_kv_fork``, ``pi_kv_copy``  pages given back, shared and copied

All compute runs in ``libpi.so``; torch only provides device memory and streams.
"""
from ._abi import (PI_F16, PI_MAX_BATCH, PI_Q4_0, PiError, make_ffn, make_predictor, pi_compact, pi_ffn_layer,
                   pi_ffn_layer_from_hidden, pi_predict, pi_predict_hidden, pi_sparse_ffn,
                   pi_status_string, pi_version, pi_workspace_bytes)
from ._kv import (PI_KV_BF16, PI_KV_F16, PI_ROPE_HALF, PI_ROPE_PAIRS, make_kv_batch, make_kv_cache, make_kv_drafts, make_kv_pages,
                  make_kv_rope, make_kv_tables, pi_kv_append, pi_kv_attn, pi_kv_attn_sinks,
                  pi_kv_attn_sinks_workspace_bytes, pi_kv_attn_workspace_bytes, pi_kv_copy, pi_kv_fork,
                  pi_kv_pages_workspace_bytes, pi_kv_release,
                  pi_kv_rope_append, pi_kv_step, pi_kv_verify, pi_kv_verify_workspace_bytes, pi_rope_frequencies)
from .layer import DeviceLayer

__all__ = ["PI_F16", "PI_Q4_0", "PI_MAX_BATCH", "PiError", "make_ffn", "make_predictor", "pi_compact",
           "pi_ffn_layer", "pi_ffn_layer_from_hidden", "pi_predict_hidden", "pi_predict", "pi_sparse_ffn", "pi_status_string", "pi_version", "pi_workspace_bytes",
           "DeviceLayer", "PI_KV_F16", "PI_KV_BF16", "make_kv_batch", "make_kv_cache", "make_kv_tables", "pi_kv_append",
           "pi_kv_attn", "pi_kv_attn_workspace_bytes", "pi_kv_step", "PI_ROPE_HALF", "PI_ROPE_PAIRS", "make_kv_drafts", "make_kv_pages",
           "make_kv_rope", "pi_kv_attn_sinks", "pi_kv_attn_sinks_workspace_bytes", "pi_kv_copy", "pi_kv_fork", "pi_kv_pages_workspace_bytes", "pi_kv_release",
           "pi_kv_rope_append", "pi_kv_verify", "pi_kv_verify_workspace_bytes", "pi_rope_frequencies"]
