"""Dynamic block-sparse self-attention for video DiTs on B200 (sm_100a).

Pipeline per (batch, head): mean-pooled block scores with a row softmax,
per-row Top-p block selection (optionally restricted to a candidate set),
exact block-sparse attention over the selected blocks, and the exact softmax
mass of every selected block.  Around it, what a transformer layer does with
its queries, keys and values: per-head norm with position rotation, 8-bit
activation rows, and attention over a local window with first tokens that
stay visible, trained or cached.  All arithmetic runs in ``libdsa.so``; the
Python layer only marshals arguments (see ``ops``).  The library is loaded
on the first call, and a call fails loudly if it has not been built.
"""
from . import ops, synth, window_layer  # noqa: F401
from ._lib import DSAError  # noqa: F401
from .ops import (Act8, HilbertOrder, RopePlan, attn_bwd, attn_fwd, block_mass,  # noqa: F401
                  device_status, hilbert_order, mass_to_probs, pack8, permute_tokens, pool_score,
                  pool_score_hier, qk_norm_rope, qk_norm_rope_bwd, select_topp, sparse_attention,
                  unpack8, window_attn_bwd, window_attn_decode, window_attn_fwd)

__all__ = ["ops", "synth", "DSAError", "pool_score", "select_topp", "attn_fwd",
           "block_mass", "mass_to_probs", "sparse_attention", "device_status",
           "hilbert_order", "permute_tokens", "HilbertOrder", "pool_score_hier", "attn_bwd",
           "qk_norm_rope", "qk_norm_rope_bwd", "RopePlan", "pack8", "unpack8", "Act8",
           "window_attn_fwd", "window_attn_bwd", "window_attn_decode", "window_layer"]
