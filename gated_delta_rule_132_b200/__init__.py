"""Kimi Delta Attention (KDA) on NVIDIA B200: a C-ABI CUDA library (sm_100a)
with a thin Python binding.

The compute entry points (``kda_chunk_fwd``, ``kda_decode_step``,
``kda_decode_tokens``) live in
``gated_delta_rule_132_b200.kda``, those of the full-attention layer
(``kda_attn_fwd``, ``kda_attn_bwd``, ``kda_attn_tree`` and the page calls
``kda_cache_*``) in ``gated_delta_rule_132_b200.attn``; both load the in-tree ``libkda_b200.so`` on
first use; ``inputs`` holds the seeded synthetic-input generators.
"""
import importlib

from . import inputs  # noqa: F401  (no CUDA needed)

_EXPORTS = ("kda_chunk_fwd", "kda_chunk_fwd_prepare", "kda_chunk_fwd_carry",
            "kda_decode_step", "kda_decode_tokens", "kda_gdn_chunk_fwd", "kda_chunk_bwd",
            "kda_chunk_fwd_workspace_size",
            "ChunkFwdCall", "lib", "KdaError")
_ATTN_EXPORTS = ("kda_attn_fwd", "kda_attn_bwd", "kda_attn_tree", "kda_attn_status",
                 "kda_cache_fork", "kda_cache_reserve", "kda_cache_release", "kda_cache_append",
                 "kda_cache_compact", "kda_cache_copy_pages")


def __getattr__(name):
    module = ".kda" if name in _EXPORTS else ".attn" if name in _ATTN_EXPORTS else None
    if module is None:
        raise AttributeError(name)
    value = globals()[name] = getattr(importlib.import_module(module, __name__), name)
    return value
