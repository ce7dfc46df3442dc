"""Bounded-decay chunked linear attention for GB300 (sm_103a).

The compute lives in libbdla.so (C ABI declared in include/bdla.h); this
package holds the CUDA sources (csrc/), their build script, a thin ctypes
binding and the seeded synthetic input generator.
"""
from .bdla import (BOUNDED, CHUNK, SOFTPLUS, BdlaError, Workspace, attn_bwd, attn_cached,  # noqa: F401
                   attn_fwd, attn_shared, bwd, bwd_delta, bwd_vec, cache_append, decay, decode, decode_delta, fwd, fwd_delta, fwd_vec, lib,
                   n_slots, qk_norm, qk_norm_append, qk_norm_bwd, tile_states, workspace_bytes)

__all__ = ["BOUNDED", "SOFTPLUS", "CHUNK", "BdlaError", "Workspace", "fwd", "bwd", "fwd_vec", "bwd_vec",
           "fwd_delta", "bwd_delta", "tile_states",
           "decay", "decode", "decode_delta", "lib", "n_slots", "workspace_bytes",
           "qk_norm", "qk_norm_bwd", "qk_norm_append", "attn_fwd", "attn_bwd", "cache_append", "attn_cached", "attn_shared"]
