"""GB300 (sm_103a) structured-mask attention, forward and backward, with rotary
positions and attention over an 8-bit key / value cache.

The computation lives in the CUDA library ``libattnmask.so`` (C ABI declared
in ``include/attn_block_mask.h`` and ``include/attn_cache.h``); this package is
its thin Python binding plus the seeded synthetic workloads used by the tests
and the benchmark.
"""
from .api import (AttnError, BlockMask, KVCache, MASK_KINDS, RopePlan, TILE_EMPTY, TILE_FULL,  # noqa: F401
                  TILE_PARTIAL, attn_block_mask_build, attn_block_mask_build_noalloc,
                  attn_block_mask_workspace_size, attn_bwd, attn_bwd_workspace_size,
                  attn_cache_append, attn_cache_evict, attn_cache_fwd, attn_cache_fwd_workspace_size,
                  attn_cache_get_status, attn_cache_weights, attn_fwd, attn_get_status,
                  attn_last_error_message, attn_rope, attn_rope_plan, attn_status_string, attn_version)
