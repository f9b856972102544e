"""GB300-native (sm_103a) scaled dot-product causal multi-head self-attention.

The compute path is the CUDA library ``libattn_sm103a.so`` (C ABI in
``include/attn.h``); this package is its thin Python binding.  ``attn_fwd``
runs the tcgen05/TMA prefill kernel, ``attn_decode`` the split-KV decode kernel
with its in-kernel log-sum-exp combine, ``attn_bwd`` the backward pass (given
``attn_fwd_lse``'s output and log-sum-exps).  A paged key-value cache is
written by ``attn_paged_append``, read by ``attn_decode_paged`` and shrunk by
``attn_cache_evict`` to the keys with the largest attention weights, which
``attn_key_weights`` (a prompt's) and ``attn_decode_paged`` (a step's) sum up.
Sequences of different lengths packed one behind another are attended to by
``attn_fwd_packed`` and ``attn_bwd_packed``; ``attn_rope`` turns queries and keys
by their positions, ``attn_rope_append`` writes them to the paged cache in the
same pass, and ``attn_cache_plan`` hands out the pages and slots of a serving
step.  There is no CPU or PyTorch fallback: without the built library every
call raises.
"""
from ._binding import (ATTN_ERR_CHECK, ATTN_ERR_CUDA, ATTN_ERR_INVALID_ARG, ATTN_ERR_NO_MEMORY,  # noqa: F401
                       ATTN_ERR_SCRATCH_LIMIT, ATTN_ERR_TIMEOUT, ATTN_ERR_UNSUPPORTED, ATTN_OK,
                       AttnError, RopeFrequencies, attn_bwd, attn_bwd_packed, attn_cache_evict,
                       attn_cache_plan, attn_debug_inject_fault, attn_decode, attn_decode_noalloc,
                       attn_decode_paged, attn_decode_paged_workspace,
                       attn_decode_ring, attn_fwd, attn_fwd_chunk, attn_fwd_lse, attn_fwd_packed,
                       attn_key_weights, attn_packed_workspace, attn_paged_append, attn_rope,
                       attn_rope_append, attn_rope_frequencies, attn_status, error_string, version)
