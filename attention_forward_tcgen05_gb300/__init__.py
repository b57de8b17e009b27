"""GB300 (sm_103a) attention engine: exact SDPA with online softmax, and its gradients.

Prefill FMHA on tcgen05 tensor cores (TMA-fed, TMEM accumulators) and a GQA
split-KV decode with an LSE-weighted merge, serving calls over a paged cache and the
gradients of the dense prefill, behind the C ABI of
``include/attn.h``.  ``libattn.so`` is built in-tree by ``build.build()``.
"""
from ._binding import (  # noqa: F401
    ATTN_BF16, ATTN_ERR_CUDA, ATTN_ERR_DEVICE_INPUT, ATTN_ERR_DEVICE_TIMEOUT, ATTN_ERR_INVALID_ARG,
    ATTN_ERR_SCRATCH_TOO_SMALL, ATTN_ERR_UNSUPPORTED, ATTN_F32, ATTN_OK, LIB_PATH, AttnError,
    attn_debug_wait_timeout, attn_decode, attn_decode_noalloc, attn_decode_noalloc_scratch_bytes,
    attn_decode_packed, attn_decode_split, attn_decode_split_packed, attn_merge, attn_prefill_fwd,
    attn_prefill_packed, attn_prefill_schedule, attn_prefill_varlen, attn_prefill_varlen_window,
    attn_prefill_window, attn_strerror, attn_sync_check, attn_version, decode, decode_counters,
    decode_packed, decode_split, decode_split_packed, load, merge, prefill, prefill_schedule,
    prefill_varlen, prefill_window, sync_check)
from ._serving import (  # noqa: F401
    attn_decode_paged, attn_decode_paged_splits, attn_decode_window, attn_decode_window_splits, attn_evict,
    attn_key_weights, attn_prefill_paged, attn_prefill_paged_splits, attn_rope_append, attn_rope_append_axes,
    attn_rope_rotate, decode_paged, decode_window, evict, key_weights, prefill_paged, rope_append, rope_axes,
    rope_frequencies, rope_rotate)
from ._backward import (  # noqa: F401
    attn_prefill_backward, attn_prefill_backward_workspace, attn_prefill_varlen_backward, prefill_backward,
    prefill_varlen_backward)
