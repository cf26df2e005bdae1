"""Fused scaled-dot-product attention forward for GB300 (sm_103a).

``attn_fwd`` and friends mirror the C ABI of ``include/attn_fwd.h``;
``attention_forward`` is a tensor-level convenience wrapper, and
``HostForward`` runs the forward pass on pinned host buffers with the copies
overlapped.  For serving there are ``attention_varlen`` (whole prompts, packed,
grouped heads), ``KVCache4`` (a K/V cache in 4 bits: append, read, attention
of one token per sequence, eviction) and ``PagedKVCache`` (a K/V cache in pages:
append with the head norm and rotation, attention of new tokens with a sliding
window).  ``qk_norm_rope`` and its gradient stand before attention in training, too.
The CUDA library is loaded on first use and must have been built (``build_ext``).
"""
from ._lib import (ATTN_BF16, ATTN_ERR_ALIGNMENT, ATTN_ERR_CAPACITY, ATTN_ERR_DEVICE, ATTN_ERR_INVALID_ARG, ATTN_ERR_LAUNCH,
                   ATTN_ERR_PAGE, ATTN_ERR_TIMEOUT, ATTN_ERR_UNSUPPORTED, ATTN_FP16, ATTN_FP32, ATTN_OK, EXPORTED, AttnError,
                   attn_cache4_append, attn_cache4_decode, attn_cache4_decode_workspace_bytes, attn_cache4_evict,
                   attn_cache4_evict_workspace_bytes, attn_cache4_read, attn_cache4_t, attn_fwd,
                   attn_fwd_fp8, attn_bwd, attn_bwd_workspace_bytes,
                   attn_heads_t, attn_paged_append, attn_paged_attend,
                   attn_paged_attend_workspace_bytes, attn_pages_t, attn_qk_norm_rope, attn_qk_norm_rope_bwd,
                   attn_qk_norm_rope_bwd_workspace_bytes, attn_rotary_t,
                   attn_fwd_abi_version, attn_fwd_debug_status, attn_fwd_schedule, attn_fwd_splitkv,
                   attn_fwd_splitkv_static, attn_fwd_splitkv_suggest,
                   attn_fwd_splitkv_workspace_bytes, attn_fwd_status, attn_fwd_varlen,
                   attn_fwd_varlen_workspace_bytes,
                   STATIC_SCRATCH_BYTES, attn_merge, attn_status_str, attn_watchdog_selftest, call_status,
                   load)
from .api import attention_backward, attention_forward, attention_varlen
from .cache import KVCache4
from .host import HostForward, plan_pieces
from .paged import PagedKVCache
from .rotary import Rotary, qk_norm_rope, qk_norm_rope_backward, rotary_frequencies
from .build_ext import LIB_PATH, build

__all__ = [
    "ATTN_OK", "ATTN_ERR_INVALID_ARG", "ATTN_ERR_UNSUPPORTED", "ATTN_ERR_ALIGNMENT",
    "ATTN_ERR_LAUNCH", "ATTN_ERR_TIMEOUT", "ATTN_ERR_DEVICE", "EXPORTED", "AttnError",
    "attn_fwd", "attn_fwd_fp8", "attn_bwd", "attn_bwd_workspace_bytes", "attention_backward",
    "attn_fwd_status", "attn_fwd_schedule", "attn_fwd_splitkv", "attn_fwd_splitkv_suggest",
    "attn_fwd_splitkv_workspace_bytes", "attn_fwd_splitkv_static", "STATIC_SCRATCH_BYTES",
    "attn_merge", "call_status",
    "attn_status_str",
    "attn_fwd_debug_status",
    "attn_watchdog_selftest", "attn_fwd_abi_version", "attention_forward", "load", "build",
    "LIB_PATH", "HostForward", "plan_pieces", "ATTN_ERR_CAPACITY", "ATTN_BF16", "ATTN_FP16", "ATTN_FP32",
    "attention_varlen", "KVCache4", "attn_fwd_varlen", "attn_fwd_varlen_workspace_bytes", "attn_cache4_t",
    "attn_cache4_append", "attn_cache4_read", "attn_cache4_decode", "attn_cache4_decode_workspace_bytes",
    "attn_cache4_evict", "attn_cache4_evict_workspace_bytes", "ATTN_ERR_PAGE", "Rotary", "rotary_frequencies", "qk_norm_rope",
    "qk_norm_rope_backward", "PagedKVCache", "attn_heads_t", "attn_rotary_t", "attn_pages_t", "attn_qk_norm_rope",
    "attn_qk_norm_rope_bwd", "attn_qk_norm_rope_bwd_workspace_bytes", "attn_paged_append",
    "attn_paged_attend", "attn_paged_attend_workspace_bytes",
]
