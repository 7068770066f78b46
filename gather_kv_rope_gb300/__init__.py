"""GB300-native paged KV insert (RoPE + MXFP8) and dequant-gather.

The compute runs in libgkr.so (hand-written sm_103a CUDA kernels behind a C ABI,
declared in include/gkr.h); this package builds it in-tree and binds it with
ctypes.  PyTorch supplies device memory and streams only.

    kv_insert(kv, k_cache, slot_mapping, positions, cos_sin_cache, block_size, record,
              fp8_scale=None)
    kv_gather(k_cache, indices, out, fp8_scale=None)
    rope_quant_insert(kv, k_cache, slot_mapping, positions, cos_sin_cache, block_size,
                      compress_ratio, sanitize_nans)
    qnorm_rope_kv_insert(q, kv, k_cache, slot_mapping, positions, cos_sin_cache,
                         num_heads_padded, eps, block_size, apply_q_norm)
    sparse_logits(q, k_cache, indices, sm_scale)
    sparse_attention(q, k_cache, indices, sm_scale, weights=None)     MXFP4 records
    kv_evict(indices, weights, keep, recent)
    kv_allocate(past, added, block_table, free_pages, block_size, num_tokens)
    kv_slots(block_table, lengths, block_size, width, first=None)
    kv_slots_packed(block_table, lengths, block_size, total, first=None)
    prompt_attention(q, kv, starts, sm_scale, kv_starts=None, causal=True)
    prefix_attention(q, k_cache, prefix, indices, sm_scale)           MXFP4 records

Every call takes launch_opts=LaunchOpts(...); `with launch_policy(...)` sets them for
the calls of the current thread (context).
"""
from .build import build as _build_lib
from ._binding import (CacheDesc, ERR_INDEX, ERR_POS, ERR_SCALE, ERR_SLOT, ERR_TIMEOUT, GkrError,
                       LaunchOpts, MXFP4,
                       PACKED, RECORDS, alloc_cache, cache_bytes, get_early_metadata,
                       get_insert_staged_min, get_insert_stream_min, get_pdl,
                       insert_kernel_for, kv_allocate, kv_evict, kv_gather, kv_insert, kv_slots,
                       kv_slots_packed, launch_policy, lib,
                       library_path, page_stride, prefix_attention, prefix_attention_workspace,
                       prompt_attention, prompt_attention_workspace, qnorm_rope_kv_insert,
                       record_rows,
                       rope_quant_insert, set_early_metadata, set_insert_staged_min,
                       set_insert_stream_min, set_pdl, sparse_attention,
                       sparse_attention_workspace, sparse_logits, status_string)

__all__ = ["build", "kv_insert", "kv_gather", "rope_quant_insert", "qnorm_rope_kv_insert",
           "sparse_logits", "sparse_attention", "sparse_attention_workspace", "kv_evict",
           "kv_allocate", "kv_slots", "kv_slots_packed", "prompt_attention",
           "prompt_attention_workspace", "prefix_attention", "prefix_attention_workspace",
           "ERR_TIMEOUT", "MXFP4",
           "LaunchOpts", "launch_policy", "page_stride", "record_rows",
           "alloc_cache", "cache_bytes", "status_string", "set_pdl", "get_pdl",
           "set_early_metadata", "get_early_metadata", "set_insert_stream_min",
           "get_insert_stream_min", "set_insert_staged_min", "get_insert_staged_min",
           "insert_kernel_for", "GkrError", "CacheDesc", "RECORDS", "PACKED", "ERR_SLOT",
           "ERR_POS", "ERR_INDEX", "ERR_SCALE", "lib", "library_path"]


def build(force: bool = False):
    """Compile libgkr.so for sm_103a in-tree (skipped when up to date)."""
    return _build_lib(force=force)
