"""GB300-native rotary position embedding.

Operators behind a C ABI (``include/rope_gb300.h``), implemented as
hand-written CUDA kernels for sm_103a:

* ``rope_inplace_partial`` -- in-place partial-slice interleave RoPE of a BSND
  tensor, with fp32 cos/sin allowed for fp16/bf16 x;
* ``rope_with_sin_cos_cache`` -- cos/sin-cache-indexed RoPE of query and key,
  rope or mrope mode, GPT-NeoX or GPT-J style, pass-through columns untouched;
* ``qkv_rmsnorm_rope_cache`` -- fused QKV split, RMSNorm, RoPE and paged cache write;
* ``rope_frequencies``, ``scaled_cos_sin_cache``, ``scaled_cos_sin`` -- the cos/sin
  tables that the others read, scaled for long contexts;
* ``append_paged_kv`` -- RoPE of query and key on the way to a paged KV cache;
* ``paged_attention`` -- attention over that cache, a shared prefix read once for all;
* ``append_paged_kv_8bit``, ``paged_attention_8bit`` -- the two for a cache of 8-bit codes with a
  scale for each block of tokens and head;
* ``rearrange_sequences``, ``compact_pages``, ``copy_pages`` -- sequences of a paged cache forked,
  reordered and dropped, its live pages moved to the front, pages copied in all layers' caches.

PyTorch supplies device memory and streams only.
"""
from ._capi import (  # noqa: F401
    ROPE_DEVICE_POSITION_OUT_OF_RANGE,
    ROPE_ERR_CUDA,
    ROPE_ERR_PARAM_INVALID,
    ROPE_ERR_PARAM_NULLPTR,
    ROPE_OK,
    RopeError,
    get_device_error,
    launch_count,
    PreparedCall,
    load,
    prepare_inplace_partial,
    prepare_with_sin_cos_cache,
    rope_inplace_partial,
    rope_inplace_partial_backward,
    rope_with_sin_cos_cache,
    qkv_rmsnorm_rope_cache,
    prepare_qkv_rmsnorm_rope_cache,
    ROPE_DEVICE_SLOT_OUT_OF_RANGE,
    ROPE_DEVICE_INDEX_OUT_OF_BOUNDS,
    ROPE_DEVICE_WAIT_EXPIRED,
    ROPE_DEVICE_PAGES_EXHAUSTED,
    append_paged_kv_8bit,
    compact_pages,
    copy_pages,
    paged_attention_8bit,
    prepare_append_paged_kv_8bit,
    prepare_paged_attention_8bit,
    rearrange_sequences,
    append_paged_kv,
    paged_attention,
    paged_attention_workspace,
    prepare_append_paged_kv,
    prepare_paged_attention,
    rope_frequencies,
    scaled_cos_sin,
    scaled_cos_sin_cache,
    status_string,
)

from .autograd import inplace_partial_rotary_mul  # noqa: E402,F401

__all__ = [
    "inplace_partial_rotary_mul",
    "rope_inplace_partial",
    "rope_inplace_partial_backward",
    "rope_with_sin_cos_cache",
    "qkv_rmsnorm_rope_cache",
    "rope_frequencies",
    "scaled_cos_sin_cache",
    "scaled_cos_sin",
    "append_paged_kv",
    "paged_attention",
    "paged_attention_workspace",
    "append_paged_kv_8bit",
    "paged_attention_8bit",
    "rearrange_sequences",
    "compact_pages",
    "copy_pages",
    "get_device_error",
    "launch_count",
    "status_string",
    "load",
    "RopeError",
]
