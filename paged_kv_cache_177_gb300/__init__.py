"""GB300-native PagedAttention decode.

The compute path is the CUDA library ``libpagedkv.so`` (C ABI in
``include/pagedkv.h``), reached from Python through ``binding``:
``paged_decode_attention``, ``kv_append``, ``copy_blocks`` and the checks
around them, and the serving calls beside those: the cache in 8-bit floating
point (``kv_append_e4m3``, ``paged_decode_attention_e4m3``), the pass from the
projections to the cache (``qk_norm_rope_append``) and trees of drafted tokens
(``paged_tree_attention``, ``kv_accept_layers``).  ``block_manager`` and ``scheduler`` are the host-side paging and
continuous-batching logic that produce the calls' metadata; ``workloads``
draws seeded synthetic inputs.

The binding is imported on first use, so the host-side modules work on
machines without the library or a GPU.
"""
__version__ = "0.1.0"

_BINDING_NAMES = {
    "paged_decode_attention", "kv_append", "copy_blocks", "check_copy_pairs", "validate", "validate_slots",
    "swap_blocks", "check_swap_pairs", "paged_decode_attention_shared_prefix", "paged_prefill_attention",
    "paged_decode_step", "shared_prefix_workspace_bytes", "prefix_groups", "copy_blocks_layers", "kv_append_layers",
    "layer_pointers", "device_error", "workspace_bytes", "partition_tokens", "decode_launches", "decode_persistent",
    "status_string", "version", "PagedKVError", "e4m3_cache", "kv_append_e4m3", "dequantize_blocks",
    "paged_decode_attention_e4m3", "e4m3_workspace_bytes", "qk_norm_rope_append", "tree_masks",
    "paged_tree_attention", "tree_workspace_bytes", "kv_accept_layers",
}


def __getattr__(name):
    if name in _BINDING_NAMES:
        from . import binding
        return getattr(binding, name)
    raise AttributeError(name)
