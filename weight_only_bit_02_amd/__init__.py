"""MI355X-native (gfx950) AWQ W4A16 hot path: quantize + pack, activation-aware scale
search, and the W4A16 linear, as hand-written HIP kernels behind a small C ABI
(include/awq.h, lib/libawq_mi355x.so)."""

from ._abi import AwqError, load as load_library  # noqa: F401
from .awq import (  # noqa: F401
    PackedLinear, SearchResult, SearchWorkspace, activation_stats, alloc_packed, apply_inverse_scale,
    candidate_scales, clip_search, gemv_max_m, linear_w4a16, linear_w4a16_gated_silu, quantize_pack,
    search_scales,
)
from .grouped import (  # noqa: F401
    LoraAdapters, PackedExperts, Routing, RowGroups, group_rows, group_rows_workspace_size,
    linear_w4a16_grouped, linear_w4a16_grouped_gated_silu, linear_w4a16_lora,
    linear_w4a16_lora_workspace_size, moe_combine, moe_route, moe_route_workspace_size,
    quantize_pack_experts,
)
from .kv import (  # noqa: F401
    KVBatch, KVCache, Rotary, alloc_kv_cache, attention_kv4, attention_kv4_workspace_size, kv_append, kv_read,
)
