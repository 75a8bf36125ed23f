"""B200 (sm_100a) hot path of one FreeToken-style MoE layer with FP4 experts
offloaded to pinned host memory: router, LRU expert-slot pool in HBM, copy-engine
miss streaming, FP4 SwiGLU expert FFN, router-weighted combine, the q* bandwidth
split, and beside them the grouped router and products with 4-bit matrices (a shared
expert, projections, an output head).  The work is in libmoe_fp4.so (include/moe_fp4.h); this package
is its Python binding."""
from . import _lib  # noqa: F401
from .api import (BandwidthEstimate, FP4Weight, GroupedRouting, Lookup, Pool, SharedExpert, combine,  # noqa: F401
                  decode_layer, decode_layer_routed, decode_resident,
                  dequant_slot, expert_ffn, ffn_launch_info, fp4_linear, fp4_swiglu, nvfp4_gemm,
                  nvfp4_quantize, prefill_ffn, prefill_workspace_bytes, qstar_split,
                  route, route_grouped, route_grouped_workspace_bytes, route_noalloc,
                  route_select, route_workspace_bytes, set_wait_limits, slot_lookup,
                  slot_lookup_launch, slot_lookup_result, stream_misses)
from .layer import DecodeLayer  # noqa: F401
