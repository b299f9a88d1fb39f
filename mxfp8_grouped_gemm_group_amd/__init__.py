"""MI355X-native fused MXFP8 grouped-matmul + finalize-routing (MoE combine), and
the operators around it in a MoE block: the router's choice (``moe_route``),
dense products (``linear``; with an adapter per request: ``lora_linear``), the
experts for a few tokens (``moe_decode``) and the experts' products in 16 bits with
their gradients (``grouped_linear``, ``grouped_linear_wgrad``).

The operators run in libgfr.so (HIP kernels for gfx950, C ABI in
include/gfr.h); this package is its thin Python binding plus the seeded input
generators (``workloads``).  The library is loaded on first use and its absence
is an error: there is no fallback implementation.
"""
from ._binding import (DEV_BAD_ADAPTER, DEV_BAD_EXPERT, DEV_BAD_GROUP_LIST, DEV_BAD_ROW_INDEX,
                       GfrError, gemm1_swiglu_quant, gmm_finalize_routing,
                       gmm_finalize_routing_det_noalloc, load_library, status_string,
                       w4a8_finalize_routing, workspace_size)
from ._layer import (DECODE_MAX_TOKENS, RouteResult, grouped_linear, grouped_linear_wgrad, linear,
                     lora_linear, lora_linear_workspace_size, moe_decode,
                     moe_decode_workspace_size, moe_route)

__all__ = ["gmm_finalize_routing", "gmm_finalize_routing_det_noalloc", "gemm1_swiglu_quant",
           "w4a8_finalize_routing", "workspace_size", "status_string", "load_library",
           "GfrError", "DEV_BAD_GROUP_LIST", "DEV_BAD_ROW_INDEX", "DEV_BAD_EXPERT", "linear",
           "moe_decode", "moe_decode_workspace_size", "moe_route", "RouteResult",
           "DECODE_MAX_TOKENS", "grouped_linear", "grouped_linear_wgrad",
           "lora_linear", "lora_linear_workspace_size", "DEV_BAD_ADAPTER"]
