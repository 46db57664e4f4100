"""MI355X-native SALR linear layer.

SALR (Sparsity-Aware Low-Rank Representation) serves a linear layer as
Y = X W_s^T + (X A_cat) B_cat: W_s is the frozen weight after a static
per-row magnitude prune, stored as a bitmap plus packed bf16 values, and
A_cat / B_cat stack the truncated-SVD residual adapter with the LoRA
adapters.  Encode, forward, the adapter backward, grouped experts with their
router, dispatch and combine, adapters of many requests, and the AdamW and
Muon steps run in hand-written gfx950 HIP kernels behind the C ABI of
include/salr.h (libsalr.so); this package only marshals arguments (binding.py)
and draws synthetic inputs (synth.py).
"""

from .binding import (  # noqa: F401
    ADAMW_BLOCK,
    ADAPTERS_MAX,
    EXPORTS,
    LIB_PATH,
    MOE_MAX_TOPK,
    MUON_COEFFICIENTS,
    MUON_MAX_SIDE,
    NOALLOC_SCRATCH_BYTES,
    AdamWPlan,
    AdaptersPlan,
    MuonPlan,
    SalrAdapters,
    SalrError,
    SalrLayer,
    SalrMoE,
    WaitTimeout,
    adamw_dyn,
    adamw_plan,
    adamw_states,
    adamw_step,
    adapters_backward,
    adapters_forward,
    adapters_plan,
    adapters_plan_bytes,
    adapters_workspace,
    adapters_ws_bytes,
    backward_workspace,
    backward_ws_bytes,
    encode,
    forward_workspace,
    fuse,
    lib,
    linear_backward,
    linear_forward,
    linear_forward_noalloc,
    moe_combine,
    moe_combine_backward,
    moe_dispatch,
    moe_dispatch_backward,
    moe_dispatch_workspace,
    moe_dispatch_ws_bytes,
    moe_encode_expert,
    moe_forward,
    moe_query_sizes,
    moe_route,
    moe_route_backward,
    moe_workspace,
    muon_plan,
    muon_states,
    muon_step,
    nf4_levels,
    probe_mfma,
    probe_stream_read,
    quantize_nf4,
    query_sizes,
    transpose_count,
    transpose_layer,
    transpose_ws_bytes,
    wait_error,
    workspace,
)

__all__ = [
    "ADAMW_BLOCK", "ADAPTERS_MAX", "EXPORTS", "LIB_PATH", "MOE_MAX_TOPK", "MUON_COEFFICIENTS", "MUON_MAX_SIDE",
    "NOALLOC_SCRATCH_BYTES", "AdamWPlan", "AdaptersPlan", "MuonPlan", "SalrAdapters", "SalrError", "SalrLayer",
    "SalrMoE", "WaitTimeout", "adamw_dyn", "adamw_plan", "adamw_states", "adamw_step", "adapters_backward",
    "adapters_forward", "adapters_plan", "adapters_plan_bytes", "adapters_workspace", "adapters_ws_bytes",
    "backward_workspace", "backward_ws_bytes", "encode", "forward_workspace", "fuse", "lib", "linear_backward",
    "linear_forward", "linear_forward_noalloc", "moe_combine", "moe_combine_backward", "moe_dispatch",
    "moe_dispatch_backward", "moe_dispatch_workspace", "moe_dispatch_ws_bytes", "moe_encode_expert", "moe_forward",
    "moe_query_sizes", "moe_route", "moe_route_backward", "moe_workspace", "muon_plan", "muon_states", "muon_step",
    "nf4_levels", "probe_mfma", "probe_stream_read", "quantize_nf4", "query_sizes", "transpose_count",
    "transpose_layer", "transpose_ws_bytes", "wait_error", "workspace",
]
