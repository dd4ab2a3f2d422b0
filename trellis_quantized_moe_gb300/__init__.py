"""GB300 (sm_103a) fused EXL3 routed-expert MoE layer.

The compute runs in the CUDA library built from csrc/ (see include/exl3.h);
this package holds its build script and a thin ctypes binding.
"""
from .binding import (  # noqa: F401
    DeviceExperts, DeviceProjection, DeviceStages, Exl3Error,
    exl3_abi_version, exl3_linear, exl3_linear_workspace_bytes, exl3_moe_additive,
    exl3_moe_forward, exl3_moe_workspace_bytes, exl3_route_pack, exl3_route_pack_max_tiles,
    exl3_workspace_error, DeviceAdapters, exl3_lora_backward, exl3_lora_forward,
    exl3_lora_h_cols, exl3_lora_plan, exl3_lora_plan_bytes, exl3_lora_workspace_bytes,
    exl3_router_backward, exl3_router_forward, exl3_router_workspace_bytes, DeviceAdamW, exl3_adamw,
    exl3_adamw_workspace_bytes, exl3_combine, exl3_combine_backward, exl3_dispatch, exl3_dispatch_plan,
    exl3_dispatch_workspace_bytes, EXL3_E4M3, EXL3_E4M3_RANDOM, EXL3_F16, EXL3_BF16, EXL3_F32, EXL3_I32, EXL3_I64,
)
