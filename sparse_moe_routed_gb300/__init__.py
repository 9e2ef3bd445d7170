"""GB300-native routed-expert MoE layer (sm_103a CUDA kernels behind a C ABI).

Importing this package does not load the CUDA library; the first call does
(building it in-tree if needed).  There is no CPU path.
"""
from . import _lib
from ._lib import (MoEError, moe_cache_fetch, moe_cache_plan, moe_combine, moe_expert_down, moe_expert_gateup,
                   moe_expert_swiglu_cached, moe_grouped_swiglu, moe_permute, moe_rmsnorm, moe_route,
                   moe_route_noalloc, moe_route_recall, route_block_dedup)
from ._block import (moe_block_norm, moe_block_norm_backward, moe_block_norm_workspace_size, moe_checkpoint_load,
                     moe_checkpoint_save, moe_collect, moe_collect_backward, moe_dispatch, moe_dispatch_backward,
                     moe_ffn, moe_ffn_backward, moe_ffn_backward_workspace_size, moe_route_backward,
                     moe_route_backward_workspace_size)
from .layer import CachedMoELayer, MoELayer, MoEStack, PrefillRing, pack_layer_experts
from .train import MoETrainLayer

__all__ = ["_lib", "MoEError", "MoELayer", "CachedMoELayer", "MoEStack", "MoETrainLayer", "PrefillRing", "pack_layer_experts",
           "moe_cache_plan", "moe_cache_fetch", "moe_expert_swiglu_cached", "moe_route", "moe_permute", "moe_expert_gateup", "moe_expert_down",
           "moe_grouped_swiglu", "moe_combine", "route_block_dedup", "moe_rmsnorm", "moe_route_noalloc",
           "moe_route_recall", "moe_dispatch", "moe_dispatch_backward", "moe_collect", "moe_collect_backward",
           "moe_block_norm", "moe_block_norm_backward", "moe_block_norm_workspace_size", "moe_route_backward",
           "moe_route_backward_workspace_size", "moe_checkpoint_save", "moe_checkpoint_load", "moe_ffn",
           "moe_ffn_backward", "moe_ffn_backward_workspace_size"]
