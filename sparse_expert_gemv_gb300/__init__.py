"""Output-centric small-batch MoE decode layer for GB300 (sm_103a).

The layer of the warp-decode post (cursor.com/blog/warp-decode): tokens are
routed to k of E experts; a gate/up kernel computes SiLU(gate) * up per
(token, routed expert, neuron) and a down kernel computes the routing-weighted
sum over the top-k experts per (token, output dimension). Weights are MXFP8
(E4M3 codes with one UE8M0 scale per 32 elements along the reduction axis),
decoded to FP32 in registers, one warp per output.

For calls of many tokens, prompt.py has the operators of the whole block with
MXFP8 activations (residual norm, grouping by expert, ragged expert products
on the tensor cores, weighted combination), and MoEDecode.prompt runs them.
block.py has what stands between the routed experts, for prompts and decode
batches alike: the router's choice, the norms around a block's end, dense
products with their epilogues.

The compute lives in libmoe_decode.so (C ABI, include/moe_decode.h,
include/moe_prompt.h and include/moe_block.h). This package is a thin ctypes binding: PyTorch supplies device memory and streams.
"""
from ._lib import (LIB_PATH, MOE_DEVICE_BAD_ID, MOE_DEVICE_TIMEOUT, MOE_FLAG_HOST_COPY,
                   MOE_FLAG_MXFP4, MOE_FLAG_NO_PDL, MOE_FLAG_WARP_MMA, MoEConfig, MoEError, check,
                   lib)
from .block import DenseProduct, norm_add_norm, route_experts
from .layer import MoEDecode
from .prompt import GroupedProduct, RmsNorm, add_rms_norm, combine, group_by_expert

__all__ = ["MoEDecode", "GroupedProduct", "RmsNorm", "add_rms_norm", "combine", "group_by_expert",
           "DenseProduct", "norm_add_norm", "route_experts", "MoEError", "MoEConfig", "lib", "check", "LIB_PATH",
           "MOE_DEVICE_BAD_ID", "MOE_DEVICE_TIMEOUT", "MOE_FLAG_HOST_COPY", "MOE_FLAG_MXFP4",
           "MOE_FLAG_NO_PDL", "MOE_FLAG_WARP_MMA"]
