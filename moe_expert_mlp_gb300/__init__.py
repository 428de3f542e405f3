"""Routed-expert MLP (grouped GEMM over ragged expert groups, forward and
backward) for one NVIDIA GB300, as a C-ABI CUDA library with a thin Python
binding.  See include/moe.h for the boundary."""
from ._lib import (  # noqa: F401
    EXPORTS,
    GradList,
    MoeError,
    lib,
    make_block_norm_desc,
    make_desc,
    moe_block_norm_workspace_size,
    moe_block_post_norm_bwd,
    moe_block_post_norm_fwd,
    moe_block_pre_norm_bwd,
    moe_block_pre_norm_fwd,
    moe_clip_grads,
    moe_fc1_padded_width,
    moe_grad_norm,
    moe_grad_norm_workspace_size,
    moe_group_offsets,
    moe_mlp_bwd,
    moe_mlp_fwd,
    moe_mlp_desc_t,
    moe_permute_bwd,
    moe_read_device_status,
    moe_repack_fc1,
    moe_route_bwd,
    moe_route_permute,
    moe_unpack_fc1,
    moe_unpermute_combine,
    moe_unpermute_combine_bwd,
    moe_workspace_size,
)
from .block import MoEResidualBlock  # noqa: F401
from .layer import MoEExpertMLP  # noqa: F401
