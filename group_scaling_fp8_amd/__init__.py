"""MI355X (gfx950) per-group fp8 scaling: Python binding of libmgs.so.

The functions below carry the names of the C entry points in include/mgs.h
and only marshal arguments: they check torch tensors, allocate outputs the
caller did not pass, and call the library on the current HIP stream. Every
step of the computation runs in the library's HIP kernels. There is no CPU
fallback: if libmgs.so is missing, the first call raises.
"""
from __future__ import annotations

from ._lib import (  # noqa: F401
    MGS_ERR_HIP, MGS_ERR_INVALID_ARG, MGS_ERR_UNSUPPORTED, MGS_FLAG_ACCUMULATE, MGS_FLAG_FAST_ACCUM,
    MGS_FLAG_POW2_SCALE, MGS_FLAG_VALIDATE, MGS_MAX_GROUPS, MGS_MOE_MAX_TOP_K,
    MGS_MX_FLOOR, MGS_MX_RCEIL, MGS_OK, MGS_OUT_BF16, MGS_OUT_F32, MgsError, lib, library_path,
)
from .api import (  # noqa: F401
    dim0_workspace, mgs_cast_e4m3, mgs_copy, mgs_dim0_workspace_bytes, mgs_mx_dequant_dim0,
    mgs_mx_quant_dim0, mgs_mx_quant_dim1, mgs_quant_experts_dim1, mgs_quant_groups_dim0,
    mgs_quant_groups_dim0_noalloc, mgs_quant_groups_dim0_t, mgs_quant_groups_dim1,
)
from .experts import (  # noqa: F401
    mgs_mm_block128, mgs_mm_wgrad, mgs_moe_combine, mgs_moe_combine_grad, mgs_moe_dispatch, mgs_moe_rows,
    mgs_moe_sort, mgs_quant_blocks128, mgs_quant_rows128,
)
