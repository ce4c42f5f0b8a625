"""MI355X (gfx950) per-group fp8 scaling: Python binding of libmgs.so.

The functions below carry the names of the C entry points in include/mgs.h
and only marshal arguments: they check torch tensors, allocate outputs the
caller did not pass, and call the library on the current HIP stream. Every
step of the computation runs in the library's HIP kernels. There is no CPU
fallback: if libmgs.so is missing, the first call raises. The calls of gated
feed-forward layers and of 8-bit integers stand in the module ``feedforward``
and are found here by their names too.
"""
from __future__ import annotations

from ._lib import (  # noqa: F401
    MGS_ACT_GELU, MGS_ACT_SILU, MGS_ERR_HIP, MGS_ERR_INVALID_ARG, MGS_ERR_UNSUPPORTED, MGS_FLAG_ACCUMULATE,
    MGS_FLAG_FAST_ACCUM, MGS_FLAG_POW2_SCALE, MGS_FLAG_VALIDATE, MGS_I8_MAX_K, MGS_MAX_GROUPS, MGS_MOE_MAX_TOP_K,
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
from . import feedforward  # noqa: E402,F401

_FEEDFORWARD = ("mgs_mm_gated_block128", "mgs_mm_gated_grad_block128", "mgs_quant_rows_i8", "mgs_mm_i8", "mgs_mm_gated_i8")


def __getattr__(name):
    if name in _FEEDFORWARD:
        return getattr(feedforward, name)
    raise AttributeError("module %r has no attribute %r" % (__name__, name))


def __dir__():
    return sorted([*globals(), *_FEEDFORWARD])
