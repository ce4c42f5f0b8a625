"""Torch-tensor front end of the gated feed-forward calls and of the 8-bit
integer ones (argument marshalling only).

A training step of gated experts, w1 (E, 2 F, K) the gate's and the other
projection's rows, w2 (E, K, F), F % 128 == 0, with what mgs_moe_dispatch gives:

    b1, s1, b1_t, s1_t = mgs_quant_blocks128(w1)
    b2, s2, b2_t, s2_t = mgs_quant_blocks128(w2)
    h, gu = mgs_mm_gated_block128(a, sa, b1.view(2 * E, F, K), s1.view(2 * E, -1, s1.shape[2]), offsets, keep=True)
    yp = mgs_mm_block128(*mgs_quant_rows128(h), b2, s2, offsets)
    # backward, from dyp
    dgu, h = mgs_mm_gated_grad_block128(*mgs_quant_rows128(dyp), b2_t, s2_t, gu, offsets, hidden=True)
    dxp = mgs_mm_block128(*mgs_quant_rows128(dgu), b1_t, s1_t, offsets)
    t = lambda v: mgs_quant_groups_dim0_t(v, offsets)
    dw1, dw2 = mgs_mm_wgrad(*t(dgu), *t(xp), offsets), mgs_mm_wgrad(*t(dyp), *t(h), offsets)

and the same layer in serving, on 8-bit integers (w1 as (2 E, F, K), offsets and
rows sorted with `mgs_moe_sort` or taken from a dispatch with `permuted`):

    b1, s1, b2, s2 = *mgs_quant_rows_i8(w1), *mgs_quant_rows_i8(w2)
    h = mgs_mm_gated_i8(*mgs_quant_rows_i8(xp), b1, s1, offsets)
    yp = mgs_mm_i8(*mgs_quant_rows_i8(h), b2, s2, offsets)
"""
from __future__ import annotations

from typing import Optional, Tuple

import torch

from ._lib import MGS_ACT_GELU, MGS_ACT_SILU, MGS_FLAG_FAST_ACCUM, check, lib
from .api import _BF16_LIKE, _U8_LIKE, _need, _out, _stream_handle
from .experts import _input, _out_type, _ptr

_I8, _F32, _I32 = (torch.int8,), (torch.float32,), (torch.int32,)
_ZEROS_SCALE = 127000001904640.0            # 127 / 1e-12 in float32, the scale of a row of zeros


def _run(name: str, t: torch.Tensor, *args):
    """Calls the entry point with t's device current: kernels are launched there."""
    if t.get_device() == torch.cuda.current_device():
        st = getattr(lib(), name)(*args)
    else:
        with torch.cuda.device(t.device):
            st = getattr(lib(), name)(*args)
    check(name, st)


def _stream(stream, device):
    """`stream`, or the device's current one, as torch's own object."""
    if stream is None:
        return torch.cuda.current_stream(device)
    return stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(_stream_handle(stream), device=device)


def _given(t, first, name: str, dtypes, shape):
    """_input, with its checks in one expression: a call's host time counts where its kernel takes microseconds."""
    if not (type(t) is torch.Tensor and t.is_cuda and t.dtype in dtypes and t.shape == shape and t.is_contiguous() and
            t.get_device() == first.get_device()):
        _input(t, first, name, dtypes, shape)


def _operands(a, a_scales, b, b_scales, offsets, dtypes, matrices: int) -> Tuple[int, ...]:
    """Checks rows a (M, K) and weights b (matrices * E, N, K), their scales
    (of blocks of 128, or of rows of 8-bit integers) and the E end offsets;
    M, K, E, N."""
    _need(a, "a", dtypes, 2)
    M, K = a.shape
    _need(b, "b", dtypes, 3)
    W, N = b.shape[:2]
    if W % matrices:
        raise ValueError("b has %d matrices, %d for each group" % (W, matrices))
    _given(b, a, "b", dtypes, (W, N, K))
    if dtypes is _I8:
        _given(a_scales, a, "a_scales", _F32, (M,))
        _given(b_scales, a, "b_scales", _F32, (W, N))
    else:
        kb = (K + 127) // 128
        _given(a_scales, a, "a_scales", _F32, (M, kb))
        _given(b_scales, a, "b_scales", _F32, (W, (N + 127) // 128, kb))
    if offsets is not None:
        _given(offsets, a, "offsets", _I32, (W // matrices,))
    return M, K, W // matrices, N


def _act(act: int) -> int:
    if act not in (MGS_ACT_SILU, MGS_ACT_GELU):
        raise ValueError("act must be MGS_ACT_SILU or MGS_ACT_GELU")
    return int(act)


def mgs_mm_gated_block128(a: torch.Tensor, a_scales: torch.Tensor, b: torch.Tensor, b_scales: torch.Tensor,
                          offsets: Optional[torch.Tensor] = None, act: int = MGS_ACT_SILU, fast_accum: bool = False,
                          keep: bool = False, h: Optional[torch.Tensor] = None, gu: Optional[torch.Tensor] = None,
                          stream=None):
    """Both projections of a gated layer, its activation and their product:
    rows a (M, K) E4M3 with scales (M, ceil(K/128)) times the group's two
    weights b (2 E, F, K) E4M3, matrix 2 e the gate and 2 e + 1 the other,
    scales (2 E, ceil(F/128), ceil(K/128)). Returns h (M, F) bf16, act(g) * u,
    and with `keep` (or a passed gu) also gu (M, 2 F) bf16, g then u of each
    row. offsets and fast_accum are mgs_mm_block128's."""
    M, K, E, F = _operands(a, a_scales, b, b_scales, offsets, _U8_LIKE, 2)
    act = _act(act)
    h = _out(h, (M, F), torch.bfloat16, a.device, "h", stream)
    if keep or gu is not None:
        gu = _out(gu, (M, 2 * F), torch.bfloat16, a.device, "gu", stream)
    _run("mgs_mm_gated_block128", a, a.data_ptr(), a_scales.data_ptr(), M, K, b.data_ptr(), b_scales.data_ptr(), E, F,
         _ptr(offsets), act, MGS_FLAG_FAST_ACCUM if fast_accum else 0, h.data_ptr(),
         _ptr(gu), _stream_handle(stream, a))
    return h if gu is None else (h, gu)


def mgs_mm_gated_grad_block128(dy: torch.Tensor, dy_scales: torch.Tensor, b: torch.Tensor, b_scales: torch.Tensor,
                               gu: torch.Tensor, offsets: Optional[torch.Tensor] = None, act: int = MGS_ACT_SILU,
                               fast_accum: bool = False, hidden: bool = False, dgu: Optional[torch.Tensor] = None,
                               h: Optional[torch.Tensor] = None, stream=None):
    """The gradients of both projections from the output's, dy (M, D) E4M3
    with scales (M, ceil(D/128)): b (E, F, D) and scales (E, ceil(F/128),
    ceil(D/128)) are the transposed cast of the down weight, gu (M, 2 F) bf16
    what the forward call kept. Returns dgu (M, 2 F) bf16, dg then du of each
    row (a passed dgu may be gu), and with `hidden` (or a passed h) also h (M, F) bf16, act(g) * u."""
    M, D, E, F = _operands(dy, dy_scales, b, b_scales, offsets, _U8_LIKE, 1)
    _given(gu, dy, "gu", _BF16_LIKE, (M, 2 * F))
    act = _act(act)
    dgu = _out(dgu, (M, 2 * F), torch.bfloat16, dy.device, "dgu", stream)
    if hidden or h is not None:
        h = _out(h, (M, F), torch.bfloat16, dy.device, "h", stream)
    _run("mgs_mm_gated_grad_block128", dy, dy.data_ptr(), dy_scales.data_ptr(), M, D, b.data_ptr(), b_scales.data_ptr(),
         E, F, _ptr(offsets), act, MGS_FLAG_FAST_ACCUM if fast_accum else 0,
         gu.data_ptr(), dgu.data_ptr(), _ptr(h), _stream_handle(stream, dy))
    return dgu if h is None else (dgu, h)


def mgs_quant_rows_i8(x: torch.Tensor, q: Optional[torch.Tensor] = None, scales: Optional[torch.Tensor] = None,
                      stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """8-bit integers with one scale for each row: x (M, K) bf16, or the
    weights (E, N, K) of experts. Returns q int8 of x's shape and scales
    float32 of its leading dims; rows of no columns have the scale of rows of
    zeros."""
    _need(x, "x", _BF16_LIKE)
    if x.dim() not in (2, 3):
        raise ValueError("x must have 2 or 3 dims")
    if q is None and scales is None and stream is None:      # the cheapest way to both: one token's cast takes 2 us
        q, scales = torch.empty_like(x, dtype=torch.int8), x.new_empty(x.shape[:-1], dtype=torch.float32)
    else:
        q = _out(q, tuple(x.shape), torch.int8, x.device, "q", stream)
        scales = _out(scales, tuple(x.shape[:-1]), torch.float32, x.device, "scales", stream)
    if x.shape[-1] == 0:                                     # the call does nothing
        with torch.cuda.device(x.device), torch.cuda.stream(_stream(stream, x.device)):
            scales.fill_(_ZEROS_SCALE)
        return q, scales
    _run("mgs_quant_rows_i8", x, x.data_ptr(), scales.numel(), x.shape[-1], q.data_ptr(), scales.data_ptr(),
         _stream_handle(stream, x))
    return q, scales


def mgs_mm_i8(a: torch.Tensor, a_scales: torch.Tensor, b: torch.Tensor, b_scales: torch.Tensor,
              offsets: Optional[torch.Tensor] = None, out_dtype=torch.bfloat16, y: Optional[torch.Tensor] = None,
              stream=None) -> torch.Tensor:
    """Rows a (M, K) int8 with scales (M) times the transposed weight b
    (E, N, K) int8, scales (E, N), of the group that each row is in (int32 end
    offsets over M; None with E == 1: one dense product). Returns y (M, N);
    rows past the last group are zero. Sums are exact."""
    M, K, E, N = _operands(a, a_scales, b, b_scales, offsets, _I8, 1)
    kind = _out_type(out_dtype)
    y = _out(y, (M, N), out_dtype, a.device, "y", stream)
    _run("mgs_mm_i8", a, a.data_ptr(), a_scales.data_ptr(), M, K, b.data_ptr(), b_scales.data_ptr(), E, N,
         _ptr(offsets), kind, y.data_ptr(), _stream_handle(stream, a))
    return y


def mgs_mm_gated_i8(a: torch.Tensor, a_scales: torch.Tensor, b: torch.Tensor, b_scales: torch.Tensor,
                    offsets: Optional[torch.Tensor] = None, act: int = MGS_ACT_SILU, h: Optional[torch.Tensor] = None,
                    stream=None) -> torch.Tensor:
    """mgs_mm_gated_block128's h (M, F) bf16 of 8-bit integers: a (M, K) int8
    with scales (M), b (2 E, F, K) int8 with scales (2 E, F)."""
    M, K, E, F = _operands(a, a_scales, b, b_scales, offsets, _I8, 2)
    act = _act(act)
    h = _out(h, (M, F), torch.bfloat16, a.device, "h", stream)
    _run("mgs_mm_gated_i8", a, a.data_ptr(), a_scales.data_ptr(), M, K, b.data_ptr(), b_scales.data_ptr(), E, F,
         _ptr(offsets), act, h.data_ptr(), _stream_handle(stream, a))
    return h
