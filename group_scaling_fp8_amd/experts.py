"""Torch-tensor front end of the mixture-of-experts entry points (argument
marshalling only): tokens sorted by expert and back, the block-128 casts,
and the products that read the casts' E4M3 bytes and scales.

A training step of one expert weight w (E, N, K), for x (T, K), expert ids
and router weights (T, k):

    offsets, rows, slots, a, sa, xp = mgs_moe_dispatch(x, ids, E, permuted=True)
    b, sb, b_t, sb_t = mgs_quant_blocks128(w)
    yp = mgs_mm_block128(a, sa, b, sb, offsets)
    y = mgs_moe_combine(yp, rows, weights)
    # backward, from dy
    dyp, dweights = mgs_moe_combine_grad(dy, yp, rows, slots, weights)
    dxp = mgs_mm_block128(*mgs_quant_rows128(dyp), b_t, sb_t, offsets)
    dx = mgs_moe_combine(dxp, rows)
    dw = mgs_mm_wgrad(*mgs_quant_groups_dim0_t(dyp, offsets), *mgs_quant_groups_dim0_t(xp, offsets), offsets)
"""
from __future__ import annotations

import ctypes
import functools
from typing import Optional, Tuple

import torch

from ._lib import (MGS_ERR_INVALID_ARG, MGS_FLAG_ACCUMULATE, MGS_FLAG_FAST_ACCUM, MGS_FLAG_POW2_SCALE, MGS_OUT_BF16,
                   MGS_OUT_F32, MgsError, check, lib)
from .api import _BF16_LIKE, _U8_LIKE, _allocator, _need, _out, _stream_handle

_OUT_TYPES = {torch.bfloat16: MGS_OUT_BF16, torch.float32: MGS_OUT_F32}


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _same_device(t: torch.Tensor, first: torch.Tensor, name: str):
    if t.get_device() != first.get_device():
        raise ValueError("%s is on %s, the first input on %s" % (name, t.device, first.device))


def _shape(t: torch.Tensor, shape, name: str):
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))


def _input(t: torch.Tensor, first: torch.Tensor, name: str, dtypes, shape):
    _need(t, name, dtypes, len(shape))
    _shape(t, shape, name)
    _same_device(t, first, name)


@functools.lru_cache(maxsize=4096)
def _order_sizes(T: int, k: int, E: int, align: int) -> Tuple[int, int]:
    n, w = ctypes.c_int64(0), ctypes.c_int64(0)
    check("mgs_moe_rows", lib().mgs_moe_rows(T, k, E, align, ctypes.byref(n)))
    check("mgs_moe_workspace_bytes", lib().mgs_moe_workspace_bytes(T, k, E, ctypes.byref(w)))
    return int(n.value), int(w.value)


def mgs_moe_rows(T: int, top_k: int, n_experts: int, align: int = 16) -> int:
    """Rows that always hold T * top_k slots in n_experts groups of multiples of `align` rows."""
    return _order_sizes(int(T), int(top_k), int(n_experts), int(align))[0]


def _dispatch(x, ids, n_experts, align, pow2, cast, permuted, stream):
    _need(ids, "expert_ids", (torch.int32,), 2)
    T, k = ids.shape
    E, align = int(n_experts), int(align)
    P, need = _order_sizes(T, k, E, align)
    dev = ids.device
    D = 0
    if x is not None:
        _need(x, "x", _BF16_LIKE, 2)
        _same_device(x, ids, "x")
        if x.shape[0] != T:
            raise ValueError("x has %d tokens, expert_ids %d" % (x.shape[0], T))
        D = x.shape[1]
    empty = _allocator(stream, dev)
    offsets = empty((E,), dtype=torch.int32, device=dev)
    rows = empty((T, k), dtype=torch.int32, device=dev)
    slots = empty((P,), dtype=torch.int32, device=dev)
    q = scales = xp = ws = None
    if cast:
        q = empty((P, D), dtype=torch.uint8, device=dev)
        scales = empty((P, (D + 127) // 128), dtype=torch.float32, device=dev)
    if permuted:
        xp = empty((P, D), dtype=torch.bfloat16, device=dev)
    if need:
        ws = empty((need,), dtype=torch.uint8, device=dev)
    moves = P > 0 and D > 0
    st = lib().mgs_moe_dispatch(_ptr(x) if moves else None, T, D, ids.data_ptr(), k, E, align,
                                MGS_FLAG_POW2_SCALE if pow2 else 0, P, offsets.data_ptr(), rows.data_ptr(),
                                slots.data_ptr(), _ptr(xp) if moves else None, _ptr(q) if moves else None,
                                _ptr(scales) if moves else None, _ptr(ws), need, _stream_handle(stream, ids))
    check("mgs_moe_dispatch", st)
    return offsets, rows, slots, q, scales, xp


def mgs_moe_sort(expert_ids: torch.Tensor, n_experts: int, align: int = 16,
                 stream=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """The order alone: expert_ids (T, k) int32. Returns offsets (E) end
    offsets, rows (T, k) and slots (mgs_moe_rows) int32, -1 for none."""
    return _dispatch(None, expert_ids, n_experts, align, False, False, False, stream)[:3]


def mgs_moe_dispatch(x: torch.Tensor, expert_ids: torch.Tensor, n_experts: int, align: int = 16, pow2: bool = False,
                     permuted: bool = False, stream=None) -> Tuple[torch.Tensor, ...]:
    """Tokens x (T, D) bf16 sorted by expert and cast in blocks of 128
    columns. Returns offsets (E), rows (T, k), slots (P), q (P, D) uint8 E4M3
    and scales (P, ceil(D/128)) float32, and with `permuted` also xp (P, D)
    bf16, the rows before the cast; P = mgs_moe_rows(T, k, E, align)."""
    out = _dispatch(x, expert_ids, n_experts, align, pow2, True, permuted, stream)
    return out if permuted else out[:5]


def mgs_moe_combine(yp: torch.Tensor, rows: torch.Tensor, weights: Optional[torch.Tensor] = None,
                    y: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """y (T, D) bf16, the sum of each token's rows of yp (P, D) bf16 times its
    weights (T, k) float32 (None: 1, the gradient of the sorted copy)."""
    _need(yp, "yp", _BF16_LIKE, 2)
    _need(rows, "rows", (torch.int32,), 2)
    _same_device(rows, yp, "rows")
    P, D = yp.shape
    T, k = rows.shape
    if weights is not None:
        _input(weights, yp, "weights", (torch.float32,), (T, k))
    y = _out(y, (T, D), torch.bfloat16, yp.device, "y", stream)
    st = lib().mgs_moe_combine(yp.data_ptr(), P, D, rows.data_ptr(), T, k, _ptr(weights), y.data_ptr(),
                               _stream_handle(stream, yp))
    check("mgs_moe_combine", st)
    return y


def mgs_moe_combine_grad(dy: torch.Tensor, yp: torch.Tensor, rows: torch.Tensor, slots: torch.Tensor,
                         weights: torch.Tensor, dyp: Optional[torch.Tensor] = None,
                         dw: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """The gradient of mgs_moe_combine from dy (T, D) bf16: dyp (P, D) bf16
    and dw (T, k) float32."""
    _need(dy, "dy", _BF16_LIKE, 2)
    _need(rows, "rows", (torch.int32,), 2)
    _same_device(rows, dy, "rows")
    T, k = rows.shape
    D = dy.shape[1]
    _need(yp, "yp", _BF16_LIKE, 2)
    P = yp.shape[0]
    _input(dy, dy, "dy", _BF16_LIKE, (T, D))
    _input(yp, dy, "yp", _BF16_LIKE, (P, D))
    _input(slots, dy, "slots", (torch.int32,), (P,))
    _input(weights, dy, "weights", (torch.float32,), (T, k))
    dyp = _out(dyp, (P, D), torch.bfloat16, dy.device, "dyp", stream)
    dw = _out(dw, (T, k), torch.float32, dy.device, "dw", stream)
    st = lib().mgs_moe_combine_grad(dy.data_ptr(), yp.data_ptr(), P, D, rows.data_ptr(), slots.data_ptr(), T, k,
                                    weights.data_ptr(), dyp.data_ptr(), dw.data_ptr(), _stream_handle(stream, dy))
    check("mgs_moe_combine_grad", st)
    return dyp, dw


def mgs_quant_rows128(x: torch.Tensor, pow2: bool = False, q: Optional[torch.Tensor] = None,
                      scales: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """One scale for each row and block of 128 columns: x (M, K) bf16.
    Returns q (M, K) uint8 E4M3 and scales (M, ceil(K/128)) float32."""
    _need(x, "x", _BF16_LIKE, 2)
    M, K = x.shape
    q = _out(q, (M, K), torch.uint8, x.device, "q", stream)
    scales = _out(scales, (M, (K + 127) // 128), torch.float32, x.device, "scales", stream)
    st = lib().mgs_quant_rows128(x.data_ptr(), M, K, MGS_FLAG_POW2_SCALE if pow2 else 0, q.data_ptr(),
                                 scales.data_ptr(), _stream_handle(stream, x))
    check("mgs_quant_rows128", st)
    return q, scales


def mgs_quant_blocks128(w: torch.Tensor, pow2: bool = False, transposed: bool = True,
                        stream=None) -> Tuple[torch.Tensor, ...]:
    """One scale for each block of 128 x 128 of w (E, N, K) bf16. Returns q
    (E, N, K) uint8 E4M3 and scales (E, ceil(N/128), ceil(K/128)) float32,
    and with `transposed` also q_t (E, K, N) and scales_t."""
    _need(w, "w", _BF16_LIKE, 3)
    E, N, K = w.shape
    nb, kb = (N + 127) // 128, (K + 127) // 128
    empty = _allocator(stream, w.device)
    q = empty((E, N, K), dtype=torch.uint8, device=w.device)
    scales = empty((E, nb, kb), dtype=torch.float32, device=w.device)
    q_t = scales_t = None
    if transposed:
        q_t = empty((E, K, N), dtype=torch.uint8, device=w.device)
        scales_t = empty((E, kb, nb), dtype=torch.float32, device=w.device)
    st = lib().mgs_quant_blocks128(w.data_ptr(), E, N, K, MGS_FLAG_POW2_SCALE if pow2 else 0, q.data_ptr(),
                                   scales.data_ptr(), _ptr(q_t), _ptr(scales_t), _stream_handle(stream, w))
    check("mgs_quant_blocks128", st)
    return (q, scales, q_t, scales_t) if transposed else (q, scales)


def _out_type(dtype) -> int:
    if dtype not in _OUT_TYPES:
        raise TypeError("out_dtype must be torch.bfloat16 or torch.float32, got %s" % (dtype,))
    return _OUT_TYPES[dtype]


def mgs_mm_block128(a: torch.Tensor, a_scales: torch.Tensor, b: torch.Tensor, b_scales: torch.Tensor,
                    offsets: Optional[torch.Tensor] = None, out_dtype=torch.bfloat16,
                    fast_accum: bool = False, y: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Rows a (M, K) E4M3 with scales (M, ceil(K/128)) times the transposed
    weight b (E, N, K) E4M3, scales (E, ceil(N/128), ceil(K/128)), of the
    group that each row is in (int32 end offsets over M; None with E == 1: one
    dense product). Returns y (M, N); rows past the last group are zero.
    `fast_accum` sums in the 8-bit matrix instruction (MGS_FLAG_FAST_ACCUM)."""
    _need(a, "a", _U8_LIKE, 2)
    M, K = a.shape
    _need(b, "b", _U8_LIKE, 3)
    E, N = b.shape[:2]
    kb = (K + 127) // 128
    _input(b, a, "b", _U8_LIKE, (E, N, K))
    _input(a_scales, a, "a_scales", (torch.float32,), (M, kb))
    _input(b_scales, a, "b_scales", (torch.float32,), (E, (N + 127) // 128, kb))
    if offsets is not None:
        _input(offsets, a, "offsets", (torch.int32,), (E,))
    kind = _out_type(out_dtype)
    y = _out(y, (M, N), out_dtype, a.device, "y", stream)
    st = lib().mgs_mm_block128(a.data_ptr(), a_scales.data_ptr(), M, K, b.data_ptr(), b_scales.data_ptr(), E, N,
                               _ptr(offsets), MGS_FLAG_FAST_ACCUM if fast_accum else 0, kind, y.data_ptr(),
                               _stream_handle(stream, a))
    check("mgs_mm_block128", st)
    return y


def mgs_mm_wgrad(a_t: torch.Tensor, a_scales_t: torch.Tensor, b_t: torch.Tensor, b_scales_t: torch.Tensor,
                 offsets: torch.Tensor, out_dtype=torch.float32, fast_accum: bool = False,
                 dw: Optional[torch.Tensor] = None, accumulate: bool = False, stream=None) -> torch.Tensor:
    """Each group's weight gradient dw (G, N, K) from two outputs of
    mgs_quant_groups_dim0_t: a_t (N, M), a_scales_t (N, G) of the output
    gradient and b_t (K, M), b_scales_t (K, G) of the input, with their int32
    end offsets over M (multiples of 16). `accumulate` adds to dw (float32),
    `fast_accum` sums in the 8-bit matrix instruction (MGS_FLAG_FAST_ACCUM)."""
    _need(a_t, "a_t", _U8_LIKE, 2)
    N, M = a_t.shape
    _need(b_t, "b_t", _U8_LIKE, 2)
    K = b_t.shape[0]
    _need(offsets, "offsets", (torch.int32,), 1)
    G = offsets.shape[0]
    _input(b_t, a_t, "b_t", _U8_LIKE, (K, M))
    _input(a_scales_t, a_t, "a_scales_t", (torch.float32,), (N, G))
    _input(b_scales_t, a_t, "b_scales_t", (torch.float32,), (K, G))
    _same_device(offsets, a_t, "offsets")
    kind = _out_type(out_dtype)
    if accumulate and dw is None:
        raise MgsError("mgs_mm_wgrad", MGS_ERR_INVALID_ARG, ": accumulate needs dw")
    dw = _out(dw, (G, N, K), out_dtype, a_t.device, "dw", stream)
    flags = (MGS_FLAG_ACCUMULATE if accumulate else 0) | (MGS_FLAG_FAST_ACCUM if fast_accum else 0)
    st = lib().mgs_mm_wgrad(a_t.data_ptr(), a_scales_t.data_ptr(), b_t.data_ptr(), b_scales_t.data_ptr(), M, N, K,
                            offsets.data_ptr(), G, flags, kind, dw.data_ptr(),
                            _stream_handle(stream, a_t))
    check("mgs_mm_wgrad", st)
    return dw
