"""A layer of gated experts: training in E4M3, serving in 8-bit integers.

An expert is (act(x w1g^T) * (x w1u^T)) w2^T, with w1 (E, 2, inner, hidden) the
gate's rows and the other projection's. Each token goes to its top_k experts:

    dispatch -> both projections, activation, product -> cast -> product with w2 -> combine

In training the forward call keeps the projections in bf16; backward computes
their gradients in the product with w2's transpose, and the hidden rows once more
for w2's gradient. Where inner is a multiple of 128, one cast of w1 as
(E, 2 * inner, hidden) serves the forward call, as its 2 E matrices, and in its
transposed order the input gradient. In serving, weights are cast once to 8-bit
integers with a scale for each output channel and rows when they are multiplied,
with a scale for each token.

    python examples/gated_experts.py --tokens 4096 --hidden 4096 --inner 2048 --experts 16 --top-k 2
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import group_scaling_fp8_amd as mgs  # noqa: E402
from group_scaling_fp8_amd import feedforward as ff  # noqa: E402


def cast_weights(w1, w2):
    """What a training step keeps of w1 (E, 2, inner, hidden) and w2 (E, hidden, inner) bf16."""
    E, _, inner, hidden = w1.shape
    q, s, q_t, s_t = mgs.mgs_quant_blocks128(w1.view(E, 2 * inner, hidden))
    pairs = q.view(2 * E, inner, hidden)
    if inner % 128 == 0:
        s = s.view(2 * E, inner // 128, -1)
    else:                        # the pair's second matrix starts inside a block of the cast above
        pairs, s = mgs.mgs_quant_blocks128(w1.view(2 * E, inner, hidden), transposed=False)
    return (pairs, s, q_t, s_t), mgs.mgs_quant_blocks128(w2)


def forward(x, ids, router, weights, act=mgs.MGS_ACT_SILU, fast_accum=True):
    """x (T, hidden) bf16, ids (T, k) int32, router (T, k) float32. Returns y
    (T, hidden) bf16 and what backward needs."""
    (w1, s1, _, _), (w2, s2, _, _) = weights
    offsets, rows, slots, a, sa, xp = mgs.mgs_moe_dispatch(x, ids, w2.shape[0], permuted=True)
    h, gu = ff.mgs_mm_gated_block128(a, sa, w1, s1, offsets, act, fast_accum=fast_accum, keep=True)
    yp = mgs.mgs_mm_block128(*mgs.mgs_quant_rows128(h), w2, s2, offsets, fast_accum=fast_accum)
    return mgs.mgs_moe_combine(yp, rows, router), (offsets, rows, slots, xp, gu, yp)


def backward(dy, router, weights, saved, act=mgs.MGS_ACT_SILU, fast_accum=True):
    """Gradients of x, the router weights, w1 and w2 (float32) from dy (T, hidden) bf16."""
    (_, _, w1_t, s1_t), (_, _, w2_t, s2_t) = weights
    offsets, rows, slots, xp, gu, yp = saved
    dyp, drouter = mgs.mgs_moe_combine_grad(dy, yp, rows, slots, router)
    dgu, h = ff.mgs_mm_gated_grad_block128(*mgs.mgs_quant_rows128(dyp), w2_t, s2_t, gu, offsets, act,
                                           fast_accum=fast_accum, hidden=True)
    dxp = mgs.mgs_mm_block128(*mgs.mgs_quant_rows128(dgu), w1_t, s1_t, offsets, fast_accum=fast_accum)
    dx = mgs.mgs_moe_combine(dxp, rows)
    t = {name: mgs.mgs_quant_groups_dim0_t(v, offsets) for name, v in (("dyp", dyp), ("h", h), ("dgu", dgu), ("xp", xp))}
    dw2 = mgs.mgs_mm_wgrad(*t["dyp"], *t["h"], offsets)
    dw1 = mgs.mgs_mm_wgrad(*t["dgu"], *t["xp"], offsets)
    return dx, drouter, dw1.view(dw1.shape[0], 2, -1, dw1.shape[2]), dw2


def cast_weights_i8(w1, w2):
    """What a server keeps: w1 (E, 2, inner, hidden) and w2 (E, hidden, inner) bf16 as 8-bit integers."""
    E, _, inner, hidden = w1.shape
    return ff.mgs_quant_rows_i8(w1.view(2 * E, inner, hidden)), ff.mgs_quant_rows_i8(w2)


def serve(x, ids, router, weights, act=mgs.MGS_ACT_SILU):
    """The layer's y (T, hidden) bf16 in 8-bit integers."""
    w1, w2 = weights
    offsets, rows, _, _, _, xp = mgs.mgs_moe_dispatch(x, ids, w2[0].shape[0], permuted=True)
    h = ff.mgs_mm_gated_i8(*ff.mgs_quant_rows_i8(xp), *w1, offsets, act)
    yp = ff.mgs_mm_i8(*ff.mgs_quant_rows_i8(h), *w2, offsets)
    return mgs.mgs_moe_combine(yp, rows, router)


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--inner", type=int, default=2048)
    ap.add_argument("--experts", type=int, default=16)
    ap.add_argument("--top-k", type=int, default=2)
    ap.add_argument("--act", choices=("silu", "gelu"), default="silu")
    ap.add_argument("--steps", type=int, default=10)
    a = ap.parse_args()
    gen = torch.Generator(device="cuda")
    gen.manual_seed(0)

    def normal(*shape, sigma):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16) * sigma
    x, dy = normal(a.tokens, a.hidden, sigma=1.0), normal(a.tokens, a.hidden, sigma=1.0)
    w1, w2 = normal(a.experts, 2, a.inner, a.hidden, sigma=0.02), normal(a.experts, a.hidden, a.inner, sigma=0.02)
    top = torch.topk(torch.randn((a.tokens, a.experts), generator=gen, device="cuda"), a.top_k)
    ids, router = top.indices.to(torch.int32).contiguous(), torch.softmax(top.values, 1)
    act = mgs.MGS_ACT_SILU if a.act == "silu" else mgs.MGS_ACT_GELU

    def step():
        weights = cast_weights(w1, w2)
        y, saved = forward(x, ids, router, weights, act)
        return (y,) + backward(dy, router, weights, saved, act)

    def timed(f):
        f()
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        for _ in range(a.steps):
            f()
        end.record()
        torch.cuda.synchronize()
        return start.elapsed_time(end) / a.steps
    for name, v in zip(("y", "dx", "drouter", "dw1", "dw2"), step()):
        print("%-8s %-24s norm %.5g" % (name, tuple(v.shape), v.float().norm().item()))
    kept = cast_weights_i8(w1, w2)
    print("%-8s %-24s norm %.5g" % ("y int8", tuple(x.shape), serve(x, ids, router, kept, act).float().norm().item()))
    ms, one = timed(step), 2 * 3 * a.tokens * a.top_k * a.hidden * a.inner
    print("training %.3f ms a step, %.0f TFLOP/s in the products" % (ms, 3 * one / ms / 1e9))
    ms = timed(lambda: serve(x, ids, router, kept, act))
    print("serving  %.3f ms a pass, %.0f TOP/s in the products" % (ms, one / ms / 1e9))


if __name__ == "__main__":
    main()
