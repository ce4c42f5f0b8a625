"""A mixture-of-experts layer in E4M3, forward and backward, from the library's calls.

Each token goes to its top_k experts, an expert is relu(x w1^T) w2^T, and a
token's results are summed with its router weights:

    dispatch -> product with w1 -> relu -> cast -> product with w2 -> combine

Weights are cast once per step in blocks of 128 x 128, in both orders; rows are
cast in blocks of 128; the weight gradients read the transposed per-group casts
(mgs_quant_groups_dim0_t), which keep one scale for each column and group. The
products with bf16 results ask for the faster sums (fast_accum), whose loss is at
most 2^-10 of the sum of a result's terms in magnitude and mostly far below the
rounding to bf16; the weight gradients are summed in binary32.

    python examples/experts_layer.py --tokens 4096 --hidden 4096 --inner 2048 --experts 16 --top-k 2
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import group_scaling_fp8_amd as mgs  # noqa: E402


def cast_weights(w1, w2):
    """What a step keeps of its weights: w1 (E, inner, hidden), w2 (E, hidden, inner) bf16."""
    return mgs.mgs_quant_blocks128(w1), mgs.mgs_quant_blocks128(w2)


def forward(x, ids, router, weights, fast_accum=True):
    """x (T, hidden) bf16, ids (T, k) int32, router (T, k) float32. Returns y
    (T, hidden) bf16 and what backward needs."""
    (w1, s1, _, _), (w2, s2, _, _) = weights
    offsets, rows, slots, a, sa, xp = mgs.mgs_moe_dispatch(x, ids, w1.shape[0], permuted=True)
    h = torch.relu_(mgs.mgs_mm_block128(a, sa, w1, s1, offsets, fast_accum=fast_accum))
    yp = mgs.mgs_mm_block128(*mgs.mgs_quant_rows128(h), w2, s2, offsets, fast_accum=fast_accum)
    return mgs.mgs_moe_combine(yp, rows, router), (offsets, rows, slots, xp, h, yp)


def backward(dy, router, weights, saved, fast_accum=True):
    """Gradients of x, the router weights, w1 and w2 (float32) from dy (T, hidden) bf16."""
    (_, _, w1_t, s1_t), (_, _, w2_t, s2_t) = weights
    offsets, rows, slots, xp, h, yp = saved
    dyp, drouter = mgs.mgs_moe_combine_grad(dy, yp, rows, slots, router)
    dh = mgs.mgs_mm_block128(*mgs.mgs_quant_rows128(dyp), w2_t, s2_t, offsets, fast_accum=fast_accum)
    dh = torch.where(h > 0, dh, 0)
    dxp = mgs.mgs_mm_block128(*mgs.mgs_quant_rows128(dh), w1_t, s1_t, offsets, fast_accum=fast_accum)
    dx = mgs.mgs_moe_combine(dxp, rows)
    t = {name: mgs.mgs_quant_groups_dim0_t(v, offsets) for name, v in (("dyp", dyp), ("h", h), ("dh", dh), ("xp", xp))}
    dw2 = mgs.mgs_mm_wgrad(*t["dyp"], *t["h"], offsets)
    dw1 = mgs.mgs_mm_wgrad(*t["dh"], *t["xp"], offsets)
    return dx, drouter, dw1, dw2


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--inner", type=int, default=2048)
    ap.add_argument("--experts", type=int, default=16)
    ap.add_argument("--top-k", type=int, default=2)
    ap.add_argument("--steps", type=int, default=10)
    a = ap.parse_args()
    gen = torch.Generator(device="cuda")
    gen.manual_seed(0)

    def normal(*shape, sigma):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16) * sigma
    x, dy = normal(a.tokens, a.hidden, sigma=1.0), normal(a.tokens, a.hidden, sigma=1.0)
    w1, w2 = (normal(a.experts, *s, sigma=0.02) for s in ((a.inner, a.hidden), (a.hidden, a.inner)))
    top = torch.topk(torch.randn((a.tokens, a.experts), generator=gen, device="cuda"), a.top_k)
    ids, router = top.indices.to(torch.int32).contiguous(), torch.softmax(top.values, 1)

    def step():
        weights = cast_weights(w1, w2)
        y, saved = forward(x, ids, router, weights)
        return (y,) + backward(dy, router, weights, saved)
    out = step()
    for name, v in zip(("y", "dx", "drouter", "dw1", "dw2"), out):
        print("%-8s %-20s norm %.5g" % (name, tuple(v.shape), v.float().norm().item()))
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(a.steps):
        step()
    end.record()
    torch.cuda.synchronize()
    ms = start.elapsed_time(end) / a.steps
    flops = 3 * 2 * 2 * a.tokens * a.top_k * a.hidden * a.inner
    print("%.3f ms a step, %.0f TFLOP/s in the products" % (ms, flops / ms / 1e9))


if __name__ == "__main__":
    main()
