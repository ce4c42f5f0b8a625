"""The mixture-of-experts calls together: the layer of examples/experts_layer.py
on small integers (every cast, product and sum is exact, so the results are
too), all calls in one captured graph, and calls on another stream."""
import os
import sys

import numpy as np
import pytest
import torch

import experts_ref as ref
import oracle
import group_scaling_fp8_amd as mgs
from group_scaling_fp8_amd import workloads as wl
from gpu_util import assert_same_bytes, to_dev

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import experts_layer  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mgs.lib()


def plain_layer(x, ids, router, w1, w2, dy):
    """The layer and its gradients in 64 bits, token by token."""
    T, k = ids.shape
    y, dx, drouter = np.zeros(x.shape), np.zeros(x.shape), np.zeros((T, k))
    dw1, dw2 = np.zeros(w1.shape), np.zeros(w2.shape)
    for t in range(T):
        for s in range(k):
            e = ids[t, s]
            if not 0 <= e < len(w1):
                continue
            h = np.maximum(w1[e] @ x[t], 0)
            out = w2[e] @ h
            y[t] += router[t, s] * out
            drouter[t, s] = dy[t] @ out
            g = router[t, s] * dy[t]
            dh = (w2[e].T @ g) * (h > 0)
            dx[t] += w1[e].T @ dh
            dw2[e] += np.outer(g, h)
            dw1[e] += np.outer(dh, x[t])
    return y, dx, drouter, dw1, dw2


def signs(rng, shape, ones):
    """`ones` entries of +-1 in every row, zeros elsewhere."""
    a = np.zeros((int(np.prod(shape[:-1])), shape[-1]))
    for row in a:
        row[rng.choice(shape[-1], ones, replace=False)] = rng.choice([-1.0, 1.0], ones)
    return a.reshape(shape)


@pytest.mark.parametrize("T,k,E,hidden,inner", [(1, 2, 4, 64, 32), (45, 3, 5, 272, 144), (150, 2, 4, 144, 400)])
@pytest.mark.parametrize("fast", [False, True])
def test_layer_on_small_integers(T, k, E, hidden, inner, fast):
    """A token and its gradient have one entry of +-1, weights are 0 and +-1:
    an expert's inner values are 0 and 1, their gradients 0 and +- the router
    weight, so every cast is exact (one magnitude, a power of two, in a block)
    and results are multiples of 1/2 of at most 8 bits, exact in bf16. What is
    left are the roundings of the scales' reciprocals, at most 2^-20 of a
    result below 256: far under half a step of 1/2."""
    rng = np.random.default_rng(T)
    ids = np.argsort(rng.random((T, E)), 1)[:, :k].astype(np.int32)
    ids[rng.random((T, k)) < 0.1] = -1
    x, dy = signs(rng, (T, hidden), 1), signs(rng, (T, hidden), 1)
    w1, w2 = signs(rng, (E, inner, hidden), hidden // 4), signs(rng, (E, hidden, inner), inner // 4)
    router = rng.choice([0.5, 1.0, 2.0], (T, k))
    want = plain_layer(x, ids, router, w1, w2, dy)
    assert all(np.abs(v).max() <= 64 for v in want)
    dev = {n: to_dev(wl.f32_to_bf16_bits(v.astype(np.float32))).view(torch.bfloat16)
           for n, v in (("x", x), ("dy", dy), ("w1", w1), ("w2", w2))}
    router_d, ids_d = to_dev(router.astype(np.float32)), to_dev(ids)
    weights = experts_layer.cast_weights(dev["w1"], dev["w2"])
    y, saved = experts_layer.forward(dev["x"], ids_d, router_d, weights, fast)
    got = (y,) + experts_layer.backward(dev["dy"], router_d, weights, saved, fast)
    for name, a, b in zip(("y", "dx", "drouter", "dw1", "dw2"), got, want):
        assert np.abs(a.double().cpu().numpy() - b).max() <= 2.0 ** -12, name


def test_wgrad_reads_dim0_t_of_rows_past_the_last_group():
    """Row arrays are longer than their groups: dim0_t leaves the columns past
    the last end alone, and the weight gradient does not read them."""
    rng = np.random.default_rng(11)
    T, k, E, D = 100, 2, 6, 144
    ids = rng.integers(0, E, (T, k)).astype(np.int32)
    x = wl.randn_bf16(rng, (T, D), 0.02, 0.001, 8.0)
    off, rows, slots, q, s, xp = mgs.mgs_moe_dispatch(to_dev(x), to_dev(ids), E, permuted=True)
    P = slots.shape[0]
    end = int(off[-1])
    assert end < P
    q_t = torch.full((D, P), 0x7F, dtype=torch.uint8, device="cuda")
    q_t, s_t = mgs.mgs_quant_groups_dim0_t(xp, off, q_t=q_t)
    r_q, r_s = oracle.quant_groups_dim0_t(np.ascontiguousarray(xp.view(torch.int16).cpu().numpy().view(np.uint16)[:end]),
                                          off.cpu().numpy())
    assert_same_bytes(np.ascontiguousarray(q_t.cpu().numpy()[:, :end]), r_q, "q_t")
    assert_same_bytes(s_t.cpu().numpy(), r_s, "scales_t")
    dw = mgs.mgs_mm_wgrad(q_t, s_t, q_t, s_t, off)
    want, mag = ref.mm_wgrad(r_q, r_s, r_q, r_s, off.cpu().numpy())
    assert (np.abs(dw.cpu().numpy() - want) <= ref.mm_tolerance(want, mag, P, "f32")).all()


def inputs(seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    T, k, E, D, N = 700, 2, 6, 272, 144
    ids = torch.randint(-1, E, (T, k), generator=gen, device="cuda", dtype=torch.int32)
    return {"x": torch.randn((T, D), generator=gen, device="cuda", dtype=torch.bfloat16), "ids": ids,
            "router": torch.rand((T, k), generator=gen, device="cuda"),
            "dy": torch.randn((T, D), generator=gen, device="cuda", dtype=torch.bfloat16),
            "w1": torch.randn((E, N, D), generator=gen, device="cuda", dtype=torch.bfloat16) * 0.05,
            "w2": torch.randn((E, D, N), generator=gen, device="cuda", dtype=torch.bfloat16) * 0.05}


def all_calls(v, ws):
    """Every call once (mgs_moe_sort through the dispatch of more slots than one
    launch takes); the weight gradients' casts in a caller's workspace."""
    b1, b2 = experts_layer.cast_weights(v["w1"], v["w2"])
    off, rows, slots, a, sa, xp = mgs.mgs_moe_dispatch(v["x"], v["ids"], v["w1"].shape[0], permuted=True)
    h = torch.relu(mgs.mgs_mm_block128(a, sa, b1[0], b1[1], off, fast_accum=True))
    yp = mgs.mgs_mm_block128(*mgs.mgs_quant_rows128(h), b2[0], b2[1], off)
    y = mgs.mgs_moe_combine(yp, rows, v["router"])
    dyp, dr = mgs.mgs_moe_combine_grad(v["dy"], yp, rows, slots, v["router"])
    small = mgs.mgs_moe_dispatch(v["x"][:40], v["ids"][:40], v["w1"].shape[0])
    few = mgs.mgs_mm_block128(small[3], small[4], b1[0], b1[1], small[0], torch.float32)
    ta = mgs.mgs_quant_groups_dim0_t(dyp, off, workspace=ws)
    tb = mgs.mgs_quant_groups_dim0_t(h, off, workspace=ws)
    dw = mgs.mgs_mm_wgrad(*ta, *tb, off)
    return {"off": off, "rows": rows, "slots": slots, "a": a, "sa": sa, "h": h, "yp": yp, "y": y, "dyp": dyp, "dr": dr,
            "few": few, "dw": dw, "small": small[2]}


def test_every_call_in_one_graph():
    v = inputs(1)
    ws = mgs.dim0_workspace(4096, 512)
    want = {seed: {n: t.clone() for n, t in all_calls(inputs(seed), ws).items()} for seed in (1, 2, 3)}
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        out = all_calls(v, ws)
    torch.cuda.synchronize()
    for seed in (2, 3, 1, 2):
        for n, t in inputs(seed).items():
            v[n].copy_(t)
        for t in out.values():
            t.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for n, t in out.items():
            assert torch.equal(t.view(torch.uint8), want[seed][n].view(torch.uint8)), (seed, n)
        # eager work of the same calls between the replays
        with torch.cuda.stream(s):
            again = all_calls(inputs(seed), ws)
        torch.cuda.synchronize()
        for n, t in again.items():
            assert torch.equal(t.view(torch.uint8), want[seed][n].view(torch.uint8)), (seed, n)


def test_calls_on_another_stream():
    """With `stream` given, work runs there: behind what is queued on it, with
    nothing on the default stream to wait for."""
    v = inputs(5)
    ws = mgs.dim0_workspace(4096, 512)
    want = {n: t.clone() for n, t in all_calls(v, ws).items()}
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    x2, ids2 = torch.zeros_like(v["x"]), torch.full_like(v["ids"], -1)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        x2.copy_(v["x"])
        ids2.copy_(v["ids"])
    off, rows, slots, a, sa = mgs.mgs_moe_dispatch(x2, ids2, 6, stream=side)
    torch.cuda.synchronize()
    for n, t in (("off", off), ("rows", rows), ("slots", slots), ("a", a), ("sa", sa)):
        assert torch.equal(t.view(torch.uint8), want[n].view(torch.uint8)), n


@pytest.mark.parametrize("as_int", [False, True])
def test_workspace_of_another_stream(as_int):
    """A call's own workspace stays its own until the call has run: memory that
    the default stream takes right after the call returns is not it."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(9)
    ids = torch.randint(-1, 64, (40000, 2), generator=gen, device="cuda", dtype=torch.int32)
    want = mgs.mgs_moe_sort(ids, 64)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    got = mgs.mgs_moe_sort(ids, 64, stream=side.cuda_stream if as_int else side)
    taken = [torch.full((n,), -1, dtype=torch.uint8, device="cuda") for n in (256, 512, 1024, 2048, 4096, 8192, 16384)]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert all(int(t.min()) == 255 for t in taken)
