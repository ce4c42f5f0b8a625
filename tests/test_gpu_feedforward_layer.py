"""The gated and the 8-bit integer calls together: the layer of
examples/gated_experts.py against its formulas and gradients in 64 bits, all
calls in one captured graph, on other streams, and two at once."""
import os
import sys

import numpy as np
import pytest
import torch

import feedforward_ref as ff
import group_scaling_fp8_amd as mgs
from group_scaling_fp8_amd import feedforward, workloads as wl
from gpu_util import to_dev
from test_gpu_experts_layer import signs

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import gated_experts  # noqa: E402

pytestmark = pytest.mark.gpu

SLEEP = 20_000_000        # cycles that hold a stream back


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mgs.lib()


def plain_layer(x, ids, router, w1, w2, dy, act):
    """The layer and its gradients in 64 bits, token by token, each with the sum of its terms' magnitudes."""
    T, k = ids.shape
    out = {"y": x, "dx": x, "drouter": router, "dw1": w1, "dw2": w2}
    out = {n: (np.zeros(v.shape), np.zeros(v.shape)) for n, v in out.items()}

    def add(name, at, v, mag):
        out[name][0][at] += v
        out[name][1][at] += mag
    for t in range(T):
        for s in range(k):
            e = ids[t, s]
            if not 0 <= e < len(w1):
                continue
            g, u = w1[e, 0] @ x[t], w1[e, 1] @ x[t]
            h, slope = ff.act_of(act, g) * u, ff.slope_of(act, g)
            yt, my = w2[e] @ h, np.abs(w2[e]) @ np.abs(h)
            add("y", t, router[t, s] * yt, router[t, s] * my)
            add("drouter", (t, s), dy[t] @ yt, np.abs(dy[t]) @ my)
            d = router[t, s] * dy[t]
            dh = w2[e].T @ d
            both = np.concatenate([dh * u * slope, dh * ff.act_of(act, g)])
            w = w1[e].reshape(-1, x.shape[1])
            add("dx", t, w.T @ both, np.abs(w).T @ np.abs(both))
            add("dw2", e, np.outer(d, h), np.abs(np.outer(d, h)))
            v = np.outer(both, x[t]).reshape(w1[e].shape)
            add("dw1", e, v, np.abs(v))
    return out


@pytest.mark.parametrize("T,k,E,hidden,inner", [(1, 2, 4, 64, 32), (45, 3, 5, 272, 144), (150, 2, 4, 144, 384)])
@pytest.mark.parametrize("act", [ff.SILU, ff.GELU])
@pytest.mark.parametrize("fast", [False, True])
def test_layer_and_its_gradients(T, k, E, hidden, inner, act, fast):
    """A token and its gradient have one entry of +-1, weights are 0 and +-1:
    projections are 0 and +-1, so their casts and those of dy (times a power of
    two) are exact. h, dg and du have magnitudes within a factor of 2^6 of each
    other in a block, normal numbers of E4M3 under any block's scale: each cast
    of one rounds it by 2^-4 of itself at most, after its rounding to bf16 by
    2^-8. Everything is linear from there on; the sums' own roundings (2^-10 of
    the magnitudes with the faster sums) and one more to bf16 for yp, dxp, y and
    dx are under 2^-6 of the magnitudes together. drouter reads yp, so it has
    the same bound."""
    rng = np.random.default_rng(T)
    ids = np.argsort(rng.random((T, E)), 1)[:, :k].astype(np.int32)
    ids[rng.random((T, k)) < 0.1] = -1
    x, dy = signs(rng, (T, hidden), 1), signs(rng, (T, hidden), 1)
    w1, w2 = signs(rng, (E, 2, inner, hidden), hidden // 4), signs(rng, (E, hidden, inner), inner // 4)
    router = rng.choice([0.5, 1.0, 2.0], (T, k))
    want = plain_layer(x, ids, router, w1, w2, dy, act)
    dev = {n: to_dev(wl.f32_to_bf16_bits(v.astype(np.float32))).view(torch.bfloat16)
           for n, v in (("x", x), ("dy", dy), ("w1", w1), ("w2", w2))}
    router_d, ids_d = to_dev(router.astype(np.float32)), to_dev(ids)
    weights = gated_experts.cast_weights(dev["w1"], dev["w2"])
    y, saved = gated_experts.forward(dev["x"], ids_d, router_d, weights, act, fast)
    got = (y,) + gated_experts.backward(dev["dy"], router_d, weights, saved, act, fast)
    for name, a in zip(("y", "dx", "drouter", "dw1", "dw2"), got):
        v, mag = want[name]
        err = np.abs(a.double().cpu().numpy() - v)
        assert (err <= mag * (2.0 ** -4 * (1 + 2.0 ** -8) + 2.0 ** -8 + 2.0 ** -6) + 1e-30).all(), (name, float(err.max()))
        assert mag.max() > 0.07, name         # no expert's terms are smaller than half of |gelu(-1)| = 0.159


@pytest.mark.parametrize("T,k,E,hidden,inner", [(1, 2, 4, 64, 32), (45, 3, 5, 272, 144), (150, 2, 4, 144, 400)])
def test_serving_layer(T, k, E, hidden, inner):
    """The same in integers: tokens and weights are cast exactly, and h (rows
    whose largest magnitude scales to 127) to within half of 1 / 127 of that.
    Roundings to bf16 of h, yp and y add under 2^-6 of the magnitudes."""
    rng = np.random.default_rng(T + 1)
    ids = np.argsort(rng.random((T, E)), 1)[:, :k].astype(np.int32)
    ids[rng.random((T, k)) < 0.1] = -1
    x = signs(rng, (T, hidden), 1)
    w1, w2 = signs(rng, (E, 2, inner, hidden), hidden // 4), signs(rng, (E, hidden, inner), inner // 4)
    router = rng.choice([0.5, 1.0, 2.0], (T, k))
    v, mag = plain_layer(x, ids, router, w1, w2, np.zeros_like(x), ff.SILU)["y"]
    dev = [to_dev(wl.f32_to_bf16_bits(a.astype(np.float32))).view(torch.bfloat16) for a in (x, w1, w2)]
    weights = gated_experts.cast_weights_i8(dev[1], dev[2])
    y = gated_experts.serve(dev[0], to_dev(ids), to_dev(router.astype(np.float32)), weights)
    biggest = ff.act_of(ff.SILU, np.float64(1.0))          # of any h
    used = router.sum(1)[:, None] * (np.abs(w2).sum(2).max() * biggest * 0.51 / 127)
    err = np.abs(y.double().cpu().numpy() - v)
    assert (err <= mag * 2.0 ** -6 + used).all(), float(err.max())


def inputs(seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    T, k, E, hidden, inner = 500, 2, 6, 272, 128
    bf16 = dict(generator=gen, device="cuda", dtype=torch.bfloat16)
    return {"x": torch.randn((T, hidden), **bf16), "dy": torch.randn((T, hidden), **bf16),
            "ids": torch.randint(-1, E, (T, k), generator=gen, device="cuda", dtype=torch.int32),
            "router": torch.rand((T, k), generator=gen, device="cuda"),
            "w1": torch.randn((E, 2, inner, hidden), **bf16) * 0.05, "w2": torch.randn((E, hidden, inner), **bf16) * 0.05}


def all_calls(v):
    """Training, serving and a few tokens of each."""
    weights, kept = gated_experts.cast_weights(v["w1"], v["w2"]), gated_experts.cast_weights_i8(v["w1"], v["w2"])
    y, saved = gated_experts.forward(v["x"], v["ids"], v["router"], weights)
    out = dict(zip(("dx", "drouter", "dw1", "dw2"), gated_experts.backward(v["dy"], v["router"], weights, saved)))
    few = (v["x"][:5], v["ids"][:5], v["router"][:5])
    out.update(y=y, gu=saved[4], served=gated_experts.serve(v["x"], v["ids"], v["router"], kept),
               few=gated_experts.serve(*few, kept), few_train=gated_experts.forward(*few, weights, fast_accum=False)[0],
               wide=feedforward.mgs_mm_i8(*feedforward.mgs_quant_rows_i8(v["x"]), kept[0][0][:1], kept[0][1][:1], None,
                                          torch.float32))
    return out


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def test_every_call_in_one_graph():
    v = inputs(1)
    want = {seed: {n: t.clone() for n, t in all_calls(inputs(seed)).items()} for seed in (1, 2, 3)}
    torch.cuda.synchronize()
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        all_calls(v)                     # this stream's own workspaces are made before the capture
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        out = all_calls(v)
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
            assert same(t, want[seed][n]), (seed, n)
        again = all_calls(inputs(seed))  # eager work of the same calls between the replays
        torch.cuda.synchronize()
        assert all(same(t, want[seed][n]) for n, t in again.items())


def calls():
    v = inputs(4)
    w1, s1 = mgs.mgs_quant_blocks128(v["w1"].view(12, 128, 272), transposed=False)
    _, _, w2_t, s2_t = mgs.mgs_quant_blocks128(v["w2"])
    a, sa = mgs.mgs_quant_rows128(v["x"])
    off = torch.tensor([90, 90, 200, 310, 400, 500], dtype=torch.int32, device="cuda")
    gu = torch.randn((500, 256), device="cuda").to(torch.bfloat16)
    q, s = feedforward.mgs_quant_rows_i8(v["x"])
    q1, qs1 = feedforward.mgs_quant_rows_i8(v["w1"].view(12, 128, 272))
    return {
        "gated": lambda **kw: feedforward.mgs_mm_gated_block128(a, sa, w1, s1, off, keep=True, **kw),
        "grad": lambda **kw: feedforward.mgs_mm_gated_grad_block128(a, sa, w2_t, s2_t, gu, off, hidden=True, **kw),
        "cast": lambda **kw: feedforward.mgs_quant_rows_i8(v["x"], **kw),
        "product": lambda **kw: (feedforward.mgs_mm_i8(q, s, q1[:6], qs1[:6], off, **kw),),
        "gated8": lambda **kw: (feedforward.mgs_mm_gated_i8(q, s, q1, qs1, off, **kw),),
    }


@pytest.mark.parametrize("as_int", [False, True])
def test_calls_on_another_stream(as_int):
    """Work runs on the given stream, its outputs are that stream's memory: what
    the current stream frees or takes meanwhile is not touched."""
    side = torch.cuda.Stream()
    for name, call in calls().items():
        print(name, flush=True)
        want = [t.clone() for t in call()]
        held = [torch.full((t.numel() * t.element_size(),), 7, dtype=torch.uint8, device="cuda") for t in want]
        kept = [torch.zeros_like(h) for h in held]
        torch.cuda.synchronize()
        torch.cuda._sleep(SLEEP)
        for k, h in zip(kept, held):
            k.copy_(h)
        del h, held
        got = call(stream=side.cuda_stream if as_int else side)
        torch.cuda.synchronize()
        assert all(bool((k == 7).all()) for k in kept), name
        assert all(same(g, w) for g, w in zip(got, want)), name


def test_two_calls_at_once():
    """Calls have no state: on two streams together they give what they give alone."""
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    c = calls()
    want = {n: [t.clone() for t in f()] for n, f in c.items()}
    torch.cuda.synchronize()
    got = [(n, f(stream=s)) for _ in range(5) for s in (one, two) for n, f in c.items()]
    torch.cuda.synchronize()
    for n, outs in got:
        assert all(same(g, w) for g, w in zip(outs, want[n])), n


@pytest.mark.parametrize("M,F,D,fast", [(9, 48, 144, False), (60, 272, 272, True), (700, 1200, 400, True), (2000, 1200, 144, False),
                                        (2100, 2336, 144, True), (8200, 4000, 144, True)])
def test_gradients_in_place_of_the_projections(M, F, D, fast):
    """In every form, gu may be overwritten by its gradients."""
    rng = np.random.default_rng(M)
    gu = to_dev(wl.randn_bf16(rng, (M, 2 * F), 1.0)).view(torch.bfloat16)
    dy = mgs.mgs_quant_rows128(to_dev(wl.randn_bf16(rng, (M, D), 1.0)).view(torch.bfloat16))
    w = mgs.mgs_quant_blocks128(to_dev(wl.randn_bf16(rng, (1, F, D), 0.1)).view(torch.bfloat16), transposed=False)
    want, h = feedforward.mgs_mm_gated_grad_block128(*dy, *w, gu, fast_accum=fast, hidden=True)
    got, again = feedforward.mgs_mm_gated_grad_block128(*dy, *w, gu, fast_accum=fast, hidden=True, dgu=gu)
    assert got is gu and same(got, want) and same(again, h)


def test_front_end_refuses():
    c = calls()
    out = {n: f() for n, f in c.items()}
    i8 = torch.zeros((4, 64), dtype=torch.int8, device="cuda")
    one = torch.ones(4, device="cuda")
    w, sw = torch.zeros((1, 32, 64), dtype=torch.int8, device="cuda"), torch.ones((1, 32), device="cuda")
    off = torch.tensor([4], dtype=torch.int32, device="cuda")
    for call, error in (
            (lambda: feedforward.mgs_mm_i8(i8.view(torch.uint8), one, w, sw), TypeError),
            (lambda: feedforward.mgs_mm_i8(i8, one, w, sw, out_dtype=torch.float16), TypeError),
            (lambda: feedforward.mgs_mm_i8(i8, one[:3], w, sw), ValueError),
            (lambda: feedforward.mgs_mm_i8(i8, one, w, sw[:, :16]), ValueError),
            (lambda: feedforward.mgs_mm_i8(i8, one, w[:, :, :32].contiguous(), sw), ValueError),
            (lambda: feedforward.mgs_mm_i8(i8, one, w.transpose(1, 2), sw), ValueError),
            (lambda: feedforward.mgs_mm_i8(i8, one, w, sw, torch.cat([off, off])), ValueError),
            (lambda: feedforward.mgs_mm_i8(i8, one, w, sw, off.long()), TypeError),
            (lambda: feedforward.mgs_mm_i8(i8, one, w, sw, y=torch.zeros((4, 16), dtype=torch.bfloat16, device="cuda")), ValueError),
            (lambda: feedforward.mgs_mm_gated_i8(i8, one, w, sw), ValueError),
            (lambda: feedforward.mgs_mm_gated_i8(i8, one, w.expand(2, 32, 64).contiguous(), sw.expand(2, 32).contiguous(), act=2), ValueError),
            (lambda: feedforward.mgs_mm_i8(i8, one, w.expand(2, 32, 64).contiguous(), sw.expand(2, 32).contiguous()), mgs.MgsError),
            (lambda: feedforward.mgs_quant_rows_i8(one), TypeError),
            (lambda: feedforward.mgs_quant_rows_i8(torch.zeros(64, dtype=torch.bfloat16, device="cuda")), ValueError),
            (lambda: feedforward.mgs_quant_rows_i8(torch.zeros((2, 12), dtype=torch.bfloat16, device="cuda")), mgs.MgsError),
            (lambda: feedforward.mgs_mm_i8(torch.zeros(264, dtype=torch.int8, device="cuda")[8:].view(4, 64), one, w, sw), mgs.MgsError),
            (lambda: c["grad"](dgu=out["gated"][0]), ValueError)):
        with pytest.raises(error):
            call()
