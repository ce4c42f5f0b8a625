"""Workloads of the mixture-of-experts operators, with their plain forms.

A layer of experts in E4M3: tokens are sorted by expert and cast in blocks
of 128 (dispatch), multiplied with each expert's weight (product), and
summed back with their router weights (combine); the backward pass adds the
gradient of combine and the weight gradient (wgrad), whose operands are the
transposed per-group casts, and each step casts the weights in blocks of
128 x 128 in both orders (weights).

A case is a dict of plain values. ``prepare`` makes what a program holds
before the call, ``run`` is one call: the plain form in elementary torch
operations, or, where ``own`` is true, the library's entry points.
``exact`` computes the same outputs in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

BLOCK = 128          # columns that share a scale
ALIGN = 16           # rows of a token group come in multiples of this
FP8_MAX = 448.0
EPS = 1e-12


# ---- cases -------------------------------------------------------------------

def listed():
    return [
        # serving, one token at a time: eight of 64 experts, latency only
        dict(name="dispatch_one_token", op="dispatch", T=1, k=8, E=64, D=5120, drop=0.0),
        # a ragged prompt with dropped slots and a width that ends inside a block
        dict(name="dispatch_odd", op="dispatch", T=1117, k=6, E=61, D=4112, drop=0.1),
        # a training batch, four of 64 experts
        dict(name="dispatch_large", op="dispatch", T=16640, k=4, E=64, D=8192, drop=0.0),
        # the way back of a training batch, two of 16 experts, dropped slots
        dict(name="combine_large", op="combine", T=32771, k=2, E=16, D=5120, drop=0.05),
        # its gradient, with respect to the experts' rows and the router weights
        dict(name="combine_grad_large", op="combine_grad", T=16640, k=4, E=64, D=4096, drop=0.02),
        # the cast of one layer's weights after an optimizer step, both orders
        dict(name="weights_cast", op="weights", E=16, N=8192, K=5120),
        # serving, four tokens: two of 16 experts each, most experts unused
        dict(name="product_decode", op="product", T=4, k=2, E=16, M=0, N=8192, K=5120, cast=False, f32=False),
        # an ordinary batch of experts
        dict(name="product_ordinary", op="product", T=0, k=0, E=16, M=4096, N=4096, K=4096, cast=False, f32=False),
        # one dense product of odd sizes, rows and both other sides ending inside a block
        dict(name="product_dense_odd", op="product", T=0, k=0, E=0, M=1003, N=4176, K=4112, cast=False, f32=True),
        # the input gradient of a training batch: the output gradient is cast in the call
        dict(name="product_large", op="product", T=0, k=0, E=16, M=16640, N=5120, K=8192, cast=True, f32=False),
        # a small layer's weight gradient, few tokens in each of four groups
        dict(name="wgrad_small", op="wgrad", G=4, M=256, N=1040, K=4096, f32=True),
        # a training batch's weight gradient
        dict(name="wgrad_large", op="wgrad", G=16, M=16640, N=8192, K=5120, f32=False),
    ]


def _spread(rng, lo, hi, step=1):
    """A multiple of step in [lo, hi] but 3072, uniform in its logarithm."""
    v = int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))
    v = max(lo, min(hi, v // step * step))
    return v - step if v == 3072 else v


def draw(rng):
    op = rng.choice(["dispatch", "combine", "combine_grad", "weights", "product", "product", "product", "wgrad",
                     "wgrad"])
    if op in ("dispatch", "combine", "combine_grad"):
        E = rng.choice([4, 7, 16, 61, 64, 160, 256])
        k = rng.randint(1, min(8, E))
        D = _spread(rng, 256, 8192, 16)
        most = {"dispatch": 66560 * 8192, "combine": 65542 * 5120, "combine_grad": 66560 * 4096}[op]
        T = _spread(rng, 1, min(32768, most // (k * D)))
        return dict(op=op, T=T, k=k, E=E, D=D, drop=rng.choice([0.0, 0.0, 0.03, 0.3]))
    if op == "weights":
        N, K = _spread(rng, 256, 8192, 16), _spread(rng, 256, 8192, 16)
        return dict(op=op, E=_spread(rng, 1, max(1, min(64, 16 * 8192 * 5120 // (N * K)))), N=N, K=K)
    if op == "product":
        N, K = _spread(rng, 512, 8192, 16), _spread(rng, 512, 8192, 16)
        kind = rng.choice(["decode", "dense", "grouped", "grouped"])
        if kind == "decode":
            E = _spread(rng, 2, max(2, min(64, 16 * 8192 * 5120 // (N * K))))
            return dict(op=op, T=_spread(rng, 1, 64), k=rng.randint(1, min(8, E)), E=E, M=0, N=N, K=K, cast=False,
                        f32=False)
        if kind == "dense":
            return dict(op=op, T=0, k=0, E=0, M=_spread(rng, 1, 16640), N=N, K=K, cast=rng.random() < 0.5,
                        f32=rng.random() < 0.5)
        E = _spread(rng, 2, max(2, min(64, 16 * 8192 * 5120 // (N * K))))
        return dict(op=op, T=0, k=0, E=E, M=_spread(rng, 256, 16640, 16), N=N, K=K, cast=rng.random() < 0.5,
                    f32=rng.random() < 0.25)
    N, K = _spread(rng, 256, 8192, 16), _spread(rng, 256, 5120, 16)
    G = _spread(rng, 1, max(1, min(64, 16 * 8192 * 5120 // (N * K))))
    return dict(op=op, G=G, M=_spread(rng, 64, 16640, 16), N=N, K=K, f32=rng.random() < 0.5)


# ---- inputs --------------------------------------------------------------------

def _values(gen, shape, sigma=0.02, outlier=8.0):
    """bf16 normal values with one in a thousand at +-outlier, as trained activations have them."""
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16) * sigma
    big = torch.rand(shape, generator=gen, device="cuda", dtype=torch.bfloat16) < 0.001
    return torch.where(big, torch.sign(x) * outlier, x)


def _routing(gen, T, k, E, drop):
    """Distinct experts for each token, some of them more popular, and normalised weights."""
    score = torch.randn((T, E), generator=gen, device="cuda") + torch.randn((E,), generator=gen, device="cuda") * 0.7
    top, ids = torch.topk(score, k, dim=1)
    weights = torch.softmax(top, dim=1)
    if drop > 0:
        ids = torch.where(torch.rand((T, k), generator=gen, device="cuda") < drop, -1, ids)
    return ids.to(torch.int32).contiguous(), weights.contiguous()


def _group_ends(gen, extent, G):
    """End offsets of G groups of random multiples of ALIGN rows (empty ones among them) that fill extent."""
    units = extent // ALIGN
    cuts = torch.randint(0, units + 1, (G - 1,), generator=gen, device="cuda").sort().values
    ends = torch.cat([cuts, torch.full((1,), units, device="cuda", dtype=cuts.dtype)]) * ALIGN
    return ends.to(torch.int32)


def _rows_bound(T, k, E):
    n = T * k
    return (n + min(E, n) * (ALIGN - 1)) // ALIGN * ALIGN


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op = case["op"]
    st = {"case": case}
    if op in ("dispatch", "combine", "combine_grad"):
        T, k, E, D = case["T"], case["k"], case["E"], case["D"]
        st["ids"], st["weights"] = _routing(gen, T, k, E, case["drop"])
        if op == "dispatch":
            st["x"] = _values(gen, (T, D))
            return st
        st["offsets"], st["rows"], st["slots"] = _order(st["ids"], E)
        yp = _values(gen, (_rows_bound(T, k, E), D), 1.0, 20.0)
        yp[st["slots"] < 0] = 0
        st["yp"] = yp
        if op == "combine_grad":
            st["dy"] = _values(gen, (T, D))
    elif op == "weights":
        st["w"] = _values(gen, (case["E"], case["N"], case["K"]), 0.02, 0.5)
    elif op == "product":
        E, N, K = case["E"], case["N"], case["K"]
        M = case["M"]
        if case["T"]:
            ids, _ = _routing(gen, case["T"], case["k"], E, 0.0)
            st["offsets"], _, slots = _order(ids, E)
            M = slots.numel()
        else:
            st["offsets"] = _group_ends(gen, M, E) if E else None
        st["ends"] = st["offsets"].tolist() if E else [M]
        x = _values(gen, (M, K))
        if case["T"]:
            x[slots < 0] = 0
        if case["cast"]:
            st["x"] = x
        else:
            q, s = _cast_rows(x)
            st["a"], st["a_scales"] = q.view(torch.uint8), s
        q, s = _cast_blocks(_values(gen, (max(E, 1), N, K), 0.02, 0.5))
        st["b"], st["b_scales"] = q.view(torch.uint8), s
    else:
        G, M = case["G"], case["M"]
        st["offsets"] = _group_ends(gen, M, G)
        st["ends"] = st["offsets"].tolist()
        for name, width in (("a", case["N"]), ("b", case["K"])):
            q, s = _cast_groups_t(_values(gen, (M, width)), st["offsets"], G)
            st[name], st[name + "_scales"] = q.view(torch.uint8), s
    return st


# ---- plain forms -----------------------------------------------------------------

def _scale(amax):
    # a division of two tensors: a number over a tensor goes through the reciprocal and rounds twice
    return torch.full_like(amax, FP8_MAX) / torch.clamp(amax, min=EPS)


def _e4m3(v):
    return torch.clamp(v, -FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn)


def _pad_to_blocks(x, dim):
    over = -x.shape[dim] % BLOCK
    if not over:
        return x
    shape = list(x.shape)
    shape[dim] = over
    return torch.cat([x, x.new_zeros(shape)], dim)


def _cast_rows(x):
    """One scale for each row and block of 128 columns."""
    M, K = x.shape
    v = _pad_to_blocks(x.float(), 1).view(M, -1, BLOCK)
    s = _scale(v.abs().amax(2))
    return _e4m3(v * s[:, :, None]).reshape(M, -1)[:, :K].contiguous(), s


def _cast_blocks(w):
    """One scale for each block of 128 x 128 of every matrix."""
    E, N, K = w.shape
    v = _pad_to_blocks(_pad_to_blocks(w, 1), 2).float()
    v = v.view(E, v.shape[1] // BLOCK, BLOCK, v.shape[2] // BLOCK, BLOCK)
    s = _scale(v.abs().amax((2, 4)))
    q = _e4m3(v * s[:, :, None, :, None])
    return q.reshape(E, q.shape[1] * BLOCK, -1)[:, :N, :K].contiguous(), s


def _cast_groups_t(x, offsets, G):
    """One scale for each column and token group; values and scales transposed."""
    M, K = x.shape
    group = torch.bucketize(torch.arange(M, device=x.device), offsets, right=True)
    amax = torch.zeros((G, K), device=x.device)
    amax.scatter_reduce_(0, group[:, None].expand(M, K), x.float().abs(), "amax")
    s = _scale(amax)
    return _e4m3(x.float() * s[group]).t().contiguous(), s.t().contiguous()


def _order(ids, E):
    """End offsets of the experts' rows, the row of each slot and the slot of each row (-1: none)."""
    T, k = ids.shape
    n, P = T * k, _rows_bound(T, k, E)
    flat = ids.reshape(-1).long()
    held = (flat >= 0) & (flat < E)
    key = torch.where(held, flat, E)
    count = (key[:, None] == torch.arange(E + 1, device=ids.device)).sum(0)
    full = (count + ALIGN - 1) // ALIGN * ALIGN
    order = torch.argsort(key, stable=True)
    expert = key[order]
    before = torch.cumsum(count, 0) - count
    start = torch.cumsum(full, 0) - full
    row = torch.where(expert < E, start[expert] + torch.arange(n, device=ids.device) - before[expert], -1)
    rows = torch.empty_like(row)
    rows[order] = row
    slots = torch.full((P + 1,), -1, device=ids.device, dtype=torch.long)
    slots[torch.where(row < 0, P, row)] = order
    offsets = torch.cumsum(full[:E], 0)
    return offsets.to(torch.int32), rows.view(T, k).to(torch.int32), slots[:P].to(torch.int32)


def _plain_dispatch(st):
    x, ids = st["x"], st["ids"]
    offsets, rows, slots = _order(ids, st["case"]["E"])
    xp = torch.where((slots >= 0)[:, None], x[slots.clamp(min=0).long() // ids.shape[1]], 0)
    q, s = _cast_rows(xp)
    return {"offsets": offsets, "rows": rows, "slots": slots, "q": q, "scales": s}


def _plain_combine(st):
    rows = st["rows"]
    w = torch.where(rows >= 0, st["weights"], 0.0)
    y = (st["yp"][rows.clamp(min=0).long()].float() * w[:, :, None]).sum(1)
    return {"y": y.to(torch.bfloat16)}


def _plain_combine_grad(st):
    rows, slots, k = st["rows"], st["slots"], st["rows"].shape[1]
    slot = slots.clamp(min=0).long()
    w = torch.where(slots >= 0, st["weights"].reshape(-1)[slot], 0.0)
    dy = st["dy"].float()
    dyp = dy[slot // k] * w[:, None]
    dw = (st["yp"][rows.clamp(min=0).long()].float() * dy[:, None, :]).sum(2)
    return {"dyp": dyp.to(torch.bfloat16), "dw": torch.where(rows >= 0, dw, 0.0)}


def _plain_weights(st):
    q, s = _cast_blocks(st["w"])
    return {"q": q, "scales": s, "q_t": q.transpose(1, 2).contiguous(), "scales_t": s.transpose(1, 2).contiguous()}


def _spread_scales(s, size, dim):
    return s.repeat_interleave(BLOCK, dim).narrow(dim, 0, size)


def _plain_product(st):
    case, b = st["case"], st["b"].view(torch.float8_e4m3fn)
    if case["cast"]:
        a, a_scales = _cast_rows(st["x"])
    else:
        a, a_scales = st["a"].view(torch.float8_e4m3fn), st["a_scales"]
    (M, K), N = a.shape, b.shape[1]
    y = torch.zeros((M, N), device=a.device, dtype=torch.float32 if case["f32"] else torch.bfloat16)
    first = 0
    for e, end in enumerate(st["ends"]):        # the groups that have rows
        if end > first:
            av = a[first:end].float() / _spread_scales(a_scales[first:end], K, 1)
            bv = b[e].float() / _spread_scales(_spread_scales(st["b_scales"][e], N, 0), K, 1)
            y[first:end] = av @ bv.t()
        first = end
    return {"y": y}


def _plain_wgrad(st):
    a, b = st["a"].view(torch.float8_e4m3fn), st["b"].view(torch.float8_e4m3fn)
    dw = torch.zeros((len(st["ends"]), a.shape[0], b.shape[0]), device=a.device,
                     dtype=torch.float32 if st["case"]["f32"] else torch.bfloat16)
    first = 0
    for g, end in enumerate(st["ends"]):
        if end > first:
            av = a[:, first:end].float() / st["a_scales"][:, g:g + 1]
            bv = b[:, first:end].float() / st["b_scales"][:, g:g + 1]
            dw[g] = av @ bv.t()
        first = end
    return {"dw": dw}


# ---- one pass --------------------------------------------------------------------

def _own_run(st):
    import group_scaling_fp8_amd as mgs
    case, op = st["case"], st["case"]["op"]
    out_dtype = torch.float32 if case.get("f32") else torch.bfloat16
    fast = not case.get("f32")       # where the output is rounded to bf16, the faster sums' loss does not show
    if op == "dispatch":
        offsets, rows, slots, q, s = mgs.mgs_moe_dispatch(st["x"], st["ids"], case["E"])
        return {"offsets": offsets, "rows": rows, "slots": slots, "q": q.view(torch.float8_e4m3fn), "scales": s}
    if op == "combine":
        return {"y": mgs.mgs_moe_combine(st["yp"], st["rows"], st["weights"])}
    if op == "combine_grad":
        dyp, dw = mgs.mgs_moe_combine_grad(st["dy"], st["yp"], st["rows"], st["slots"], st["weights"])
        return {"dyp": dyp, "dw": dw}
    if op == "weights":
        q, s, q_t, s_t = mgs.mgs_quant_blocks128(st["w"])
        return {"q": q.view(torch.float8_e4m3fn), "scales": s, "q_t": q_t.view(torch.float8_e4m3fn), "scales_t": s_t}
    if op == "product":
        a, a_scales = mgs.mgs_quant_rows128(st["x"]) if case["cast"] else (st["a"], st["a_scales"])
        return {"y": mgs.mgs_mm_block128(a, a_scales, st["b"], st["b_scales"], st["offsets"], out_dtype,
                                         fast_accum=fast)}
    return {"dw": mgs.mgs_mm_wgrad(st["a"], st["a_scales"], st["b"], st["b_scales"], st["offsets"], out_dtype,
                                   fast_accum=fast)}


_PLAIN = {"dispatch": _plain_dispatch, "combine": _plain_combine, "combine_grad": _plain_combine_grad,
          "weights": _plain_weights, "product": _plain_product, "wgrad": _plain_wgrad}


def run(state):
    return _own_run(state) if own else _PLAIN[state["case"]["op"]](state)


# ---- what a pass cannot do without ---------------------------------------------------

def work(case):
    op = case["op"]
    up = lambda v: -(-v // BLOCK)  # noqa: E731
    if op in ("dispatch", "combine", "combine_grad"):
        T, k, D = case["T"], case["k"], case["D"]
        n, P = T * k, _rows_bound(T, k, case["E"])
        held = round(n * (1 - case["drop"]))
        if op == "dispatch":
            return {"bytes": T * D * 2 + n * 4 + P * (D + up(D) * 4 + 4) + n * 4 + case["E"] * 4, "flops": T * D * 3}
        if op == "combine":
            return {"bytes": held * D * 2 + T * D * 2 + n * 8, "flops": 2 * held * D}
        return {"bytes": T * D * 2 + held * D * 2 + P * D * 2 + n * 12 + P * 4, "flops": 3 * held * D}
    if op == "weights":
        E, N, K = case["E"], case["N"], case["K"]
        return {"bytes": E * N * K * 4 + E * up(N) * up(K) * 8, "flops": 2 * E * N * K}
    if op == "product":
        N, K, E = case["N"], case["K"], max(case["E"], 1)
        if case["T"]:
            rows = case["T"] * case["k"]
            M = _rows_bound(case["T"], case["k"], E)
            used = E * (1 - (1 - case["k"] / E) ** case["T"])       # experts that some token chose, on average
        else:
            rows = M = case["M"]
            used = min(E, -(-M // ALIGN))
        a = rows * (K + up(K) * 4) + (rows * K * 2 if case["cast"] else 0)
        return {"bytes": a + used * (N * K + up(N) * up(K) * 4) + M * N * (4 if case["f32"] else 2),
                "flops": 2 * rows * N * K}
    G, M, N, K = case["G"], case["M"], case["N"], case["K"]
    return {"bytes": M * (N + K) + G * (N + K) * 4 + G * N * K * (4 if case["f32"] else 2), "flops": 2 * M * N * K}


# ---- the definition in 64 bits -----------------------------------------------------------

def _e4m3_64(v):
    """The nearest E4M3 value (ties to the even code) of v, which is a binary32 value held in 64 bits."""
    v = v.clamp(-448.0, 448.0)
    e = torch.frexp(v.abs()).exponent.clamp(min=-5) - 1          # floor(log2 |v|), at least that of the subnormals
    step = torch.tensor([2.0 ** (i - 9) for i in range(15)], dtype=torch.float64, device=v.device)[e + 6]
    return torch.round(v / step) * step


def _scale_64(amax):
    # the scale is a binary32 number by definition: the 64-bit quotient rounds to it
    eps = float(torch.tensor(EPS, dtype=torch.float32))
    return (448.0 / amax.clamp(min=eps)).float().double()


def _blocks_of(size):
    return [(i, min(i + BLOCK, size)) for i in range(0, size, BLOCK)]


def _exact_rows(x):
    q, s = torch.empty(x.shape, dtype=torch.float64, device=x.device), []
    for i, j in _blocks_of(x.shape[1]):
        v = x[:, i:j].double()
        s.append(_scale_64(v.abs().amax(1)))
        q[:, i:j] = _e4m3_64((v * s[-1][:, None]).float().double())
    return q, torch.stack(s, 1)


def _exact_dispatch(st):
    ids, E, x = st["ids"].cpu(), st["case"]["E"], st["x"]
    (T, k), P = ids.shape, _rows_bound(ids.shape[0], ids.shape[1], E)
    members = [[] for _ in range(E)]
    for i, e in enumerate(ids.reshape(-1).tolist()):
        if 0 <= e < E:
            members[e].append(i)
    slots, rows, offsets = [], [-1] * (T * k), []
    for mine in members:
        for i in mine:
            rows[i] = len(slots)
            slots.append(i)
        slots += [-1] * (-len(mine) % ALIGN)
        offsets.append(len(slots))
    slots += [-1] * (P - len(slots))
    q_of, s_of = _exact_rows(x)
    zero_scale = _scale_64(torch.zeros((), dtype=torch.float64)).item()
    at = torch.tensor(slots, device=x.device)
    token = at.clamp(min=0) // k
    q = torch.where((at >= 0)[:, None], q_of[token], 0.0)
    s = torch.where((at >= 0)[:, None], s_of[token], zero_scale)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    return {"offsets": i32(offsets), "rows": i32(rows).view(T, k), "slots": i32(slots), "q": q, "scales": s}


def _exact_combine(st):
    rows, yp = st["rows"].long(), st["yp"]
    y = torch.zeros((rows.shape[0], yp.shape[1]), dtype=torch.float64, device=yp.device)
    for s in range(rows.shape[1]):
        t = torch.nonzero(rows[:, s] >= 0)[:, 0]
        y[t] += st["weights"][t, s].double()[:, None] * yp[rows[t, s]].double()
    return {"y": y}


def _exact_combine_grad(st):
    rows, yp, dy = st["rows"].long(), st["yp"], st["dy"]
    dyp = torch.zeros(yp.shape, dtype=torch.float64, device=yp.device)
    dw = torch.zeros(rows.shape, dtype=torch.float64, device=yp.device)
    for s in range(rows.shape[1]):
        t = torch.nonzero(rows[:, s] >= 0)[:, 0]
        r = rows[t, s]
        dyp[r] = st["weights"][t, s].double()[:, None] * dy[t].double()
        dw[t, s] = (dy[t].double() * yp[r].double()).sum(1)
    return {"dyp": dyp, "dw": dw}


def _exact_weights(st):
    w = st["w"]
    E, N, K = w.shape
    q = torch.empty(w.shape, dtype=torch.float32, device=w.device)      # E4M3 values: exact in 32 bits
    s = torch.empty((E, len(_blocks_of(N)), len(_blocks_of(K))), dtype=torch.float64, device=w.device)
    for a, (i, j) in enumerate(_blocks_of(N)):
        rows = w[:, i:j].double()
        for b, (c, d) in enumerate(_blocks_of(K)):
            v = rows[:, :, c:d]
            s[:, a, b] = _scale_64(v.abs().amax((1, 2)))
            q[:, i:j, c:d] = _e4m3_64((v * s[:, a, b, None, None]).float().double()).float()
    return {"q": q, "scales": s, "q_t": q.transpose(1, 2).contiguous(), "scales_t": s.transpose(1, 2).contiguous()}


def _decoded_64(code):
    """The value of each E4M3 byte, from its sign, exponent and fraction."""
    code = torch.arange(256, device=code.device)
    sign, e, f = 1.0 - 2.0 * (code >> 7).double(), (code >> 3) & 15, (code & 7).double()
    power = torch.tensor([2.0 ** max(i - 7, -6) for i in range(16)], dtype=torch.float64, device=code.device)[e]
    return sign * torch.where(e == 0, f / 8, 1 + f / 8) * power


def _exact_product(st):
    case, b = st["case"], st["b"]
    table = _decoded_64(b)
    if case["cast"]:
        a, sa = _exact_rows(st["x"])
    else:
        a, sa = table[st["a"].long()], st["a_scales"].double()
    a = a / sa.repeat_interleave(BLOCK, 1)[:, :a.shape[1]]
    N, K = b.shape[1:]
    y = torch.zeros((a.shape[0], N), dtype=torch.float64, device=b.device)
    first = 0
    for e, end in enumerate(st["ends"]):
        if end > first:
            bv = table[b[e].long()]
            bv /= st["b_scales"][e].double().repeat_interleave(BLOCK, 0)[:N].repeat_interleave(BLOCK, 1)[:, :K]
            y[first:end] = torch.matmul(a[first:end], bv.t())
        first = end
    return {"y": y}


def _exact_wgrad(st):
    a, b = st["a"], st["b"]
    table = _decoded_64(a)
    dw = torch.zeros((len(st["ends"]), a.shape[0], b.shape[0]), dtype=torch.float64, device=a.device)
    first = 0
    for g, end in enumerate(st["ends"]):
        if end > first:
            s = st["a_scales"][:, g, None].double() * st["b_scales"][None, :, g].double()
            torch.matmul(table[a[:, first:end].long()], table[b[:, first:end].long()].t(), out=dw[g])
            dw[g] /= s
        first = end
    return {"dw": dw}


_EXACT = {"dispatch": _exact_dispatch, "combine": _exact_combine, "combine_grad": _exact_combine_grad,
          "weights": _exact_weights, "product": _exact_product, "wgrad": _exact_wgrad}


def exact(case, seed):
    return _EXACT[case["op"]](prepare(case, seed))
