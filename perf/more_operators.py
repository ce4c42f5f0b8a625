"""Workloads of the gated experts and of the 8-bit integer products, with their plain forms.

An expert of a gated feed-forward layer is (act(x Wg^T) * (x Wu^T)) Wd^T. In
training its operands are E4M3 with block-128 scales: one call computes both
projections, the activation and the product (gated), one the gradients of both
projections from the output's (grad); the products around them are in
perf/operators.py. In serving, operands are 8-bit integers with one scale for
each token and each output channel: the cast (cast), the product (product) and
both projections with the activation (gated8).

A case is a dict of plain values. ``prepare`` makes what a program holds
before the call, ``run`` is one call: the plain form in elementary torch
operations, or, where ``own`` is true, the library's entry points.
``exact`` computes the same outputs in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

BLOCK = 128          # columns that share an E4M3 scale
ALIGN = 16           # rows of a token group come in multiples of this
E4M3_MAX = 448.0
I8_MAX = 127.0
EPS = 1e-12


# ---- cases -------------------------------------------------------------------

def listed():
    return [
        # decoding four tokens, two of 16 experts each: most experts unused
        dict(name="gated_decode", op="gated", T=4, k=2, E=16, M=0, F=8192, K=5120, act="silu", keep=False, fast=True),
        # a dense layer of odd sizes, binary32 sums, what the gradient needs kept
        dict(name="gated_dense_odd", op="gated", T=0, k=0, E=0, M=1003, F=2096, K=4112, act="gelu", keep=True,
             fast=False),
        # a training batch of 16 experts
        dict(name="gated_large", op="gated", T=0, k=0, E=16, M=16640, F=8192, K=5120, act="silu", keep=True, fast=True),
        # few tokens in four experts of an odd width
        dict(name="grad_small", op="grad", E=4, M=256, F=1040, D=4096, act="gelu", hidden=True, fast=True),
        # the training batch's way back, the hidden rows computed again for the weight gradient
        dict(name="grad_large", op="grad", E=16, M=16640, F=8192, D=5120, act="silu", hidden=True, fast=True),
        # one token's activations before a product: latency only
        dict(name="cast_one_token", op="cast", M=1, K=5120),
        # a long prompt's activations
        dict(name="cast_large", op="cast", M=16640, K=8192),
        # decoding one token through one projection
        dict(name="product_one_token", op="product", T=0, k=0, E=0, M=1, N=8192, K=8192, f32=False),
        # a ragged batch in 16 experts of odd sizes
        dict(name="product_odd", op="product", T=0, k=0, E=16, M=4096, N=4112, K=4176, f32=True),
        # a long prompt through one dense projection
        dict(name="product_large", op="product", T=0, k=0, E=0, M=16640, N=8192, K=8192, f32=False),
        # decoding four tokens in integers
        dict(name="gated8_decode", op="gated8", T=4, k=2, E=16, M=0, F=8192, K=5120, act="silu"),
        # a long prompt in 16 experts in integers
        dict(name="gated8_large", op="gated8", T=0, k=0, E=16, M=16640, F=8192, K=5120, act="silu"),
    ]


def _spread(rng, lo, hi, step=1):
    """A multiple of step in [lo, hi], uniform in its logarithm."""
    v = int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))
    return max(lo, min(hi, v // step * step))


def _batch(rng, experts):
    """Few tokens routed to experts, one dense batch, or ragged groups."""
    kind = rng.choice(["decode", "dense", "grouped", "grouped"])
    if kind == "dense":
        return dict(T=0, k=0, E=0, M=_spread(rng, 1, 16640))
    E = _spread(rng, 2, max(2, experts))
    if kind == "decode":
        return dict(T=_spread(rng, 1, 64), k=rng.randint(1, min(8, E)), E=E, M=0)
    return dict(T=0, k=0, E=E, M=_spread(rng, 256, 16640, 16))


def draw(rng):
    op = rng.choice(["gated", "gated", "grad", "grad", "cast", "product", "product", "gated8", "gated8"])
    if op == "cast":
        K = _spread(rng, 128, 16384, 8)
        return dict(op=op, M=_spread(rng, 1, 16640 * 8192 // K), K=K)
    wide, deep = _spread(rng, 256, 8192, 16), _spread(rng, 256, 5120 if op != "product" else 8192, 16)
    experts = min(64, 16 * 8192 * 5120 // (wide * deep))
    act = rng.choice(["silu", "gelu"])
    if op == "product":
        return dict(op=op, **_batch(rng, experts), N=wide, K=deep, f32=rng.random() < 0.25)
    if op == "gated8":
        return dict(op=op, **_batch(rng, experts), F=wide, K=deep, act=act)
    if op == "gated":
        return dict(op=op, **_batch(rng, experts), F=wide, K=deep, act=act, keep=rng.random() < 0.6,
                    fast=rng.random() < 0.75)
    E = _spread(rng, 1, max(1, experts))
    return dict(op=op, E=E if E > 1 else 0, M=_spread(rng, 64, 16640, 16), F=wide, D=deep, act=act,
                hidden=rng.random() < 0.6, fast=rng.random() < 0.75)


# ---- inputs --------------------------------------------------------------------

def _values(gen, shape, sigma=0.02, outlier=8.0):
    """bf16 normal values with one in a thousand at +-outlier, as trained activations have them."""
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16) * sigma
    big = torch.rand(shape, generator=gen, device="cuda", dtype=torch.bfloat16) < 0.001
    return torch.where(big, torch.sign(x) * outlier, x)


def _group_ends(gen, extent, G):
    """End offsets of G groups of random multiples of ALIGN rows (empty ones among them) that fill extent."""
    units = extent // ALIGN
    cuts = torch.randint(0, units + 1, (G - 1,), generator=gen, device="cuda").sort().values
    ends = torch.cat([cuts, torch.full((1,), units, device="cuda", dtype=cuts.dtype)]) * ALIGN
    return ends.to(torch.int32)


def _rows_bound(T, k, E):
    n = T * k
    return (n + min(E, n) * (ALIGN - 1)) // ALIGN * ALIGN


def _routed_ends(gen, T, k, E):
    """End offsets of T tokens in k distinct experts each, groups filled up to ALIGN rows, and which rows hold a token."""
    score = torch.randn((T, E), generator=gen, device="cuda") + torch.randn((E,), generator=gen, device="cuda") * 0.7
    count = torch.bincount(torch.topk(score, k, dim=1).indices.reshape(-1), minlength=E)
    full = (count + ALIGN - 1) // ALIGN * ALIGN
    ends = torch.cumsum(full, 0)
    row = torch.arange(_rows_bound(T, k, E), device="cuda")
    group = torch.bucketize(row, ends, right=True).clamp(max=E - 1)
    return ends.to(torch.int32), row - (ends - full)[group] < count[group]


def _rows(gen, case, width):
    """The batch's group ends (None: one dense batch), the same on the host, and its rows: bf16, zero where no token is."""
    if case.get("T"):
        offsets, held = _routed_ends(gen, case["T"], case["k"], case["E"])
        x = _values(gen, (held.numel(), width), 0.5, 20.0)
        x[~held] = 0
    else:
        offsets = _group_ends(gen, case["M"], case["E"]) if case["E"] else None
        x = _values(gen, (case["M"], width), 0.5, 20.0)
    return offsets, [x.shape[0]] if offsets is None else offsets.tolist(), x


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op = case["op"]
    st = {"case": case}
    if op == "cast":
        st["x"] = _values(gen, (case["M"], case["K"]), 0.5, 20.0)
        return st
    E = max(case["E"], 1)
    st["offsets"], st["ends"], x = _rows(gen, case, case["D"] if op == "grad" else case["K"])
    weights = {"gated": lambda: (2 * E, case["F"], case["K"]), "gated8": lambda: (2 * E, case["F"], case["K"]),
               "grad": lambda: (E, case["F"], case["D"]), "product": lambda: (E, case["N"], case["K"])}[op]()
    w = _values(gen, weights, 0.02, 0.5)
    if op in ("gated", "grad"):
        (q, st["a_scales"]), (b, st["b_scales"]) = _cast_rows(x), _cast_blocks(w)
        st["a"], st["b"] = q.view(torch.uint8), b.view(torch.uint8)
    else:
        (st["a"], st["a_scales"]), (st["b"], st["b_scales"]) = _cast_i8(x), _cast_i8(w)
    if op == "grad":
        # projections as the forward call keeps them
        st["gu"] = _values(gen, (x.shape[0], 2 * case["F"]), 1.5, 12.0)
    return st


# ---- plain forms -----------------------------------------------------------------

def _scale(amax, most):
    # a division of two tensors: a number over a tensor goes through the reciprocal and rounds twice
    return torch.full_like(amax, most) / torch.clamp(amax, min=EPS)


def _e4m3(v):
    return torch.clamp(v, -E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _pad_to_blocks(x, dim):
    over = -x.shape[dim] % BLOCK
    if not over:
        return x
    shape = list(x.shape)
    shape[dim] = over
    return torch.cat([x, x.new_zeros(shape)], dim)


def _cast_rows(x):
    """E4M3 with one scale for each row and block of 128 columns."""
    M, K = x.shape
    v = _pad_to_blocks(x.float(), 1).view(M, -1, BLOCK)
    s = _scale(v.abs().amax(2), E4M3_MAX)
    return _e4m3(v * s[:, :, None]).reshape(M, -1)[:, :K].contiguous(), s


def _cast_blocks(w):
    """E4M3 with one scale for each block of 128 x 128 of every matrix."""
    E, N, K = w.shape
    v = _pad_to_blocks(_pad_to_blocks(w, 1), 2).float()
    v = v.view(E, v.shape[1] // BLOCK, BLOCK, v.shape[2] // BLOCK, BLOCK)
    s = _scale(v.abs().amax((2, 4)), E4M3_MAX)
    q = _e4m3(v * s[:, :, None, :, None])
    return q.reshape(E, q.shape[1] * BLOCK, -1)[:, :N, :K].contiguous(), s


def _cast_i8(x):
    """8-bit integers with one scale for each row, to the nearest, ties to the even one."""
    v = x.float()
    s = _scale(v.abs().amax(-1), I8_MAX)
    return torch.round(v * s[..., None]).to(torch.int8), s


def _sigmoid_of(act, g):
    """The logistic factor of g * sigmoid(t(g)), and the derivative of t."""
    if act == "silu":
        t, dt = g, torch.ones_like(g)
    else:
        c = 2 * math.sqrt(2 / math.pi)
        t, dt = c * (g + 0.044715 * g * g * g), c * (1 + 3 * 0.044715 * g * g)
    return 1 / (1 + torch.exp(-t)), dt


def _spread_scales(s, size, dim):
    return s.repeat_interleave(BLOCK, dim).narrow(dim, 0, size)


def _products(st, matrices):
    """Each group's rows times its `matrices` weights, in 32 bits: (rows, matrices, N)."""
    a, b = st["a"].view(torch.float8_e4m3fn), st["b"].view(torch.float8_e4m3fn)
    (M, K), N = a.shape, b.shape[1]
    y = torch.zeros((M, matrices, N), device=a.device)
    first = 0
    for e, end in enumerate(st["ends"]):        # the groups that have rows
        if end > first:
            av = a[first:end].float() / _spread_scales(st["a_scales"][first:end], K, 1)
            for j in range(matrices):
                s = st["b_scales"][e * matrices + j]
                bv = b[e * matrices + j].float() / _spread_scales(_spread_scales(s, N, 0), K, 1)
                y[first:end, j] = av @ bv.t()
        first = end
    return y


def _products_i8(st, matrices):
    """The same of 8-bit integers: sums pass 24 bits, so they are held in 64."""
    a, b = st["a"], st["b"]
    M, N = a.shape[0], b.shape[1]
    y = torch.zeros((M, matrices, N), device=a.device)
    first = 0
    for e, end in enumerate(st["ends"]):
        if end > first:
            av = a[first:end].double()
            for j in range(matrices):
                s = st["a_scales"][first:end, None].double() * st["b_scales"][e * matrices + j].double()
                y[first:end, j] = (av @ b[e * matrices + j].double().t() / s).float()
        first = end
    return y


def _plain_gated(st):
    case = st["case"]
    y = (_products if case["op"] == "gated" else _products_i8)(st, 2)
    g, u = y[:, 0], y[:, 1]
    s, _ = _sigmoid_of(case["act"], g)
    out = {"h": (g * s * u).to(torch.bfloat16)}
    if case.get("keep"):
        out["gu"] = y.reshape(y.shape[0], -1).to(torch.bfloat16)
    return out


def _plain_grad(st):
    case = st["case"]
    F = case["F"]
    dh = _products(st, 1)[:, 0]
    g, u = st["gu"][:, :F].float(), st["gu"][:, F:].float()
    s, dt = _sigmoid_of(case["act"], g)
    dg = dh * u * (s + g * s * (1 - s) * dt)
    out = {"dgu": torch.cat([dg, dh * g * s], 1).to(torch.bfloat16)}
    if case["hidden"]:
        out["h"] = (g * s * u).to(torch.bfloat16)
    return out


def _plain_cast(st):
    q, s = _cast_i8(st["x"])
    return {"q": q, "scales": s}


def _plain_product(st):
    return {"y": _products_i8(st, 1)[:, 0].to(torch.float32 if st["case"]["f32"] else torch.bfloat16)}


# ---- one pass --------------------------------------------------------------------

def _own_run(st):
    import group_scaling_fp8_amd as mgs
    from group_scaling_fp8_amd import feedforward
    case, op = st["case"], st["case"]["op"]
    if op == "cast":
        q, s = feedforward.mgs_quant_rows_i8(st["x"])
        return {"q": q, "scales": s}
    args = (st["a"], st["a_scales"], st["b"], st["b_scales"])
    if op == "product":
        return {"y": feedforward.mgs_mm_i8(*args, st["offsets"], torch.float32 if case["f32"] else torch.bfloat16)}
    act = mgs.MGS_ACT_SILU if case["act"] == "silu" else mgs.MGS_ACT_GELU
    if op == "gated8":
        return {"h": feedforward.mgs_mm_gated_i8(*args, st["offsets"], act)}
    if op == "gated":
        out = feedforward.mgs_mm_gated_block128(*args, st["offsets"], act, fast_accum=case["fast"],
                                                keep=case["keep"])
        return {"h": out[0], "gu": out[1]} if case["keep"] else {"h": out}
    out = feedforward.mgs_mm_gated_grad_block128(*args, st["gu"], st["offsets"], act, fast_accum=case["fast"],
                                                 hidden=case["hidden"])
    return {"dgu": out[0], "h": out[1]} if case["hidden"] else {"dgu": out}


_PLAIN = {"gated": _plain_gated, "gated8": _plain_gated, "grad": _plain_grad, "cast": _plain_cast,
          "product": _plain_product}


def run(state):
    return _own_run(state) if own else _PLAIN[state["case"]["op"]](state)


# ---- what a pass cannot do without ---------------------------------------------------

def work(case):
    op = case["op"]
    if op == "cast":
        return {"bytes": case["M"] * (case["K"] * 3 + 4), "flops": 3 * case["M"] * case["K"]}
    up = lambda v: -(-v // BLOCK)  # noqa: E731
    N, K, E = case.get("N") or case["F"], case.get("K") or case["D"], max(case["E"], 1)
    if case.get("T"):
        rows = case["T"] * case["k"]
        M = _rows_bound(case["T"], case["k"], E)
        used = E * (1 - (1 - case["k"] / E) ** case["T"])       # experts that some token chose, on average
    else:
        rows = M = case["M"]
        used = min(E, -(-M // ALIGN))
    matrices = 2 if op in ("gated", "gated8") else 1
    if op in ("gated", "grad"):
        a, b = rows * (K + up(K) * 4), N * K + up(N) * up(K) * 4
    else:
        a, b = rows * (K + 4), N * K + N * 4
    out = {"gated": 6 if case.get("keep") else 2, "gated8": 2, "grad": 8 + (2 if case.get("hidden") else 0),
           "product": 4 if case.get("f32") else 2}[op]          # bytes for each row and column, grad: also gu
    return {"bytes": a + used * matrices * b + M * N * out, "flops": 2 * rows * matrices * N * K}


# ---- the definition in 64 bits -----------------------------------------------------------

def _decoded_64(code):
    """The value of each E4M3 byte, from its sign, exponent and fraction."""
    code = torch.arange(256, device=code.device)
    sign, e, f = 1.0 - 2.0 * (code >> 7).double(), (code >> 3) & 15, (code & 7).double()
    power = torch.tensor([2.0 ** max(i - 7, -6) for i in range(16)], dtype=torch.float64, device=code.device)[e]
    return sign * torch.where(e == 0, f / 8, 1 + f / 8) * power


def _over_blocks(s, rows, cols, dim):
    """v / s of a block's values, spread over the whole matrix (dim 0: blocks down and across, 1: across)."""
    s = s.double()
    if dim == 0:
        s = s[torch.arange(rows, device=s.device) // BLOCK]
    return s[:, torch.arange(cols, device=s.device) // BLOCK]


def _matrices_64(st, e, matrices):
    b, s = st["b"], st["b_scales"]
    N, K = b.shape[1:]
    if st["case"]["op"] in ("gated", "grad"):
        table = _decoded_64(b)
        return [table[b[i].long()] / _over_blocks(s[i], N, K, 0) for i in range(e * matrices, (e + 1) * matrices)]
    return [b[i].double() / s[i].double()[:, None] for i in range(e * matrices, (e + 1) * matrices)]


def _rows_64(st, first, end):
    a, s = st["a"][first:end], st["a_scales"][first:end]
    if st["case"]["op"] in ("gated", "grad"):
        return _decoded_64(a)[a.long()] / _over_blocks(s, a.shape[0], a.shape[1], 1)
    return a.double() / s.double()[:, None]


def _activation_64(act, g):
    """act(g) and its derivative, from the hyperbolic tangent."""
    if act == "silu":
        s = 0.5 * (1 + torch.tanh(g / 2))
        return g * s, s * (1 + g * (1 - s))
    r = math.sqrt(2 / math.pi)
    th = torch.tanh(r * (g + 0.044715 * g ** 3))
    return 0.5 * g * (1 + th), 0.5 * (1 + th) + 0.5 * g * (1 - th * th) * r * (1 + 3 * 0.044715 * g * g)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "cast":
        v = st["x"].double()
        s = (I8_MAX / v.abs().amax(1).clamp(min=float(torch.tensor(EPS)))).float()     # a binary32 number by definition
        near = (v * s.double()[:, None]).float().double()                              # and so is the scaled value
        q = torch.floor(near + 0.5)
        return {"q": torch.where((near + 0.5 == q) & (q % 2 != 0), q - 1, q).to(torch.int8), "scales": s.double()}
    matrices = 2 if op in ("gated", "gated8") else 1
    M, N = st["a"].shape[0], st["b"].shape[1]
    out = {}
    f64 = lambda cols: torch.zeros((M, cols), dtype=torch.float64, device=st["a"].device)  # noqa: E731
    out[{"product": "y", "grad": "dgu"}.get(op, "h")] = main = f64(2 * N if op == "grad" else N)
    if case.get("keep"):
        out["gu"] = f64(2 * N)
    if op == "grad" and case["hidden"]:
        out["h"] = f64(N)
    first = 0
    for e, end in enumerate(st["ends"]):
        if end > first:
            y = [torch.matmul(_rows_64(st, first, end), w.t()) for w in _matrices_64(st, e, matrices)]
            if op == "product":
                main[first:end] = y[0]
            elif op == "grad":
                g, u = st["gu"][first:end, :N].double(), st["gu"][first:end, N:].double()
                act, slope = _activation_64(case["act"], g)
                main[first:end, :N] = y[0] * u * slope
                main[first:end, N:] = y[0] * act
                if case["hidden"]:
                    out["h"][first:end] = act * u
            else:
                main[first:end] = _activation_64(case["act"], y[0])[0] * y[1]
                if case.get("keep"):
                    out["gu"][first:end, :N], out["gu"][first:end, N:] = y
        first = end
    return out
