"""CPU checks of the mixture-of-experts calls: arguments they refuse (before
any GPU work), the host-only size queries, the Python front end's own
checks, and the plain 64-bit forms against small worked cases."""
import ctypes
import inspect
import os

import numpy as np
import pytest

import experts_ref as ref
import group_scaling_fp8_amd as mgs
from group_scaling_fp8_amd import workloads as wl

OK, INVALID, UNSUPPORTED = mgs.MGS_OK, mgs.MGS_ERR_INVALID_ARG, mgs.MGS_ERR_UNSUPPORTED
A = 1 << 20          # a fake, well-aligned "device" address; never dereferenced


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(mgs.library_path()):
        from group_scaling_fp8_amd import build
        build.build()
    return mgs.lib()


def with_defaults(fn, order, **defaults):
    return lambda **kw: fn(*[dict(defaults, **kw)[name] for name in order])


def test_size_queries(L):
    n = ctypes.c_int64(-1)

    def rows(*a):
        return L.mgs_moe_rows(*a, ctypes.byref(n))
    for T, k, E, align in ((0, 1, 4, 16), (1, 8, 64, 16), (7, 2, 1, 16), (33, 3, 8, 32), (5000, 8, 1024, 128)):
        assert rows(T, k, E, align) == OK
        m = T * k
        assert n.value == (m + min(E, m) * (align - 1)) // align * align
        assert n.value == mgs.mgs_moe_rows(T, k, E, align)
        # the worst split: as many groups as possible hold one row more than a multiple
        used = min(E, m)
        worst = sum(-(-c // align) * align for c in
                    [1] * max(0, used - 1) + ([m - used + 1] if used else []))
        assert worst <= n.value
    assert rows(-1, 1, 4, 16) == INVALID
    assert rows(1, 0, 4, 16) == INVALID
    assert rows(1, 1, 0, 16) == INVALID
    assert rows(1, 1, 4, 8) == INVALID
    assert rows(1, 1, 4, 24) == INVALID
    assert rows(1, 65, 4, 16) == UNSUPPORTED
    assert rows(1, 1, 1025, 16) == UNSUPPORTED
    assert rows(1 << 30, 2, 4, 16) == UNSUPPORTED
    assert L.mgs_moe_rows(1, 1, 4, 16, None) == INVALID
    assert L.mgs_moe_workspace_bytes(1, 8, 64, ctypes.byref(n)) == OK and n.value == 0
    assert L.mgs_moe_workspace_bytes(1 << 20, 8, 64, ctypes.byref(n)) == OK and 0 < n.value <= 256 * 64
    assert L.mgs_moe_workspace_bytes(1, 8, 64, None) == INVALID


def test_dispatch_refusals(L):
    f = with_defaults(L.mgs_moe_dispatch,
                      ("x", "T", "D", "ids", "k", "E", "align", "flags", "P", "off", "rows", "slots", "xp", "q", "s",
                       "ws", "wsb", "stream"),
                      x=A, T=4, D=64, ids=A, k=2, E=8, align=16, flags=0, P=128, off=A, rows=A, slots=A, xp=A, q=A,
                      s=A, ws=None, wsb=0, stream=None)
    for bad in (dict(T=-1), dict(k=0), dict(E=0), dict(align=0), dict(align=20), dict(flags=2), dict(flags=4),
                dict(D=-8), dict(D=12), dict(P=112), dict(P=-1), dict(off=None), dict(off=A + 2), dict(ids=None),
                dict(ids=A + 1), dict(rows=None), dict(rows=A + 2), dict(slots=None), dict(slots=A + 2),
                dict(q=None), dict(s=None), dict(x=None), dict(x=A + 8), dict(xp=A + 8), dict(q=A + 4), dict(s=A + 2),
                dict(wsb=-1)):
        assert f(**bad) == INVALID, bad
    for bad in (dict(k=65), dict(E=1025), dict(align=8192), dict(D=1 << 31), dict(P=1 << 31), dict(T=1 << 30)):
        assert f(**bad) == UNSUPPORTED, bad
    # more slots than one workgroup counts need a workspace
    big = dict(T=100000, P=200000 + 8 * 15)
    assert f(**big) == INVALID
    assert f(ws=A, wsb=64, **big) == INVALID
    assert f(ws=A + 8, wsb=1 << 20, **big) == INVALID


def test_combine_refusals(L):
    f = with_defaults(L.mgs_moe_combine, ("yp", "P", "D", "rows", "T", "k", "w", "y", "stream"),
                      yp=A, P=64, D=64, rows=A, T=4, k=2, w=A, y=A, stream=None)
    for bad in (dict(P=-1), dict(D=12), dict(D=-8), dict(T=-1), dict(k=0), dict(rows=None), dict(rows=A + 2),
                dict(y=None), dict(y=A + 8), dict(yp=None), dict(yp=A + 8), dict(w=A + 2)):
        assert f(**bad) == INVALID, bad
    for bad in (dict(k=65), dict(P=1 << 31), dict(D=1 << 31)):
        assert f(**bad) == UNSUPPORTED, bad
    assert f(T=0) == OK and f(D=0) == OK
    g = with_defaults(L.mgs_moe_combine_grad,
                      ("dy", "yp", "P", "D", "rows", "slots", "T", "k", "w", "dyp", "dw", "stream"),
                      dy=A, yp=A, P=64, D=64, rows=A, slots=A, T=4, k=2, w=A, dyp=A, dw=A, stream=None)
    for bad in (dict(P=-1), dict(D=12), dict(T=-1), dict(k=0), dict(rows=None), dict(slots=None), dict(slots=A + 2),
                dict(w=None), dict(dw=None), dict(dw=A + 2), dict(dy=None), dict(dy=A + 8), dict(yp=None),
                dict(yp=A + 8), dict(dyp=None), dict(dyp=A + 8)):
        assert g(**bad) == INVALID, bad
    assert g(k=65) == UNSUPPORTED
    assert g(T=0, P=0) == OK


def test_cast_refusals(L):
    f = with_defaults(L.mgs_quant_rows128, ("x", "M", "K", "flags", "q", "s", "stream"),
                      x=A, M=4, K=64, flags=0, q=A, s=A, stream=None)
    for bad in (dict(M=-1), dict(K=12), dict(K=-8), dict(flags=2), dict(x=None), dict(q=None), dict(s=None),
                dict(x=A + 8), dict(q=A + 4), dict(s=A + 2)):
        assert f(**bad) == INVALID, bad
    assert f(K=1 << 31) == UNSUPPORTED
    assert f(M=0) == OK and f(K=0) == OK
    g = with_defaults(L.mgs_quant_blocks128, ("w", "E", "N", "K", "flags", "q", "s", "qt", "st", "stream"),
                      w=A, E=2, N=64, K=64, flags=0, q=A, s=A, qt=A, st=A, stream=None)
    for bad in (dict(E=-1), dict(N=8), dict(K=24), dict(N=-16), dict(flags=4), dict(w=None), dict(q=None),
                dict(s=None), dict(qt=None), dict(st=None), dict(w=A + 8), dict(q=A + 8), dict(qt=A + 8),
                dict(s=A + 2), dict(st=A + 2)):
        assert g(**bad) == INVALID, bad
    assert g(K=1 << 31) == UNSUPPORTED
    assert g(E=1 << 30, N=1 << 20, K=1 << 20) == UNSUPPORTED
    assert g(E=0) == OK and g(N=0) == OK and g(K=0) == OK


def test_product_refusals(L):
    f = with_defaults(L.mgs_mm_block128, ("a", "sa", "M", "K", "b", "sb", "G", "N", "off", "flags", "out", "y", "stream"),
                      a=A, sa=A, M=64, K=64, b=A, sb=A, G=2, N=64, off=A, flags=0, out=0, y=A, stream=None)
    for bad in (dict(M=-1), dict(N=-16), dict(K=-16), dict(N=24), dict(K=24), dict(G=0), dict(out=2), dict(out=-1), dict(flags=4), dict(flags=1),
                dict(off=None), dict(off=A + 2), dict(y=None), dict(y=A + 8), dict(a=None), dict(a=A + 8),
                dict(b=None), dict(b=A + 8), dict(sa=None), dict(sa=A + 2), dict(sb=None), dict(sb=A + 2)):
        assert f(**bad) == INVALID, bad
    for bad in (dict(G=1025), dict(M=1 << 31), dict(N=1 << 31), dict(K=1 << 23), dict(M=1 << 30, N=1 << 20)):
        assert f(**bad) == UNSUPPORTED, bad
    assert f(M=0) == OK and f(N=0) == OK
    g = with_defaults(L.mgs_mm_wgrad,
                      ("a", "sa", "b", "sb", "M", "N", "K", "off", "G", "flags", "out", "dw", "stream"),
                      a=A, sa=A, b=A, sb=A, M=64, N=64, K=64, off=A, G=2, flags=0, out=1, dw=A, stream=None)
    for bad in (dict(M=-16), dict(M=24), dict(N=8), dict(K=8), dict(G=0), dict(flags=1), dict(flags=2),
                dict(flags=4, out=0), dict(out=3), dict(off=None), dict(off=A + 1), dict(dw=None), dict(dw=A + 8),
                dict(a=None), dict(a=A + 8), dict(b=None), dict(b=A + 8), dict(sa=None), dict(sb=A + 2)):
        assert g(**bad) == INVALID, bad
    for bad in (dict(G=1025), dict(M=1 << 23), dict(N=1 << 31), dict(N=1 << 30, K=1 << 30)):
        assert g(**bad) == UNSUPPORTED, bad
    assert g(N=0) == OK and g(K=0) == OK


def test_python_front_end_rejects_cpu_tensors():
    torch = pytest.importorskip("torch")
    x = torch.zeros((16, 64), dtype=torch.bfloat16)
    ids = torch.zeros((16, 2), dtype=torch.int32)
    u8, f32 = torch.zeros((16, 64), dtype=torch.uint8), torch.zeros((16, 1))
    off = torch.tensor([16], dtype=torch.int32)
    for call in (lambda: mgs.mgs_moe_sort(ids, 4), lambda: mgs.mgs_moe_dispatch(x, ids, 4),
                 lambda: mgs.mgs_moe_combine(x, ids), lambda: mgs.mgs_quant_rows128(x),
                 lambda: mgs.mgs_quant_blocks128(x[None]),
                 lambda: mgs.mgs_mm_block128(u8, f32, u8[None], f32[None], off),
                 lambda: mgs.mgs_mm_wgrad(u8, f32, u8, f32, off),
                 lambda: mgs.mgs_moe_combine_grad(x, x, ids, ids[:, 0], ids.float())):
        with pytest.raises(ValueError):
            call()


def test_every_call_takes_a_stream():
    for name in ("mgs_moe_sort", "mgs_moe_dispatch", "mgs_moe_combine", "mgs_moe_combine_grad", "mgs_quant_rows128",
                 "mgs_quant_blocks128", "mgs_mm_block128", "mgs_mm_wgrad"):
        assert "stream" in inspect.signature(getattr(mgs, name)).parameters, name


# ---- the plain forms themselves -------------------------------------------------

def test_order_by_hand():
    ids = np.array([[1, 3], [3, -1], [1, 1], [9, 0]], np.int32)
    off, rows, slots = ref.order(ids, 4, 16)
    assert off.tolist() == [16, 32, 32, 48]
    assert rows.tolist() == [[16, 32], [33, -1], [17, 18], [-1, 0]]
    assert slots[0] == 7 and slots[16:19].tolist() == [0, 4, 5] and slots[32:34].tolist() == [1, 2]
    assert (slots >= 0).sum() == 6 and len(slots) == 64


def test_casts_by_hand():
    x = np.zeros((2, 144), np.float32)
    x[0, 5], x[0, 130], x[1, 0] = 2.0, -0.5, 448.0
    q, s = ref.rows128(wl.f32_to_bf16_bits(x))
    assert s.tolist() == [[224.0, 896.0], [1.0, np.float32(448.0) / np.float32(1e-12)]]
    assert ref.DECODE[q[0, 5]] == 448 and ref.DECODE[q[0, 130]] == -448 and ref.DECODE[q[1, 0]] == 448
    w = np.zeros((1, 144, 144), np.float32)
    w[0, 0, 0], w[0, 143, 143], w[0, 143, 0] = 4.0, 1.0, 448.0
    q, s = ref.blocks128(wl.f32_to_bf16_bits(w))
    assert s[0, 0, 0] == 112 and s[0, 1, 1] == 448 and s[0, 1, 0] == 1
    assert ref.DECODE[q[0, 143, 143]] == 448 and q.astype(int).sum() == 3 * 0x7E


def test_products_by_hand():
    one = int(np.argmin(np.abs(np.nan_to_num(ref.DECODE, nan=9) - 1)))
    a, b = np.full((3, 144), one, np.uint8), np.full((2, 16, 144), one, np.uint8)
    sa, sb = np.array([[1, 2]] * 3, np.float32), np.array([[[1, 4]], [[2, 2]]], np.float32)
    y, mag = ref.mm_block128(a, sa, b, sb, [1, 2])
    assert (y[0] == 128 + 16 / 8).all() and (y[1] == 64 + 16 / 4).all() and (y[2] == 0).all() and (mag == y).all()
    dw, _ = ref.mm_wgrad(a[:, :32], np.array([[2, 1]] * 3, np.float32), b[0, :, :32], np.array([[1, 4]] * 16, np.float32),
                         [16, 32])
    assert (dw[0] == 8).all() and (dw[1] == 4).all()


def test_gradient_of_combine_by_differences():
    """The formula of the gradient against central differences of the sum."""
    rng = np.random.default_rng(3)
    ids = np.array([[0, 2], [2, -1], [1, 0]], np.int32)
    _, rows, slots = ref.order(ids, 3, 16)
    yp, w, dy = rng.standard_normal((len(slots), 5)), rng.random((3, 2)), rng.standard_normal((3, 5))
    dyp, dw, _ = ref.combine_grad(dy, yp, rows, w)

    def loss(yp, w):
        return float((ref.combine(yp, rows, w)[0] * dy).sum())
    h = 1e-6
    for at in [(0, 1), (1, 4), (16, 0), (32, 2), (33, 3), (47, 0)]:
        up, down = yp.copy(), yp.copy()
        up[at] += h
        down[at] -= h
        assert abs((loss(up, w) - loss(down, w)) / (2 * h) - dyp[at]) < 1e-7
    for at in np.ndindex(w.shape):
        up, down = w.copy(), w.copy()
        up[at] += h
        down[at] -= h
        assert abs((loss(yp, up) - loss(yp, down)) / (2 * h) - dw[at]) < 1e-7
