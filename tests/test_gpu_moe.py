"""Tokens sorted by expert and back on the GPU: orders and cast bytes equal
to the plain form's, sums and gradients within the roundings they make."""
import numpy as np
import pytest
import torch

import experts_ref as ref
import group_scaling_fp8_amd as mgs
from group_scaling_fp8_amd import workloads as wl
from gpu_util import Guarded, assert_same_bytes, dev, to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mgs.lib()


def bf16(a):
    return to_dev(wl.f32_to_bf16_bits(a)).view(torch.bfloat16)


def bits(t):
    return t.view(torch.int16).cpu().numpy().view(np.uint16)


def draw_ids(rng, T, k, E, kind="mixed"):
    if kind == "dropped":
        return np.full((T, k), -1, np.int32)
    if kind == "one":
        return np.full((T, k), E - 1, np.int32)
    ids = rng.integers(0, E, size=(T, k)).astype(np.int32)
    if kind == "skewed":
        ids[rng.random((T, k)) < 0.8] = E // 2
    if kind == "mixed":      # dropped slots: ids outside the experts on both sides
        ids[rng.random((T, k)) < 0.1] = -1
        ids[rng.random((T, k)) < 0.05] = E
        ids[rng.random((T, k)) < 0.02] = np.iinfo(np.int32).min
        ids[rng.random((T, k)) < 0.02] = np.iinfo(np.int32).max
    return ids


@pytest.mark.parametrize("T,k,E,align,kind", [
    (0, 2, 4, 16, "mixed"), (1, 1, 1, 16, "plain"), (1, 8, 64, 16, "plain"), (1, 8, 64, 16, "dropped"),
    (3, 64, 5, 32, "mixed"), (65, 3, 7, 16, "mixed"), (129, 2, 1024, 48, "mixed"), (1000, 4, 61, 16, "skewed"),
    (4096, 2, 16, 128, "one"), (4097, 2, 16, 16, "mixed"), (5000, 8, 256, 16, "mixed"),
    (40001, 7, 1023, 64, "mixed"), (100000, 8, 64, 16, "skewed")])
def test_order(T, k, E, align, kind):
    rng = np.random.default_rng(T * 31 + E)
    ids = draw_ids(rng, T, k, E, kind)
    off, rows, slots = mgs.mgs_moe_sort(to_dev(ids), E, align)
    torch.cuda.synchronize()
    r_off, r_rows, r_slots = ref.order(ids, E, align)
    assert np.array_equal(off.cpu().numpy(), r_off)
    assert np.array_equal(rows.cpu().numpy(), r_rows)
    assert np.array_equal(slots.cpu().numpy(), r_slots)


@pytest.mark.parametrize("T,k,E,D,kind,pow2", [
    (0, 2, 4, 64, "mixed", False), (1, 1, 1, 8, "plain", False), (1, 8, 64, 5120, "plain", False),
    (1, 3, 8, 1048, "dropped", True), (37, 4, 9, 136, "mixed", False), (300, 6, 61, 520, "mixed", True),
    (1100, 2, 4, 4112, "skewed", False), (5000, 3, 16, 264, "mixed", False)])
def test_dispatch(T, k, E, D, kind, pow2):
    rng = np.random.default_rng(T + D)
    ids = draw_ids(rng, T, k, E, kind)
    x = wl.randn_bf16(rng, (T, D), 0.02, 0.001, 8.0)
    if T > 2:
        x[1] = 0
        x[2, :128] = 1          # the least subnormal: amax below the scale's floor
    off, rows, slots, q, s, xp = mgs.mgs_moe_dispatch(to_dev(x), to_dev(ids), E, pow2=pow2, permuted=True)
    torch.cuda.synchronize()
    r_off, r_rows, r_slots = ref.order(ids, E, 16)
    assert np.array_equal(off.cpu().numpy(), r_off)
    assert np.array_equal(rows.cpu().numpy(), r_rows)
    assert np.array_equal(slots.cpu().numpy(), r_slots)
    r_xp = ref.permuted(x, r_slots, k)
    assert_same_bytes(bits(xp), r_xp, "xp")
    r_q, r_s = ref.rows128(r_xp, pow2)
    assert_same_bytes(q.cpu().numpy(), r_q, "q")
    assert_same_bytes(s.cpu().numpy(), r_s, "scales")


def test_dispatch_into_larger_row_arrays_stays_inside_them():
    """The C call with more rows than it needs, guard bands around every
    output, and an n_rows that is no multiple of the alignment."""
    rng = np.random.default_rng(8)
    T, k, E, D = 70, 3, 5, 200
    P = mgs.mgs_moe_rows(T, k, E) + 37
    ids, x = draw_ids(rng, T, k, E), wl.randn_bf16(rng, (T, D), 1.0)
    out = {"off": Guarded((E,), torch.int32), "rows": Guarded((T, k), torch.int32),
           "slots": Guarded((P,), torch.int32), "xp": Guarded((P, D), torch.int16),
           "q": Guarded((P, D), torch.uint8), "s": Guarded((P, 2), torch.float32)}
    o = {n: g.view.data_ptr() for n, g in out.items()}
    ids_d, x_d = to_dev(ids), to_dev(x)
    st = mgs.lib().mgs_moe_dispatch(x_d.data_ptr(), T, D, ids_d.data_ptr(), k, E, 16, 0, P, o["off"], o["rows"],
                                    o["slots"], o["xp"], o["q"], o["s"], None, 0, None)
    assert st == mgs.MGS_OK
    torch.cuda.synchronize()
    for g in out.values():
        g.check()
    r_off, r_rows, r_slots = ref.order(ids, E, 16)
    r_slots = np.concatenate([r_slots, np.full(P - len(r_slots), -1, np.int32)])
    r_xp = ref.permuted(x, r_slots, k)
    r_q, r_s = ref.rows128(r_xp)
    for name, want in (("off", r_off), ("rows", r_rows), ("slots", r_slots), ("xp", r_xp.view(np.int16)), ("q", r_q),
                       ("s", r_s)):
        assert np.array_equal(out[name].numpy(), want), name


@pytest.mark.parametrize("T,k,E,D,kind", [
    (1, 1, 1, 8, "plain"), (1, 8, 64, 5120, "plain"), (5, 2, 4, 2056, "dropped"), (37, 4, 9, 136, "mixed"),
    (130, 6, 61, 520, "mixed"), (33, 64, 16, 72, "mixed"), (257, 2, 4, 4112, "skewed")])
@pytest.mark.parametrize("weighted", [True, False])
def test_combine(T, k, E, D, kind, weighted):
    rng = np.random.default_rng(T * 7 + D)
    ids = draw_ids(rng, T, k, E, kind)
    _, rows, slots = ref.order(ids, E, 16)
    yp = wl.randn_bf16(rng, (len(slots), D), 1.0, 0.001, 20.0)
    yp[slots < 0] = 0x7FC0          # NaN in the rows that no slot reads
    w = rng.random((T, k)).astype(np.float32)
    got = mgs.mgs_moe_combine(to_dev(yp), to_dev(rows), to_dev(w) if weighted else None)
    torch.cuda.synchronize()
    want, mag = ref.combine(ref.bf16_to_f64(yp), rows, w if weighted else np.ones_like(w))
    # k additions in binary32, each off by at most half a step of a partial
    # sum, then one rounding to bf16
    tol = mag * k * 2.0 ** -24 * 1.01 + np.abs(want) * ref.HALF_STEP["bf16"] * 1.01
    err = np.abs(ref.bf16_to_f64(bits(got)) - want)
    assert (err <= tol).all(), float((err - tol).max())


@pytest.mark.parametrize("T,k,E,D,kind", [
    (1, 1, 1, 8, "plain"), (1, 8, 64, 5120, "plain"), (5, 2, 4, 2056, "dropped"), (37, 4, 9, 136, "mixed"),
    (130, 6, 61, 520, "mixed"), (33, 64, 16, 72, "mixed"), (70, 2, 4, 8200, "skewed")])
def test_combine_grad(T, k, E, D, kind):
    rng = np.random.default_rng(T * 11 + D)
    ids = draw_ids(rng, T, k, E, kind)
    _, rows, slots = ref.order(ids, E, 16)
    yp = wl.randn_bf16(rng, (len(slots), D), 1.0, 0.001, 20.0)
    yp[slots < 0] = 0x7F80          # infinity in the rows that no slot reads
    dy = wl.randn_bf16(rng, (T, D), 0.02, 0.001, 8.0)
    w = rng.random((T, k)).astype(np.float32)
    dyp, dw = Guarded(yp.shape, torch.bfloat16), Guarded((T, k), torch.float32)
    mgs.mgs_moe_combine_grad(to_dev(dy).view(torch.bfloat16), to_dev(yp), to_dev(rows), to_dev(slots), to_dev(w),
                             dyp=dyp.view, dw=dw.view)
    torch.cuda.synchronize()
    dyp.check()
    dw.check()
    want_p, want_w, mag = ref.combine_grad(ref.bf16_to_f64(dy), ref.bf16_to_f64(np.where(yp == 0x7F80, 0, yp)), rows, w)
    # dyp: one binary32 product and one rounding; dw: a sum of D terms in binary32
    got = ref.bf16_to_f64(bits(dyp.view))
    assert (np.abs(got - want_p) <= np.abs(want_p) * (ref.HALF_STEP["bf16"] * 1.01 + 2.0 ** -23)).all()
    err = np.abs(dw.numpy() - want_w)
    assert (err <= mag * D * 2.0 ** -24 * 1.01).all()


def test_bad_rows_and_slots_stay_in_bounds():
    """Rows and slots outside their arrays add nothing and are not followed."""
    rng = np.random.default_rng(5)
    P, D, T, k = 64, 64, 9, 3
    yp = wl.randn_bf16(rng, (P, D), 1.0)
    rows = rng.choice(P, size=(T, k), replace=False).astype(np.int32)
    rows[0] = [-5, P, np.iinfo(np.int32).max]
    rows[1, 0] = np.iinfo(np.int32).min
    slots = np.full(P, -1, np.int32)
    for i, p in enumerate(rows.reshape(-1)):
        if 0 <= p < P:
            slots[p] = i
    slots[slots < 0] = rng.choice([-1, -7, T * k, np.iinfo(np.int32).max], size=(slots < 0).sum())
    w = rng.random((T, k)).astype(np.float32)
    dy = wl.randn_bf16(rng, (T, D), 1.0)
    y = mgs.mgs_moe_combine(to_dev(yp), to_dev(rows), to_dev(w))
    dyp, dw = mgs.mgs_moe_combine_grad(to_dev(dy), to_dev(yp), to_dev(rows), to_dev(slots), to_dev(w))
    torch.cuda.synchronize()
    want, _ = ref.combine(ref.bf16_to_f64(yp), rows, w)
    assert (bits(y)[0] == 0).all()
    assert np.abs(ref.bf16_to_f64(bits(y)) - want).max() < 0.05
    want_p, want_w, _ = ref.combine_grad(ref.bf16_to_f64(dy), ref.bf16_to_f64(yp), rows, w)
    assert (dw.cpu().numpy()[0] == 0).all() and np.abs(dw.cpu().numpy() - want_w).max() < 1e-3
    assert np.abs(ref.bf16_to_f64(bits(dyp)) - want_p).max() < 0.05


def test_gradient_against_differences():
    """<dy, combine> as a function of the weights and of the rows: its
    central differences, with steps that bf16 and binary32 hold exactly."""
    rng = np.random.default_rng(12)
    T, k, E, D = 6, 2, 3, 16
    ids = draw_ids(rng, T, k, E, "plain")
    _, rows, slots = ref.order(ids, E, 16)
    # few enough bits that every product and sum is exact in binary32
    yp = np.where((slots >= 0)[:, None], rng.integers(-8, 9, (len(slots), D)), 0).astype(np.float32)
    dy = rng.integers(-4, 5, (T, D)).astype(np.float32)
    w = (rng.integers(1, 5, (T, k)) / 4).astype(np.float32)
    rows_d, slots_d = to_dev(rows), to_dev(slots)

    def loss(yp, w):
        y = mgs.mgs_moe_combine(bf16(yp), rows_d, to_dev(w))
        return float((y.double().cpu().numpy() * dy).sum())
    dyp, dw = mgs.mgs_moe_combine_grad(bf16(dy), bf16(yp), rows_d, slots_d, to_dev(w))
    dyp, dw = dyp.double().cpu().numpy(), dw.double().cpu().numpy()
    h = 0.25
    for t in range(T):
        for s in range(k):
            up, down = w.copy(), w.copy()
            up[t, s] += h
            down[t, s] -= h
            assert (loss(yp, up) - loss(yp, down)) / (2 * h) == dw[t, s]
    for p in range(0, len(slots), 5):
        for c in (0, D - 1):
            up, down = yp.copy(), yp.copy()
            up[p, c] += 1
            down[p, c] -= 1
            assert (loss(up, w) - loss(down, w)) / 2 == dyp[p, c]


def test_repeats_are_identical():
    rng = np.random.default_rng(4)
    T, k, E, D = 3000, 4, 16, 520
    ids, x = to_dev(draw_ids(rng, T, k, E)), to_dev(wl.randn_bf16(rng, (T, D), 1.0))
    w = torch.rand((T, k), device=dev())
    first = None
    for _ in range(3):
        off, rows, slots, q, s, xp = mgs.mgs_moe_dispatch(x, ids, E, permuted=True)
        y = mgs.mgs_moe_combine(xp, rows, w)
        dyp, dw = mgs.mgs_moe_combine_grad(y, xp, rows, slots, w)
        now = [t.view(torch.uint8).clone() if t.dtype != torch.int32 else t.clone()
               for t in (off, rows, slots, q, s, xp, y, dyp, dw)]
        if first is not None:
            assert all(torch.equal(a, b) for a, b in zip(first, now))
        first = now


def test_past_two_to_the_31_elements():
    """Row arrays of more than 2^31 elements: the last rows arrive."""
    T, k, E, D = 33000, 8, 8, 8192
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GiB")
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    x = torch.randn((T, D), generator=gen, device="cuda", dtype=torch.bfloat16)
    ids = (torch.arange(k, device="cuda", dtype=torch.int32)[None] + torch.arange(T, device="cuda", dtype=torch.int32)[:, None]) % E
    off, rows, slots, q, s, xp = mgs.mgs_moe_dispatch(x, ids.contiguous(), E, permuted=True)
    assert xp.numel() > 1 << 31
    for p in (0, 1, 262144, 262145, int(off[-1]) - 1, int(off[-1]) // 2):
        slot = int(slots[p])
        if slot >= 0:
            assert torch.equal(xp[p], x[slot // k]), p
    last = int(torch.nonzero(slots >= 0)[-1])
    assert last > 262144 and torch.equal(xp[last], x[int(slots[last]) // k])
    back = mgs.mgs_moe_combine(xp, rows, torch.full((T, k), 0.125, device="cuda"))
    assert torch.equal(back, x)
    dyp, dw = mgs.mgs_moe_combine_grad(x, xp, rows, slots, torch.ones((T, k), device="cuda"))
    assert torch.equal(dyp[last], xp[last]) and torch.equal(dyp[262150], xp[262150])


def test_more_workgroups_than_one_grid_dimension_holds():
    """17 million tokens of eight columns: a workgroup each passes 2^32 threads."""
    T, E, D = 17_000_000, 4, 8
    t = torch.arange(T, device="cuda")
    ids = (t % E).to(torch.int32)[:, None].contiguous()
    x = (t[:, None] % 251 - 125).to(torch.bfloat16).expand(T, D).contiguous()
    off, rows, slots, q, s, xp = mgs.mgs_moe_dispatch(x, ids, E, permuted=True)
    per = T // E
    full = (per + 15) // 16 * 16
    assert off.tolist() == [full * (e + 1) for e in range(E)]
    assert torch.equal(rows[:, 0].long(), t % E * full + t // E)
    assert torch.equal(xp[rows[:, 0].long()], x)
    assert torch.equal(slots[rows[:, 0].long()].long(), t)
    pads = slots < 0
    assert int(pads.sum()) == slots.shape[0] - T and not bool(xp[pads].any())
    w = torch.full((T, 1), 2.0, device="cuda")
    assert torch.equal(mgs.mgs_moe_combine(xp, rows, w), 2 * x)
    dyp, dw = mgs.mgs_moe_combine_grad(x, xp, rows, slots, w)
    assert torch.equal(dyp[rows[:, 0].long()], 2 * x) and not bool(dyp[pads].any())
    assert torch.equal(dw[:, 0], (t % 251 - 125).float() ** 2 * D)


@pytest.mark.parametrize("T,k,E,align,kind", [
    (32768, 1, 5, 16, "mixed"), (4681, 7, 300, 32, "mixed"), (32769, 1, 1024, 16, "skewed"), (16400, 2, 513, 16, "mixed"),
    (9000, 4, 512, 16, "one"), (300001, 2, 3, 16, "mixed"), (10900, 3, 7, 4096, "mixed"), (513, 1, 2, 16, "dropped")])
def test_order_around_the_limit_of_one_launch(T, k, E, align, kind):
    """32768 slots are the last that one launch takes; runs past 524288 slots are
    ranked in several parts a wave."""
    test_order(T, k, E, align, kind)


@pytest.mark.parametrize("T,k,E,D,kind,pow2", [
    (520, 64, 70, 4104, "mixed", False), (33001, 1, 9, 72, "skewed", True), (4096, 8, 33, 1040, "mixed", False),
    (3000, 1, 40, 2072, "dropped", False)])
def test_dispatch_around_the_limit_of_one_launch(T, k, E, D, kind, pow2):
    test_dispatch(T, k, E, D, kind, pow2)
