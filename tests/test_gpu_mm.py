"""The products of cast matrices against sums in 64 bits, with tolerances
from the number of roundings (experts_ref.mm_tolerance)."""
import numpy as np
import pytest
import torch

import experts_ref as ref
import group_scaling_fp8_amd as mgs
from gpu_util import Guarded, dev, to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mgs.lib()


OUT = {"bf16": torch.bfloat16, "f32": torch.float32}


def codes(rng, shape):
    """E4M3 bytes of every exponent and both signs, zeros among them, without NaN."""
    c = rng.integers(0, 127, size=shape).astype(np.uint8)
    c[rng.random(shape) < 0.05] = 0
    return c | (rng.integers(0, 2, size=shape) << 7).astype(np.uint8)


def scales(rng, shape):
    """Scales as the casts give them, over many binades."""
    return np.exp2(rng.uniform(-6, 14, size=shape)).astype(np.float32)


def ends_of(kind, M, G, rng):
    if kind == "none":
        return None
    if kind == "even":
        return np.array([M * (g + 1) // G for g in range(G)], np.int32)
    if kind == "tail":          # rows past the last group, and empty groups
        e = np.sort(rng.integers(0, M * 2 // 3 + 1, size=G)).astype(np.int32)
        return e
    if kind == "empty":
        return np.zeros(G, np.int32)
    if kind == "one":           # every row in one group in the middle
        return np.array([0] * (G // 2) + [M] * (G - G // 2), np.int32)
    if kind == "bad":           # decreasing, negative and past the end
        e = rng.integers(-50, M + 50, size=G).astype(np.int32)
        return e
    raise AssertionError(kind)


def check(got, want, tol, what):
    err = np.abs(got.astype(np.float64) - want)
    bad = ~(err <= tol)
    assert not bad.any(), (what, int(bad.sum()), float(np.nanmax(err[bad] if bad.any() else err)),
                           tuple(np.argwhere(bad)[0]))


MM = [
    # M, N, K, groups, ends
    (1, 16, 16, 1, "none"), (1, 128, 128, 1, "none"), (2, 272, 1040, 1, "none"), (16, 48, 144, 1, "none"),
    (17, 144, 256, 1, "none"), (100, 528, 2064, 1, "none"), (129, 256, 384, 1, "none"), (300, 400, 656, 1, "none"),
    (520, 1040, 272, 1, "none"),
    (1, 32, 64, 3, "one"), (8, 160, 384, 8, "even"), (64, 272, 528, 4, "tail"), (128, 512, 1040, 8, "tail"),
    (80, 80, 160, 70, "even"), (200, 96, 144, 65, "tail"), (257, 272, 528, 3, "even"), (512, 144, 272, 2, "empty"),
    (700, 528, 400, 5, "one"), (1300, 272, 1168, 9, "even"), (900, 144, 144, 6, "bad"), (96, 272, 400, 12, "bad"),
]


@pytest.mark.parametrize("M,N,K,G,kind", MM)
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("fast", [False, True])
def test_mm_block128(M, N, K, G, kind, out, fast):
    rng = np.random.default_rng(M * 13 + N + K)
    off = ends_of(kind, M, G, rng)
    ends = ref.clean_ends(off if off is not None else [M], M)
    a, b = codes(rng, (M, K)), codes(rng, (G, N, K))
    kb = -(-K // 128)
    sa, sb = scales(rng, (M, kb)), scales(rng, (G, -(-N // 128), kb))
    # what no group holds is not a number
    a[ends[-1]:] = 0x7F
    sa[ends[-1]:] = np.nan
    y = Guarded((M, N), OUT[out])
    mgs.mgs_mm_block128(to_dev(a), to_dev(sa), to_dev(b), to_dev(sb), None if off is None else to_dev(off), OUT[out],
                        fast, y=y.view)
    torch.cuda.synchronize()
    y.check()
    want, mag = ref.mm_block128(np.where(a == 0x7F, 0, a), np.nan_to_num(sa, nan=1.0), b, sb, ends)
    check(y.view.float().cpu().numpy(), want, ref.mm_tolerance(want, mag, K, out, fast), (M, N, K, G, kind))


def test_mm_block128_rows_do_not_depend_on_others():
    """A row that is not a number leaves the others alone, and an
    expert's weights that are not numbers reach its own rows only."""
    rng = np.random.default_rng(77)
    M, N, K, G = 150, 272, 272, 3
    off = np.array([50, 90, 150], np.int32)
    a, b = codes(rng, (M, K)), codes(rng, (G, N, K))
    sa, sb = scales(rng, (M, 3)), scales(rng, (G, 3, 3))
    clean = mgs.mgs_mm_block128(to_dev(a), to_dev(sa), to_dev(b), to_dev(sb), to_dev(off)).float().cpu().numpy()
    a[[0, 49, 60, 149]] = 0x7F
    b[1] = 0xFF
    got = mgs.mgs_mm_block128(to_dev(a), to_dev(sa), to_dev(b), to_dev(sb), to_dev(off)).float().cpu().numpy()
    keep = np.ones(M, bool)
    keep[[0, 49, 149]] = False
    keep[50:90] = False
    assert np.array_equal(got[keep], clean[keep])
    assert np.isnan(got[~keep]).all()


WG = [
    # M, N, K, groups, ends
    (0, 48, 32, 2, "empty"), (16, 16, 16, 1, "even"), (16, 144, 272, 3, "one"), (48, 272, 144, 2, "even"),
    (128, 128, 128, 1, "even"), (160, 528, 272, 4, "tail"), (1040, 272, 400, 3, "even"), (2064, 144, 144, 5, "tail"),
    (272, 160, 1040, 70, "tail"), (512, 400, 528, 6, "bad"), (4096, 272, 256, 2, "one"), (256, 1040, 656, 4, "tail"),
]


@pytest.mark.parametrize("M,N,K,G,kind", WG)
@pytest.mark.parametrize("out", ["bf16", "f32", "accumulate"])
@pytest.mark.parametrize("fast", [False, True])
def test_mm_wgrad(M, N, K, G, kind, out, fast):
    rng = np.random.default_rng(M * 17 + N + K)
    off = ends_of(kind, M, G, rng)
    if kind != "bad":
        off = off // 16 * 16
    ends = ref.clean_ends(off, M, 16)
    a, b = codes(rng, (N, M)), codes(rng, (K, M))
    a[:, ends[-1]:] = 0x7F
    b[:, ends[-1]:] = 0xFF
    sa, sb = scales(rng, (N, G)), scales(rng, (K, G))
    f32 = out != "bf16"
    dw = Guarded((G, N, K), torch.float32 if f32 else torch.bfloat16)
    before = np.zeros((G, N, K))
    if out == "accumulate":
        start = rng.standard_normal((G, N, K)).astype(np.float32)
        dw.view.copy_(to_dev(start))
        before = start.astype(np.float64)
    mgs.mgs_mm_wgrad(to_dev(a), to_dev(sa), to_dev(b), to_dev(sb), to_dev(off), OUT["f32" if f32 else "bf16"],
                     fast, dw=dw.view, accumulate=out == "accumulate")
    torch.cuda.synchronize()
    dw.check()
    want, mag = ref.mm_wgrad(a, sa, b, sb, ends)
    tol = ref.mm_tolerance(want, mag, M, "f32" if f32 else "bf16", fast)
    if out == "accumulate":
        want = want + before
        tol = tol + np.abs(want) * 2.0 ** -24 * 1.01
    check(dw.view.float().cpu().numpy(), want, tol, (M, N, K, G, kind))


def test_wgrad_groups_do_not_see_each_other():
    """Columns of another group that are not numbers, inside the same
    128-byte lines, do not reach a group's gradient."""
    rng = np.random.default_rng(6)
    M, N, K, G = 160, 32, 48, 3
    off = np.array([48, 112, 160], np.int32)
    a, b = codes(rng, (N, M)), codes(rng, (K, M))
    sa, sb = scales(rng, (N, G)), scales(rng, (K, G))
    clean = mgs.mgs_mm_wgrad(to_dev(a), to_dev(sa), to_dev(b), to_dev(sb), to_dev(off)).cpu().numpy()
    a[:, 48:112], b[:, 48:112] = 0x7F, 0x7F
    got = mgs.mgs_mm_wgrad(to_dev(a), to_dev(sa), to_dev(b), to_dev(sb), to_dev(off)).cpu().numpy()
    assert np.array_equal(got[[0, 2]], clean[[0, 2]]) and np.isnan(got[1]).all()


def test_repeats_are_identical():
    rng = np.random.default_rng(10)
    M, N, K, G = 640, 400, 1168, 5
    off = to_dev(ends_of("even", M, G, rng) // 16 * 16)
    a, b, sa, sb = (to_dev(v) for v in (codes(rng, (M, K)), codes(rng, (G, N, K)), scales(rng, (M, 10)),
                                        scales(rng, (G, 4, 10))))
    at, bt, sat, sbt = (to_dev(v) for v in (codes(rng, (N, M)), codes(rng, (K, M)), scales(rng, (N, G)),
                                            scales(rng, (K, G))))
    ys = [mgs.mgs_mm_block128(a, sa, b, sb, off, torch.float32) for _ in range(3)]
    ds = [mgs.mgs_mm_wgrad(at, sat, bt, sbt, off) for _ in range(3)]
    assert all(torch.equal(ys[0], y) for y in ys) and all(torch.equal(ds[0], d) for d in ds)


def test_float8_tensors_and_refusals_in_python():
    rng = np.random.default_rng(2)
    a, b = to_dev(codes(rng, (32, 64))), to_dev(codes(rng, (2, 16, 64)))
    sa, sb, off = torch.ones((32, 1), device=dev()), torch.ones((2, 1, 1), device=dev()), to_dev(np.array([16, 32], np.int32))
    f8 = torch.float8_e4m3fn
    assert torch.equal(mgs.mgs_mm_block128(a, sa, b, sb, off), mgs.mgs_mm_block128(a.view(f8), sa, b.view(f8), sb, off))
    for bad in (lambda: mgs.mgs_mm_block128(a, sa[:16], b, sb, off), lambda: mgs.mgs_mm_block128(a, sa, b, sb, off[:1]),
                lambda: mgs.mgs_mm_block128(a[:, ::2], sa, b, sb, off), lambda: mgs.mgs_mm_block128(a, sa, b, sb.cpu(), off)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        mgs.mgs_mm_block128(a, sa, b, sb, off, torch.float16)
    with pytest.raises(mgs.MgsError):
        mgs.mgs_mm_block128(a, sa, b, sb)           # two weights, no groups
    with pytest.raises(mgs.MgsError):
        mgs.mgs_mm_wgrad(a, torch.ones((32, 1), device=dev()), a, torch.ones((32, 1), device=dev()),
                         to_dev(np.array([64], np.int32)), accumulate=True)


def test_past_two_to_the_31_elements():
    """Outputs and weights of more than 2^31 elements."""
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GiB")
    rng = np.random.default_rng(3)
    M, N, K = 70000, 32768, 144
    a, b = codes(rng, (M, K)), codes(rng, (1, N, K))
    sa, sb = scales(rng, (M, 2)), scales(rng, (1, N // 128, 2))
    y = mgs.mgs_mm_block128(to_dev(a), to_dev(sa), to_dev(b), to_dev(sb))
    assert y.numel() > 1 << 31
    at = [0, 65535, 65536, 69999]
    want, mag = ref.mm_block128(a[at], sa[at], b, sb, [len(at)])
    check(y[at].float().cpu().numpy(), want, ref.mm_tolerance(want, mag, K, "bf16"), "y")
    del y
    G, N, K = 9, 16384, 16400
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    w = torch.randint(0, 127, (G, N, K), generator=gen, device="cuda", dtype=torch.uint8)
    a, sa = codes(rng, (18, K)), scales(rng, (18, 129))
    sb = scales(rng, (G, 128, 129))
    off = np.arange(2, 20, 2).astype(np.int32)
    y = mgs.mgs_mm_block128(to_dev(a), to_dev(sa), w, to_dev(sb), to_dev(off))
    cols = np.r_[0:16, N - 16:N]
    want, mag = ref.mm_block128(a[16:], sa[16:], w[8:][:, cols].cpu().numpy(), sb[8:][:, [0] + [127]][:, [0]], [2])
    want2, mag2 = ref.mm_block128(a[16:], sa[16:], w[8:][:, cols].cpu().numpy(), sb[8:][:, [127]], [2])
    want[:, 16:], mag[:, 16:] = want2[:, 16:], mag2[:, 16:]
    check(y[16:][:, cols].float().cpu().numpy(), want, ref.mm_tolerance(want, mag, K, "bf16"), "last weight")
    dw = mgs.mgs_mm_wgrad(to_dev(codes(rng, (N, 32))), torch.ones((N, G), device=dev()), to_dev(codes(rng, (K, 32))),
                          torch.ones((K, G), device=dev()), to_dev(np.array([0] * 8 + [32], np.int32)), torch.bfloat16)
    assert dw.numel() > 1 << 31 and (dw[:8, ::997, ::31] == 0).all() and (dw[8] != 0).any(1).all()


@pytest.mark.parametrize("M,N,K,G,kind", [
    (640, 400, 400, 1, "even"), (1120, 16, 16, 70, "tail"), (4112, 48, 32, 3, "bad"), (16, 16, 16, 1, "even"),
    (2048, 272, 272, 2, "one"), (336, 32, 48, 130, "tail"), (1296, 528, 496, 1, "tail")])
@pytest.mark.parametrize("out", ["bf16", "f32", "accumulate"])
@pytest.mark.parametrize("fast", [False, True])
def test_mm_wgrad_of_few_outputs(M, N, K, G, kind, out, fast):
    """Weights so small that each workgroup takes a group's whole contraction."""
    test_mm_wgrad(M, N, K, G, kind, out, fast)
