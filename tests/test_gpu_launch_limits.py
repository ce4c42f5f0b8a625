"""Sizes that the expert calls accept and whose work passes what one
dimension of a launch, or 32 bits, can count."""
import numpy as np
import pytest
import torch

import experts_ref as ref
import group_scaling_fp8_amd as mgs
from gpu_util import dev, to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GiB")
    mgs.lib()


def whole(gen, shape, most=8):
    """Whole numbers as bf16."""
    return torch.randint(-most, most + 1, shape, generator=gen, device="cuda", dtype=torch.int8).to(torch.bfloat16)


def generator(seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return gen


def test_weight_cast_of_more_than_2_to_the_24_matrices():
    """A workgroup of 256 threads for each: more than 2^32 threads."""
    E = (1 << 24) + 5
    w = whole(generator(1), (E, 16, 16))
    q, s, q_t, s_t = mgs.mgs_quant_blocks128(w)
    assert torch.equal(s, s_t)
    for lo in (0, E // 2, E - 4096):
        v = w[lo:lo + 4096].float()
        amax = v.abs().amax((1, 2), keepdim=True)
        want = torch.full_like(amax, 448) / amax
        assert torch.equal(s[lo:lo + 4096], want)
        assert torch.equal(q[lo:lo + 4096], (v * want).to(torch.float8_e4m3fn).view(torch.uint8))
        assert torch.equal(q_t[lo:lo + 4096], q[lo:lo + 4096].transpose(1, 2))
    # amax is a whole number from 1 to 8 (256 values: never 0 here), so s holds one of eight values
    values = torch.full((8,), 448.0, device="cuda") / torch.arange(1, 9, device="cuda")
    assert bool(torch.isin(s.view(-1), values).all())


def test_few_rows_of_more_tiles_than_2_to_the_23():
    """A workgroup of 512 threads for each: more than 2^32 threads."""
    G, M, N, K = 1024, 20480, 120000, 16
    rng = np.random.default_rng(2)
    a = rng.integers(0x30, 0x48, (M, K)).astype(np.uint8)
    b = torch.randint(0x30, 0x48, (G, N, K), generator=generator(2), device="cuda", dtype=torch.uint8)
    sa = np.exp2(rng.integers(-3, 4, (M, 1))).astype(np.float32)
    sb = np.exp2(rng.integers(-3, 4, (G, -(-N // 128), 1))).astype(np.float32)
    ends = np.arange(20, M + 1, 20).astype(np.int32)
    y = mgs.mgs_mm_block128(to_dev(a), to_dev(sa), b, to_dev(sb), to_dev(ends))
    for first in (0, 59904, N - 64):      # starts of blocks of 128 columns
        cols = slice(first, min(first + 128, N))
        part = np.ascontiguousarray(sb[:, first // 128:first // 128 + 1])
        want, mag = ref.mm_block128(a, sa, b[:, cols].cpu().numpy(), part, ends)
        err = np.abs(y[:, cols].double().cpu().numpy() - want)
        assert (err <= ref.mm_tolerance(want, mag, K, "bf16")).all(), first


def test_combine_of_wide_rows():
    """More than 65536 runs of 2048 columns."""
    D = (1 << 27) + 2056
    yp = whole(generator(3), (3, D))
    rows, slots = to_dev(np.array([[2], [0]], np.int32)), to_dev(np.array([1, -1, 0], np.int32))
    w = torch.full((2, 1), 2.0, device=dev())
    y = mgs.mgs_moe_combine(yp, rows, w)
    assert torch.equal(y[0], 2 * yp[2]) and torch.equal(y[1], 2 * yp[0])
    dyp, dw = mgs.mgs_moe_combine_grad(y, yp, rows, slots, w)
    assert torch.equal(dyp[2], 4 * yp[2]) and torch.equal(dyp[0], 4 * yp[0]) and not bool(dyp[1].any())


def test_dispatch_of_wide_rows():
    """More than 65536 pieces of 1024 columns."""
    D = (1 << 26) + 1032
    x = whole(generator(4), (1, D))
    off, rows, slots, q, s, xp = mgs.mgs_moe_dispatch(x, torch.zeros((1, 1), dtype=torch.int32, device="cuda"), 1,
                                                      permuted=True)
    assert off.tolist() == [16] and rows.tolist() == [[0]] and slots.tolist() == [0] + [-1] * 15
    want_q, want_s = mgs.mgs_quant_rows128(x)
    assert torch.equal(xp[:1], x) and torch.equal(q[:1], want_q) and torch.equal(s[:1], want_s)
    assert not bool(xp[1:].any()) and not bool(q[1:].any())


@pytest.mark.parametrize("T", [3, 40000])
def test_order_into_nearly_2_to_the_31_rows(T):
    """The C call with as many rows as it takes, by one launch and ranked: every
    row past the groups is marked as empty."""
    k, E, align, P = 1, 1024, 4096, (1 << 31) - 1
    rng = np.random.default_rng(T)
    ids = rng.integers(0, E, (T, k)).astype(np.int32)
    ids_d, slots = to_dev(ids), torch.zeros((P,), dtype=torch.int32, device="cuda")
    off, rows = torch.empty((E,), dtype=torch.int32, device="cuda"), torch.empty((T, k), dtype=torch.int32, device="cuda")
    ws = torch.empty((256 * E,), dtype=torch.uint8, device="cuda")
    st = mgs.lib().mgs_moe_dispatch(None, T, 0, ids_d.data_ptr(), k, E, align, 0, P, off.data_ptr(), rows.data_ptr(),
                                    slots.data_ptr(), None, None, None, ws.data_ptr(), ws.numel(), None)
    assert st == mgs.MGS_OK
    r_off, r_rows, r_slots = ref.order(ids, E, align)
    assert np.array_equal(off.cpu().numpy(), r_off) and np.array_equal(rows.cpu().numpy(), r_rows)
    assert np.array_equal(slots[:len(r_slots)].cpu().numpy(), r_slots)
    assert all(bool((part == -1).all()) for part in slots[len(r_slots):].split(1 << 28))
