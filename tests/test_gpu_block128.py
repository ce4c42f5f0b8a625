"""The casts with one scale per block of 128, byte for byte against the
oracle's cast."""
import numpy as np
import pytest
import torch

import experts_ref as ref
import group_scaling_fp8_amd as mgs
from group_scaling_fp8_amd import workloads as wl
from gpu_util import Guarded, assert_same_bytes, to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mgs.lib()


def values(rng, shape):
    x = wl.randn_bf16(rng, shape, 0.02, 0.001, 8.0)
    flat = x.reshape(-1)
    if flat.size > 64:
        # signed zeros, subnormals and the largest magnitudes
        at = rng.choice(flat.size, size=min(40, flat.size // 4), replace=False)
        flat[at] = rng.choice(np.array([0, 0x8000, 1, 0x8001, 0x7F, 0x7F7F, 0xFF7F], np.uint16), size=len(at))
    return x


@pytest.mark.parametrize("M,K", [(1, 8), (1, 128), (3, 120), (16, 136), (129, 520), (77, 4112), (1000, 1024)])
@pytest.mark.parametrize("pow2", [False, True])
def test_rows128(M, K, pow2):
    rng = np.random.default_rng(M + K)
    x = values(rng, (M, K))
    q, s = Guarded((M, K), torch.uint8), Guarded((M, -(-K // 128)), torch.float32)
    mgs.mgs_quant_rows128(to_dev(x), pow2, q=q.view, scales=s.view)
    torch.cuda.synchronize()
    q.check()
    s.check()
    r_q, r_s = ref.rows128(x, pow2)
    assert_same_bytes(q.numpy(), r_q, "q")
    assert_same_bytes(s.numpy(), r_s, "scales")


def test_rows128_is_the_rowwise_cast_with_those_groups():
    rng = np.random.default_rng(9)
    x = to_dev(values(rng, (65, 1040)))
    q, s = mgs.mgs_quant_rows128(x)
    q1, s1 = mgs.mgs_quant_groups_dim1(x, to_dev(ref.block_ends(1040)))
    assert torch.equal(q, q1) and torch.equal(s.view(torch.int32), s1.view(torch.int32))


@pytest.mark.parametrize("E,N,K", [(1, 16, 16), (2, 128, 128), (3, 144, 112), (1, 400, 656), (2, 256, 512),
                                   (5, 16, 1040), (2, 1040, 48)])
@pytest.mark.parametrize("pow2", [False, True])
def test_blocks128(E, N, K, pow2):
    rng = np.random.default_rng(N + K)
    w = values(rng, (E, N, K))
    w[0, :128, :128] = 0
    nb, kb = -(-N // 128), -(-K // 128)
    shapes = (((E, N, K), torch.uint8), ((E, nb, kb), torch.float32), ((E, K, N), torch.uint8),
              ((E, kb, nb), torch.float32))
    out = [Guarded(*s) for s in shapes]
    w_d = to_dev(w)
    st = mgs.lib().mgs_quant_blocks128(w_d.data_ptr(), E, N, K, int(pow2), *[o.view.data_ptr() for o in out], None)
    assert st == mgs.MGS_OK
    torch.cuda.synchronize()
    for o in out:
        o.check()
    r_q, r_s = ref.blocks128(w, pow2)
    assert_same_bytes(out[0].numpy(), r_q, "q")
    assert_same_bytes(out[1].numpy(), r_s, "scales")
    assert_same_bytes(out[2].numpy(), np.ascontiguousarray(r_q.transpose(0, 2, 1)), "q_t")
    assert_same_bytes(out[3].numpy(), np.ascontiguousarray(r_s.transpose(0, 2, 1)), "scales_t")
    q, s = mgs.mgs_quant_blocks128(w_d, pow2, transposed=False)
    torch.cuda.synchronize()
    assert_same_bytes(q.cpu().numpy(), r_q, "q alone")
    assert_same_bytes(s.cpu().numpy(), r_s, "scales alone")


def test_past_two_to_the_31_elements():
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GiB")
    gen = torch.Generator(device="cuda")
    gen.manual_seed(2)
    w = torch.randn((9, 16384, 16400), generator=gen, device="cuda", dtype=torch.bfloat16)
    q, s, q_t, s_t = mgs.mgs_quant_blocks128(w)
    qr, sr = mgs.mgs_quant_rows128(w.view(-1, 16400))
    assert w.numel() > 1 << 31
    last = w[8, -128:, -16:].float().abs().amax()
    assert s[8, -1, -1] == (torch.full_like(last, 448) / last)
    got = q[8, -128:].view(torch.float8_e4m3fn).float() / s[8, -1].repeat_interleave(128)[:16400]
    # half a step of a normal E4M3 value, or of the subnormals' 2^-9
    tol = w[8, -128:].float().abs() * 2.0 ** -4 * 1.01 + 2.0 ** -10 / s[8, -1].repeat_interleave(128)[:16400]
    assert ((got - w[8, -128:].float()).abs() <= tol).all()
    assert torch.equal(q_t[8, -1], q[8, :, -1]) and torch.equal(s_t[8, -1], s[8, :, -1])
    row = w[8, -1, -16:].float()
    assert sr[-1, -1] == torch.full_like(row[0], 448) / row.abs().amax()
    assert torch.equal(qr[-1, -16:], (row * sr[-1, -1]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
