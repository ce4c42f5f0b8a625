"""Groups without rows in every form of the products: zeros (or what dw
held), whatever the bytes and scales that belong to them are."""
import numpy as np
import pytest
import torch

import experts_ref as ref
import group_scaling_fp8_amd as mgs
from gpu_util import Guarded, to_dev
from test_gpu_mm import OUT, check, codes, scales

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mgs.lib()


# few rows a tile, two sets of waves, 128 x 128, 256 x 256
@pytest.mark.parametrize("M,N,K,G", [(96, 48, 32, 3), (96, 400, 528, 3), (96, 1040, 1168, 3), (96, 2064, 2064, 16)])
@pytest.mark.parametrize("out", ["bf16", "f32", "accumulate"])
@pytest.mark.parametrize("fast", [False, True])
def test_wgrad(M, N, K, G, out, fast):
    rng = np.random.default_rng(N + K)
    off = np.full(G, M, np.int32)
    off[0] = 0                     # the second group has all rows
    a, b, sa, sb = codes(rng, (N, M)), codes(rng, (K, M)), scales(rng, (N, G)), scales(rng, (K, G))
    sa[:, 0], sb[:, 0] = np.nan, 1.0
    sa[:, 2:], sb[:, 2:] = 0.0, np.inf
    f32 = out != "bf16"
    dw = Guarded((G, N, K), OUT["f32" if f32 else "bf16"])
    before = np.full((N, K), 3.0 if out == "accumulate" else 0.0)
    dw.view.fill_(3.0)
    mgs.mgs_mm_wgrad(to_dev(a), to_dev(sa), to_dev(b), to_dev(sb), to_dev(off), OUT["f32" if f32 else "bf16"], fast,
                     dw=dw.view, accumulate=out == "accumulate")
    torch.cuda.synchronize()
    dw.check()
    got = dw.view.float().cpu().numpy()
    assert (got[0] == before).all() and (got[2:] == before).all()
    want, mag = ref.mm_wgrad(a, sa[:, 1:2], b, sb[:, 1:2], [M])
    tol = ref.mm_tolerance(want, mag, M, "f32" if f32 else "bf16", fast)
    if out == "accumulate":
        want = want + before
        tol = tol + np.abs(want) * 2.0 ** -24 * 1.01
    check(got[1], want[0], tol[0], (N, K))


@pytest.mark.parametrize("M,N,K,G", [(40, 48, 272, 3), (400, 272, 272, 3), (4000, 1936, 272, 3), (8200, 4240, 272, 3)])
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("fast", [False, True])
def test_block128(M, N, K, G, out, fast):
    """An expert without rows, and rows without an expert."""
    rng = np.random.default_rng(N + K)
    last = M // 2
    off = np.array([0, last, last], np.int32)
    a, b = codes(rng, (M, K)), codes(rng, (G, N, K))
    sa, sb = scales(rng, (M, 3)), scales(rng, (G, -(-N // 128), 3))
    a[last:], b[0], b[2] = 0x7F, 0xFF, 0x7F
    sa[last:], sb[0], sb[2] = np.nan, 0.0, np.inf
    y = Guarded((M, N), OUT[out])
    mgs.mgs_mm_block128(to_dev(a), to_dev(sa), to_dev(b), to_dev(sb), to_dev(off), OUT[out], fast, y=y.view)
    torch.cuda.synchronize()
    y.check()
    got = y.view.float().cpu().numpy()
    assert (got[last:] == 0).all()
    want, mag = ref.mm_block128(a[:last], sa[:last], b[1:2], sb[1:2], [last])
    check(got[:last], want, ref.mm_tolerance(want, mag, K, out, fast), (M, N))
