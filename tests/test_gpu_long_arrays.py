"""Arrays whose casts need 2^32 threads or more: one launch cannot hold them."""
import pytest
import torch

import group_scaling_fp8_amd as mgs

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _memory():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mgs.lib()
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


def need(gib):
    if torch.cuda.mem_get_info()[0] < gib << 30:
        pytest.skip("needs %d GiB" % gib)


def test_cast():
    need(90)
    n = (1 << 34) + 1028           # four values a thread
    x = torch.ones((n,), device="cuda")
    at = [0, 1023, (1 << 33) - 1, 1 << 33, (1 << 34) - 1, 1 << 34, n - 1]
    x[at] = -2.0
    out = torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda")
    mgs.mgs_cast_e4m3(x, out)
    assert (out[at] == 0xC0).all()
    out[at] = 0x38
    assert all(bool((part == 0x38).all()) for part in out.split(1 << 31))


def test_mx():
    need(215)
    mode = mgs.MGS_MX_RCEIL
    M, K = (1 << 21) + 3, 1 << 15  # 16 values a thread
    x = torch.empty((M, K), dtype=torch.bfloat16, device="cuda")
    x.fill_(1.0)
    small = torch.ones((1, 32), dtype=torch.bfloat16, device="cuda")
    small_q, small_s = mgs.mgs_mx_quant_dim0(small, mode)
    want_q, want_s = int(small_q[0, 0]), int(small_s[0, 0])
    small[0, :4] = torch.tensor([-6.0, 0.3, 5.0, 0.0], dtype=torch.bfloat16)
    small_q, small_s = mgs.mgs_mx_quant_dim0(small, mode)
    at = [(0, 0), (1 << 20, 0), ((1 << 21) - 1, K - 32), (1 << 21, 0), (M - 1, K - 32)]
    for r, c in at:
        x[r, c:c + 32] = small[0]
    q = torch.full((M, K), 0xA5, dtype=torch.uint8, device="cuda")
    s = torch.full((M, K // 32), 0xA5, dtype=torch.uint8, device="cuda")
    mgs.mgs_mx_quant_dim0(x, mode, q=q, scales=s)
    for r, c in at:
        assert torch.equal(q[r, c:c + 32], small_q[0]) and int(s[r, c // 32]) == int(small_s[0, 0]), (r, c)
        q[r, c:c + 32], s[r, c // 32] = want_q, want_s
    assert all(bool((part == want_q).all()) for part in q.view(-1).split(1 << 31))
    assert all(bool((part == want_s).all()) for part in s.view(-1).split(1 << 31))
