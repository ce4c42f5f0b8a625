"""CPU check of launches that would hold 2^32 threads or more: they are
refused before HIP is asked, since such a launch runs only a part of its
grid without an error."""
import os

import pytest

import group_scaling_fp8_amd as mgs

A = 1 << 20          # a fake, well-aligned "device" address; never dereferenced
HIP_INVALID_VALUE = 1


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(mgs.library_path()):
        from group_scaling_fp8_amd import build
        build.build()
    return mgs.lib()


@pytest.mark.parametrize("M,K", [(1 << 31, 8), (1 << 24, 16384), (1 << 40, 8)])
def test_mx_dim1(L, M, K):
    """512 rows by 128 columns and 1024 threads a tile: 2^22 tiles."""
    assert L.mgs_mx_quant_dim1(A, M, K, mgs.MGS_MX_FLOOR, A, A, None) == mgs.MGS_ERR_HIP
    assert L.mgs_last_hip_error() == HIP_INVALID_VALUE
