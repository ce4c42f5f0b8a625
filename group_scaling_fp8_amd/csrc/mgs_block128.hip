// mgs_block128.hip — casts with one scale per block of 128 (gfx950).
//
// The framework's cast, s = fl32(448 / max(amax, 1e-12)) and
// q = E4M3(fl32(x * s)), over blocks that the block-128 product reads:
// 1 x 128 for activations and gradients, 128 x 128 for weights. One pass: a
// block's values stay in registers between its maximum and its cast, so both
// kernels are bound by memory traffic. Times are of launches back to back on
// MI355X.
#include "mgs_block128_device.hpp"
#include "mgs_experts.hpp"

namespace mgs {

namespace {

// A wave casts 512 columns of one row: 16 lanes hold one block of 128. 16640 x
// 8192, 0.41 GB: 70 us, 5.9 TB/s (streaming stores: 74).
__global__ __launch_bounds__(256) void rows128_kernel(const uint16_t* __restrict__ x, int64_t M, int64_t K,
                                                      int units, int pow2, uint8_t* __restrict__ q,
                                                      float* __restrict__ scales) {
    const int lane = threadIdx.x & (kWave - 1);
    const int64_t nb = (K + 127) / 128, total = M * units;
    for (int64_t it = (int64_t)blockIdx.x * 4 + threadIdx.x / kWave; it < total; it += (int64_t)gridDim.x * 4) {
        const int64_t r = it / units, col = (it - r * units) * 512 + lane * 8;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (col < K) v = load_stream(x + r * K + col);
        const float s = group_scale(row16_max(mag_fold(mag_max8(0u, v))), pow2 != 0);
        if (col < K) {
            *reinterpret_cast<uint2*>(q + r * K + col) = cast8_group(v, s);
            if ((lane & 15) == 0) scales[r * nb + col / 128] = s;
        }
    }
}

// One block of 128 x 128 a workgroup: thread t holds 8 columns (t & 15) of the
// rows 4 (t / 16) + j and 64 + 4 (t / 16) + j, j < 4, so that loads and stores of a
// row are whole lines. The transposed order goes through LDS, four rows of a
// column at a time: both orders cost one read of w. Streaming stores: the
// outputs are larger than the caches. 16 x 8192 x 5120, 2.68 GB with both orders:
// 530 us back to back, 5.1 TB/s (plain stores of q: 557).
__global__ __launch_bounds__(256) void blocks128_kernel(const uint16_t* __restrict__ w, int64_t E, int64_t N,
                                                        int64_t K, int pow2, uint8_t* __restrict__ q,
                                                        float* __restrict__ scales, uint8_t* __restrict__ q_t,
                                                        float* __restrict__ scales_t) {
    __shared__ uint32_t s_max[4];
    __shared__ uint32_t s_t[128][32 + 1];
    const int64_t nbk = (K + 127) / 128, nbn = (N + 127) / 128;
    const uint32_t block = (uint32_t)workgroup_xz();        // the host has checked that 31 bits hold E nbn nbk
    const int64_t bk = block % nbk, rest = block / nbk, bn = rest % nbn, e = rest / nbn;
    if (e >= E) return;
    const int cv = threadIdx.x & 15, rq = threadIdx.x / 16;
    const int64_t col = bk * 128 + cv * 8, row0 = bn * 128;
    auto row_of = [&](int j) { return row0 + rq * 4 + (j & 3) + (j >> 2) * 64; };
    const uint16_t* we = w + e * N * K;
    uint4 v[8];
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        v[j] = make_uint4(0, 0, 0, 0);
        if (row_of(j) < N && col < K) v[j] = load_stream(we + row_of(j) * K + col);
        m = mag_max8(m, v[j]);
    }
    m = mag_fold(m);
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d, kWave));
    if ((threadIdx.x & (kWave - 1)) == 0) s_max[threadIdx.x / kWave] = m;
    __syncthreads();
    m = max(max(s_max[0], s_max[1]), max(s_max[2], s_max[3]));
    const float s = group_scale(m, pow2 != 0);
    if (threadIdx.x == 0) {
        scales[(e * nbn + bn) * nbk + bk] = s;
        if (scales_t) scales_t[(e * nbk + bk) * nbn + bn] = s;
    }
    uint2 c[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        c[j] = cast8_group(v[j], s);
        if (row_of(j) < N && col < K) store_stream(q + (e * N + row_of(j)) * K + col, c[j]);
    }
    if (!q_t) return;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t lo[4], hi[4];
        transpose4x4(c[4 * h].x, c[4 * h + 1].x, c[4 * h + 2].x, c[4 * h + 3].x, lo);
        transpose4x4(c[4 * h].y, c[4 * h + 1].y, c[4 * h + 2].y, c[4 * h + 3].y, hi);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            s_t[cv * 8 + i][h * 16 + rq] = lo[i];
            s_t[cv * 8 + 4 + i][h * 16 + rq] = hi[i];
        }
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int i = j * 256 + threadIdx.x, k = i / 8, r = (i & 7) * 16;
        if (bk * 128 + k >= K || row0 + r >= N) continue;
        const uint32_t* t = &s_t[k][r / 4];
        store_stream16(q_t + (e * K + bk * 128 + k) * N + row0 + r, make_uint4(t[0], t[1], t[2], t[3]));
    }
}

}  // namespace

hipError_t launch_rows128(const uint16_t* x, int64_t M, int64_t K, bool pow2, uint8_t* q, float* scales,
                          hipStream_t stream) {
    const int units = (int)((K + 511) / 512);
    const int64_t want = (M * units + 3) / 4, blocks = want < (1 << 20) ? want : (1 << 20);
    hipLaunchKernelGGL(rows128_kernel, dim3((unsigned)blocks), dim3(256), 0, stream, x, M, K, units, pow2 ? 1 : 0, q,
                       scales);
    return hipGetLastError();
}

hipError_t launch_blocks128(const uint16_t* w, int64_t E, int64_t N, int64_t K, bool pow2, uint8_t* q,
                            float* scales, uint8_t* q_t, float* scales_t, hipStream_t stream) {
    const int64_t blocks = E * ((N + 127) / 128) * ((K + 127) / 128);
    hipLaunchKernelGGL(blocks128_kernel, grid_xz(blocks), dim3(256), 0, stream, w, E, N, K, pow2 ? 1 : 0, q, scales,
                       q_t, scales_t);
    return hipGetLastError();
}

}  // namespace mgs
