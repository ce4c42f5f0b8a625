// mgs_block128.hip — casts with one scale per block of 128 (gfx950).
//
// The framework's cast, s = fl32(448 / max(amax, 1e-12)) and
// q = E4M3(fl32(x * s)), over blocks that the block-128 product reads:
// 1 x 128 for activations and gradients, 128 x 128 for weights. One pass: a
// block's values stay in registers between its maximum and its cast, so both
// kernels are bound by memory traffic. Times are of single launches on MI355X.
#include "mgs_block128_device.hpp"
#include "mgs_experts.hpp"

namespace mgs {

namespace {

// A wave casts 512 columns of one row: 16 lanes hold one block of 128. 16640 x
// 8192, 0.41 GB: 70 us, 5.9 TB/s.
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
// rows t / 16 + 16 j. The transposed order goes through LDS: both orders cost one
// read of w. 16 x 8192 x 5120, 2.68 GB with both orders: 500 us, 5.4 TB/s.
__global__ __launch_bounds__(256) void blocks128_kernel(const uint16_t* __restrict__ w, int64_t N, int64_t K,
                                                        int pow2, uint8_t* __restrict__ q, float* __restrict__ scales,
                                                        uint8_t* __restrict__ q_t, float* __restrict__ scales_t) {
    __shared__ uint32_t s_max[4];
    __shared__ uint8_t s_t[128][128 + 4];
    const int64_t nbk = (K + 127) / 128, nbn = (N + 127) / 128;
    const int64_t bk = blockIdx.x % nbk, rest = blockIdx.x / nbk, bn = rest % nbn, e = rest / nbn;
    const int cv = threadIdx.x & 15, r0 = threadIdx.x / 16;
    const int64_t col = bk * 128 + cv * 8, row0 = bn * 128;
    const uint16_t* we = w + e * N * K;
    uint4 v[8];
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int64_t r = row0 + r0 + 16 * j;
        v[j] = make_uint4(0, 0, 0, 0);
        if (r < N && col < K) v[j] = load_stream(we + r * K + col);
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
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int r = r0 + 16 * j;
        const uint2 c = cast8_group(v[j], s);
        if (row0 + r < N && col < K) *reinterpret_cast<uint2*>(q + (e * N + row0 + r) * K + col) = c;
        if (q_t) {
#pragma unroll
            for (int i = 0; i < 8; ++i) s_t[cv * 8 + i][r] = (uint8_t)((i < 4 ? c.x : c.y) >> (8 * (i & 3)));
        }
    }
    if (!q_t) return;
    __syncthreads();
    for (int i = threadIdx.x; i < 128 * 16; i += 256) {
        const int c = i / 16, r = (i & 15) * 8;
        if (bk * 128 + c >= K || row0 + r >= N) continue;
        uint2 o;
        o.x = *reinterpret_cast<const uint32_t*>(&s_t[c][r]);
        o.y = *reinterpret_cast<const uint32_t*>(&s_t[c][r + 4]);
        *reinterpret_cast<uint2*>(q_t + (e * K + bk * 128 + c) * N + row0 + r) = o;
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
    hipLaunchKernelGGL(blocks128_kernel, dim3((unsigned)blocks), dim3(256), 0, stream, w, N, K, pow2 ? 1 : 0, q,
                       scales, q_t, scales_t);
    return hipGetLastError();
}

}  // namespace mgs
