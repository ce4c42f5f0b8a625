// mgs_i8.hip — 8-bit integers with one scale for each row (gfx950): the cast, and
// the products of its bytes.
//
//   cast     s = fl32(127 / max(amax of the row, 1e-12)), q = rint(fl32(x * s))
//   product  y[m, n] = sum_k a[m, k] b[e, n, k] / (sa[m] sb[e, n])
//   gated    h = act(g) u of the products g and u with matrices 2 e and 2 e + 1
//
// Sums of products of bytes are exact: the matrix cores add them in 32-bit
// integers, which hold 131071 products of any two bytes. A sum is rounded to
// binary32 once and scaled once, so a result does not depend on the form, the
// tile or the order of its sum.
//
// The products are the tiles of mgs_mm_tile.hpp with sums in place: two 16 x 16 x 64
// instructions for a step's 128 bytes, scales once at the end. Dense products run at
// 2623 TOP/s (16384^3; the library's at 2391), the gated pair at 2586 (16384 x 2 x
// 8192 x 8192), bound by the matrix cores; in 16 ragged groups (16640 rows, 2 x 8192
// x 5120) 1335 us, of which the rows of tiles past a group's end are 12%. One row by
// 8192 x 8192 12.5 us, bound by the weights' bytes at 5.4 TB/s. Rows whose length is no
// multiple of 128 cross a line in every step: 4096 rows in 16 groups by 4096 x 4176
// take 164 us, by 4096 x 4096 126.
#include "mgs_experts.hpp"
#include "mgs_kernels.hpp"
#include "mgs_mm_tile.hpp"

namespace mgs {

namespace {

// |x s| <= 127 (1 + 2^-23) for a row's own scale. Adding 1.5 * 2^23 rounds
// fl32(x s) to the nearest integer, ties to even, and leaves it in the low byte.
__device__ __forceinline__ uint32_t i8x4(float a, float b, float c, float d, float s) {
#pragma clang fp contract(off)      // x s is rounded before it is rounded to an integer
    constexpr float kOne = 12582912.0f;
    const uint32_t x = __float_as_uint(a * s + kOne), y = __float_as_uint(b * s + kOne);
    const uint32_t z = __float_as_uint(c * s + kOne), w = __float_as_uint(d * s + kOne);
    return __builtin_amdgcn_perm(__builtin_amdgcn_perm(w, z, 0x0C0C0400u), __builtin_amdgcn_perm(y, x, 0x0C0C0400u),
                                 0x05040100u);
}

__device__ __forceinline__ uint2 i8x8(uint4 v, float s) {
    return make_uint2(i8x4(bf16_lo(v.x), bf16_hi(v.x), bf16_lo(v.y), bf16_hi(v.y), s),
                      i8x4(bf16_lo(v.z), bf16_hi(v.z), bf16_lo(v.w), bf16_hi(v.w), s));
}

// The maximum over the LANES threads that share a row, in each of them.
template <int LANES>
__device__ __forceinline__ uint32_t row_max(uint32_t m, uint32_t* s_max) {
    m = row16_max(m);
    if constexpr (LANES >= kWave) {
        m = max(m, (uint32_t)__shfl_xor((int)m, 16, kWave));
        m = max(m, (uint32_t)__shfl_xor((int)m, 32, kWave));
    }
    if constexpr (LANES > kWave) {
        __syncthreads();             // the last row's maxima are read
        if ((threadIdx.x & (kWave - 1)) == 0) s_max[threadIdx.x / kWave] = m;
        __syncthreads();
        m = s_max[0];
#pragma unroll
        for (int w = 1; w < LANES / kWave; ++w) m = max(m, s_max[w]);
    }
    return m;
}

// Threads of a workgroup where LANES of them cast a row.
template <int LANES>
constexpr int kThreads = LANES > 256 ? LANES : 256;

// LANES threads cast a row; up to LANES * V * 8 columns stay in registers between the
// maximum and the cast (HELD), longer rows are read again. Bound by memory: 16640 x
// 8192, 0.41 GB, 61 us, 6.7 TB/s.
template <int LANES, int V, bool HELD>
__global__ __launch_bounds__(kThreads<LANES>) void rows_i8_kernel(const uint16_t* __restrict__ x, int64_t M, int64_t K,
                                                      uint8_t* __restrict__ q, float* __restrict__ scales) {
    __shared__ uint32_t s_max[kThreads<LANES> / kWave];
    constexpr int ROWS = kThreads<LANES> / LANES;
    const int lane = threadIdx.x % LANES;
    for (int64_t r0 = (int64_t)blockIdx.x * ROWS; r0 < M; r0 += (int64_t)gridDim.x * ROWS) {
        const int64_t r = r0 + threadIdx.x / LANES;
        const bool mine = r < M;
        const uint16_t* xr = x + (mine ? r : 0) * K;
        uint4 v[V];
        uint32_t m = 0;
        for (int64_t c0 = 0;; c0 += LANES * V * 8) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int64_t c = c0 + (j * LANES + lane) * 8;
                v[j] = make_uint4(0, 0, 0, 0);
                if (mine && c < K) v[j] = HELD ? load_stream(xr + c) : *reinterpret_cast<const uint4*>(xr + c);
            }
#pragma unroll
            for (int j = 0; j < V; ++j) m = mag_max8(m, v[j]);
            if (HELD || c0 + LANES * V * 8 >= K) break;
        }
        // the largest magnitude as bits is a NaN's if the row holds one, and the scale then NaN
        const float amax = __uint_as_float(row_max<LANES>(mag_fold(m), s_max) << 16);
        const float s = 127.0f / (amax < 1e-12f ? 1e-12f : amax);
        if (mine && lane == 0) scales[r] = s;
        for (int64_t c0 = 0; c0 < K; c0 += LANES * V * 8) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int64_t c = c0 + (j * LANES + lane) * 8;
                if (!mine || c >= K) continue;
                if constexpr (!HELD) v[j] = *reinterpret_cast<const uint4*>(xr + c);
                *reinterpret_cast<uint2*>(q + r * K + c) = i8x8(v[j], s);
            }
            if (HELD) break;
        }
    }
}

template <int LANES, int V, bool HELD>
hipError_t launch_rows(const uint16_t* x, int64_t M, int64_t K, uint8_t* q, float* scales, hipStream_t stream) {
    constexpr int ROWS = kThreads<LANES> / LANES;
    const int64_t want = (M + ROWS - 1) / ROWS, blocks = want < (1 << 20) ? want : (1 << 20);
    hipLaunchKernelGGL((rows_i8_kernel<LANES, V, HELD>), dim3((unsigned)blocks), dim3(kThreads<LANES>), 0, stream, x, M,
                       K, q, scales);
    return hipGetLastError();
}

}  // namespace

// The fewest lanes whose registers hold a row (us of 136 M values, MI355X): rows of 512
// with 16 lanes 62, with 64 73; of 2048 with 64 61, with 256 73; of 2560 with 64 lanes of
// eight pieces 62, with 256 of four 67; of 32768 with 256 lanes 63, read twice 103; of
// 65536 with 1024 lanes 72, read twice 103.
hipError_t launch_rows_i8(const uint16_t* x, int64_t M, int64_t K, uint8_t* q, float* scales, hipStream_t stream) {
    if (K <= 512) return launch_rows<16, 4, true>(x, M, K, q, scales, stream);
    if (K <= 2048) return launch_rows<64, 4, true>(x, M, K, q, scales, stream);
    if (K <= 4096) return launch_rows<64, 8, true>(x, M, K, q, scales, stream);
    if (K <= 8192) return launch_rows<256, 4, true>(x, M, K, q, scales, stream);
    if (K <= 16384) return launch_rows<256, 8, true>(x, M, K, q, scales, stream);
    if (K <= 32768) return launch_rows<256, 16, true>(x, M, K, q, scales, stream);
    if (K <= 131072) return launch_rows<1024, 16, true>(x, M, K, q, scales, stream);      // every length a product takes
    return launch_rows<1024, 8, false>(x, M, K, q, scales, stream);
}

hipError_t launch_mm_i8(const uint8_t* a, const float* a_scales, int64_t M, int64_t K, const uint8_t* b,
                        const float* b_scales, int64_t E, int64_t N, const int32_t* offsets, bool f32, void* y,
                        int cus, hipStream_t stream) {
    if (K == 0) return launch_zero(y, (size_t)M * N * (f32 ? 4 : 2), stream);
    const MmArgs p{a, a_scales, b, b_scales, offsets, M, N, K, N, (int)E, 0, y, nullptr, nullptr, {}};
    return f32 ? launch_sized<Kind<Job::Rows, Num::Int8, true>>(p, cus, stream)
               : launch_sized<Kind<Job::Rows, Num::Int8, false>>(p, cus, stream);
}

hipError_t launch_mm_gated_i8(const uint8_t* a, const float* a_scales, int64_t M, int64_t K, const uint8_t* b,
                              const float* b_scales, int64_t E, int64_t F, const int32_t* offsets, int act, void* h,
                              int cus, hipStream_t stream) {
    if (K == 0) return launch_zero(h, (size_t)M * F * 2, stream);
    const MmArgs p{a, a_scales, b, b_scales, offsets, M, F, K, F, (int)E, 0, h, nullptr, nullptr, activation(act)};
    return launch_sized<Kind<Job::Gated, Num::Int8, false>>(p, cus, stream);
}

}  // namespace mgs
