// mgs_block128_device.hpp — device helpers of the block-128 casts and the
// token-order kernels.
#pragma once

#include "mgs_device.hpp"

namespace mgs {

// A launch has fewer than 2^32 threads along x (with more, the count wraps and
// the rest of the grid does not run): more workgroups go on along z. The last
// run along x may pass the end.
__device__ __forceinline__ int64_t workgroup_xz() { return blockIdx.x + (int64_t)gridDim.x * blockIdx.z; }
inline dim3 grid_xz(int64_t blocks, unsigned y = 1) {
    constexpr int64_t kMaxX = 1 << 22;       // of at most 512 threads
    const int64_t x = blocks < kMaxX ? blocks : kMaxX;
    return dim3((unsigned)x, y, (unsigned)((blocks + x - 1) / x));
}

// Max over the 16 lanes of a DPP row, in every lane of it (rotations by 8, 4,
// 2 and 1): with 8 columns a lane, the maximum of a block of 128.
__device__ __forceinline__ uint32_t row16_max(uint32_t v) {
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x128, 0xF, 0xF, false));
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x124, 0xF, 0xF, false));
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x122, 0xF, 0xF, false));
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x121, 0xF, 0xF, false));
    return v;
}

// Two binary32 values as a bf16 pair, rounded to nearest even.
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    b2 r;
    r.x = (__bf16)lo;
    r.y = (__bf16)hi;
    return __builtin_bit_cast(uint32_t, r);
}

__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
    return make_uint4(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]), bf16x2(v[4], v[5]), bf16x2(v[6], v[7]));
}

// acc += w * (eight bf16)
__device__ __forceinline__ void add8(float (&acc)[8], uint4 v, float w) {
    acc[0] = fmaf(bf16_lo(v.x), w, acc[0]);
    acc[1] = fmaf(bf16_hi(v.x), w, acc[1]);
    acc[2] = fmaf(bf16_lo(v.y), w, acc[2]);
    acc[3] = fmaf(bf16_hi(v.y), w, acc[3]);
    acc[4] = fmaf(bf16_lo(v.z), w, acc[4]);
    acc[5] = fmaf(bf16_hi(v.z), w, acc[5]);
    acc[6] = fmaf(bf16_lo(v.w), w, acc[6]);
    acc[7] = fmaf(bf16_hi(v.w), w, acc[7]);
}

__device__ __forceinline__ float dot8(float acc, uint4 a, uint4 b) {
    acc = fmaf(bf16_lo(a.x), bf16_lo(b.x), acc);
    acc = fmaf(bf16_hi(a.x), bf16_hi(b.x), acc);
    acc = fmaf(bf16_lo(a.y), bf16_lo(b.y), acc);
    acc = fmaf(bf16_hi(a.y), bf16_hi(b.y), acc);
    acc = fmaf(bf16_lo(a.z), bf16_lo(b.z), acc);
    acc = fmaf(bf16_hi(a.z), bf16_hi(b.z), acc);
    acc = fmaf(bf16_lo(a.w), bf16_lo(b.w), acc);
    return fmaf(bf16_hi(a.w), bf16_hi(b.w), acc);
}

// Sum over the wave, in every lane, in a fixed order.
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int d = kWave / 2; d > 0; d >>= 1) v += __shfl_xor(v, d, kWave);
    return v;
}

}  // namespace mgs
