// mgs_mm.hip — products of E4M3 matrices with fp32 scales on the matrix cores
// (gfx950).
//
// Both products contract the contiguous dim of two row-major operands:
//   block128:  y[m, n] = sum_b 1 / (sa[m, b] sb[e, n / 128, b])
//                        * sum_{k in block b} a[m, k] b[e, n, k]
//   wgrad:     dw[g][n, k] = 1 / (sa[n, g] sb[k, g]) * sum_{m in g} a_t[n, m] b_t[k, m]
// block128 sums every block of 128 from zero and adds the scaled partial sum to
// its fp32 accumulators; wgrad accumulates in place and scales once at the end.
//
// Two forms of the inner sums:
//   exact  the bytes become bf16 (every E4M3 value is one) and go through the
//          16 x 16 x 32 bf16 instruction, whose sums are binary32.
//   fast   one 16 x 16 x 128 instruction on the bytes themselves, at twice the
//          rate. It aligns the products of each eight consecutive k to the
//          largest of the eight and drops what lies below 2^-13 of it (measured
//          bit by bit on the card); the sums of the eights are binary32. The
//          loss is at most 2^-10 of the sum of the terms' magnitudes (where one
//          of eight is far larger than the rest) and about 5e-5 of a typical
//          sum, a thirtieth of a bf16 output's own rounding.
#include "mgs_experts.hpp"
#include "mgs_kernels.hpp"
#include "mgs_mm_tile.hpp"

namespace mgs {

namespace {

template <Job JOB>
hipError_t launch_typed(const MmArgs& p, bool fast, bool f32, int cus, hipStream_t stream) {
    if (fast)
        return f32 ? launch_sized<Kind<JOB, Num::Fast, true>>(p, cus, stream)
                   : launch_sized<Kind<JOB, Num::Fast, false>>(p, cus, stream);
    return f32 ? launch_sized<Kind<JOB, Num::Exact, true>>(p, cus, stream)
               : launch_sized<Kind<JOB, Num::Exact, false>>(p, cus, stream);
}

}  // namespace

hipError_t launch_mm_block128(const uint8_t* a, const float* a_scales, int64_t M, int64_t K, const uint8_t* b,
                              const float* b_scales, int64_t E, int64_t N, const int32_t* offsets, bool fast,
                              bool f32, void* y, int cus, hipStream_t stream) {
    if (K == 0) return launch_zero(y, (size_t)M * N * (f32 ? 4 : 2), stream);
    const MmArgs p{a, a_scales, b, b_scales, offsets, M, N, K, N, (int)E, 0, y};
    return launch_typed<Job::Rows>(p, fast, f32, cus, stream);
}

hipError_t launch_mm_wgrad(const uint8_t* a_t, const float* a_scales_t, const uint8_t* b_t,
                           const float* b_scales_t, int64_t M, int64_t N, int64_t K, const int32_t* offsets,
                           int64_t G, bool fast, bool f32, bool accumulate, void* dw, int cus, hipStream_t stream) {
    const MmArgs p{a_t, a_scales_t, b_t, b_scales_t, offsets, M, N, K, K, (int)G, accumulate ? 1 : 0, dw};
    return launch_typed<Job::Wgrad>(p, fast, f32, cus, stream);
}

}  // namespace mgs
