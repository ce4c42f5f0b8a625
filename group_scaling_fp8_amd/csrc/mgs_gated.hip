// mgs_gated.hip — the gated feed-forward layer on E4M3 operands (gfx950).
//
// Forward, for rows m of group e with its two weights (matrices 2 e and 2 e + 1):
//   g = sum_b 1 / (sa[m, b] sb[2 e, n / 128, b])     * sum_{k in b} a[m, k] b[2 e, n, k]
//   u = the same with matrix 2 e + 1
//   h = act(g) u,   act(g) = g sigmoid(t(g))
// and backward, from the output's gradient dy and the down weight:
//   dh = sum_b 1 / (sa[m, b] sb[e, n / 128, b]) * sum_{k in b} dy[m, k] b[e, n, k]
//   du = dh act(g),   dg = dh u act'(g)
// One launch each: both projections of a column are sums of the same lane, so
// the activation is applied to binary32 values in registers and neither
// projections nor dh make a way through memory.
//
// Measured (us, MI355X; 16640 rows in 16 ragged groups, 2 x 8192 x 5120): forward
// with the projections kept 1600, of which the products alone are about 1430 at
// block128's dense rate of 2190 TFLOP/s, their tiles' rows past a group's end counted;
// the rest is 0.8 GB of output, which the next tile's first two steps do not cover
// (left out: 1520 of 1720 at the time). The activation itself is 1%. Backward with
// the hidden rows 980: products 714, reading the projections 62, output 115, and the
// arithmetic of the gradients. Dense sizes: 2155 TFLOP/s without the projections
// kept, 2055 with them, backward 1921; with binary32 sums 1082, 1048 and 1002, where
// the widening's instructions bound it. Four tokens to 2 of 16 experts take 116, the
// used experts' weights at 4.7 TB/s.
#include "mgs_experts.hpp"
#include "mgs_kernels.hpp"
#include "mgs_mm_tile.hpp"

namespace mgs {

namespace {

template <Job JOB, bool MORE>
hipError_t launch_summed(const MmArgs& p, bool fast, int cus, hipStream_t stream) {
    return fast ? launch_sized<Kind<JOB, Num::Fast, false, MORE>>(p, cus, stream)
                : launch_sized<Kind<JOB, Num::Exact, false, MORE>>(p, cus, stream);
}

}  // namespace

hipError_t launch_mm_gated(const uint8_t* a, const float* a_scales, int64_t M, int64_t K, const uint8_t* b,
                           const float* b_scales, int64_t E, int64_t F, const int32_t* offsets, int act, bool fast,
                           void* h, void* gu, int cus, hipStream_t stream) {
    if (K == 0) {
        const hipError_t e = gu ? launch_zero(gu, (size_t)M * F * 4, stream) : hipSuccess;
        return e != hipSuccess ? e : launch_zero(h, (size_t)M * F * 2, stream);
    }
    const MmArgs p{a, a_scales, b, b_scales, offsets, M, F, K, F, (int)E, 0, h, nullptr, gu, activation(act)};
    return gu ? launch_summed<Job::Gated, true>(p, fast, cus, stream)
              : launch_summed<Job::Gated, false>(p, fast, cus, stream);
}

hipError_t launch_mm_gated_grad(const uint8_t* dy, const float* dy_scales, int64_t M, int64_t D, const uint8_t* b,
                                const float* b_scales, int64_t E, int64_t F, const int32_t* offsets, int act,
                                bool fast, const uint16_t* gu, void* dgu, void* h, int cus, hipStream_t stream) {
    const MmArgs p{dy, dy_scales, b, b_scales, offsets, M, F, D, F, (int)E, 0, dgu, gu, h, activation(act)};
    return h ? launch_summed<Job::Grad, true>(p, fast, cus, stream)
             : launch_summed<Job::Grad, false>(p, fast, cus, stream);
}

}  // namespace mgs
