// mgs_experts.hpp — host-side launchers of the mixture-of-experts kernels:
// token order, block-128 casts and the products (internal).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mgs {

// ---- token order (mgs_moe.hip) ---------------------------------------------------

struct DispatchArgs {
    const uint16_t* x;      // (T, D) bf16, or null: only the order
    const int32_t* ids;     // (T, k)
    int64_t T, D;
    int k, E, align;
    int64_t P;              // rows of the outputs, at least moe_rows_bound
    int pow2;
    int32_t* offsets;       // (E)
    int32_t* rows;          // (T, k)
    int32_t* slots;         // (P)
    uint16_t* xp;           // (P, D) bf16 or null
    uint8_t* q;             // (P, D) E4M3 or null
    float* scales;          // (P, ceil(D / 128))
    int32_t* hist;          // workspace: slot counts (moe_runs, E), or null
};

// An upper bound on the rows that the experts' groups take (a multiple of align).
inline int64_t moe_rows_bound(int64_t n, int64_t E, int64_t align) {
    const int64_t used = n < E ? n : E;
    return (n + used * (align - 1)) / align * align;
}

// Up to this many slots one launch does everything (us with it and, in
// parentheses, ranked first: 1024 slots 6.3 (11.8), 6702 12.7 (20.4), 32768 to
// 16 experts 26 (32); 65536 45.6 (45.4)).
constexpr int64_t kMoeFusedSlots = 32768;
// More are ranked in runs of moe_run slots, one workgroup each; the runs'
// counts go through the workspace (moe_runs, E).
inline int64_t moe_run(int64_t n) {
    const int64_t s = (n + 63) / 64;
    return s < 8192 ? 8192 : s;
}
inline int64_t moe_runs(int64_t n) { return (n + moe_run(n) - 1) / moe_run(n); }
inline int64_t moe_workspace(int64_t n, int64_t E) { return n > kMoeFusedSlots ? moe_runs(n) * E * 4 : 0; }

hipError_t launch_dispatch(const DispatchArgs& a, int cus, hipStream_t stream);

// y[t] = sum over the k slots of weights (null: 1) times yp[rows[t, s]].
hipError_t launch_combine(const uint16_t* yp, int64_t P, int64_t D, const int32_t* rows, int64_t T, int k,
                          const float* weights, uint16_t* y, int cus, hipStream_t stream);

hipError_t launch_combine_grad(const uint16_t* dy, const uint16_t* yp, int64_t P, int64_t D,
                               const int32_t* rows, const int32_t* slots, int64_t T, int k,
                               const float* weights, uint16_t* dyp, float* dw, int cus, hipStream_t stream);

// ---- block-128 casts (mgs_block128.hip) ------------------------------------------

hipError_t launch_rows128(const uint16_t* x, int64_t M, int64_t K, bool pow2, uint8_t* q, float* scales,
                          hipStream_t stream);

// q_t and scales_t may be null (both): only the first order.
hipError_t launch_blocks128(const uint16_t* w, int64_t E, int64_t N, int64_t K, bool pow2, uint8_t* q,
                            float* scales, uint8_t* q_t, float* scales_t, hipStream_t stream);

// ---- products (mgs_mm.hip) ---------------------------------------------------------

// fast: sums in the 8-bit matrix instruction (see mgs_mm.hip). offsets null: one
// group of all M rows.
hipError_t launch_mm_block128(const uint8_t* a, const float* a_scales, int64_t M, int64_t K, const uint8_t* b,
                              const float* b_scales, int64_t E, int64_t N, const int32_t* offsets, bool fast,
                              bool f32, void* y, int cus, hipStream_t stream);

hipError_t launch_mm_wgrad(const uint8_t* a_t, const float* a_scales_t, const uint8_t* b_t,
                           const float* b_scales_t, int64_t M, int64_t N, int64_t K, const int32_t* offsets,
                           int64_t G, bool fast, bool f32, bool accumulate, void* dw, int cus, hipStream_t stream);

}  // namespace mgs
