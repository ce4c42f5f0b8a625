// mgs_experts_api.hip — the C ABI of the mixture-of-experts calls (declared in
// include/mgs.h): host-side argument checks and stream-ordered launches.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mgs.h"
#include "mgs_experts.hpp"
#include "mgs_status.hpp"

namespace {

using mgs::aligned;
using mgs::hip_status;

// Rows of one operand's tile are addressed with 32-bit offsets: 256 rows of
// up to this many bytes.
constexpr int64_t kMaxRowBytes = (int64_t(1) << 31) / 256 - 256;
constexpr int64_t kMaxCols = kMaxRowBytes / 4;       // of an output

int check_order(int64_t T, int32_t top_k, int32_t n_experts, int32_t align) {
    if (T < 0 || top_k < 1 || n_experts < 1 || align < 16 || align % 16 != 0) return MGS_ERR_INVALID_ARG;
    if (top_k > MGS_MOE_MAX_TOP_K || n_experts > MGS_MAX_GROUPS || align > 4096) return MGS_ERR_UNSUPPORTED;
    if (T > INT32_MAX / 2 / top_k) return MGS_ERR_UNSUPPORTED;      // slots and rows are int32
    return MGS_OK;
}

hipStream_t as_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }

}  // namespace

extern "C" {

int mgs_moe_rows(int64_t T, int32_t top_k, int32_t n_experts, int32_t align, int64_t* n_rows) {
    const int st = check_order(T, top_k, n_experts, align);
    if (st != MGS_OK) return st;
    if (!n_rows) return MGS_ERR_INVALID_ARG;
    *n_rows = mgs::moe_rows_bound(T * top_k, n_experts, align);
    return MGS_OK;
}

int mgs_moe_workspace_bytes(int64_t T, int32_t top_k, int32_t n_experts, int64_t* bytes) {
    const int st = check_order(T, top_k, n_experts, 16);
    if (st != MGS_OK) return st;
    if (!bytes) return MGS_ERR_INVALID_ARG;
    *bytes = mgs::moe_workspace(T * top_k, n_experts);
    return MGS_OK;
}

int mgs_moe_dispatch(const void* x, int64_t T, int64_t D, const int32_t* expert_ids, int32_t top_k,
                     int32_t n_experts, int32_t align, uint32_t flags, int64_t n_rows, int32_t* offsets,
                     int32_t* rows, int32_t* slots, void* xp, void* q, float* scales, void* workspace,
                     int64_t workspace_bytes, void* stream) {
    const int st = check_order(T, top_k, n_experts, align);
    if (st != MGS_OK) return st;
    if (flags & ~MGS_FLAG_POW2_SCALE) return MGS_ERR_INVALID_ARG;
    if (D < 0 || D % 8 != 0) return MGS_ERR_INVALID_ARG;
    if (D > INT32_MAX || n_rows > INT32_MAX) return MGS_ERR_UNSUPPORTED;
    if (n_rows < mgs::moe_rows_bound(T * top_k, n_experts, align)) return MGS_ERR_INVALID_ARG;
    if (!offsets || !aligned(offsets, 4)) return MGS_ERR_INVALID_ARG;
    if (T > 0 && (!expert_ids || !rows || !aligned(expert_ids, 4) || !aligned(rows, 4))) return MGS_ERR_INVALID_ARG;
    if (n_rows > 0 && (!slots || !aligned(slots, 4))) return MGS_ERR_INVALID_ARG;
    const bool moves = (xp || q) && n_rows > 0 && D > 0;
    if ((q != nullptr) != (scales != nullptr)) return MGS_ERR_INVALID_ARG;
    if (moves && ((T > 0 && !x) || !aligned(x, 16) || !aligned(xp, 16) || !aligned(q, 8) || !aligned(scales, 4)))
        return MGS_ERR_INVALID_ARG;
    const int64_t need = mgs::moe_workspace(T * top_k, n_experts);
    if (workspace_bytes < 0 || workspace_bytes < need || !aligned(workspace, 16) || (need > 0 && !workspace))
        return MGS_ERR_INVALID_ARG;
    const mgs::DispatchArgs a{static_cast<const uint16_t*>(x), expert_ids, T, moves ? D : 0, top_k, n_experts, align,
                              n_rows, (flags & MGS_FLAG_POW2_SCALE) ? 1 : 0, offsets, rows, slots,
                              moves ? static_cast<uint16_t*>(xp) : nullptr, moves ? static_cast<uint8_t*>(q) : nullptr,
                              scales, static_cast<int32_t*>(workspace)};
    return hip_status(mgs::launch_dispatch(a, mgs::device_cus(), as_stream(stream)));
}

int mgs_moe_combine(const void* yp, int64_t n_rows, int64_t D, const int32_t* rows, int64_t T, int32_t top_k,
                    const float* weights, void* y, void* stream) {
    const int st = check_order(T, top_k, 1, 16);
    if (st != MGS_OK) return st;
    if (n_rows < 0 || D < 0 || D % 8 != 0) return MGS_ERR_INVALID_ARG;
    if (D > INT32_MAX || n_rows > INT32_MAX) return MGS_ERR_UNSUPPORTED;
    if (T == 0 || D == 0) return MGS_OK;
    if (!rows || !y || (n_rows > 0 && !yp) || !aligned(rows, 4) || !aligned(y, 16) || !aligned(yp, 16) ||
        !aligned(weights, 4))
        return MGS_ERR_INVALID_ARG;
    return hip_status(mgs::launch_combine(static_cast<const uint16_t*>(yp), n_rows, D, rows, T, top_k, weights,
                                          static_cast<uint16_t*>(y), mgs::device_cus(), as_stream(stream)));
}

int mgs_moe_combine_grad(const void* dy, const void* yp, int64_t n_rows, int64_t D, const int32_t* rows,
                         const int32_t* slots, int64_t T, int32_t top_k, const float* weights, void* dyp, float* dw,
                         void* stream) {
    const int st = check_order(T, top_k, 1, 16);
    if (st != MGS_OK) return st;
    if (n_rows < 0 || D < 0 || D % 8 != 0) return MGS_ERR_INVALID_ARG;
    if (D > INT32_MAX || n_rows > INT32_MAX) return MGS_ERR_UNSUPPORTED;
    if (T == 0 && n_rows == 0) return MGS_OK;
    if (n_rows > 0 && (!slots || !aligned(slots, 4))) return MGS_ERR_INVALID_ARG;
    if (T > 0 && (!rows || !weights || !dw || !aligned(rows, 4) || !aligned(weights, 4) || !aligned(dw, 4)))
        return MGS_ERR_INVALID_ARG;
    if (D > 0 && ((T > 0 && !dy) || (n_rows > 0 && (!yp || !dyp)) || !aligned(dy, 16) || !aligned(yp, 16) ||
                  !aligned(dyp, 16)))
        return MGS_ERR_INVALID_ARG;
    return hip_status(mgs::launch_combine_grad(static_cast<const uint16_t*>(dy), static_cast<const uint16_t*>(yp),
                                               n_rows, D, rows, slots, T, top_k, weights, static_cast<uint16_t*>(dyp),
                                               dw, mgs::device_cus(), as_stream(stream)));
}

int mgs_quant_rows128(const void* x, int64_t M, int64_t K, uint32_t flags, void* q, float* scales, void* stream) {
    if (M < 0 || K < 0 || K % 8 != 0 || (flags & ~MGS_FLAG_POW2_SCALE)) return MGS_ERR_INVALID_ARG;
    if (K > INT32_MAX || M > INT32_MAX) return MGS_ERR_UNSUPPORTED;
    if (M == 0 || K == 0) return MGS_OK;
    if (!x || !q || !scales || !aligned(x, 16) || !aligned(q, 8) || !aligned(scales, 4)) return MGS_ERR_INVALID_ARG;
    return hip_status(mgs::launch_rows128(static_cast<const uint16_t*>(x), M, K, (flags & MGS_FLAG_POW2_SCALE) != 0,
                                          static_cast<uint8_t*>(q), scales, as_stream(stream)));
}

int mgs_quant_blocks128(const void* w, int64_t E, int64_t N, int64_t K, uint32_t flags, void* q, float* scales,
                        void* q_t, float* scales_t, void* stream) {
    if (E < 0 || N < 0 || K < 0 || N % 16 != 0 || K % 16 != 0 || (flags & ~MGS_FLAG_POW2_SCALE))
        return MGS_ERR_INVALID_ARG;
    if (E > INT32_MAX || N > INT32_MAX || K > INT32_MAX) return MGS_ERR_UNSUPPORTED;
    if (E == 0 || N == 0 || K == 0) return MGS_OK;
    if (((N + 127) / 128) * ((K + 127) / 128) > INT32_MAX / E) return MGS_ERR_UNSUPPORTED;
    if ((q_t != nullptr) != (scales_t != nullptr)) return MGS_ERR_INVALID_ARG;
    if (!w || !q || !scales || !aligned(w, 16) || !aligned(q, 16) || !aligned(scales, 4) || !aligned(q_t, 16) ||
        !aligned(scales_t, 4))
        return MGS_ERR_INVALID_ARG;
    return hip_status(mgs::launch_blocks128(static_cast<const uint16_t*>(w), E, N, K,
                                            (flags & MGS_FLAG_POW2_SCALE) != 0, static_cast<uint8_t*>(q), scales,
                                            static_cast<uint8_t*>(q_t), scales_t, as_stream(stream)));
}

int mgs_mm_block128(const void* a, const float* a_scales, int64_t M, int64_t K, const void* b, const float* b_scales,
                    int32_t n_groups, int64_t N, const int32_t* offsets, uint32_t flags, int out_type, void* y,
                    void* stream) {
    if (M < 0 || N < 0 || K < 0 || n_groups < 1 || N % 16 != 0 || K % 16 != 0) return MGS_ERR_INVALID_ARG;
    if (out_type != MGS_OUT_BF16 && out_type != MGS_OUT_F32) return MGS_ERR_INVALID_ARG;
    if (flags & ~MGS_FLAG_FAST_ACCUM) return MGS_ERR_INVALID_ARG;
    if (!offsets && n_groups != 1) return MGS_ERR_INVALID_ARG;
    if (n_groups > MGS_MAX_GROUPS || M > INT32_MAX || N > kMaxCols || K > kMaxRowBytes) return MGS_ERR_UNSUPPORTED;
    if (M == 0 || N == 0) return MGS_OK;
    if (!y || !aligned(y, 16) || !aligned(offsets, 4)) return MGS_ERR_INVALID_ARG;
    if (K > 0 && (!a || !a_scales || !b || !b_scales || !aligned(a, 16) || !aligned(b, 16) || !aligned(a_scales, 4) ||
                  !aligned(b_scales, 4)))
        return MGS_ERR_INVALID_ARG;
    if ((M / 16 + n_groups + 1) * ((N + 15) / 16) > INT32_MAX) return MGS_ERR_UNSUPPORTED;
    return hip_status(mgs::launch_mm_block128(static_cast<const uint8_t*>(a), a_scales, M, K,
                                              static_cast<const uint8_t*>(b), b_scales, n_groups, N, offsets,
                                              (flags & MGS_FLAG_FAST_ACCUM) != 0, out_type == MGS_OUT_F32, y,
                                              mgs::device_cus(), as_stream(stream)));
}

int mgs_mm_wgrad(const void* a_t, const float* a_scales_t, const void* b_t, const float* b_scales_t, int64_t M,
                 int64_t N, int64_t K, const int32_t* offsets, int32_t n_groups, uint32_t flags, int out_type,
                 void* dw, void* stream) {
    if (M < 0 || N < 0 || K < 0 || n_groups < 1 || M % 16 != 0 || N % 16 != 0 || K % 16 != 0)
        return MGS_ERR_INVALID_ARG;
    if (flags & ~(MGS_FLAG_ACCUMULATE | MGS_FLAG_FAST_ACCUM)) return MGS_ERR_INVALID_ARG;
    if (out_type != MGS_OUT_BF16 && out_type != MGS_OUT_F32) return MGS_ERR_INVALID_ARG;
    if ((flags & MGS_FLAG_ACCUMULATE) && out_type != MGS_OUT_F32) return MGS_ERR_INVALID_ARG;
    if (n_groups > MGS_MAX_GROUPS || N > INT32_MAX || K > kMaxCols || M > kMaxRowBytes) return MGS_ERR_UNSUPPORTED;
    if (N == 0 || K == 0) return MGS_OK;
    if (!offsets || !aligned(offsets, 4) || !dw || !aligned(dw, 16)) return MGS_ERR_INVALID_ARG;
    if (!a_scales_t || !b_scales_t || !aligned(a_scales_t, 4) || !aligned(b_scales_t, 4)) return MGS_ERR_INVALID_ARG;
    if (M > 0 && (!a_t || !b_t || !aligned(a_t, 16) || !aligned(b_t, 16))) return MGS_ERR_INVALID_ARG;
    if (((N + 63) / 64) * ((K + 63) / 64) > INT32_MAX / n_groups) return MGS_ERR_UNSUPPORTED;
    return hip_status(mgs::launch_mm_wgrad(static_cast<const uint8_t*>(a_t), a_scales_t,
                                           static_cast<const uint8_t*>(b_t), b_scales_t, M, N, K, offsets, n_groups,
                                           (flags & MGS_FLAG_FAST_ACCUM) != 0, out_type == MGS_OUT_F32,
                                           (flags & MGS_FLAG_ACCUMULATE) != 0, dw, mgs::device_cus(),
                                           as_stream(stream)));
}

}  // extern "C"
