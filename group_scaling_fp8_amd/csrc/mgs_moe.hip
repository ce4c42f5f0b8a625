// mgs_moe.hip — tokens sorted by expert and back (gfx950).
//
// A slot i = t * k + s is the s-th choice of token t. Expert e's c_e slots
// take consecutive rows in slot order, and its group is filled up to a
// multiple of `align` rows, so
//   row(i) = sum_{e' < e} up(c_e') + #{j < i : id(j) = e},
// a counting sort whose ranks need no atomics in the data's order: the
// result is the same on every run.
#include "mgs_block128_device.hpp"
#include "mgs_experts.hpp"

namespace mgs {

namespace {

constexpr int kDispatchThreads = 256;
constexpr int kDispatchWaves = kDispatchThreads / kWave;

__global__ __launch_bounds__(1024) void hist_kernel(const int32_t* __restrict__ ids, int64_t n, int64_t run, int E,
                                                    int32_t* __restrict__ hist) {
    extern __shared__ int s_hist[];
    for (int e = threadIdx.x; e < E; e += blockDim.x) s_hist[e] = 0;
    __syncthreads();
    const int64_t lo = blockIdx.x * run, hi = min(lo + run, n);
    for (int64_t i = lo + threadIdx.x; i < hi; i += blockDim.x) {
        const int e = ids[i];
        if (e >= 0 && e < E) atomicAdd(&s_hist[e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += blockDim.x) hist[(int64_t)blockIdx.x * E + e] = s_hist[e];
}

// One row of padding: zeros and the scale of an empty block.
__device__ __forceinline__ void zero_row(const DispatchArgs& a, int64_t p, int u0, int ustep, int units,
                                         float empty_scale) {
    const int lane = threadIdx.x & (kWave - 1);
    const int64_t nb = (a.D + 127) / 128;
    for (int u = u0; u < units; u += ustep) {
        const int64_t col = (int64_t)u * 512 + lane * 8;
        if (col < a.D) {
            if (a.xp) *reinterpret_cast<uint4*>(a.xp + p * a.D + col) = make_uint4(0, 0, 0, 0);
            if (a.q) {
                *reinterpret_cast<uint2*>(a.q + p * a.D + col) = make_uint2(0, 0);
                if ((lane & 15) == 0) a.scales[p * nb + col / 128] = empty_scale;
            }
        }
    }
}

// Workgroup (b, c): tokens b * tb .. of the columns c, c + CS, ... in units of
// 512. Every workgroup finds the row of each of its slots by itself.
__global__ __launch_bounds__(kDispatchThreads) void dispatch_kernel(DispatchArgs a, int tb, int64_t run, int runs) {
    extern __shared__ int smem[];
    int* s_total = smem;                // (E) slots of each expert
    int* s_next = smem + a.E;           // (E) next row of each expert
    int* s_start = smem + 2 * a.E;      // (E + 1) first row of each expert's group
    int* s_row = smem + 3 * a.E + 1;    // (tb * k) rows of this workgroup's slots
    const int E = a.E, k = a.k, tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
    const int64_t t0 = (int64_t)blockIdx.x * tb, t1 = min(t0 + tb, a.T);
    const int64_t n = a.T * k, first = t0 * k, last = t1 * k;
    for (int e = tid; e < E; e += kDispatchThreads) s_total[e] = s_next[e] = 0;
    __syncthreads();
    if (runs == 0) {
        for (int64_t i = tid; i < n; i += kDispatchThreads) {
            const int e = a.ids[i];
            if (e >= 0 && e < E) {
                atomicAdd(&s_total[e], 1);
                if (i < first) atomicAdd(&s_next[e], 1);
            }
        }
    } else {
        const int mine = (int)(first / run);
        for (int i = tid; i < runs * E; i += kDispatchThreads) {
            const int j = i / E, e = i - j * E, v = a.hist[i];
            atomicAdd(&s_total[e], v);
            if (j < mine) atomicAdd(&s_next[e], v);
        }
        for (int64_t i = mine * run + tid; i < first; i += kDispatchThreads) {
            const int e = a.ids[i];
            if (e >= 0 && e < E) atomicAdd(&s_next[e], 1);
        }
    }
    __syncthreads();
    if (wave == 0) {
        int carry = 0;
        for (int base = 0; base < E; base += kWave) {
            const int e = base + lane;
            const int full = e < E ? (s_total[e] + a.align - 1) / a.align * a.align : 0;
            const int end = carry + wave_prefix_sum(full);
            if (e < E) {
                s_start[e] = end - full;
                s_next[e] += end - full;
            }
            carry = __shfl(end, kWave - 1, kWave);
        }
        if (lane == 0) s_start[E] = carry;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "workgroup");
        // ranks in slot order, 64 slots at a time: lanes of the same expert
        // find each other with one ballot for each bit of the id
        for (int64_t base = first; base < last; base += kWave) {
            const int64_t i = base + lane;
            const int e = i < last ? a.ids[i] : -1;
            const bool held = e >= 0 && e < E;
            uint64_t same = __ballot(held);
            for (int bit = 1; bit < E; bit <<= 1) {
                const uint64_t set = __ballot(held && (e & bit));
                same &= (e & bit) ? set : ~set;
            }
            const int rank = __popcll(same & ((1ull << lane) - 1));
            int row = -1;
            if (held) row = s_next[e] + rank;
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            if (held && rank == 0) s_next[e] = row + __popcll(same);
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            if (i < last) {
                if (row >= a.P) row = -1;
                s_row[i - first] = row;
                if (blockIdx.y == 0) {
                    a.rows[i] = row;
                    if (row >= 0) a.slots[row] = (int)i;
                }
            }
        }
    }
    __syncthreads();
    if (blockIdx.x == 0 && blockIdx.y == 0)
        for (int e = tid; e < E; e += kDispatchThreads) a.offsets[e] = s_start[e + 1];

    const int units = a.x ? (int)((a.D + 511) / 512) : 0;
    const int CS = gridDim.y, own_units = units > (int)blockIdx.y ? (units - blockIdx.y + CS - 1) / CS : 0;
    const int64_t nb = (a.D + 127) / 128;
    const bool pow2 = a.pow2 != 0;

    // padding rows: the end of each expert's group, and the rows past the last group
    const float empty_scale = group_scale(0u, pow2);
    for (int e = blockIdx.x * kDispatchWaves + wave; e < E; e += gridDim.x * kDispatchWaves) {
        for (int64_t p = s_start[e] + s_total[e]; p < s_start[e + 1]; ++p) {
            if (blockIdx.y == 0 && lane == 0) a.slots[p] = -1;
            zero_row(a, p, blockIdx.y, CS, units, empty_scale);
        }
    }
    for (int64_t p = s_start[E] + (int64_t)blockIdx.x * kDispatchWaves + wave; p < a.P;
         p += (int64_t)gridDim.x * kDispatchWaves) {
        if (blockIdx.y == 0 && lane == 0) a.slots[p] = -1;
        zero_row(a, p, blockIdx.y, CS, units, empty_scale);
    }

    // each token is read and cast once and written to its k rows
    const int items = (int)(t1 - t0) * own_units;
    for (int it = wave; it < items; it += kDispatchWaves) {
        const int t = it / own_units, u = blockIdx.y + (it - t * own_units) * CS;
        const int64_t col = (int64_t)u * 512 + lane * 8;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (col < a.D) v = load_stream(a.x + (t0 + t) * a.D + col);
        const float s = group_scale(row16_max(mag_fold(mag_max8(0u, v))), pow2);
        const uint2 c = cast8_group(v, s);
        if (col < a.D) {
            for (int j = 0; j < k; ++j) {
                const int64_t p = s_row[t * k + j];
                if (p < 0) continue;
                if (a.xp) *reinterpret_cast<uint4*>(a.xp + p * a.D + col) = v;
                if (a.q) {
                    *reinterpret_cast<uint2*>(a.q + p * a.D + col) = c;
                    if ((lane & 15) == 0) a.scales[p * nb + col / 128] = s;
                }
            }
        }
    }
}

// y[t] over the columns of one workgroup; fp32 sums in slot order, one
// rounding to bf16.
__global__ __launch_bounds__(256) void combine_kernel(const uint16_t* __restrict__ yp, int64_t P, int64_t D,
                                                      const int32_t* __restrict__ rows, int64_t T, int k,
                                                      const float* __restrict__ weights,
                                                      uint16_t* __restrict__ y) {
    const int64_t col = ((int64_t)blockIdx.y * 256 + threadIdx.x) * 8;
    if (col >= D) return;
    for (int64_t t = blockIdx.x; t < T; t += gridDim.x) {
        float acc[8] = {};
        for (int s = 0; s < k; ++s) {
            const int64_t p = rows[t * k + s];
            if (p < 0 || p >= P) continue;
            const float w = weights ? weights[t * k + s] : 1.0f;
            add8(acc, load_stream(yp + p * D + col), w);
        }
        *reinterpret_cast<uint4*>(y + t * D + col) = pack8(acc);
    }
}

// Workgroups below T: dyp[rows[t, s]] = w[t, s] * dy[t] and
// dw[t, s] = <dy[t], yp[rows[t, s]]>; the others zero the padding rows.
__global__ __launch_bounds__(256) void combine_grad_kernel(
        const uint16_t* __restrict__ dy, const uint16_t* __restrict__ yp, int64_t P, int64_t D,
        const int32_t* __restrict__ rows, const int32_t* __restrict__ slots, int64_t T, int k,
        const float* __restrict__ weights, uint16_t* __restrict__ dyp, float* __restrict__ dw) {
    __shared__ float s_part[64][4];
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int64_t t = blockIdx.x;
    if (t >= T) {
        const int64_t n = T * k;
        const int64_t lo = (t - T) * 64, hi = min(lo + 64, P);
        for (int64_t p = lo + wave; p < hi; p += 4) {
            const int slot = slots[p];
            if (slot >= 0 && slot < n) continue;
            for (int64_t col = lane * 8; col < D; col += 512)
                *reinterpret_cast<uint4*>(dyp + p * D + col) = make_uint4(0, 0, 0, 0);
        }
        return;
    }
    for (int s = 0; s < k; ++s) {
        const int64_t p = rows[t * k + s];
        float dot = 0.0f;
        if (p >= 0 && p < P) {
            const float w = weights[t * k + s];
            for (int64_t col = (int64_t)threadIdx.x * 8; col < D; col += 2048) {
                const uint4 g = *reinterpret_cast<const uint4*>(dy + t * D + col);
                dot = dot8(dot, g, load_stream(yp + p * D + col));
                float r[8] = {};
                add8(r, g, w);
                *reinterpret_cast<uint4*>(dyp + p * D + col) = pack8(r);
            }
        }
        dot = wave_sum(dot);
        if (lane == 0) s_part[s][wave] = dot;
    }
    __syncthreads();
    if (threadIdx.x < k) {
        const int s = threadIdx.x;
        dw[t * k + s] = (s_part[s][0] + s_part[s][1]) + (s_part[s][2] + s_part[s][3]);
    }
}

}  // namespace

hipError_t launch_dispatch(const DispatchArgs& a, int cus, hipStream_t stream) {
    const int64_t n = a.T * a.k;
    const int64_t runs = moe_superblocks(n), run = moe_superblock(n);
    if (runs > 0) {
        hipLaunchKernelGGL(hist_kernel, dim3((unsigned)runs), dim3(1024), a.E * sizeof(int), stream, a.ids, n,
                           run, a.E, a.hist);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    // about four workgroups per CU before a workgroup takes more than one token
    int64_t tb = a.T / (4 * (int64_t)cus);
    tb = tb < 1 ? 1 : tb > 16 ? 16 : tb;
    const int64_t blocks = a.T > 0 ? (a.T + tb - 1) / tb : 1;
    const int64_t units = a.x ? (a.D + 511) / 512 : 1;
    int64_t cs = 2 * (int64_t)cus / blocks;
    cs = cs < 1 ? 1 : cs > (units + 3) / 4 ? (units + 3) / 4 : cs;
    const size_t shmem = (3 * (size_t)a.E + 1 + (size_t)tb * a.k) * sizeof(int);
    hipLaunchKernelGGL(dispatch_kernel, dim3((unsigned)blocks, (unsigned)cs), dim3(kDispatchThreads), shmem, stream,
                       a, (int)tb, run, (int)runs);
    return hipGetLastError();
}

hipError_t launch_combine(const uint16_t* yp, int64_t P, int64_t D, const int32_t* rows, int64_t T, int k,
                          const float* weights, uint16_t* y, int, hipStream_t stream) {
    const int64_t blocks = T < (1 << 20) ? T : (1 << 20);
    hipLaunchKernelGGL(combine_kernel, dim3((unsigned)blocks, (unsigned)((D + 2047) / 2048)), dim3(256), 0, stream,
                       yp, P, D, rows, T, k, weights, y);
    return hipGetLastError();
}

hipError_t launch_combine_grad(const uint16_t* dy, const uint16_t* yp, int64_t P, int64_t D,
                               const int32_t* rows, const int32_t* slots, int64_t T, int k,
                               const float* weights, uint16_t* dyp, float* dw, int, hipStream_t stream) {
    const int64_t blocks = T + (P + 63) / 64;
    hipLaunchKernelGGL(combine_grad_kernel, dim3((unsigned)blocks), dim3(256), 0, stream, dy, yp, P, D, rows, slots,
                       T, k, weights, dyp, dw);
    return hipGetLastError();
}

}  // namespace mgs
