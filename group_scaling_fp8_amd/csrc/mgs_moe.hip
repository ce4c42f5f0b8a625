// mgs_moe.hip — tokens sorted by expert and back (gfx950).
//
// A slot i = t * k + s is the s-th choice of token t. Expert e's c_e slots
// take consecutive rows in slot order, and its group is filled up to a
// multiple of `align` rows, so
//   row(i) = sum_{e' < e} up(c_e') + #{j < i : id(j) = e},
// a counting sort whose ranks need no atomics in the data's order: the
// result is the same on every run.
//
// All of it is bound by memory traffic, and with few tokens by a launch's fixed
// cost. Times are of MI355X.
#include "mgs_block128_device.hpp"
#include "mgs_experts.hpp"

namespace mgs {

namespace {

// ---- the order ---------------------------------------------------------------
//
// Up to kMoeFusedSlots slots, every workgroup of the one dispatch kernel counts
// all of them for itself (1 token, 8 of 64 experts, 5120 columns: 5.2 us; 1117
// tokens, 6 of 61, 4112 columns: 12.7). More are ranked first, by one workgroup
// of 16 waves for each run of slots: hist_kernel counts, rank_kernel writes rows
// and slots, and dispatch_kernel reads them (66560 slots: 6 and 13 us).

// The lanes (of those with `held`) whose expert is this lane's: one ballot for
// each bit of the id.
__device__ __forceinline__ uint64_t same_expert(int e, bool held, int E) {
    uint64_t same = __ballot(held);
    for (int bit = 1; bit < E; bit <<= 1) {
        const uint64_t set = __ballot(held && (e & bit));
        same &= (e & bit) ? set : ~set;
    }
    return same;
}

__device__ __forceinline__ uint64_t lanes_below() {
    return (1ull << (threadIdx.x & (kWave - 1))) - 1;
}

// First row of every expert's group from the slots of each, by one wave:
// start[e] for e <= E.
__device__ __forceinline__ void group_starts(const int* total, int* start, int E, int align) {
    const int lane = threadIdx.x & (kWave - 1);
    int carry = 0;
    for (int base = 0; base < E; base += kWave) {
        const int e = base + lane;
        const int full = e < E ? (total[e] + align - 1) / align * align : 0;
        const int end = carry + wave_prefix_sum(full);
        if (e < E) start[e] = end - full;
        carry = __shfl(end, kWave - 1, kWave);
    }
    if (lane == 0) start[E] = carry;
}

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

// Rows of run blockIdx.x's slots. Wave w takes the run's w-th part and ranks its
// slots among themselves, 64 at a time; then its counts are summed over the runs
// and waves before it.
template <int WAVES>
__global__ __launch_bounds__(WAVES * 64) void rank_kernel(DispatchArgs a, int64_t run) {
    extern __shared__ int smem[];
    const int E = a.E, tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
    int* s_total = smem;                     // (E) slots of each expert
    int* s_start = s_total + E;              // (E + 1) first row of each group
    int* s_wave = s_start + E + 1;           // (waves, E) slots of each wave, then the row its first one takes
    const int64_t n = a.T * a.k, lo = blockIdx.x * run, hi = min(lo + run, n);
    const int64_t part = (run + WAVES - 1) / WAVES, first = min(lo + wave * part, hi), last = min(first + part, hi);
    int* mine = s_wave + wave * E;
    for (int e = lane; e < E; e += kWave) mine[e] = 0;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    // place[c]: how many slots of its expert come before the lane's, in its wave
    constexpr int C = 8;        // 8 x 64 slots at a time
    int id[C], place[C];
    const bool once = last - first <= C * kWave;      // they stay in registers, else in rows
    for (int64_t base = first; base < last; base += C * kWave) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int64_t i = base + c * kWave + lane;
            id[c] = i < last ? a.ids[i] : -1;
        }
        uint64_t same[C];
#pragma unroll
        for (int c = 0; c < C; ++c) same[c] = same_expert(id[c], id[c] >= 0 && id[c] < E, E);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int e = id[c], below = __popcll(same[c] & lanes_below());
            const bool held = e >= 0 && e < E;
            place[c] = held ? mine[e] + below : -1;
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            if (held && below == 0) mine[e] = place[c] + __popcll(same[c]);
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        }
        if (!once) {
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int64_t i = base + c * kWave + lane;
                if (i < last) a.rows[i] = place[c];
            }
        }
    }
    __syncthreads();
    for (int e = tid; e < E; e += WAVES * 64) {
        int count[WAVES], sum = 0, prior = 0;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) count[w] = s_wave[w * E + e];
        for (int r = 0; r < (int)gridDim.x; ++r) {
            const int c = a.hist[(int64_t)r * E + e];
            if (r < (int)blockIdx.x) prior += c;
            sum += c;
        }
        int before = prior;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
            s_wave[w * E + e] = before;
            before += count[w];
        }
        s_total[e] = sum;
    }
    __syncthreads();
    if (wave == 0) group_starts(s_total, s_start, E, a.align);
    __syncthreads();
    for (int64_t base = first; base < last; base += C * kWave) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int64_t i = base + c * kWave + lane;
            if (i >= last) continue;
            const int e = once ? id[c] : a.ids[i];
            int row = once ? place[c] : a.rows[i];
            if (row >= 0) row += s_start[e] + mine[e];
            if (row >= a.P) row = -1;
            a.rows[i] = row;
            if (row >= 0) a.slots[row] = (int)i;
        }
    }
    // offsets, and the rows that no slot takes
    const int step = gridDim.x * WAVES * 64, at = blockIdx.x * WAVES * 64 + tid;
    for (int e = at; e < E; e += step) a.offsets[e] = s_start[e + 1];
    for (int i = at; i < E * a.align; i += step) {
        const int e = i / a.align, p = s_start[e] + s_total[e] + i - e * a.align;
        if (p < s_start[e + 1]) a.slots[p] = -1;
    }
    for (int64_t p = (int64_t)s_start[E] + at; p < a.P; p += step) a.slots[p] = -1;
}

// ---- copy and cast -------------------------------------------------------------

constexpr int kDispatchThreads = 256;
constexpr int kDispatchWaves = kDispatchThreads / kWave;
constexpr int kUnit = 1024;              // columns of a wave's piece: two halves of eight a lane, 16 lanes a block of 128

__device__ __forceinline__ int64_t column(int u, int h) {
    return (int64_t)u * kUnit + h * (kUnit / 2) + (threadIdx.x & (kWave - 1)) * 8;
}

// Eight columns of row p. A wave's stores are whole lines: with 16 columns a lane,
// every second 16 bytes a store, xp came at half the rate.
__device__ __forceinline__ void put(const DispatchArgs& a, int64_t p, int64_t col, uint4 x, uint2 q, float scale) {
    if (a.xp) store_stream16(a.xp + p * a.D + col, x);
    if (a.q) {
        store_stream(a.q + p * a.D + col, q);
        if ((threadIdx.x & 15) == 0) a.scales[p * ((a.D + 127) / 128) + col / 128] = scale;
    }
}

// The units u0, u0 + ustep, ... of a row that no slot takes: zeros and the
// scale of an empty block.
__device__ __forceinline__ void zero_row(const DispatchArgs& a, int64_t p, int u0, int ustep, int units) {
    const float scale = group_scale(0u, a.pow2 != 0);
    for (int u = u0; u < units; u += ustep)
#pragma unroll
        for (int h = 0; h < 2; ++h)
            if (column(u, h) < a.D) put(a, p, column(u, h), make_uint4(0, 0, 0, 0), make_uint2(0, 0), scale);
}

// Unit u of token t, zeros past its end.
__device__ __forceinline__ void load_piece(const DispatchArgs& a, int64_t t, int u, uint4 (&x)[2]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        x[h] = make_uint4(0, 0, 0, 0);
        if (column(u, h) < a.D) x[h] = *reinterpret_cast<const uint4*>(a.x + t * a.D + column(u, h));
    }
}

// Its cast, made once, to the rows of the token's k slots.
__device__ __forceinline__ void put_piece(const DispatchArgs& a, const int* rows, int u, const uint4 (&x)[2]) {
    float s[2];
    uint2 q[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        s[h] = group_scale(row16_max(mag_fold(mag_max8(0u, x[h]))), a.pow2 != 0);
        q[h] = cast8_group(x[h], s[h]);
    }
    for (int j = 0; j < a.k; ++j) {
        const int row = rows[j];
        if (row < 0) continue;
#pragma unroll
        for (int h = 0; h < 2; ++h)
            if (column(u, h) < a.D) put(a, row, column(u, h), x[h], q[h], s[h]);
    }
}

// Everything in one launch, for few slots: workgroups below `groups` take `per`
// consecutive tokens each, all take a share of the rows without a slot, and
// grid.y splits the columns. Every workgroup finds the order by itself, while
// its first loads of x are on their way.
constexpr int kFusedThreads = 512;
constexpr int kFusedWaves = kFusedThreads / kWave;

__global__ __launch_bounds__(kFusedThreads) void dispatch_fused_kernel(DispatchArgs a, int groups, int per) {
    extern __shared__ int smem[];
    const int E = a.E, k = a.k, tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
    int* s_before = smem;               // (E) slots of each expert before this workgroup's tokens
    int* s_total = s_before + E;        // (E) all the others, then all
    int* s_start = s_total + E;         // (E + 1) first row of each group
    int* s_row = s_start + E + 1;       // (per, k) rows of this workgroup's tokens
    const int n = (int)(a.T * k), t0 = blockIdx.x * per;
    const int tokens = (int)blockIdx.x < groups ? min(per, (int)a.T - t0) : 0;
    const int first = tokens ? t0 * k : n, last = first + tokens * k;
    const int units = (int)((a.D + kUnit - 1) / kUnit), u0 = blockIdx.y;
    const int mine = (units - u0 + (int)gridDim.y - 1) / (int)gridDim.y;
    // a wave's pieces: (token, unit) pairs of this workgroup, one in kFusedWaves
    const int pieces = tokens * mine;
    auto unit_of = [&](int i) { return u0 + i % mine * (int)gridDim.y; };
    uint4 x[2][2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int i = wave + j * kFusedWaves;
        if (i < pieces) load_piece(a, t0 + i / mine, unit_of(i), x[j]);
    }
    for (int e = tid; e < 2 * E; e += kFusedThreads) s_before[e] = 0;
    __syncthreads();
    for (int base = tid; base < n; base += 8 * kFusedThreads) {
        int e[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) e[c] = base + c * kFusedThreads < n ? a.ids[base + c * kFusedThreads] : -1;
#pragma unroll
        for (int c = 0; c < 8; ++c)
            if (e[c] >= 0 && e[c] < E) atomicAdd(&smem[base + c * kFusedThreads < first ? e[c] : E + e[c]], 1);
    }
    __syncthreads();
    for (int e = tid; e < E; e += kFusedThreads) s_total[e] += s_before[e];
    __syncthreads();
    if (wave == 0) {
        group_starts(s_total, s_start, E, a.align);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "workgroup");
        for (int base = first; base < last; base += kWave) {
            const int i = base + lane, e = i < last ? a.ids[i] : -1;
            const bool held = e >= 0 && e < E;
            const uint64_t same = same_expert(e, held, E);
            const int below = __popcll(same & lanes_below());
            int row = -1;
            if (held) row = s_start[e] + s_before[e] + below;
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            if (held && below == 0) s_before[e] += __popcll(same);
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            if (row >= a.P) row = -1;
            if (i < last) {
                s_row[i - first] = row;
                if (u0 == 0) {
                    a.rows[i] = row;
                    if (row >= 0) a.slots[row] = i;
                }
            }
        }
    }
    __syncthreads();
    if (blockIdx.x == 0 && u0 == 0)
        for (int e = tid; e < E; e += kFusedThreads) a.offsets[e] = s_start[e + 1];

    for (int i = wave; i < pieces; i += 2 * kFusedWaves) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int at = i + j * kFusedWaves;
            if (at < pieces) put_piece(a, s_row + at / mine * k, unit_of(at), x[j]);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int at = i + (j + 2) * kFusedWaves;
            if (at < pieces) load_piece(a, t0 + at / mine, unit_of(at), x[j]);
        }
    }

    // rows without a slot: place r of every group, dealt out over all waves
    const int waves = gridDim.x * kFusedWaves, w = blockIdx.x * kFusedWaves + wave;
    const int places = E * a.align;
    const int64_t all = places + a.P - s_start[E];       // P may be near 2^31: 64 bits
    for (int64_t base = w; base < all; base += waves * kWave) {
        const int64_t i = base + lane * waves;
        int p = -1;
        if (i < places) {
            const int e = (int)i / a.align;
            p = s_start[e] + s_total[e] + (int)i - e * a.align;
            if (p >= s_start[e + 1]) p = -1;
        } else if (i < all) {
            p = (int)(s_start[E] + i - places);
        }
        for (uint64_t left = __ballot(p >= 0); left; left &= left - 1) {
            const int row = __shfl(p, __builtin_ctzll(left), kWave);
            if (u0 == 0 && lane == 0) a.slots[row] = -1;
            zero_row(a, row, u0, gridDim.y, units);
        }
    }
}

// Copy and cast by a known order: workgroups below `tokens` take one token each,
// so that x is read once however many experts a token has; the others take
// kZeroRows rows each and zero those without a slot (few rows a workgroup, since
// the rows past the last group come together). A row of more than 4096 columns
// has two pieces a wave, loaded together. 16640 tokens to 4 of 64 experts, 8192
// columns, 0.84 GB: 154 us, 5.5 TB/s.
constexpr int kZeroRows = 16;

template <int U>
__global__ __launch_bounds__(kDispatchThreads) void dispatch_kernel(DispatchArgs a, int tokens) {
    __shared__ int s_row[kWave];
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int units = (int)((a.D + kUnit - 1) / kUnit);
    const int64_t t = workgroup_xz();
    if (t < tokens) {
        if ((int)threadIdx.x < a.k) {
            const int p = a.rows[t * a.k + threadIdx.x];
            s_row[threadIdx.x] = p;
        }
        __syncthreads();
        for (int u = wave; u < units; u += U * kDispatchWaves) {
            uint4 x[U][2];
#pragma unroll
            for (int i = 0; i < U; ++i)
                if (u + i * kDispatchWaves < units) load_piece(a, t, u + i * kDispatchWaves, x[i]);
#pragma unroll
            for (int i = 0; i < U; ++i)
                if (u + i * kDispatchWaves < units) put_piece(a, s_row, u + i * kDispatchWaves, x[i]);
        }
    } else {
        const int64_t lo = (t - tokens) * kZeroRows + wave * (kZeroRows / kDispatchWaves), p = lo + lane;
        const int slot = lane < kZeroRows / kDispatchWaves && p < a.P ? a.slots[p] : 0;
        for (uint64_t left = __ballot(slot < 0); left; left &= left - 1)
            zero_row(a, lo + __builtin_ctzll(left), 0, 1, units);
    }
}

// y[t] over the columns of one workgroup; fp32 sums in slot order, one
// rounding to bf16. Rows of yp are read once and y is written once: neither is kept
// in the caches. 32771 tokens, 2 rows of 5120 columns each, 0.97 GB: 171 us back to
// back, 5.7 TB/s (plain stores: 198; 4096 tokens, 2 rows of 2048: 10.1 and 9.8).
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
        store_stream16(y + t * D + col, pack8(acc));
    }
}

// Workgroups (t, y) with t below T take the slots y, y + grid.y, ... of token t:
// dyp[rows[t, s]] = w[t, s] * dy[t] and dw[t, s] = <dy[t], yp[rows[t, s]]>; the
// others zero the rows without a slot. dy comes from the caches after its first
// reading; the dot products are fp32 sums in a fixed order. 16640 tokens, 4 rows
// of 4096 columns each, 1.22 GB: 216 us back to back, 5.6 TB/s (plain stores: 245).
__global__ __launch_bounds__(256) void combine_grad_kernel(
        const uint16_t* __restrict__ dy, const uint16_t* __restrict__ yp, int64_t P, int64_t D,
        const int32_t* __restrict__ rows, const int32_t* __restrict__ slots, int64_t T, int k,
        const float* __restrict__ weights, uint16_t* __restrict__ dyp, float* __restrict__ dw) {
    __shared__ float s_part[64][4];
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int64_t t = workgroup_xz();
    if (t >= T) {
        if (blockIdx.y > 0) return;
        const int64_t n = T * k, lo = (t - T) * kZeroRows + wave * (kZeroRows / 4), p = lo + lane;
        const bool mine = lane < kZeroRows / 4 && p < P;
        const int slot = mine ? slots[p] : 0;
        for (uint64_t left = __ballot(mine && (slot < 0 || slot >= n)); left; left &= left - 1) {
            uint16_t* row = dyp + (lo + __builtin_ctzll(left)) * D;
            for (int64_t col = lane * 8; col < D; col += 512)
                *reinterpret_cast<uint4*>(row + col) = make_uint4(0, 0, 0, 0);
        }
        return;
    }
    for (int s = blockIdx.y; s < k; s += gridDim.y) {
        const int64_t p = rows[t * k + s];
        float dot = 0.0f;
        if (p >= 0 && p < P) {
            const float w = weights[t * k + s];
            for (int64_t col = (int64_t)threadIdx.x * 8; col < D; col += 2048) {
                const uint4 g = *reinterpret_cast<const uint4*>(dy + t * D + col);
                dot = dot8(dot, g, load_stream(yp + p * D + col));
                float r[8] = {};
                add8(r, g, w);
                store_stream16(dyp + p * D + col, pack8(r));
            }
        }
        dot = wave_sum(dot);
        if (lane == 0) s_part[s][wave] = dot;
    }
    __syncthreads();
    const int s = blockIdx.y + threadIdx.x * gridDim.y;
    if (s < k) dw[t * k + s] = (s_part[s][0] + s_part[s][1]) + (s_part[s][2] + s_part[s][3]);
}

}  // namespace

hipError_t launch_dispatch(const DispatchArgs& a, int cus, hipStream_t stream) {
    const int64_t n = a.T * a.k, units = (a.D + kUnit - 1) / kUnit;
    const bool moves = a.xp || a.q;
    if (n <= kMoeFusedSlots) {
        // two workgroups a CU, and at least so many that a wave has about one row
        // to zero
        const int64_t per = a.T > 2 * cus ? (a.T + 2 * cus - 1) / (2 * cus) : 1, groups = (a.T + per - 1) / per;
        const int64_t spare = (a.P - n + kFusedWaves - 1) / kFusedWaves;
        int64_t blocks = spare < cus ? spare : cus;
        blocks = blocks > groups ? blocks : groups;
        blocks = blocks > 1 ? blocks : 1;
        const size_t shmem = (3 * (size_t)a.E + 1 + (size_t)(per * a.k)) * sizeof(int);
        int64_t split = cus / blocks;
        split = split > units ? units : split;
        hipLaunchKernelGGL(dispatch_fused_kernel, dim3((unsigned)blocks, (unsigned)(split > 1 ? split : 1)),
                           dim3(kFusedThreads), shmem, stream, a, (int)groups, (int)per);
        return hipGetLastError();
    }
    const int64_t runs = moe_runs(n), run = moe_run(n);
    hipLaunchKernelGGL(hist_kernel, dim3((unsigned)runs), dim3(1024), a.E * sizeof(int), stream, a.ids, n, run, a.E,
                       a.hist);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int waves = a.E > 512 ? 8 : 16;        // their counts take at most 32 KiB of LDS
    const size_t shmem = (2 * (size_t)a.E + 1 + (size_t)waves * a.E) * sizeof(int);
    if (waves == 8)
        hipLaunchKernelGGL(rank_kernel<8>, dim3((unsigned)runs), dim3(512), shmem, stream, a, run);
    else
        hipLaunchKernelGGL(rank_kernel<16>, dim3((unsigned)runs), dim3(1024), shmem, stream, a, run);
    e = hipGetLastError();
    if (e != hipSuccess || !moves) return e;
    const int64_t blocks = a.T + (a.P + kZeroRows - 1) / kZeroRows;
    if (units > kDispatchWaves)
        hipLaunchKernelGGL(dispatch_kernel<2>, grid_xz(blocks, 1), dim3(kDispatchThreads), 0, stream, a, (int)a.T);
    else
        hipLaunchKernelGGL(dispatch_kernel<1>, grid_xz(blocks, 1), dim3(kDispatchThreads), 0, stream, a, (int)a.T);
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
                               const float* weights, uint16_t* dyp, float* dw, int cus, hipStream_t stream) {
    const int64_t blocks = T + (P + kZeroRows - 1) / kZeroRows;
    if (blocks == 0) return hipSuccess;
    // few tokens: a workgroup for each slot instead of each token
    const int64_t split = T < 4 * (int64_t)cus ? k : 1;
    hipLaunchKernelGGL(combine_grad_kernel, grid_xz(blocks, (unsigned)split), dim3(256), 0, stream, dy, yp, P, D, rows,
                       slots, T, k, weights, dyp, dw);
    return hipGetLastError();
}

}  // namespace mgs
