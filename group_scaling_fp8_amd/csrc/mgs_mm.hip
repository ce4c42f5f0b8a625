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
//
// An instruction's K order is free as long as both operands use the same one,
// so a lane holds the 16-byte chunks g and g + 4 (g = lane / 16) of its row's
// 128 bytes.
#include "mgs_block128_device.hpp"
#include "mgs_experts.hpp"
#include "mgs_kernels.hpp"
#include "mgs_mm_form.hpp"

namespace mgs {

namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef __bf16 v2b __attribute__((ext_vector_type(2)));
typedef __bf16 v8b __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));

constexpr int kBK = 128;                     // bytes of the contraction a step
constexpr uint32_t kOutOfRange = 0x80000000u;   // an offset past every tile: the load gives zeros

struct MmArgs {
    const uint8_t* a;        // block128: (M, K); wgrad: (N, M)
    const float* a_scales;   // block128: (M, nkb); wgrad: (N, G)
    const uint8_t* b;        // block128: (E, N, K); wgrad: (K, M)
    const float* b_scales;   // block128: (E, nnb, nkb); wgrad: (K, G)
    const int32_t* offsets;  // group ends, or null (block128: one group of M rows)
    int64_t M, N, K;
    int64_t cols;            // columns of the output
    int G;
    int accumulate;
    void* out;
};

// One output tile: rows of operand A down, rows of operand B across.
struct Tile {
    v4i a, b;                // descriptors that start at the tile's first row
    int len;                 // bytes of the contraction
    int skip;                // leading bytes of it that belong to another group
    int steps;               // at least kMinSteps: the ones past len multiply zeros
    int m0, n0;              // block128: first row and column; wgrad: first n and k
    int row_end;             // rows past it are not stored
    int g;
    const float* scales;     // block128: of the first row, or of the columns, as the wave fetches
};

// Loads run two steps ahead of the sums, and block128's scales three, at most
// one tile on: so many steps a tile has at least.
template <bool WGRAD>
constexpr int kMinSteps = WGRAD ? 2 : 3;

// The buffer descriptor of the bytes from p + at to the end of an array of size
// bytes: base, size, raw 32-bit data. Loads past the end give zeros.
__device__ __forceinline__ v4i descriptor(const uint8_t* p, int64_t at, int64_t size) {
    const uint64_t base = reinterpret_cast<uint64_t>(p) + (uint64_t)at;
    return v4i{(int)base, (int)(base >> 32) & 0xFFFF, (int)min(size - at, (int64_t)0x7FFFFFFF), 0x00020000};
}

// 16 bytes a lane from the descriptor's base + off into lds + 16 * lane, without
// registers between. Written out because the compiler, which cannot tell the two
// buffers of a tile apart, otherwise waits for these loads before every read of
// the other one; load_wait() stands where the bytes are needed.
__device__ __forceinline__ void load16_lds(v4i rsrc, uint32_t off, uint32_t lds) {
#ifdef __HIP_DEVICE_COMPILE__
    // (the compiler does not see what the instruction reads: five wait states
    // stand for a descriptor that a vector instruction has just written)
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 3\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds"
                 :
                 : "v"(off), "s"(rsrc), "s"(lds)
                 : "memory");
#endif
}

// 4 bytes a lane, likewise, into lds + 4 * lane.
__device__ __forceinline__ void load4_lds(v4i rsrc, uint32_t off, uint32_t lds) {
#ifdef __HIP_DEVICE_COMPILE__
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 3\n\tbuffer_load_dword %0, %1, 0 offen lds"
                 :
                 : "v"(off), "s"(rsrc), "s"(lds)
                 : "memory");
#endif
}

// 16 bytes a lane to the descriptor's base + off, as output written once; with
// `add`, added to the four binary32 values there.
__device__ __forceinline__ void store16(v4i rsrc, uint32_t off, v4i v, bool add) {
#ifdef __HIP_DEVICE_COMPILE__
    typedef unsigned int v4u __attribute__((ext_vector_type(4)));
    const uint64_t base = (uint32_t)rsrc[0] | (uint64_t)(uint32_t)rsrc[1] << 32;
    const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(base), 0, rsrc[2], rsrc[3]);
    if (add) v = __builtin_bit_cast(v4i, __builtin_bit_cast(v4f, v) +
                                             __builtin_bit_cast(v4f, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0)));
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(v4u, v), r, off, 0, kLoadNontemporal);
#endif
}

// All of this wave's loads are done (vmcnt(0)).
__device__ __forceinline__ void load_wait() { __builtin_amdgcn_s_waitcnt(0x0f70); }

__device__ __forceinline__ uint32_t lds_address(const void* p) {
    return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void*)p;
}

// A tile's rows sit in LDS as 128-byte lines whose 16-byte chunks are permuted
// by the row (chunk c of a line stands at c ^ key), so that the eight rows that
// eight lanes read at one chunk fall on different banks: the key is the row
// modulo 8, or for B's rows of a bf16 output, which lanes read in runs of four
// out of eight, the row's bits 0, 1 and 3.

// A wave's share of the loads of one step's rows of 128 bytes into LDS, 16 bytes
// a lane straight from memory. Rows past the tile's last one are whatever follows
// in the array (the next group's rows, the next expert's weight: perhaps not
// numbers) and zeros past its end; a sum holds one row of A and one of B, and the
// output descriptor's size drops those of the surplus rows. Bytes outside the
// contraction are zero.
struct Loads {
    v4i src;
    uint32_t voff, step, lds;        // of the lane's first row, to the next load's, of the wave's first line
    bool inside;

    __device__ __forceinline__ Loads(v4i src, uint32_t voff, uint32_t step, int chunk, int kk, int len, int skip,
                                     uint32_t lds)
        : src(src), step(step), lds(lds) {
#ifdef __HIP_DEVICE_COMPILE__
        asm volatile("" : "+s"(kk));        // offsets are made here, not kept in registers for each kk
#endif
        const int at = kk + chunk * 16;
        inside = at < len && at >= skip;
        this->voff = voff + (uint32_t)kk;
    }
    template <int WAVES>
    __device__ __forceinline__ void start(int j) const {
        load16_lds(src, inside ? voff + j * step : kOutOfRange, lds + j * WAVES * 1024);
    }
};

// A lane's two chunks of the line at p.
__device__ __forceinline__ v8i fragment(const uint8_t* p, int lo, int hi) {
    return __builtin_shufflevector(*reinterpret_cast<const v4i*>(p + lo), *reinterpret_cast<const v4i*>(p + hi), 0, 1, 2,
                                   3, 4, 5, 6, 7);
}

// Eight E4M3 bytes as bf16.
__device__ __forceinline__ v8b widen(int lo, int hi) {
    v8b r;
#ifdef __HIP_DEVICE_COMPILE__
    const v2b a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
    const v2b b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
    const v2b c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
    const v2b d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
    r = v8b{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
#endif
    return r;
}

// A fragment as an instruction of the form takes it.
template <bool FAST>
struct Operand;

template <>
struct Operand<true> {
    v8i v;
    __device__ __forceinline__ Operand() {}
    __device__ __forceinline__ explicit Operand(v8i x) : v(x) {}
    // c[j] += a[j] b, instruction by instruction over the j
    template <int N>
    __device__ __forceinline__ static void mfma(const Operand (&a)[N], const Operand& b, v4f (&c)[N]) {
#pragma unroll
        for (int j = 0; j < N; ++j) mfma(a[j], b, c[j]);
    }
    __device__ __forceinline__ static void mfma(const Operand& a, const Operand& b, v4f& c) {
        c = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a.v, b.v, c, 0, 0, 0, 0, 0, 0);
    }
};

template <>
struct Operand<false> {
    v8b v[4];
    __device__ __forceinline__ Operand() {}
    __device__ __forceinline__ explicit Operand(v8i x) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = widen(x[2 * i], x[2 * i + 1]);
    }
    template <int N>
    __device__ __forceinline__ static void mfma(const Operand (&a)[N], const Operand& b, v4f (&c)[N]) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < N; ++j) c[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[j].v[i], b.v[i], c[j], 0, 0, 0);
    }
};

// A value that every lane holds, in scalar registers (tile addresses, so that a
// load's base is one scalar descriptor).
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int64_t uniform(int64_t v) {
    return (int64_t)(((uint64_t)(uint32_t)uniform((int)(v >> 32)) << 32) | (uint32_t)uniform((int)v));
}

// The groups as the casts read their ends (a running maximum, clamped to [0, M],
// rounded down to `align`; offsets null: one group of all rows), and the number
// of tiles of `rows` rows up to each. One wave writes them, 64 groups a turn.
struct Groups {
    int end[kMaxGroups];
    int upto[kMaxGroups];

    __device__ __forceinline__ void fill(const int32_t* offsets, int G, int M, int align, int rows) {
        const int lane = threadIdx.x & (kWave - 1);
        int carry = 0, tiles = 0;
        for (int g = lane; g - lane < G; g += kWave) {
            int raw = 0;
            if (g < G) raw = offsets ? min(max(offsets[g], 0), M) / align * align : M;
            const int e = max(wave_prefix_imax(raw), carry);
            int b = __shfl_up(e, 1, kWave);
            if (lane == 0) b = carry;
            const int u = tiles + wave_prefix_sum((e - b + rows - 1) / rows);
            if (g < G) {
                end[g] = e;
                upto[g] = u;
            }
            carry = __shfl(e, kWave - 1, kWave);
            tiles = __shfl(u, kWave - 1, kWave);
        }
    }
    // The first group with more than `tiles` row tiles up to it, or -1.
    __device__ __forceinline__ int find(int tiles, int G) const {
        const int lane = threadIdx.x & (kWave - 1);
        for (int base = 0; base < G; base += kWave) {
            const uint64_t past = __ballot(base + lane < G && upto[min(base + lane, G - 1)] > tiles);
            if (past) return base + __builtin_ctzll(past);
        }
        return -1;
    }
};

// Workgroups go to the eight XCDs in turn. Each XCD takes 32 consecutive tiles
// (one a CU), which share rows and columns in its L2, then the 32 that are eight
// such runs on: groups of unequal length spread over all XCDs. What is left of
// the last 256 is dealt out in eight equal runs.
__device__ __forceinline__ int tile_of(int b, int tiles) {
    const int whole = tiles & ~255, x = b & 7;
    if (b < whole) return (b & ~255) + x * 32 + ((b & 255) >> 3);
    const int left = tiles - whole;
    return whole + x * (left >> 3) + min(x, left & 7) + ((b - whole) >> 3);
}

// Tile `local` of rows x cols tiles, in bands of eight rows walked column by
// column: 32 consecutive tiles, the workgroups of one XCD at a time, are a patch
// of 8 x 4 that reads 12 distinct operand tiles (33 as a single column).
__device__ __forceinline__ void patch(int local, int rows, int cols, int& row, int& col) {
    const int band = local / (8 * cols);
    const int r = local - band * 8 * cols, high = min(8, rows - band * 8);
    col = r / high;
    row = band * 8 + r - col * high;
}

// Waits until at most `some` (not `none`) or no memory operations of this wave
// are outstanding. A branch that the compiler does not see keeps a step's body
// one block.
template <int SOME>
__device__ __forceinline__ void wait_some_or_none(int some) {
    static_assert(SOME < 64, "six bits");
#ifdef __HIP_DEVICE_COMPILE__
    // (a lane read needs a wait state after the instruction that wrote the lane)
    asm volatile("s_nop 1\n\tv_readfirstlane_b32 vcc_lo, %0\n\ts_cmp_eq_u32 vcc_lo, 0\n\ts_cbranch_scc1 0f\n\t"
                 "s_waitcnt vmcnt(%1)\n\ts_branch 1f\n0:\n\ts_waitcnt vmcnt(0)\n1:"
                 :
                 : "v"(some), "n"(SOME)
                 : "memory", "scc", "vcc");
#endif
}

// As many workgroups as the CUs hold at a time (one of 256 x 256 tiles, two of
// 128 x 128) walk tiles b, b + grid, ...: the first loads of a tile are issued
// before the stores of the one before it, which then drain under the tile's
// first steps. With PARTS > 1 a workgroup has one tile, whose steps are dealt
// out to as many sets of waves, each with buffers of its own; their sums are
// added in LDS at the end.
//
// What bounds it, by form (rates of dense products of 16384 x 8192 x 8192, MI355X;
// the library's plain products reach 3240 TFLOP/s in E4M3 and 1600 in bf16 at
// 16384^3, with the matrix cores busy 91% of the time):
//   256 x 256 fast    block128 2190 TFLOP/s, wgrad 2910. A step's 32 matrix
//                     instructions a wave, two waves a SIMD, take 2048 cycles;
//                     block128 adds 128 fmas a wave for the scaled sums, which
//                     stand in the gaps between them, and the eight waves read
//                     192 KiB of LDS in about 1500 cycles beside the 512 that the
//                     loads write. In a layer of ragged groups (32768 rows, 8192 x
//                     5120) the matrix cores are busy 49% of the time.
//   exact             block128 1110 TFLOP/s, wgrad 1590: the bf16 instructions
//                     take twice the cycles, and every wave widens the bytes of
//                     its fragments itself, which takes issue slots.
//   outputs           a tile's stores drain under one step of the next tile: from
//                     its second step on, each wait is for all that came before.
//                     Short contractions (eight steps a tile: wgrad of 16640 rows
//                     in 16 groups) pay for output and sums one after the other.
//   few tiles         latency: two steps' loads (64 KiB a CU) are in flight. 128 x
//                     128 tiles of 4096 rows in 16 groups by 4096 x 4096 take in 39
//                     KB/us a CU, with the matrix cores busy 26% of the time.
// (The clock falls as the matrix cores are used more: 1.9 to 2.0 GHz in the large
// products here, 1.5 to 1.6 under the library's.)
template <int BM, int BN, int WM, int WN, int PARTS, bool WGRAD, bool FAST, bool F32>
__global__ __launch_bounds__(BM / WM * (BN / WN) * 64 * PARTS, 2) void mm_kernel(MmArgs p) {
    constexpr int WAVES = BM / WM * (BN / WN);             // of one part
    constexpr int MT = WM / 16, NT = WN / 16;
    constexpr int LOADS = (BM + BN) / 8 / WAVES;           // a wave's loads a step
    constexpr int STORES = MT * NT / (F32 ? 1 : 2);        // a wave's stores of a whole tile
    static_assert(WN <= 128 && 128 % WN == 0, "a wave's columns share one scale block");
    __shared__ __align__(128) uint8_t s_all_a[PARTS][2][BM * kBK];
    __shared__ __align__(128) uint8_t s_all_b[PARTS][2][BN * kBK];
    // block128: a ring of four steps' reciprocal scales of the rows (the first BM
    // of each) and columns; wgrad: the scales of the last, this and the next
    // tile's rows and columns
    __shared__ __align__(16) float s_all_scale[PARTS][(WGRAD ? 3 : 4) * WAVES * 64];
    // block128: the scale each thread fetches, of two steps
    __shared__ float s_all_raw[PARTS][2][WGRAD ? 1 : WAVES * 64];
    __shared__ Groups s_groups;
    const int lane = threadIdx.x & (kWave - 1);
    const int part_of = PARTS > 1 ? uniform((int)(threadIdx.x / (WAVES * kWave))) : 0;
    const int tid = (int)threadIdx.x - part_of * (WAVES * kWave);
    const int wave = uniform(tid / kWave);
    uint8_t(*const s_a)[BM * kBK] = s_all_a[part_of];
    uint8_t(*const s_b)[BN * kBK] = s_all_b[part_of];
    float* const s_scale = s_all_scale[part_of];
    float(*const s_raw)[WGRAD ? 1 : WAVES * 64] = s_all_raw[part_of];
    const int wm = wave / (BN / WN) * WM, wn = wave % (BN / WN) * WN;
    const int64_t nkb = (p.K + kBK - 1) / kBK, nnb = (p.N + 127) / 128;
    const bool down = wave * 64 < BM;        // this wave fetches scales of rows, else of columns

    // ---- the tiles ----
    const int row_tiles = (int)((p.N + BM - 1) / BM);                            // wgrad: down one matrix
    const int col_tiles = (int)(((WGRAD ? p.K : p.N) + BN - 1) / BN);
    if (threadIdx.x < kWave) s_groups.fill(p.offsets, p.G, (int)p.M, WGRAD ? 16 : 1, BM);
    __syncthreads();
    auto end_of = [&](int g) { return g < 0 ? 0 : uniform(s_groups.end[g]); };
    int total;       // tiles; the host has checked that 32 bits hold them
    if constexpr (WGRAD) {
        total = p.G * row_tiles * col_tiles;
    } else {
        // the rows past the last group are one more group whose tiles are zeros
        total = (uniform(s_groups.upto[p.G - 1]) + ((int)p.M - end_of(p.G - 1) + BM - 1) / BM) * col_tiles;
    }
    auto tile = [&](int b) {
        const int L = tile_of(b, total);
        Tile t;
        int row, col;
        if constexpr (WGRAD) {
            const int per = row_tiles * col_tiles;
            t.g = uniform(L / per);
            patch(L - t.g * per, row_tiles, col_tiles, row, col);
            const int begin = end_of(t.g - 1), end = end_of(t.g);
            // steps start on 128-byte lines: a step across two lines of every
            // row takes twice as long to fetch
            const int from = (p.M & 127) == 0 ? begin & ~127 : begin;
            t.skip = begin - from;
            t.len = end > begin ? end - from : 0;
            t.m0 = uniform(row) * BM;
            t.n0 = uniform(col) * BN;
            t.row_end = (int)p.N;
            t.a = descriptor(p.a, t.m0 * p.M + from, p.N * p.M);
            t.b = descriptor(p.b, t.n0 * p.M + from, p.K * p.M);
            t.scales = nullptr;
        } else {
            // tiles are numbered by group, then in patches
            t.g = uniform(s_groups.find(uniform(L / col_tiles), p.G));
            const int last = t.g < 0 ? p.G - 1 : t.g - 1;      // the group before
            const int begin = end_of(last), end = t.g < 0 ? (int)p.M : end_of(t.g);
            const int first = last < 0 ? 0 : uniform(s_groups.upto[last]);
            patch(L - first * col_tiles, (end - begin + BM - 1) / BM, col_tiles, row, col);
            t.m0 = begin + uniform(row) * BM;
            t.n0 = uniform(col) * BN;
            t.row_end = end;
            t.skip = 0;
            t.len = t.g < 0 ? 0 : (int)p.K;
            const int64_t e = max(t.g, 0);
            t.a = descriptor(p.a, t.m0 * p.K, p.M * p.K);
            t.b = descriptor(p.b, (e * p.N + t.n0) * p.K, p.G * p.N * p.K);
            const int64_t block = min((int64_t)t.n0 / 128 + (wave - BM / 64) % (BN / 128), nnb - 1);
            t.scales = down ? p.a_scales + t.m0 * nkb : p.b_scales + (e * nnb + block) * nkb;
        }
        t.steps = max((t.len + kBK * PARTS - 1) / (kBK * PARTS), kMinSteps<WGRAD>);
        return t;
    };
    int b = blockIdx.x;
    if (b >= total) return;

    // ---- loads ----
    const int lrow = lane / 8;
    // lanes of one load instruction write 8 lines of 128 bytes in lane order;
    // lane l fetches the chunk that belongs at its place
    const int chunk_a = (lane & 7) ^ lrow;
    const int chunk_b = (lane & 7) ^ (F32 ? lrow : (lrow & 3) | (wave & 1) << 2);
    const uint32_t stride = (uint32_t)(WGRAD ? p.M : p.K);
    const uint32_t va = (wave * 8 + lrow) * stride + chunk_a * 16, vb = (wave * 8 + lrow) * stride + chunk_b * 16;
    const uint32_t lds_a = uniform((int)lds_address(s_a)), lds_b = uniform((int)lds_address(s_b));
    // step k of t, which is past its end where it is one of the next tile
    auto loads_a = [&](const Tile& t, const Tile& next, int k, int buf) {
        const bool over = k >= t.steps;
        const v4i a{over ? next.a[0] : t.a[0], over ? next.a[1] : t.a[1], over ? next.a[2] : t.a[2], t.a[3]};
        return Loads(a, va, WAVES * 8 * stride, chunk_a, ((over ? k - t.steps : k) * PARTS + part_of) * kBK,
                     over ? next.len : t.len, over ? next.skip : t.skip, lds_a + buf * (BM * kBK) + wave * 1024);
    };
    auto loads_b = [&](const Tile& t, const Tile& next, int k, int buf) {
        const bool over = k >= t.steps;
        const v4i b{over ? next.b[0] : t.b[0], over ? next.b[1] : t.b[1], over ? next.b[2] : t.b[2], t.b[3]};
        return Loads(b, vb, WAVES * 8 * stride, chunk_b, ((over ? k - t.steps : k) * PARTS + part_of) * kBK,
                     over ? next.len : t.len, over ? next.skip : t.skip, lds_b + buf * (BN * kBK) + wave * 1024);
    };
    auto start_loads = [&](const Tile& t, const Tile& next, int k, int buf) {
        const Loads a = loads_a(t, next, k, buf), b = loads_b(t, next, k, buf);
#pragma unroll
        for (int j = 0; j < BM / 8 / WAVES; ++j) a.template start<WAVES>(j);
#pragma unroll
        for (int j = 0; j < BN / 8 / WAVES; ++j) b.template start<WAVES>(j);
    };
    // block128: a thread fetches one scale, three steps ahead: the first BM of a
    // row, the waves behind them of a block of columns, one for all lanes. One
    // step ahead, when it has come, it puts the reciprocal into a ring of four
    // steps. wgrad: a thread fetches one scale of the next tile's rows and columns.
    // Like the tiles, the scales come by loads that the compiler does not wait for:
    // a wait for one of them alone would also be a wait for the stores before it.
    int ring = 0;            // steps of the tiles before this one
    const int nkb32 = (int)nkb;
    const int srow = WGRAD ? tid % (BM + BN) : tid % BM;
    const uint32_t lds_raw = uniform((int)lds_address(s_raw)) + wave * 256;
    const uint32_t lds_scale = uniform((int)lds_address(s_scale)) + wave * 256;
    const float *p_sa = p.a_scales, *p_sb = p.b_scales;
    const uint32_t scale_pitch = down ? (uint32_t)nkb : 0;
    auto scale_offset = [&](const Tile& t, const Tile& next, int k) {
        const int rows = (int)p.M - 1 - (k >= t.steps ? next.m0 : t.m0);
        return (uint32_t)min(srow, rows) * scale_pitch;
    };
    auto scales = [&](const Tile& t, const Tile& next, int k) {
        const bool over = k >= t.steps;
        return (over ? next.scales : t.scales) + min((over ? k - t.steps : k) * PARTS + part_of, nkb32 - 1);
    };
    auto start_scales = [&](const Tile& t, const Tile& next, int k) {
        const float* s = scales(t, next, k);
        load4_lds(descriptor(reinterpret_cast<const uint8_t*>(s), 0, 0x7FFFFFFF), scale_offset(t, next, k) * 4,
                  lds_raw + ((ring + k) & 1) * (WAVES * 256));
    };
    auto start_tile_scales = [&](const Tile& t, int third) {
        static_assert(!WGRAD || BM + BN <= WAVES * 64, "a thread fetches one scale");
        const int64_t first = down ? t.m0 : t.n0;
        const int at = min(down ? srow : srow - BM, (int)min((down ? p.N : p.K) - 1 - first, (int64_t)BM + BN));
        const float* s = (down ? p_sa : p_sb) + first * p.G + t.g;
        load4_lds(descriptor(reinterpret_cast<const uint8_t*>(s), 0, 0x7FFFFFFF), (uint32_t)at * (uint32_t)p.G * 4,
                  lds_scale + third * (WAVES * 256));
    };

    // ---- fragments ----
    const int fr = lane & 15, fg = lane / 16;
    // Lane row fr of B's fragment j is column col(j, fr) of the tile. For fp32
    // that is j * 16 + fr: a lane's four sums are 16 bytes. For bf16 it takes two
    // fragments to make 16 bytes: fragments 2h and 2h + 1 share out 32 columns,
    // four each in turn.
    const int a_at = (wm + fr) * kBK;
    const int b_at = (wn + (F32 ? fr : (fr >> 2) * 8 + (fr & 3))) * kBK;
    auto b_row = [](int j) { return F32 ? j * 16 : (j >> 1) * 32 + (j & 1) * 4; };
    const int lo = (fg ^ (fr & 7)) * 16, hi = ((fg + 4) ^ (fr & 7)) * 16;
    using Op = Operand<FAST>;

    Tile t = tile(b);
    if constexpr (WGRAD) {
        start_tile_scales(t, 0);
    } else {
        s_scale[tid] = 1.0f / scales(t, t, 0)[scale_offset(t, t, 0)];
        s_raw[1][tid] = scales(t, t, 1)[scale_offset(t, t, 0)];
        s_raw[0][tid] = scales(t, t, 2)[scale_offset(t, t, 0)];
    }
    start_loads(t, t, 0, 0);
    start_loads(t, t, 1, 1);
    wait_some_or_none<LOADS>(1);
    __syncthreads();
    // fa and fa1 hold the bytes of A's first two rows of fragments, ob B's
    // fragments; where registers allow it (kAhead), oa holds the first row already
    // as bf16 and fa the second row's bytes.
    constexpr bool kAhead = !FAST && MT <= 4;
    v8i fa = fragment(s_a[0] + a_at + (kAhead ? 16 * kBK : 0), lo, hi);
    v8i fa1 = {};
    if constexpr (!kAhead) fa1 = fragment(s_a[0] + a_at + 16 * kBK, lo, hi);
    Op oa, ob[NT];
    if constexpr (kAhead) oa = Op(fragment(s_a[0] + a_at, lo, hi));
#pragma unroll
    for (int j = 0; j < NT; ++j) ob[j] = Op(fragment(s_b[0] + b_at + b_row(j) * kBK, lo, hi));

    int third = 0;           // of s_scale: tiles walked modulo 3
    int drain = 0;           // whether a tile's stores (and nothing else) follow the loads of this tile's second step
    for (;;) {
    const bool more = b + (int)gridDim.x < total;
    Tile next = t;
    next.len = 0;            // after the last tile, loads bring zeros
    if (more) next = tile(b + gridDim.x);
    const int steps = t.steps;
    v4f acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = v4f{0, 0, 0, 0};
    float* const scale = s_scale + (WGRAD ? third * (WAVES * 64) : 0);
    if constexpr (WGRAD) start_tile_scales(next, third == 2 ? 0 : third + 1);
    // The scaled sums of a row's blocks are added while the next row's
    // instructions run.
    v4f part[NT];
    float part_scale = 0.0f;
#pragma unroll
    for (int j = 0; j < NT; ++j) part[j] = v4f{0, 0, 0, 0};
    auto promote = [&](int i, int j) {
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[i][j][c] = fmaf(part[j][c], part_scale, acc[i][j][c]);
    };
    // One step: the rows of fragments of A in turn, each read while the two
    // before it are multiplied. The barrier stands before the last two rows,
    // whose fragments are already in registers: behind it the other buffer is
    // complete and this one free, so the loads of the step after next and the
    // first fragments of the next step are on their way during the rest; at a
    // tile's end these are the next tile's. The body has no branch, which keeps
    // each row's sums next to its instructions.
#pragma clang loop unroll(disable)
    for (int k = 0; k < steps; ++k) {
        const int cur = (ring + k) & 1;
        const uint8_t *ta = s_a[cur] + a_at, *na = s_a[cur ^ 1] + a_at, *nb = s_b[cur ^ 1] + b_at;
        float sb_inv = 0.0f, raw = 0.0f;
        if constexpr (!WGRAD) {
            sb_inv = scale[((ring + k) & 3) * (WAVES * 64) + BM + wn / 128 * 64];
            raw = s_raw[(ring + k + 1) & 1][tid];
        }
        auto publish = [&] {
            if constexpr (!WGRAD) scale[((ring + k + 1) & 3) * (WAVES * 64) + tid] = 1.0f / raw;
        };
        // Row i of fragments. Between the instructions stand the additions of the
        // row before it and, exact, the conversions of the row after it.
        auto multiply = [&](int i, const Op& a) {
            if constexpr (WGRAD) {
                Op::mfma(ob, a, acc[i]);
            } else {
                const float f = scale[((ring + k) & 3) * (WAVES * 64) + wm + i * 16 + fr] * sb_inv;
                v4f now[NT];
#pragma unroll
                for (int j = 0; j < NT; ++j) now[j] = v4f{0, 0, 0, 0};
                Op::mfma(ob, a, now);
#pragma unroll
                for (int j = 0; j < NT; ++j) promote((i + MT - 1) % MT, j);
#pragma unroll
                for (int j = 0; j < NT; ++j) part[j] = now[j];
                part_scale = f;
            }
            // reads first: what they bring is waited for in the next row
            if constexpr (FAST) __builtin_amdgcn_sched_group_barrier(0x100, WGRAD ? 2 : 3, 0);
            if constexpr (!WGRAD || !FAST) {
#pragma unroll
                for (int j = 0; j < NT * (FAST ? 1 : 4); ++j) {
                    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                    __builtin_amdgcn_sched_group_barrier(0x002, FAST ? 5 : WGRAD ? 1 : 2, 0);
                }
            }
        };
        // Fast: the same with then(j) after each instruction.
        auto multiply_and = [&](int i, const Op& a, auto&& then) {
            float f = 0.0f;
            v4f now[NT];
            if constexpr (!WGRAD) f = scale[((ring + k) & 3) * (WAVES * 64) + wm + i * 16 + fr] * sb_inv;
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                if constexpr (WGRAD && FAST) {
                    Op::mfma(ob[j], a, acc[i][j]);
                } else if constexpr (FAST) {
                    now[j] = v4f{0, 0, 0, 0};
                    Op::mfma(ob[j], a, now[j]);
                    promote((i + MT - 1) % MT, j);
                }
                then(j);
                __builtin_amdgcn_sched_barrier(0);
            }
            if constexpr (!WGRAD) {
#pragma unroll
                for (int j = 0; j < NT; ++j) part[j] = now[j];
                part_scale = f;
            }
        };
        auto next_step = [&] {
            // the next step's bytes are in LDS
            wait_some_or_none<STORES + (WGRAD ? 1 : 0)>(k == 0 ? drain : 0);
            __syncthreads();
            if constexpr (!WGRAD) {
                start_scales(t, next, k + 3);
            }
            if constexpr (!FAST) start_loads(t, next, k + 2, cur);
        };
        if constexpr (!kAhead) {
#pragma unroll
            for (int i = 0; i < MT - 2; ++i) {
                const v8i ahead = fragment(ta + (i + 2) * 16 * kBK, lo, hi);
                if (i == 1) publish();
                multiply(i, Op(fa));
                fa = fa1;
                fa1 = ahead;
                __builtin_amdgcn_sched_barrier(0);
            }
            next_step();
            if constexpr (FAST) {
                // a load, or in the last row a load and the next step's fragment of
                // B, after each instruction: eight in a row would hold the wave up
                static_assert(NT == BM / 8 / WAVES && NT == BN / 8 / WAVES, "as many loads as instructions a row");
                const Loads a = loads_a(t, next, k + 2, cur);
                multiply_and(MT - 2, Op(fa), [&](int j) { a.template start<WAVES>(j); });
                fa = fragment(na, lo, hi);
                const Loads b = loads_b(t, next, k + 2, cur);
                multiply_and(MT - 1, Op(fa1), [&](int j) {
                    b.template start<WAVES>(j);
                    ob[j] = Op(fragment(nb + b_row(j) * kBK, lo, hi));
                });
                fa1 = fragment(na + 16 * kBK, lo, hi);
            } else {
                multiply(MT - 2, Op(fa));
                __builtin_amdgcn_sched_barrier(0);
                fa = fragment(na, lo, hi);
                multiply(MT - 1, Op(fa1));
#pragma unroll
                for (int j = 0; j < NT; ++j) ob[j] = Op(fragment(nb + b_row(j) * kBK, lo, hi));
                fa1 = fragment(na + 16 * kBK, lo, hi);
            }
        } else {
            // fa: bytes of the row after oa's
            v8i fb[NT];
#pragma unroll
            for (int i = 0; i < MT - 1; ++i) {
                const v8i ahead = i < MT - 2 ? fragment(ta + (i + 2) * 16 * kBK, lo, hi) : fragment(na, lo, hi);
                const Op after(fa);
                if (i == 1) publish();
                multiply(i, oa);
                oa = after;
                fa = ahead;
                __builtin_amdgcn_sched_barrier(0);
                if (i == MT - 3) next_step();
            }
#pragma unroll
            for (int j = 0; j < NT; ++j) fb[j] = fragment(nb + b_row(j) * kBK, lo, hi);
            const v8i ahead = fragment(na + 16 * kBK, lo, hi);
            const Op after(fa);
            multiply(MT - 1, oa);
#pragma unroll
            for (int j = 0; j < NT; ++j) ob[j] = Op(fb[j]);
            oa = after;
            fa = ahead;
        }
        __builtin_amdgcn_sched_barrier(0);
    }
    if constexpr (!WGRAD) {
#pragma unroll
        for (int j = 0; j < NT; ++j) promote(MT - 1, j);
    }
    if constexpr (PARTS > 1) {
        static_assert(PARTS == 2 && sizeof(s_all_b) >= sizeof(acc) * WAVES * 64, "the second part's sums");
        v4f* const sums = reinterpret_cast<v4f*>(s_all_b) + tid;
        load_wait();         // no load into the buffers is left, the last ones past the tile's end among them
        __syncthreads();
        if (part_of == 1) {
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int j = 0; j < NT; ++j) sums[(i * NT + j) * (WAVES * 64)] = acc[i][j];
        }
        __syncthreads();
        if (part_of == 1) return;
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j) acc[i][j] += sums[(i * NT + j) * (WAVES * 64)];
    }
    const bool empty = t.len == 0;
    if (empty) {             // whatever the scales of no rows are: here, and where wgrad scales below
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j) acc[i][j] = v4f{0, 0, 0, 0};
    }

    // ---- store: 16 bytes a lane, whole 128-byte lines by eight lanes ----
    // A lane has two pieces of 16 bytes of a line: the first of lanes fr + 8 and
    // the second of lanes fr change places, so that one store holds rows 0-7 of
    // sixteen and the other rows 8-15. Stores outside the output are dropped by
    // the descriptor's bounds, so every tile issues the same number of them.
    const uint32_t pitch = (uint32_t)p.cols * (F32 ? 4 : 2);
    const int64_t row0 = WGRAD ? t.g * p.N : 0;
    const v4i out = descriptor(static_cast<uint8_t*>(p.out), (row0 + t.m0) * pitch + t.n0 * (F32 ? 4 : 2),
                               (row0 + t.row_end) * pitch);
    uint32_t at[NT / (F32 ? 2 : 4)];
#pragma unroll
    for (int j = 0; j < NT / (F32 ? 2 : 4); ++j) {
        const int c = wn + (fg + (fr >> 3) * 4) * (F32 ? 4 : 8) + j * (F32 ? 32 : 64);
        at[j] = t.n0 + c < p.cols ? (wm + (fr & 7)) * pitch + c * (F32 ? 4 : 2) : kOutOfRange;
    }
    v4f ib[NT];
    if constexpr (WGRAD) {
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            ib[j] = *reinterpret_cast<const v4f*>(
                scale + BM + wn + (F32 ? j * 16 + fg * 4 : (j >> 1) * 32 + fg * 8 + (j & 1) * 4));
#pragma unroll
            for (int c = 0; c < 4; ++c) ib[j][c] = empty ? 0.0f : 1.0f / ib[j][c];
        }
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        if constexpr (WGRAD) {
            const float ia = empty ? 0.0f : 1.0f / scale[wm + fr + i * 16];
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int c = 0; c < 4; ++c) acc[i][j][c] = acc[i][j][c] * ia * ib[j][c];
        }
#pragma unroll
        for (int j = 0; j < NT / (F32 ? 2 : 4); ++j) {
            v4i v[2], w[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if constexpr (F32) {
                    v[h] = __builtin_bit_cast(v4i, acc[i][2 * j + h]);
                } else {
                    const v4f x = acc[i][4 * j + 2 * h], y = acc[i][4 * j + 2 * h + 1];
                    v[h] = v4i{(int)bf16x2(x[0], x[1]), (int)bf16x2(x[2], x[3]), (int)bf16x2(y[0], y[1]),
                               (int)bf16x2(y[2], y[3])};
                }
            }
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                // row_ror:8 into the upper, then the lower half of 16 lanes
                w[0][c] = __builtin_amdgcn_update_dpp(v[0][c], v[1][c], 0x128, 0xF, 0xC, false);
                w[1][c] = __builtin_amdgcn_update_dpp(v[1][c], v[0][c], 0x128, 0xF, 0x3, false);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) store16(out, at[j] + (i * 16 + h * 8) * pitch, w[h], WGRAD && F32 && p.accumulate);
        }
    }
    if (!more) break;
    t = next;
    b += gridDim.x;
    ring += steps;
    third = third == 2 ? 0 : third + 1;
    drain = p.accumulate ? 0 : 1;
    }
    load_wait();            // no load into LDS is left behind
}

// ---- few output rows, or few outputs of a long contraction -----------------------
//
// With a handful of rows the weights' bytes are block128's whole cost, and with a
// small weight wgrad has few tiles of a long contraction: a tile is BM rows by 32
// columns, and its eight waves take the contraction's blocks in turn (wave w: w,
// w + 8, ...), so that even one small product has enough loads in flight on every
// CU. Fragments come straight from memory, four lanes a line, the next block's
// while this one is multiplied; sums are exact (the matrix cores have nothing else
// to do). The waves' sums meet in LDS and are added in wave order. Bound by the
// loads: one row by 8192 x 8192 17 us, 4 TB/s.
constexpr int kFewWaves = 8;

// The 32 bytes at p + at of a row of len bytes (a multiple of 16, not 0), zeros
// past its end.
__device__ __forceinline__ v8i load32(const uint8_t* p, int64_t at, int64_t len) {
    const bool first = at < len, second = at + 16 < len;
    const v4i lo = *reinterpret_cast<const v4i*>(p + (first ? at : 0));
    const v4i hi = *reinterpret_cast<const v4i*>(p + (second ? at + 16 : 0));
    const v4i zero = {};
    return __builtin_shufflevector(first ? lo : zero, second ? hi : zero, 0, 1, 2, 3, 4, 5, 6, 7);
}

template <int BM, bool WGRAD, bool F32>
__global__ __launch_bounds__(kFewWaves * 64) void mm_few_kernel(MmArgs p) {
    constexpr int MT = BM / 16, NT = kFewCols / 16;
    __shared__ __align__(16) float s_sum[kFewWaves][BM][kFewCols + 4];
    const int lane = threadIdx.x & (kWave - 1), wave = uniform((int)(threadIdx.x / kWave));
    const int64_t nnb = (p.N + 127) / 128;
    const int col_tiles = (int)((p.cols + kFewCols - 1) / kFewCols), M = (int)p.M;

    // ---- which tile: every wave finds it, 64 groups at a time ----
    constexpr int kAlign = WGRAD ? 16 : 1;
    int carry = 0, tiles = 0;
    int e = 0, b = 0;                      // this lane's group
    auto group = [&](int g, int from) {
        int raw = 0;
        if (g < p.G) raw = p.offsets ? min(max(p.offsets[g], 0), M) / kAlign * kAlign : M;
        e = max(wave_prefix_imax(raw), from);
        b = __shfl_up(e, 1, kWave);
        if (lane == 0) b = from;
        return wave_prefix_sum((e - b + BM - 1) / BM);
    };
    int g = -1, begin, end;                // the group and its rows, wgrad: its part of the contraction
    int m0, n0;
    const int64_t wg = workgroup_xz();     // may pass the last tile
    if constexpr (WGRAD) {
        const int row_tiles = (int)((p.N + BM - 1) / BM), per = row_tiles * col_tiles;
        if (wg >= p.G * per) return;
        const int L = tile_of((int)wg, p.G * per);
        g = uniform(L / per);
        for (int base = 0; base <= g; base += kWave) {
            group(base + lane, carry);
            carry = uniform(__shfl(e, kWave - 1, kWave));
        }
        begin = uniform(__shfl(b, g % kWave, kWave));
        end = uniform(__shfl(e, g % kWave, kWave));
        m0 = uniform(L - g * per) % row_tiles * BM;
        n0 = uniform(L - g * per) / row_tiles * kFewCols;
    } else {
        int upto = 0;
        for (int base = 0; base < p.G; base += kWave) {
            upto = tiles + group(base + lane, carry);
            tiles = uniform(__shfl(upto, kWave - 1, kWave));
            carry = uniform(__shfl(e, kWave - 1, kWave));
        }
        const int last_end = carry, total = (tiles + (M - last_end + BM - 1) / BM) * col_tiles;
        if (wg >= total) return;
        const int L = tile_of((int)wg, total);
        int before = tiles;
        begin = last_end;
        end = M;
        if (L < tiles * col_tiles) {
            if (p.G > kWave) {
                carry = tiles = 0;
                for (int base = 0;; base += kWave) {
                    upto = tiles + group(base + lane, carry);
                    g = base;
                    const int now = uniform(__shfl(upto, kWave - 1, kWave));
                    if (L < now * col_tiles) break;
                    tiles = now;
                    carry = uniform(__shfl(e, kWave - 1, kWave));
                }
            } else {
                g = 0;
            }
            const int at = __builtin_ctzll(__ballot(upto * col_tiles > L));
            g = uniform(g + at);
            begin = uniform(__shfl(b, at, kWave));
            end = uniform(__shfl(e, at, kWave));
            before = uniform(__shfl(upto, at, kWave)) - (end - begin + BM - 1) / BM;
        }
        const int rows = (end - begin + BM - 1) / BM, local = L - before * col_tiles;
        m0 = begin + local % rows * BM;
        n0 = local / rows * kFewCols;
    }
    const int64_t row_end = WGRAD ? p.N : end;
    const int64_t stride = WGRAD ? p.M : p.K, len = WGRAD ? end - begin : p.K;
    const int nkb = (int)((len + kBK - 1) / kBK);

    // ---- the contraction ----
    const int fr = lane & 15, fg = lane / 16;
    v4f acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = v4f{0, 0, 0, 0};
    if (g >= 0 && len > 0) {
        const uint8_t *pa[MT], *pb[NT];
        const float *psa[MT], *psb = p.b_scales + (g * nnb + n0 / 128) * nkb;
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const int64_t r = min((int64_t)m0 + i * 16 + fr, row_end - 1);
            pa[i] = p.a + r * stride + (WGRAD ? begin : 0);
            psa[i] = p.a_scales + r * nkb;
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const int64_t r = min((int64_t)n0 + j * 16 + fr, p.cols - 1);
            pb[j] = WGRAD ? p.b + r * stride + begin : p.b + (g * p.N + r) * stride;
        }
        v8i fa[MT], fb[NT];
        float sa[MT], sb;
        auto fetch = [&](int k) {
            const int64_t at = (int64_t)k * kBK + fg * 32;
            auto get = [&](const uint8_t* q) { return load32(q, at, len); };
#pragma unroll
            for (int j = 0; j < NT; ++j) fb[j] = get(pb[j]);
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                fa[i] = get(pa[i]);
                if constexpr (!WGRAD) sa[i] = psa[i][k];
            }
            if constexpr (!WGRAD) sb = psb[k];
        };
        if (wave < nkb) fetch(wave);
        for (int k = wave; k < nkb; k += kFewWaves) {
            v8i na[MT], nb[NT];
            float f[MT];
#pragma unroll
            for (int j = 0; j < NT; ++j) nb[j] = fb[j];
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                na[i] = fa[i];
                if constexpr (!WGRAD) f[i] = (1.0f / sa[i]) * (1.0f / sb);
            }
            if (k + kFewWaves < nkb) fetch(k + kFewWaves);
            using Op = Operand<false>;
            Op ob[NT];
#pragma unroll
            for (int j = 0; j < NT; ++j) ob[j] = Op(nb[j]);
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                if constexpr (WGRAD) {
                    Op::mfma(ob, Op(na[i]), acc[i]);
                    continue;
                }
                v4f part[NT] = {};
                Op::mfma(ob, Op(na[i]), part);
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int c = 0; c < 4; ++c) acc[i][j][c] = fmaf(part[j][c], f[i], acc[i][j][c]);
            }
        }
    }

    // ---- join and store ----
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
            *reinterpret_cast<v4f*>(&s_sum[wave][i * 16 + fr][j * 16 + fg * 4]) = acc[i][j];
    __syncthreads();
    for (int x = threadIdx.x; x < BM * kFewCols / 4; x += kFewWaves * 64) {
        const int r = x / (kFewCols / 4), c = x % (kFewCols / 4) * 4;
        if (m0 + r >= row_end || n0 + c >= p.cols) continue;
        v4f v = *reinterpret_cast<const v4f*>(&s_sum[0][r][c]);
#pragma unroll
        for (int w = 1; w < kFewWaves; ++w) v += *reinterpret_cast<const v4f*>(&s_sum[w][r][c]);
        int64_t at = (int64_t)(m0 + r) * p.cols + n0 + c;
        if constexpr (WGRAD) {
            at += g * p.N * p.cols;
            if (len > 0) {
                const float ia = 1.0f / p.a_scales[(int64_t)(m0 + r) * p.G + g];
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = v[i] * ia * (1.0f / p.b_scales[(int64_t)(n0 + c + i) * p.G + g]);
            }
            if (F32 && p.accumulate) v += *reinterpret_cast<const v4f*>(static_cast<const float*>(p.out) + at);
        }
        if constexpr (F32)
            *reinterpret_cast<v4f*>(static_cast<float*>(p.out) + at) = v;
        else
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at) =
                make_uint2(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]));
    }
}

template <int BM, bool WGRAD>
hipError_t launch_few(const MmArgs& p, bool f32, hipStream_t stream) {
    const int64_t groups = p.offsets ? p.G + 1 : 1, spare = groups < p.M ? groups : p.M;
    const int64_t down = WGRAD ? p.G * ((p.N + BM - 1) / BM) : (p.M + spare * (BM - 1)) / BM;
    const int64_t blocks = down * ((p.cols + kFewCols - 1) / kFewCols);
    if (blocks > INT32_MAX) return hipErrorInvalidValue;
    if (f32)
        hipLaunchKernelGGL((mm_few_kernel<BM, WGRAD, true>), grid_xz(blocks), dim3(kFewWaves * 64), 0, stream, p);
    else
        hipLaunchKernelGGL((mm_few_kernel<BM, WGRAD, false>), grid_xz(blocks), dim3(kFewWaves * 64), 0, stream, p);
    return hipGetLastError();
}

template <int BM, int BN, int WM, int WN, int PARTS, bool WGRAD, bool FAST>
hipError_t launch(const MmArgs& p, bool f32, int cus, hipStream_t stream) {
    constexpr int threads = BM / WM * (BN / WN) * 64 * PARTS;
    constexpr int per_cu = 512 / threads;        // workgroups of at most 256 registers a lane
    // block128: every group, and the rows past the last one, may end inside a tile
    const int64_t down = WGRAD ? p.G * ((p.N + BM - 1) / BM) : p.M / BM + (p.offsets ? p.G + 1 : 1);
    const int64_t tiles = down * ((p.cols + BN - 1) / BN);
    if (tiles > INT32_MAX) return hipErrorInvalidValue;
    const int64_t blocks = PARTS > 1 || tiles < cus * per_cu ? tiles : cus * per_cu;
    if (f32)
        hipLaunchKernelGGL((mm_kernel<BM, BN, WM, WN, PARTS, WGRAD, FAST, true>), dim3((unsigned)blocks), dim3(threads), 0,
                           stream, p);
    else
        hipLaunchKernelGGL((mm_kernel<BM, BN, WM, WN, PARTS, WGRAD, FAST, false>), dim3((unsigned)blocks), dim3(threads), 0,
                           stream, p);
    return hipGetLastError();
}

template <bool WGRAD, bool FAST>
hipError_t launch_sized(const MmArgs& p, bool f32, int cus, hipStream_t stream) {
    const MmForm form = mm_form(WGRAD, FAST, p.offsets != nullptr, p.M, p.N, p.K, p.G, cus);
    if (form.few == 16) return launch_few<16, WGRAD>(p, f32, stream);
    if (form.few == 32) return launch_few<32, WGRAD>(p, f32, stream);
    if (form.few == 64) return launch_few<64, WGRAD>(p, f32, stream);
    if constexpr (WGRAD || FAST) {
        if (form.tile == 256) return launch<256, 256, 128, 64, 1, WGRAD, FAST>(p, f32, cus, stream);
        if (form.sets == 2) return launch<128, 128, 64, 64, 2, WGRAD, FAST>(p, f32, cus, stream);
    }
    return launch<128, 128, 64, 64, 1, WGRAD, FAST>(p, f32, cus, stream);
}

}  // namespace

hipError_t launch_mm_block128(const uint8_t* a, const float* a_scales, int64_t M, int64_t K, const uint8_t* b,
                              const float* b_scales, int64_t E, int64_t N, const int32_t* offsets, bool fast,
                              bool f32, void* y, int cus, hipStream_t stream) {
    if (K == 0) return launch_zero(y, (size_t)M * N * (f32 ? 4 : 2), stream);
    const MmArgs p{a, a_scales, b, b_scales, offsets, M, N, K, N, (int)E, 0, y};
    return fast ? launch_sized<false, true>(p, f32, cus, stream) : launch_sized<false, false>(p, f32, cus, stream);
}

hipError_t launch_mm_wgrad(const uint8_t* a_t, const float* a_scales_t, const uint8_t* b_t,
                           const float* b_scales_t, int64_t M, int64_t N, int64_t K, const int32_t* offsets,
                           int64_t G, bool fast, bool f32, bool accumulate, void* dw, int cus, hipStream_t stream) {
    const MmArgs p{a_t, a_scales_t, b_t, b_scales_t, offsets, M, N, K, K, (int)G, accumulate ? 1 : 0, dw};
    return fast ? launch_sized<true, true>(p, f32, cus, stream) : launch_sized<true, false>(p, f32, cus, stream);
}

}  // namespace mgs
