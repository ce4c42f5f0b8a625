// mgs_mm_tile.hpp — tiles of products on the matrix cores, and the forms that a
// product takes (internal; included by the files of the products).
//
// Every product contracts the contiguous dim of two row-major operands of 8-bit
// values; what the operands are and what is done with the sums is a Kind. What
// each product computes stands in the file that launches it.
//
// An instruction's K order is free as long as both operands use the same one,
// so a lane holds the 16-byte chunks g and g + 4 (g = lane / 16) of its row's
// 128 bytes.
#pragma once

#include "mgs_activation.hpp"
#include "mgs_block128_device.hpp"
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
    const uint8_t* a;        // rows: (M, K); wgrad: (N, M)
    const float* a_scales;   // rows: (M, nkb), 8-bit integers (M); wgrad: (N, G)
    const uint8_t* b;        // rows: (E, N, K), gated (2 E, N, K); wgrad: (K, M)
    const float* b_scales;   // rows: (E, nnb, nkb), 8-bit integers (E, N); wgrad: (K, G)
    const int32_t* offsets;  // group ends, or null (rows: one group of M rows)
    int64_t M, N, K;
    int64_t cols;            // columns of the output
    int G;
    int accumulate;
    void* out;
    const uint16_t* gu;      // gradient: (M, 2 N), both projections
    void* more;              // gated: gu (M, 2 N), gradient: h (M, N); stored where Kind::more
    Activation act;
};

// What a product is of: rows of each group with the group's weight, or wgrad;
// rows with the epilogues of a gated pair of projections or of their gradient.
enum class Job { Rows, Wgrad, Gated, Grad };
// How its sums are formed.
enum class Num { Exact, Fast, Int8 };

template <Job JOB, Num NUM, bool F32, bool MORE = false>
struct Kind {
    static constexpr bool wgrad = JOB == Job::Wgrad, gated = JOB == Job::Gated, grad = JOB == Job::Grad;
    static constexpr Num num = NUM;
    static constexpr bool eight = NUM != Num::Exact;                // the instruction reads the bytes themselves
    static constexpr bool scaled = !wgrad && NUM != Num::Int8;      // every block of 128 has scales of its own
    static constexpr bool f32 = F32, more = MORE;
    // The form for few rows: with the matrix cores idle, block128 and wgrad sum exactly. The
    // gated pair and its gradient take the faster sums where the caller allows them, which
    // widen nothing (us, fast and exact: pair of 4 tokens to 2 of 16 experts, 2 x 8192 x 5120,
    // 131 and 133, one row 16.1 and 16.8, 500 rows by 2 x 1024 x 2048 16.8 and 19.5; gradient of
    // 256 rows, 2048 x 4096, 17.0 and 17.7). Rounded to bf16 both are equally far from the exact result.
    using few = Kind<JOB, NUM == Num::Fast && !gated && !grad ? Num::Exact : NUM, F32, MORE>;
    static constexpr bool halves = gated || grad || NUM == Num::Int8;    // which 16 bytes of a line a lane takes (few rows)
};

// One output tile: rows of operand A down, rows of operand B across.
struct Tile {
    v4i a, b;                // descriptors that start at the tile's first row
    int len;                 // bytes of the contraction
    int skip;                // leading bytes of it that belong to another group
    int steps;               // at least kMinSteps: the ones past len multiply zeros
    int m0, n0;              // rows: first row and column; wgrad: first n and k
    int row_end;             // rows past it are not stored
    int g;
    const float* scales;     // blocks: of the first row, or of the columns, as the wave fetches
};

// Loads run two steps ahead of the sums, and the scales of blocks three, at most
// one tile on: so many steps a tile has at least.
template <bool SCALED>
constexpr int kMinSteps = SCALED ? 3 : 2;

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

// 16 bytes a lane to the descriptor's base + off, as output written once or, in
// halves of lines, through L2 (POLICY 0); with `add`, added to the four binary32
// values there.
template <int POLICY = kLoadNontemporal>
__device__ __forceinline__ void store16(v4i rsrc, uint32_t off, v4i v, bool add) {
#ifdef __HIP_DEVICE_COMPILE__
    typedef unsigned int v4u __attribute__((ext_vector_type(4)));
    const uint64_t base = (uint32_t)rsrc[0] | (uint64_t)(uint32_t)rsrc[1] << 32;
    const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(base), 0, rsrc[2], rsrc[3]);
    if (add) v = __builtin_bit_cast(v4i, __builtin_bit_cast(v4f, v) +
                                             __builtin_bit_cast(v4f, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0)));
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(v4u, v), r, off, 0, POLICY);
#endif
}

// 16 bytes a lane from the descriptor's base + off; past its end zeros.
__device__ __forceinline__ v4i load16(v4i rsrc, uint32_t off) {
    v4i v = {};
#ifdef __HIP_DEVICE_COMPILE__
    const uint64_t base = (uint32_t)rsrc[0] | (uint64_t)(uint32_t)rsrc[1] << 32;
    const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(base), 0, rsrc[2], rsrc[3]);
    v = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, kLoadNontemporal));
#endif
    return v;
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
    // Of a gated tile's weights (mm_kernel).
    template <int WAVES>
    __device__ __forceinline__ void start_gated(int j) const {
        static_assert(WAVES == 8 || WAVES == 4, "the waves of a tile");
        load16_lds(src, inside ? voff + j * step : kOutOfRange,
                   lds + (WAVES == 8 ? j * 8192 : (j >> 1) * 8192 + (j & 1) * 2048));
    }
};

// A lane's two chunks of the line at p.
__device__ __forceinline__ v8i fragment(const uint8_t* p, int lo, int hi) {
    return __builtin_shufflevector(*reinterpret_cast<const v4i*>(p + lo), *reinterpret_cast<const v4i*>(p + hi), 0, 1, 2,
                                   3, 4, 5, 6, 7);
}

// Eight E4M3 bytes as bf16.
__device__ __forceinline__ v8b widen(int lo, int hi) {
    v8b r = {};
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
template <Num NUM>
struct Operand;

template <>
struct Operand<Num::Fast> {
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
struct Operand<Num::Int8> {
    v8i v;
    __device__ __forceinline__ Operand() {}
    __device__ __forceinline__ explicit Operand(v8i x) : v(x) {}
    template <int N>
    __device__ __forceinline__ static void mfma(const Operand (&a)[N], const Operand& b, v4i (&c)[N]) {
#pragma unroll
        for (int j = 0; j < N; ++j) mfma(a[j], b, c[j]);
    }
    __device__ __forceinline__ static void mfma(const Operand& a, const Operand& b, v4i& c) {
        c = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_shufflevector(a.v, a.v, 0, 1, 2, 3),
                                                  __builtin_shufflevector(b.v, b.v, 0, 1, 2, 3), c, 0, 0, 0);
        c = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_shufflevector(a.v, a.v, 4, 5, 6, 7),
                                                  __builtin_shufflevector(b.v, b.v, 4, 5, 6, 7), c, 0, 0, 0);
    }
};

template <>
struct Operand<Num::Exact> {
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

// The type of a product's sums.
template <bool INT8>
struct Sum {
    typedef v4f type;
};
template <>
struct Sum<true> {
    typedef v4i type;
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
            const int u = tiles + wave_prefix_sum(tiles_down(e - b, rows));
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
//   few tiles         128 x 128 tiles of 4096 rows in 16 groups by 4096 x 4096 take in
//                     39 KB/us a CU, with the matrix cores busy 26% of the time. Where
//                     a CU has one workgroup, a wave a SIMD waits for its own reads of
//                     LDS: 256 x 4096 x 4096 in integers takes 25.7 us, 24.9 with the
//                     loads from memory left out, and deeper buffers (four steps) gain
//                     nothing.
//   epilogues         of a gated pair and its gradient: mgs_gated.hip.
// (The clock falls as the matrix cores are used more: 1.9 to 2.0 GHz in the large
// products here, 1.5 to 1.6 under the library's.)
template <int BM, int BN, int WM, int WN, int PARTS, class KIND>
__global__ __launch_bounds__(BM / WM * (BN / WN) * 64 * PARTS, 2) void mm_kernel(MmArgs p) {
    constexpr bool WGRAD = KIND::wgrad, GATED = KIND::gated, GRAD = KIND::grad, MORE = KIND::more;
    constexpr bool FAST = KIND::eight, SCALED = KIND::scaled, F32 = KIND::f32, INT8 = KIND::num == Num::Int8;
    constexpr int WAVES = BM / WM * (BN / WN);             // of one part
    constexpr int MT = WM / 16, NT = WN / 16;
    constexpr int LOADS = (BM + BN) / 8 / WAVES;           // a wave's loads a step
    // a wave's stores of a whole tile
    constexpr int STORES = GATED ? MT * (MORE ? 3 : 1) : GRAD ? MT * NT / 2 * (MORE ? 3 : 2) : MT * NT / (F32 ? 1 : 2);
    constexpr int COLS = GATED ? BN / 2 : BN;              // a tile's columns of the output
    static_assert(WN <= 128 && 128 % WN == 0, "a wave's columns share one scale block");
    static_assert(!(GATED || GRAD) || (!F32 && NT == 4), "epilogues of bf16 outputs, in pairs of fragments");
    using Acc = typename Sum<INT8>::type;
    __shared__ __align__(128) uint8_t s_all_a[PARTS][2][BM * kBK];
    __shared__ __align__(128) uint8_t s_all_b[PARTS][2][BN * kBK];
    // blocks: a ring of four steps' reciprocal scales of the rows (the first BM
    // of each) and columns; else the scales of the last, this and the next
    // tile's rows and columns
    __shared__ __align__(16) float s_all_scale[PARTS][(SCALED ? 4 : 3) * WAVES * 64];
    // blocks: the scale each thread fetches, of two steps
    __shared__ float s_all_raw[PARTS][2][SCALED ? WAVES * 64 : 1];
    __shared__ Groups s_groups;
    const int lane = threadIdx.x & (kWave - 1);
    const int part_of = PARTS > 1 ? uniform((int)(threadIdx.x / (WAVES * kWave))) : 0;
    const int tid = (int)threadIdx.x - part_of * (WAVES * kWave);
    const int wave = uniform(tid / kWave);
    uint8_t(*const s_a)[BM * kBK] = s_all_a[part_of];
    uint8_t(*const s_b)[BN * kBK] = s_all_b[part_of];
    float* const s_scale = s_all_scale[part_of];
    float(*const s_raw)[SCALED ? WAVES * 64 : 1] = s_all_raw[part_of];
    const int wm = wave / (BN / WN) * WM, wn = wave % (BN / WN) * WN;
    const int64_t nkb = (p.K + kBK - 1) / kBK, nnb = (p.N + 127) / 128;
    const bool down = wave * 64 < BM;        // this wave fetches scales of rows, else of columns

    // ---- the tiles ----
    const int row_tiles = (int)((p.N + BM - 1) / BM);                            // wgrad: down one matrix
    const int col_tiles = (int)(((WGRAD ? p.K : p.N) + COLS - 1) / COLS);
    if (threadIdx.x < kWave) s_groups.fill(p.offsets, p.G, (int)p.M, WGRAD ? 16 : 1, BM);
    __syncthreads();
    auto end_of = [&](int g) { return g < 0 ? 0 : uniform(s_groups.end[g]); };
    int total;       // tiles; the host has checked that 32 bits hold them
    if constexpr (WGRAD) {
        total = p.G * row_tiles * col_tiles;
    } else {
        // the rows past the last group are one more group whose tiles are zeros
        total = (uniform(s_groups.upto[p.G - 1]) + tiles_down((int)p.M - end_of(p.G - 1), BM)) * col_tiles;
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
            patch(L - first * col_tiles, tiles_down(end - begin, BM), col_tiles, row, col);
            t.m0 = begin + uniform(row) * BM;
            t.n0 = uniform(col) * COLS;
            t.row_end = end;
            t.skip = 0;
            t.len = t.g < 0 ? 0 : (int)p.K;
            const int64_t e = max(t.g, 0);
            t.a = descriptor(p.a, t.m0 * p.K, p.M * p.K);
            if constexpr (GATED) {
                // the lower half of the waves loads the gate's rows, the upper half the other projection's
                const int64_t w = 2 * e + (wave >= WAVES / 2 ? 1 : 0);
                t.b = descriptor(p.b, (w * p.N + t.n0) * p.K, 2 * p.G * p.N * p.K);
            } else {
                t.b = descriptor(p.b, (e * p.N + t.n0) * p.K, p.G * p.N * p.K);
            }
            if constexpr (SCALED) {
                const int at = wave - BM / 64;
                const int64_t block = min((int64_t)t.n0 / 128 + (GATED ? 0 : at % (BN / 128)), nnb - 1);
                const int64_t w = GATED ? 2 * e + (at & 1) : e;
                t.scales = down ? p.a_scales + t.m0 * nkb : p.b_scales + (w * nnb + block) * nkb;
            } else {
                t.scales = down ? p.a_scales + t.m0 : p.b_scales + (GATED ? 2 : 1) * e * p.N + t.n0;
            }
        }
        t.steps = max((t.len + kBK * PARTS - 1) / (kBK * PARTS), kMinSteps<SCALED>);
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
    // Gated: of 64 lines of B, one wave's columns, the first 32 are the gate's rows
    // and the others the same rows of the other projection, so that a lane's sums
    // hold both of a column. A wave loads eight lines of one of them at a time,
    // every WAVES * 4th row: with eight waves into every 64 lines in turn, with
    // four twice into each.
    const int wave_b = GATED ? wave % (WAVES / 2) : wave;
    const uint32_t va = (wave * 8 + lrow) * stride + chunk_a * 16, vb = (wave_b * 8 + lrow) * stride + chunk_b * 16;
    const uint32_t step_b = WAVES * (GATED ? 4 : 8) * stride;
    const uint32_t lds_a = uniform((int)lds_address(s_a)), lds_b = uniform((int)lds_address(s_b));
    const uint32_t lines_b = (GATED ? wave_b + (wave >= WAVES / 2 ? 4 : 0) : wave) * 1024;
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
        return Loads(b, vb, step_b, chunk_b, ((over ? k - t.steps : k) * PARTS + part_of) * kBK,
                     over ? next.len : t.len, over ? next.skip : t.skip, lds_b + buf * (BN * kBK) + lines_b);
    };
    auto start_b = [&](const Loads& b, int j) {
        if constexpr (GATED)
            b.template start_gated<WAVES>(j);
        else
            b.template start<WAVES>(j);
    };
    auto start_loads = [&](const Tile& t, const Tile& next, int k, int buf) {
        const Loads a = loads_a(t, next, k, buf), b = loads_b(t, next, k, buf);
#pragma unroll
        for (int j = 0; j < BM / 8 / WAVES; ++j) a.template start<WAVES>(j);
#pragma unroll
        for (int j = 0; j < BN / 8 / WAVES; ++j) start_b(b, j);
    };
    // Blocks: a thread fetches one scale, three steps ahead: the first BM of a
    // row, the waves behind them of a block of columns, one for all lanes. One
    // step ahead, when it has come, it puts the reciprocal into a ring of four
    // steps. Else a thread fetches one scale of the next tile's rows and columns.
    // Like the tiles, the scales come by loads that the compiler does not wait for:
    // a wait for one of them alone would also be a wait for the stores before it.
    int ring = 0;            // steps of the tiles before this one
    const int nkb32 = (int)nkb;
    const int srow = SCALED ? tid % BM : tid % (BM + BN);
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
        static_assert(SCALED || BM + BN <= WAVES * 64, "a thread fetches one scale");
        if constexpr (!WGRAD) {
            const int r = srow - BM;         // a line of B
            const int col = GATED ? (r >> 6) * 32 + (r & 31) : r;
            int at = down ? min(srow, (int)p.M - 1 - t.m0) : min(col, (int)p.N - 1 - t.n0);
            if (GATED && !down) at += (r >> 5 & 1) * (int)p.N;
            load4_lds(descriptor(reinterpret_cast<const uint8_t*>(t.scales), 0, 0x7FFFFFFF), (uint32_t)at * 4,
                      lds_scale + third * (WAVES * 256));
            return;
        }
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
    using Op = Operand<KIND::num>;

    Tile t = tile(b);
    if constexpr (!SCALED) {
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
    Acc acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = Acc{0, 0, 0, 0};
    float* const scale = s_scale + (SCALED ? 0 : third * (WAVES * 64));
    if constexpr (!SCALED) start_tile_scales(next, third == 2 ? 0 : third + 1);
    // The scaled sums of a row's blocks are added while the next row's
    // instructions run.
    v4f part[NT];
    float part_scale[GATED ? 2 : 1] = {};        // gated: of the gate's columns and of the other's
#pragma unroll
    for (int j = 0; j < NT; ++j) part[j] = v4f{0, 0, 0, 0};
    auto promote = [&](int i, int j) {
        if constexpr (SCALED) {
#pragma unroll
            for (int c = 0; c < 4; ++c)
                acc[i][j][c] = fmaf(part[j][c], part_scale[GATED ? j / (NT / 2) : 0], acc[i][j][c]);
        }
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
        float sb_inv[GATED ? 2 : 1] = {}, raw = 0.0f;
        if constexpr (SCALED) {
            sb_inv[0] = scale[((ring + k) & 3) * (WAVES * 64) + BM + (GATED ? 0 : wn / 128 * 64)];
            if constexpr (GATED) sb_inv[1] = scale[((ring + k) & 3) * (WAVES * 64) + BM + 64];
            raw = s_raw[(ring + k + 1) & 1][tid];
        }
        auto publish = [&] {
            if constexpr (SCALED) scale[((ring + k + 1) & 3) * (WAVES * 64) + tid] = 1.0f / raw;
        };
        // Row i of fragments. Between the instructions stand the additions of the
        // row before it and, exact, the conversions of the row after it.
        auto multiply = [&](int i, const Op& a) {
            if constexpr (!SCALED) {
                Op::mfma(ob, a, acc[i]);
            } else {
                const float f = scale[((ring + k) & 3) * (WAVES * 64) + wm + i * 16 + fr];
                v4f now[NT];
#pragma unroll
                for (int j = 0; j < NT; ++j) now[j] = v4f{0, 0, 0, 0};
                Op::mfma(ob, a, now);
#pragma unroll
                for (int j = 0; j < NT; ++j) promote((i + MT - 1) % MT, j);
#pragma unroll
                for (int j = 0; j < NT; ++j) part[j] = now[j];
                part_scale[0] = f * sb_inv[0];
                if constexpr (GATED) part_scale[1] = f * sb_inv[1];
            }
            // reads first: what they bring is waited for in the next row
            if constexpr (FAST) __builtin_amdgcn_sched_group_barrier(0x100, SCALED ? 3 : 2, 0);
            if constexpr (SCALED || !FAST) {
#pragma unroll
                for (int j = 0; j < NT * (FAST ? 1 : 4); ++j) {
                    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                    __builtin_amdgcn_sched_group_barrier(0x002, FAST ? 5 : SCALED ? 2 : 1, 0);
                }
            }
        };
        // Fast: the same with then(j) after each instruction.
        auto multiply_and = [&](int i, const Op& a, auto&& then) {
            float f = 0.0f;
            v4f now[NT];
            if constexpr (SCALED) f = scale[((ring + k) & 3) * (WAVES * 64) + wm + i * 16 + fr];
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                if constexpr (!SCALED && FAST) {
                    Op::mfma(ob[j], a, acc[i][j]);
                } else if constexpr (FAST) {
                    now[j] = v4f{0, 0, 0, 0};
                    Op::mfma(ob[j], a, now[j]);
                    promote((i + MT - 1) % MT, j);
                }
                then(j);
                __builtin_amdgcn_sched_barrier(0);
            }
            if constexpr (SCALED) {
#pragma unroll
                for (int j = 0; j < NT; ++j) part[j] = now[j];
                part_scale[0] = f * sb_inv[0];
                if constexpr (GATED) part_scale[1] = f * sb_inv[1];
            }
        };
        auto next_step = [&] {
            // the next step's bytes are in LDS
            wait_some_or_none<STORES + (SCALED ? 0 : 1)>(k == 0 ? drain : 0);
            __syncthreads();
            if constexpr (SCALED) {
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
                    start_b(b, j);
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
    if constexpr (SCALED) {
#pragma unroll
        for (int j = 0; j < NT; ++j) promote(MT - 1, j);
    }
    if constexpr (PARTS > 1) {
        static_assert(PARTS == 2 && sizeof(s_all_b) >= sizeof(acc) * WAVES * 64, "the second part's sums");
        Acc* const sums = reinterpret_cast<Acc*>(s_all_b) + tid;
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
    if (empty) {             // whatever the scales of no rows are: here, and where a tile's are applied below
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j) acc[i][j] = Acc{0, 0, 0, 0};
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
    v4f ib[NT];
    if constexpr (!SCALED) {
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            ib[j] = *reinterpret_cast<const v4f*>(
                scale + BM + wn + (F32 ? j * 16 + fg * 4 : (j >> 1) * 32 + fg * 8 + (j & 1) * 4));
#pragma unroll
            for (int c = 0; c < 4; ++c) ib[j][c] = empty ? 0.0f : 1.0f / ib[j][c];
        }
    }
    // a row of fragments with the scales that are not in its sums yet
    auto scaled_row = [&](int i, v4f (&r)[NT]) {
#pragma unroll
        for (int j = 0; j < NT; ++j) r[j] = __builtin_convertvector(acc[i][j], v4f);
        if constexpr (!SCALED) {
            const float ia = empty ? 0.0f : 1.0f / scale[wm + fr + i * 16];
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int c = 0; c < 4; ++c) r[j][c] = r[j][c] * ia * ib[j][c];
        }
    };
    auto packed = [](const v4f& x, const v4f& y) {
        return v4i{(int)bf16x2(x[0], x[1]), (int)bf16x2(x[2], x[3]), (int)bf16x2(y[0], y[1]), (int)bf16x2(y[2], y[3])};
    };
    if constexpr (GATED) {
        // A lane holds eight columns of both projections: 16 bytes of each output. A
        // wave's 32 columns are half a line, whose other half the next wave stores: L2
        // joins them (16640 x 8192 x 5120 in 16 groups 1691 us, streaming stores 1758).
        const uint32_t pitch2 = pitch * 2;
        const int c = wn / 2 + fg * 8;
        const uint32_t inside = t.n0 + c < p.cols ? 0 : kOutOfRange;
        const uint32_t at = (wm + fr) * pitch + c * 2 + inside, at2 = (wm + fr) * pitch2 + c * 2 + inside;
        v4i kept = {};
        if constexpr (MORE)
            kept = descriptor(static_cast<uint8_t*>(p.more), t.m0 * (int64_t)pitch2 + t.n0 * 2, t.row_end * (int64_t)pitch2);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            v4f r[NT], h[2];
            scaled_row(i, r);
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) h[j][e] = p.act.of(r[j][e]) * r[j + 2][e];
            store16<0>(out, at + i * 16 * pitch, packed(h[0], h[1]), false);
            if constexpr (MORE) {
                store16<0>(kept, at2 + i * 16 * pitch2, packed(r[0], r[1]), false);
                store16<0>(kept, at2 + i * 16 * pitch2 + pitch, packed(r[2], r[3]), false);
            }
        }
    } else if constexpr (GRAD) {
        // 64 columns as they are stored below: the first piece of a lane is of rows
        // 0-7 of sixteen, the second of rows 8-15, so that eight lanes load and
        // store whole lines of both projections and of the outputs
        const uint32_t pitch2 = pitch * 2;
        const v4i gu = descriptor(reinterpret_cast<const uint8_t*>(p.gu), t.m0 * (int64_t)pitch2 + t.n0 * 2,
                                  p.M * (int64_t)pitch2);
        const v4i both = descriptor(static_cast<uint8_t*>(p.out), t.m0 * (int64_t)pitch2 + t.n0 * 2,
                                    t.row_end * (int64_t)pitch2);
        v4i hidden = {};
        if constexpr (MORE)
            hidden = descriptor(static_cast<uint8_t*>(p.more), t.m0 * (int64_t)pitch + t.n0 * 2,
                                t.row_end * (int64_t)pitch);
        const int c = wn + (fg + (fr >> 3) * 4) * 8;
        const uint32_t inside = t.n0 + c < p.cols ? 0 : kOutOfRange;
        const uint32_t at = (wm + (fr & 7)) * pitch + c * 2 + inside, at2 = (wm + (fr & 7)) * pitch2 + c * 2 + inside;
        v4i g[MT][2], u[MT][2];
        // rows down an output, made where they are used: the compiler would keep every row's offset in registers
        auto down = [](int rows, uint32_t pitch) {
#ifdef __HIP_DEVICE_COMPILE__
            asm volatile("" : "+s"(pitch));
#endif
            return rows * pitch;
        };
        auto fetch = [&](int i) {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const uint32_t off = at2 + down(i * 16 + q * 8, pitch2);
                g[i][q] = load16(gu, off);
                u[i][q] = load16(gu, off + pitch);
            }
            __builtin_amdgcn_sched_barrier(0);
        };
        fetch(0);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            v4f r[NT];
            scaled_row(i, r);
            float dh[2][8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int first = __float_as_int(r[e >> 2][e & 3]), second = __float_as_int(r[2 + (e >> 2)][e & 3]);
                dh[0][e] = __int_as_float(__builtin_amdgcn_update_dpp(first, second, 0x128, 0xF, 0xC, false));
                dh[1][e] = __int_as_float(__builtin_amdgcn_update_dpp(second, first, 0x128, 0xF, 0x3, false));
            }
            if (i + 1 < MT) fetch(i + 1);        // more rows ahead spill: two 1059 us, three 1196, one 1010
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                v4i dg, du, h;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const GatedGrad lo = p.act.grad(dh[q][2 * e], bf16_lo(g[i][q][e]), bf16_lo(u[i][q][e]));
                    const GatedGrad hi = p.act.grad(dh[q][2 * e + 1], bf16_hi(g[i][q][e]), bf16_hi(u[i][q][e]));
                    dg[e] = (int)bf16x2(lo.dg, hi.dg);
                    du[e] = (int)bf16x2(lo.du, hi.du);
                    h[e] = (int)bf16x2(lo.h, hi.h);
                }
                const v4i zero = {};             // rows of no group, whatever their projections are
                const uint32_t off = at2 + down(i * 16 + q * 8, pitch2);
                store16(both, off, empty ? zero : dg, false);
                store16(both, off + pitch, empty ? zero : du, false);
                if constexpr (MORE) store16(hidden, at + down(i * 16 + q * 8, pitch), empty ? zero : h, false);
            }
        }
    } else {
        uint32_t at[NT / (F32 ? 2 : 4)];
#pragma unroll
        for (int j = 0; j < NT / (F32 ? 2 : 4); ++j) {
            const int c = wn + (fg + (fr >> 3) * 4) * (F32 ? 4 : 8) + j * (F32 ? 32 : 64);
            at[j] = t.n0 + c < p.cols ? (wm + (fr & 7)) * pitch + c * (F32 ? 4 : 2) : kOutOfRange;
        }
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            v4f r[NT];
            scaled_row(i, r);
#pragma unroll
            for (int j = 0; j < NT / (F32 ? 2 : 4); ++j) {
                v4i v[2], w[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if constexpr (F32)
                        v[h] = __builtin_bit_cast(v4i, r[2 * j + h]);
                    else
                        v[h] = packed(r[4 * j + 2 * h], r[4 * j + 2 * h + 1]);
                }
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    // row_ror:8 into the upper, then the lower half of 16 lanes
                    w[0][c] = __builtin_amdgcn_update_dpp(v[0][c], v[1][c], 0x128, 0xF, 0xC, false);
                    w[1][c] = __builtin_amdgcn_update_dpp(v[1][c], v[0][c], 0x128, 0xF, 0x3, false);
                }
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    store16(out, at[j] + (i * 16 + h * 8) * pitch, w[h], WGRAD && F32 && p.accumulate);
            }
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
// With a handful of rows the weights' bytes are a product's whole cost, and with a
// small weight there are few tiles of a long contraction: a tile is BM rows by LINES
// rows of weights (gated: half of them of each projection), and its eight waves take
// the contraction's blocks in turn (wave w: w, w + 8, ...), so that even one small
// product has enough loads in flight on every CU. Fragments come straight from memory,
// four lanes a line, DEPTH blocks while one is multiplied; block128 and wgrad sum
// exactly (the matrix cores have nothing else to do). The waves' sums meet in LDS and
// are added in wave order. Workgroups walk tiles (wgrad: one each) and load the next
// one's first blocks before they join (decode of four tokens in integers 143 to 121
// us). A lane takes 16 bytes of both halves of a line; block128 and wgrad, whose order
// of sums stays, 32 in a row. Bound by the loads: one row by 8192 x 8192 13 us in
// E4M3 and in integers, 5.3 TB/s.
constexpr int kFewWaves = 8;

// The 16 bytes at p + at and those at APART bytes from them, of a row of len bytes
// (a multiple of 16, not 0); past its end its first bytes, which within() clears.
template <int APART>
__device__ __forceinline__ v8i load32(const uint8_t* p, int64_t at, int64_t len) {
    const v4i lo = *reinterpret_cast<const v4i*>(p + (at < len ? at : 0));
    const v4i hi = *reinterpret_cast<const v4i*>(p + (at + APART < len ? at + APART : 0));
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}

template <int APART>
__device__ __forceinline__ v8i within(v8i v, int64_t at, int64_t len) {
    const v4i zero = {};
    const v4i lo = __builtin_shufflevector(v, v, 0, 1, 2, 3), hi = __builtin_shufflevector(v, v, 4, 5, 6, 7);
    return __builtin_shufflevector(at < len ? lo : zero, at + APART < len ? hi : zero, 0, 1, 2, 3, 4, 5, 6, 7);
}

// Workgroups of eight waves that a CU holds at a time: two of at most 128 registers a lane,
// which the smallest tiles need no more than (the gradient with binary32 sums 130).
template <int BM, int LINES, class KIND>
constexpr int kFewPerCu = BM == 16 && LINES == 32 && !(KIND::grad && !KIND::eight) ? 2 : 1;

template <int BM, int LINES, int DEPTH, bool WALKS, class KIND>
__global__ __launch_bounds__(kFewWaves * 64, (kFewPerCu<BM, LINES, KIND> * kFewWaves / 4)) void mm_few_kernel(MmArgs p) {
    constexpr bool WGRAD = KIND::wgrad, GATED = KIND::gated, GRAD = KIND::grad, F32 = KIND::f32;
    constexpr bool SCALED = KIND::scaled, INT8 = KIND::num == Num::Int8;
    constexpr int MT = BM / 16, NT = LINES / 16;
    constexpr int COLS = GATED ? LINES / 2 : LINES;            // gated: the same columns of both projections
    constexpr int BLOCKS = GATED ? 2 : 1;                      // weights that have scales of their own
    using Op = Operand<KIND::num>;
    using Acc = typename Sum<INT8>::type;
    __shared__ __align__(16) float s_sum[kFewWaves][BM][LINES + 4];
    const int lane = threadIdx.x & (kWave - 1), wave = uniform((int)(threadIdx.x / kWave));
    const int64_t nnb = (p.N + 127) / 128;
    const int col_tiles = (int)((p.cols + COLS - 1) / COLS), M = (int)p.M;

    // ---- the tiles: every wave finds them, 64 groups at a time ----
    constexpr int kAlign = WGRAD ? 16 : 1;
    int e = 0, b = 0, upto = 0;            // of this lane's group: its rows, and the row tiles up to its end
    auto group = [&](int g, int from, int before) {
        int raw = 0;
        if (g < p.G) raw = p.offsets ? min(max(p.offsets[g], 0), M) / kAlign * kAlign : M;
        e = max(wave_prefix_imax(raw), from);
        b = __shfl_up(e, 1, kWave);
        if (lane == 0) b = from;
        upto = before + wave_prefix_sum(tiles_down(e - b, BM));
    };
    const int row_tiles = (int)((p.N + BM - 1) / BM);                  // wgrad: down one matrix
    int last_end = 0, tiles = 0, total;
    if constexpr (WGRAD) {
        total = p.G * row_tiles * col_tiles;
    } else {
        for (int base = 0; base < p.G; base += kWave) {
            group(base + lane, last_end, tiles);
            tiles = uniform(__shfl(upto, kWave - 1, kWave));
            last_end = uniform(__shfl(e, kWave - 1, kWave));
        }
        total = (tiles + tiles_down(M - last_end, BM)) * col_tiles;    // the rows past the last group give zeros
    }
    struct FewTile {
        int g, begin, end;                 // the group (-1: none) and its rows, wgrad: its part of the contraction
        int m0, n0;
    };
    auto locate = [&](int w) {
        const int L = tile_of(w, total);
        FewTile t;
        if constexpr (WGRAD) {
            const int per = row_tiles * col_tiles;
            t.g = uniform(L / per);
            int carry = 0;
            for (int base = 0; base <= t.g; base += kWave) {
                group(base + lane, carry, 0);
                carry = uniform(__shfl(e, kWave - 1, kWave));
            }
            t.begin = uniform(__shfl(b, t.g % kWave, kWave));
            t.end = uniform(__shfl(e, t.g % kWave, kWave));
            t.m0 = uniform(L - t.g * per) % row_tiles * BM;
            t.n0 = uniform(L - t.g * per) / row_tiles * COLS;
            return t;
        }
        int before = tiles;
        t.g = -1;
        t.begin = last_end;
        t.end = M;
        if (L < tiles * col_tiles) {
            int base = 0;
            if (p.G > kWave) {
                for (int carry = 0, passed = 0;; base += kWave) {
                    group(base + lane, carry, passed);
                    passed = uniform(__shfl(upto, kWave - 1, kWave));
                    if (L < passed * col_tiles) break;
                    carry = uniform(__shfl(e, kWave - 1, kWave));
                }
            }
            const int at = __builtin_ctzll(__ballot(upto * col_tiles > L));
            t.g = uniform(base + at);
            t.begin = uniform(__shfl(b, at, kWave));
            t.end = uniform(__shfl(e, at, kWave));
            before = uniform(__shfl(upto, at, kWave)) - tiles_down(t.end - t.begin, BM);
        }
        const int rows = tiles_down(t.end - t.begin, BM), local = L - before * col_tiles;
        t.m0 = t.begin + local % rows * BM;
        t.n0 = local / rows * COLS;
        return t;
    };
    const int64_t grid = (int64_t)gridDim.x * gridDim.z;
    int64_t wg = workgroup_xz();           // may pass the last tile
    if (wg >= total) return;

    // ---- the contraction ----
    const int fr = lane & 15, fg = lane / 16;
    int64_t len;
    int nkb;
    const uint8_t *pa[MT], *pb[NT];
    const float *psa[MT], *psb[BLOCKS];
    // A block of the contraction: its bytes and scales, in registers from their loads to their products.
    struct Block {
        v8i a[MT], b[NT];
        float sa[MT], sb[BLOCKS];
    };
    constexpr int APART = KIND::halves ? 64 : 16;
    // What lies past the rows' end is cleared where a block is multiplied: behind its
    // loads the selects wait for them, before the block at hand is multiplied (one row by
    // 8192 x 8192 12.9 us, so 14.2; wgrad of 4 x 512 x 512 31, 33; gradient of one row,
    // 8192 x 5120, 9.9 and 11.1). Sixteen rows of a gated pair do wait there: tiles in
    // turn read two weights each, and lose with more of their loads under way (four tokens
    // to 2 of 16 experts, 2 x 8192 x 5120, 118 us, without the wait 124; integers, to 8 of
    // 64 of 2 x 2048 x 4096, 85 and 87).
    constexpr bool WAITS = GATED && BM == 16;
    auto place = [&](int k) { return (int64_t)k * kBK + fg * (KIND::halves ? 16 : 32); };
    auto fetch = [&](Block& x, int k) {
        const int64_t at = place(k);
        auto get = [&](const uint8_t* q) {
            const v8i v = load32<APART>(q, at, len);
            return WAITS ? within<APART>(v, at, len) : v;
        };
#pragma unroll
        for (int j = 0; j < NT; ++j) x.b[j] = get(pb[j]);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            x.a[i] = get(pa[i]);
            if constexpr (SCALED) x.sa[i] = psa[i][k];
        }
        if constexpr (SCALED)
#pragma unroll
            for (int w = 0; w < BLOCKS; ++w) x.sb[w] = psb[w][k];
    };
    Acc acc[MT][NT];
    auto multiply = [&](Block& x, int k) {
        if (!WAITS && (int64_t)(k + 1) * kBK > len) {          // the rows end in this block
#pragma unroll
            for (int j = 0; j < NT; ++j) x.b[j] = within<APART>(x.b[j], place(k), len);
#pragma unroll
            for (int i = 0; i < MT; ++i) x.a[i] = within<APART>(x.a[i], place(k), len);
        }
        float f[MT][BLOCKS];
        if constexpr (SCALED)
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int w = 0; w < BLOCKS; ++w) f[i][w] = (1.0f / x.sa[i]) * (1.0f / x.sb[w]);
        Op ob[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) ob[j] = Op(x.b[j]);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            if constexpr (!SCALED) {
                Op::mfma(ob, Op(x.a[i]), acc[i]);
            } else {
                v4f part[NT] = {};
                Op::mfma(ob, Op(x.a[i]), part);
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        acc[i][j][c] = fmaf(part[j][c], f[i][GATED ? j / (NT / 2) : 0], acc[i][j][c]);
            }
        }
    };
    Block x[DEPTH];
    // Where t's operands are, and the loads of each wave's first blocks.
    auto begin = [&](const FewTile& t) {
        len = t.g < 0 ? 0 : WGRAD ? t.end - t.begin : p.K;
        nkb = (int)((len + kBK - 1) / kBK);
        if (len == 0) return;
        const int64_t row_end = WGRAD ? p.N : t.end, stride = WGRAD ? p.M : p.K;
#pragma unroll
        for (int w = 0; w < BLOCKS; ++w) psb[w] = p.b_scales + (((int64_t)t.g * BLOCKS + w) * nnb + t.n0 / 128) * nkb;
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const int64_t r = min((int64_t)t.m0 + i * 16 + fr, row_end - 1);
            pa[i] = p.a + r * stride + (WGRAD ? t.begin : 0);
            psa[i] = p.a_scales + r * nkb;
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const int64_t r = min((int64_t)t.n0 + (GATED ? j % (NT / 2) : j) * 16 + fr, p.cols - 1);
            pb[j] = WGRAD ? p.b + r * stride + t.begin
                          : p.b + (((int64_t)t.g * BLOCKS + (GATED ? j / (NT / 2) : 0)) * p.N + r) * stride;
        }
#pragma unroll
        for (int d = 0; d < DEPTH; ++d)
            if (wave + d * kFewWaves < nkb) fetch(x[d], wave + d * kFewWaves);
    };
    FewTile t = locate((int)wg);
    begin(t);
    for (;;) {
    const int64_t row_end = WGRAD ? p.N : t.end;
    const int g = t.g, m0 = t.m0, n0 = t.n0;
    const bool none = len == 0;
    // A thread stores four columns of one or two rows. What their results take besides the
    // sums is loaded first: at the end it would come behind the next tile's blocks.
    constexpr int PIECES = BM * COLS / 4, TURNS = (PIECES + kFewWaves * 64 - 1) / (kFewWaves * 64);
    auto piece = [&](int turn, int& r, int& c) {
        const int x = threadIdx.x + turn * (kFewWaves * 64);
        r = x / (COLS / 4);
        c = x % (COLS / 4) * 4;
        return x < PIECES && m0 + r < row_end && n0 + c < p.cols;
    };
    float sa[INT8 ? TURNS : 1], sb[INT8 ? TURNS : 1][BLOCKS][4];
    uint2 kept[GRAD ? TURNS : 1][2];
#pragma unroll
    for (int turn = 0; turn < TURNS; ++turn) {
        int r, c;
        if (!piece(turn, r, c) || g < 0) continue;
        if constexpr (INT8) {
            sa[turn] = p.a_scales[m0 + r];
#pragma unroll
            for (int w = 0; w < BLOCKS; ++w)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    sb[turn][w][i] = p.b_scales[((int64_t)g * BLOCKS + w) * p.N + n0 + c + i];
        }
        if constexpr (GRAD) {
            const uint16_t* gu = p.gu + (int64_t)(m0 + r) * 2 * p.cols + n0 + c;
            kept[turn][0] = *reinterpret_cast<const uint2*>(gu);
            kept[turn][1] = *reinterpret_cast<const uint2*>(gu + p.cols);
        }
    }
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = Acc{0, 0, 0, 0};
    for (int k = wave; k < nkb; k += DEPTH * kFewWaves) {
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) {
            const int now = k + d * kFewWaves;
            if (now >= nkb) break;
            Block y = x[d];
            if (now + DEPTH * kFewWaves < nkb) fetch(x[d], now + DEPTH * kFewWaves);
            multiply(y, now);
        }
    }
    // the next tile's first loads are on their way while this one is joined
    bool more = false;
    if constexpr (WALKS) {
        wg += grid;
        more = wg < total;
        if (more) {
            t = locate((int)wg);
            begin(t);
        }
    }

    // ---- join and store ----
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
            *reinterpret_cast<Acc*>(&s_sum[wave][i * 16 + fr][j * 16 + fg * 4]) = acc[i][j];
    __syncthreads();
    // four sums of the tile's row r from its line c on, added in wave order
    auto joined = [&](int r, int c) {
        Acc v = *reinterpret_cast<const Acc*>(&s_sum[0][r][c]);
#pragma unroll
        for (int w = 1; w < kFewWaves; ++w) v += *reinterpret_cast<const Acc*>(&s_sum[w][r][c]);
        return __builtin_convertvector(v, v4f);
    };
    // and the scales that are not in the sums yet, of output columns col to col + 3 of weight w
    auto scaled = [&](v4f v, int64_t row, int64_t col, int turn, int w) {
        if constexpr (WGRAD) {
            if (!none) {
                const float ia = 1.0f / p.a_scales[row * p.G + g];
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = v[i] * ia * (1.0f / p.b_scales[(col + i) * p.G + g]);
            }
        } else if constexpr (INT8) {
            if (g >= 0) {
                const float ia = 1.0f / sa[turn];
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = v[i] * ia * (1.0f / sb[turn][w][i]);
            }
        }
        return v;
    };
    auto store4 = [](void* out, int64_t at, v4f v) {
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + at) = make_uint2(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]));
    };
#pragma unroll
    for (int turn = 0; turn < TURNS; ++turn) {
        int r, c;
        if (!piece(turn, r, c)) continue;
        const int64_t row = m0 + r, col = n0 + c;
        v4f v = scaled(joined(r, c), row, col, turn, 0);
        const int64_t at = row * p.cols + col, at2 = at + row * p.cols;
        if constexpr (GATED) {
            const v4f u = scaled(joined(r, COLS + c), row, col, turn, 1);
            if constexpr (KIND::more) {
                store4(p.more, at2, v);
                store4(p.more, at2 + p.cols, u);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = p.act.of(v[i]) * u[i];
            store4(p.out, at, v);
        } else if constexpr (GRAD) {
            const uint2 gw = kept[turn][0], uw = kept[turn][1];
            const float gs[4] = {bf16_lo(gw.x), bf16_hi(gw.x), bf16_lo(gw.y), bf16_hi(gw.y)};
            const float us[4] = {bf16_lo(uw.x), bf16_hi(uw.x), bf16_lo(uw.y), bf16_hi(uw.y)};
            v4f dg = {}, du = {}, h = {};
            if (g >= 0) {                 // rows of no group give zeros, whatever their projections are
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const GatedGrad d = p.act.grad(v[i], gs[i], us[i]);
                    dg[i] = d.dg;
                    du[i] = d.du;
                    h[i] = d.h;
                }
            }
            store4(p.out, at2, dg);
            store4(p.out, at2 + p.cols, du);
            if constexpr (KIND::more) store4(p.more, at, h);
        } else if constexpr (F32) {
            const int64_t to = (WGRAD ? g * p.N * p.cols : 0) + at;
            if (WGRAD && p.accumulate) v += *reinterpret_cast<const v4f*>(static_cast<const float*>(p.out) + to);
            *reinterpret_cast<v4f*>(static_cast<float*>(p.out) + to) = v;
        } else {
            store4(p.out, (WGRAD ? g * p.N * p.cols : 0) + at, v);
        }
    }
    if (!more) break;
    __syncthreads();         // the sums are read before the next tile's are written
    }
}

template <int BM, int LINES, class KIND>
hipError_t launch_few(const MmArgs& p, int cus, hipStream_t stream) {
    constexpr bool WGRAD = KIND::wgrad;
    constexpr int COLS = KIND::gated ? LINES / 2 : LINES;
    const int64_t groups = p.offsets ? p.G + 1 : 1, spare = groups < p.M ? groups : p.M;
    const int64_t down = WGRAD ? p.G * ((p.N + BM - 1) / BM) : (p.M + spare * (BM - 1)) / BM;
    const int64_t tiles = down * ((p.cols + COLS - 1) / COLS);
    if (tiles > INT32_MAX) return hipErrorInvalidValue;
    // Two blocks ahead pay for integers only, which have the registers (4 tokens to 2 of
    // 16 experts, 2 x 8192 x 5120: 140 to 117 us at the time; E4M3 116 to 125).
    constexpr int DEPTH = KIND::num == Num::Int8 && BM == 16 && LINES == 64 ? 2 : 1;
    const int64_t most = cus * kFewPerCu<BM, LINES, KIND>;
    const int64_t blocks = WGRAD || tiles < most ? tiles : most;
    // block128 and wgrad without the code that walks, which costs 0.3 us a call (one row by
    // 1024 x 1024: 4.7, without it 4.4).
    if constexpr (WGRAD || !KIND::halves) {
        if (blocks == tiles) {
            hipLaunchKernelGGL((mm_few_kernel<BM, LINES, DEPTH, false, KIND>), grid_xz(blocks), dim3(kFewWaves * 64), 0,
                               stream, p);
            return hipGetLastError();
        }
    }
    if constexpr (!WGRAD)
        hipLaunchKernelGGL((mm_few_kernel<BM, LINES, DEPTH, true, KIND>), grid_xz(blocks), dim3(kFewWaves * 64), 0, stream,
                           p);
    return hipGetLastError();
}

template <int BM, int BN, int WM, int WN, int PARTS, class KIND>
hipError_t launch(const MmArgs& p, int cus, hipStream_t stream) {
    constexpr bool WGRAD = KIND::wgrad;
    constexpr int COLS = KIND::gated ? BN / 2 : BN;
    constexpr int threads = BM / WM * (BN / WN) * 64 * PARTS;
    constexpr int per_cu = 512 / threads;        // workgroups of at most 256 registers a lane
    // rows: every group, and the rows past the last one, may end inside a tile
    const int64_t down = WGRAD ? p.G * ((p.N + BM - 1) / BM) : p.M / BM + (p.offsets ? p.G + 1 : 1);
    const int64_t tiles = down * ((p.cols + COLS - 1) / COLS);
    if (tiles > INT32_MAX) return hipErrorInvalidValue;
    const int64_t blocks = PARTS > 1 || tiles < cus * per_cu ? tiles : cus * per_cu;
    hipLaunchKernelGGL((mm_kernel<BM, BN, WM, WN, PARTS, KIND>), dim3((unsigned)blocks), dim3(threads), 0, stream, p);
    return hipGetLastError();
}

// The form by the rules of mgs_mm_form.hpp; a gated pair of projections counts as one
// product of twice the columns.
template <class KIND>
hipError_t launch_sized(const MmArgs& p, int cus, hipStream_t stream) {
    const bool grouped = p.offsets != nullptr;
    const MmForm form = KIND::halves
                            ? mm_form_rows(KIND::num == Num::Int8, KIND::eight, grouped, p.M,
                                           (KIND::gated ? 2 : 1) * p.N, p.K, p.G, cus)
                            : mm_form(KIND::wgrad, KIND::eight, grouped, p.M, p.N, p.K, p.G, cus);
    using Few = typename KIND::few;
    if constexpr (KIND::halves) {
        if (form.few == 16 && form.tile == 64) return launch_few<16, 64, Few>(p, cus, stream);
        if (form.few == 32 && form.tile == 64) return launch_few<32, 64, Few>(p, cus, stream);
        if constexpr (KIND::num == Num::Int8)
            if (form.few == 64) return launch_few<64, 64, Few>(p, cus, stream);
    } else {
        if (form.few == 64) return launch_few<64, 32, Few>(p, cus, stream);
    }
    if (form.few == 16) return launch_few<16, 32, Few>(p, cus, stream);
    if (form.few == 32) return launch_few<32, 32, Few>(p, cus, stream);
    if constexpr (KIND::wgrad || KIND::eight) {
        if (form.tile == 256) return launch<256, 256, 128, 64, 1, KIND>(p, cus, stream);
    }
    if constexpr (KIND::wgrad || KIND::eight || KIND::halves) {
        if (form.sets == 2) return launch<128, 128, 64, 64, 2, KIND>(p, cus, stream);
    }
    return launch<128, 128, 64, 64, 1, KIND>(p, cus, stream);
}

}  // namespace

}  // namespace mgs
