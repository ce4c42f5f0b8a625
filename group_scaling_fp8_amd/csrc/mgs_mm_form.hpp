// mgs_mm_form.hpp — which form a product takes, and how many tiles rows take
// (internal; no HIP).
#pragma once

#include <stdint.h>

namespace mgs {

constexpr int kFewCols = 32;      // columns of a tile of the form for few rows

// Tiles of `high` rows that hold `rows` rows, of which there are up to 2^31 - 1: the sum
// passes 31 bits.
constexpr int tiles_down(int rows, int high) { return (int)(((uint32_t)rows + (uint32_t)high - 1) / (uint32_t)high); }

struct MmForm {
    int few;      // rows of a tile of the form for few rows or few outputs, or 0:
    int tile;     // tiles of 256 x 256 or 128 x 128 through LDS (few rows: mm_form_rows),
    int sets;     // with this many sets of waves on one tile's contraction
};

// Which form a product takes, from the sizes the host knows (us, MI355X):
// - few rows: up to 20 rows a group on average, one row of fragments (M = 1 by
//   8192 x 8192: 13, against 50 on tiles of 128 x 128; more rows a group only
//   where there is one group: 512 rows in 16 groups by 2048 x 4096 take 51, and
//   39 on tiles); up to 40 rows two, and four where that is at most one
//   workgroup a CU (64 rows by 8192 x 8192: 33 and 40; 256 rows by 4096 x 4096,
//   two a CU: 35 and 24).
// - few outputs of wgrad: the same form with the fewest rows a tile that still
//   leaves one workgroup a CU (16640 x 256 x 272: 25 with 16 rows, 47 with 64, and
//   66 on tiles of 128 x 128 in two parts; 16384 x 1024 x 512: 48 and 60, twice as
//   many outputs 92 and 61; with binary32 sums 92 and 95, and 32 and 52 in four
//   groups of 512 x 512).
// - 256 x 256 tiles where they fill the CUs, twice if groups end inside them
//   (block128 16640 x 5120 x 8192 in 16 groups: 780, and about 1000 with 128 x
//   128; 2048 x 4096 x 4096, half the CUs: 66 and 48) and, for wgrad, where the
//   contraction is long or the tiles are many (16640 x 8192 x 5120 in 16 groups:
//   745, and about 950; 4096 x 2048 x 2048 in 8 groups, four steps a tile: 40 and
//   32).
// - 128 x 128 tiles otherwise, two workgroups a CU (block128 with binary32 sums
//   has no registers for more: 256 x 128 took 1591, 128 x 128 1491; 128 x 64,
//   three a CU, did not gain on 1003 x 4176 x 4112, and lost a third on
//   8192 x 8192 x 4096); where they leave half the CUs idle, two sets of waves
//   share a tile's contraction (256 x 4096 x 4096: 27 to 22; wgrad 8192 x 1024 x
//   1024 in two groups: 44 to 37; with binary32 sums block128 does not gain).
inline MmForm mm_form(bool wgrad, bool fast, bool grouped, int64_t M, int64_t N, int64_t K, int64_t G, int cus) {
    auto up = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
    const int64_t groups = grouped ? G : 1;
    if (wgrad) {
        const int64_t across = groups * up(K, kFewCols);
        if (across * up(N, 16) <= cus) return {16, 0, 0};
        if (across * up(N, 32) <= cus) return {32, 0, 0};
        if (across * up(N, 64) <= (fast ? cus : 2 * cus)) return {64, 0, 0};
        const int64_t tiles = groups * up(N, 256) * up(K, 256);
        if (tiles >= cus && (M / groups >= 2048 || tiles >= 4 * cus)) return {0, 256, 1};
    } else {
        const int64_t rows = up(M, groups);
        if (rows <= 20) return {16, 0, 0};
        if (groups == 1 && rows <= 40) return {32, 0, 0};
        if (groups == 1 && up(M, 64) * up(N, kFewCols) <= cus) return {64, 0, 0};
        if (fast && (up(M, 256) + groups / 2) * up(N, 256) >= (groups == 1 ? cus : 2 * cus)) return {0, 256, 1};
    }
    if (wgrad || fast) {
        const int64_t tiles = wgrad ? groups * up(N, 128) * up(K, 128) : (M / 128 + (grouped ? G + 1 : 1)) * up(N, 128);
        if (2 * tiles <= cus) return {0, 128, 2};
    }
    return {0, 128, 1};
}

// Which form the gated products, their gradient and the 8-bit integer ones take; N
// counts both projections' columns, `ints` and `eight` that operands are integers and
// that the instruction reads the bytes themselves. In the form for few rows `tile` is
// the lines of weights a tile has. Groups end inside tiles: half a row of tiles more
// for each. (us, MI355X; I: integers, E: E4M3, X: E4M3 with binary32 sums.)
// - the form for few rows with the smallest tile that leaves one workgroup a CU at
//   most: its eight waves share a contraction however few tiles there are (I, 64 rows by
//   4096 x 4096: 10.9 with 32 rows and 32 lines, 14.4 with 16, 20.6 on tiles of 128 x 128;
//   1000 rows by 800 x 8192: 33 with 64 and 64, 36 on tiles; gradient of 256 rows,
//   2048 x 4096: E 17 with 32 and 64, 28 on tiles, X 18 and 39; E has no registers for 64
//   and 64). X takes 32 and 64 for two rounds of them too (64 rows, 2 x 8192 x 5120: 38, on
//   tiles 43; three rounds, 96 rows, 55 and 43).
// - up to 20 rows a group 16 rows a tile, whatever the weights: with 64 lines, which read a
//   row half as often (E, 4 tokens to 2 of 16 experts of 2 x 8192 x 5120: 118, with 32
//   lines 137, on tiles 138; 16 tokens to 4 of 64 of 2 x 2048 x 4096: 109, 111, 115). I
//   takes 64 lines only where every wave has enough blocks to run two ahead, three and a
//   half of them where workgroups walk eight tiles and five where they walk fewer (32 lines
//   | 64; 4 tokens to 2 of 16, 2 x 8192 columns, by the contraction: 2560 68 | 70, 3584 90 |
//   89, 4608 112 | 111, 5632 135 | 130, 7168 166 | 161; 16 to 4 of 64, one product of 4096:
//   2560 77 | 78, 3584 99 | 98, 4608 125 | 120, 7168 185 | 178; 16 to 2 of 16, 2 x 2048: 3584
//   48 | 49, 4608 59 | 60, 5632 66 | 67; 16 rows by 32768: 4608 34 | 30, 5632 44 | 40). Rows of
//   a multiple of 4096 bytes, of which 64 lines begin on the same channels, take 32
//   whatever their length (4096: 99 | 108, 99 | 105, 111 | 113; 8192: 188 | 195, 94 | 103).
// - up to 40 rows 32 and 64, for I only where there is one group (64 tokens to 8 of 64
//   experts of 2 x 2048 x 4096: E 223, on tiles 231, I 202 and 215. Groups of unlike lengths
//   lose, of which the rule knows nothing, and I the more: 640 rows in 16 random groups,
//   2 x 8192 x 5120, E 428 and 273, I 387 and 238).
// - tiles of 256 x 256, one a CU, or 128 x 128, two a CU: by the time of their
//   rounds, in hundredths of a round of two tiles of 128 x 128 a CU. A tile of
//   256 x 256 takes 1.47 of it and one of 128 x 128 alone on its CU 0.65 (I, 2048 x
//   4096 x 4096: 37 on tiles of 128 and 52; 2048 rows in 8 groups: 69 and 58; 4096
//   rows in 16 groups, 4112 x 4176: 187 and 164).
// - two sets of waves on a tile of 128 x 128 where there is one a CU at most (256 rows,
//   2 x 8192 x 5120: 33, one set 39, X 49 and 55; 128 rows, X 44 and 51; with 264 tiles 52
//   and 37).
inline MmForm mm_form_rows(bool ints, bool eight, bool grouped, int64_t M, int64_t N, int64_t K, int64_t G, int cus) {
    auto up = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
    const int64_t groups = grouped ? G : 1, extra = grouped ? G / 2 : 0, rows = up(M, groups);
    constexpr int kFew[5][2] = {{16, 32}, {32, 32}, {16, 64}, {32, 64}, {64, 64}};
    for (int i = 0; i < (ints ? 5 : 4); ++i)
        if ((up(M, kFew[i][0]) + extra) * up(N, kFew[i][1]) <= cus) return {kFew[i][0], kFew[i][1], 0};
    if (rows <= 20) {
        const bool walks = (up(M, 16) + extra) * up(N, 64) >= 8 * cus;
        const bool longer = K / 128 >= (walks ? 28 : 40) && K % 4096 != 0;
        return {16, ints && !longer ? 32 : 64, 0};
    }
    if (rows <= 40 && (groups == 1 || !ints)) return {32, 64, 0};
    if (!eight && (up(M, 32) + extra) * up(N, 64) <= 2 * cus) return {32, 64, 0};
    const int64_t large = (up(M, 256) + extra) * up(N, 256), small = (up(M, 128) + extra) * up(N, 128);
    if (small <= cus) return {0, 128, 2};
    if (!eight) return {0, 128, 1};
    const int64_t left = small % (2 * cus);
    const int64_t small_time = small / (2 * cus) * 100 + (left == 0 ? 0 : left <= cus ? 65 : 100);
    return {0, up(large, cus) * 147 < small_time ? 256 : 128, 1};
}

}  // namespace mgs
