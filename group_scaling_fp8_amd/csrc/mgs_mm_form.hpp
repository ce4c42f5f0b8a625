// mgs_mm_form.hpp — which form a product takes (internal; host only, no HIP).
#pragma once

#include <stdint.h>

namespace mgs {

constexpr int kFewCols = 32;      // columns of a tile of the form for few rows

struct MmForm {
    int few;      // rows of a tile of the form for few rows or few outputs, or 0:
    int tile;     // tiles of 256 x 256 or 128 x 128 through LDS,
    int sets;     // with this many sets of waves on one tile's contraction
};

// Which form a product takes, from the sizes the host knows (us, MI355X):
// - few rows: up to 20 rows a group on average, one row of fragments (M = 1 by
//   8192 x 8192: 17, against 66 on tiles of 128 x 128; more rows a group only
//   where there is one group: 512 rows in 16 groups by 2048 x 4096 take 58, and
//   33 on tiles); up to 40 rows two, and four where that is at most one
//   workgroup a CU (64 rows by 8192 x 8192: 39 and 66; 256 rows by 4096 x 4096,
//   two a CU: 36 and 32).
// - few outputs of wgrad: the same form with the fewest rows a tile that still
//   leaves one workgroup a CU (16640 x 256 x 272: 25 with 16 rows, 48 with 64, and
//   66 on tiles of 128 x 128 in two parts; 16384 x 1024 x 512: 48 and 60, twice as
//   many outputs 93 and 61; with binary32 sums still 93 and 94, and 43 and 52 in
//   four groups of 512 x 512).
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

}  // namespace mgs
