// Which tiles each product of the orthogonalisation takes, and how many matrices
// go through at once (ep_muon.hip).  Plain integers.  Not installed; callers use
// include/ep_layout.h.
#pragma once

#include <stdint.h>

namespace epk {
namespace {

// The products: G, P, the next X, and the last X into the results (of tall
// matrices through LDS, which turns it).
enum MuonOp { kGram, kPoly, kNext, kLast, kLastTall };
constexpr bool is_update(int op) { return op >= kNext; }

constexpr int kMuonProblems = 40;           // shapes of a launch: its arguments stay below 4 KiB
// Workgroups of a launch: 2^31 threads of at most 2^32 - 1.
constexpr int64_t kMuonMostBlocks = (int64_t)1 << 23;

// Tiles of one matrix.
template <int BM, int BN>
inline constexpr int64_t tiles_of(int op, int m, int ld_n) {
    const int64_t down = (m + BM - 1) / BM;
    return is_update(op) ? down * ((ld_n + BN - 1) / BN) : down * (down + 1) / 2;
}

// `mats` matrices of one shape, laid as m x n with m <= n and rows of ld_n.
struct MuonSizes {
    int32_t m, ld_n, mats;
};

// The tiles of a product: 64 x 64 for all, or the first wide_mats[i] matrices of
// each shape 256 x 256 and the others 128 x 128.
struct MuonShape {
    bool small;
    int32_t wide_mats[kMuonProblems];
};

// Rounds of wide tiles that so many middle ones cost, two on a compute unit (8
// matrices of 2048 x 7168, G: 183 us a wide round, 119 one of 512 middle tiles).
inline double muon_middle_cost(int64_t tiles, int num_cu) {
    const int64_t rest = tiles % (2 * num_cu);
    return 0.65 * (double)(tiles / (2 * num_cu)) + (rest == 0 ? 0.0 : rest <= num_cu ? 0.42 : 0.65);
}

// Wide tiles are the fastest where they come in whole rounds of the compute units;
// what is left of a last round goes to the middle ones, by whole matrices (8
// matrices, G: 252 wide and 136 middle tiles instead of two rounds of 288).  Less
// than 5/8 of a compute unit's worth of middle tiles: small ones (16 matrices of
// 256 x 512, the next X: 8.4 us, 13.0).
inline MuonShape muon_shape(int op, int count, const MuonSizes* s, int num_cu) {
    MuonShape f{};
    int64_t wide = 0, middle = 0;
    for (int i = 0; i < count; ++i) {
        wide += s[i].mats * tiles_of<256, 256>(op, s[i].m, s[i].ld_n);
        middle += s[i].mats * tiles_of<128, 128>(op, s[i].m, s[i].ld_n);
    }
    f.small = middle < (int64_t)num_cu * 5 / 8;
    if (f.small) return f;
    const double all_wide = (double)((wide + num_cu - 1) / num_cu), all_middle = muon_middle_cost(middle, num_cu);
    const bool is_wide = all_wide < all_middle;
    if (wide > num_cu && wide % num_cu != 0) {
        // the fewest matrices from the end on that leave whole rounds
        MuonShape mixed{};
        for (int i = 0; i < count; ++i) mixed.wide_mats[i] = s[i].mats;
        int64_t over = wide % num_cu, less = 0, more = 0, left = 0;
        for (int i = count - 1; i >= 0 && less < over; --i) {
            const int64_t each = tiles_of<256, 256>(op, s[i].m, s[i].ld_n);
            int64_t k = (over - less + each - 1) / each;
            k = k < s[i].mats ? k : s[i].mats;
            mixed.wide_mats[i] -= (int32_t)k;
            less += k * each;
            more += k * tiles_of<128, 128>(op, s[i].m, s[i].ld_n);
        }
        for (int i = 0; i < count; ++i) left += mixed.wide_mats[i];
        const double cost = (double)((wide - less + num_cu - 1) / num_cu) + muon_middle_cost(more, num_cu);
        // another launch costs something, too
        if (left > 0 && cost < (is_wide ? all_wide : all_middle) - 0.05) return mixed;
    }
    if (is_wide)
        for (int i = 0; i < count; ++i) f.wide_mats[i] = s[i].mats;
    return f;
}

// Workgroups that a matrix needs in any of the launches, at most: its tiles of 64 x 64
// (as many as its units in the split) and its partial sums.
inline int64_t muon_blocks_of(int m, int ld_n, int partials) { return tiles_of<64, 64>(kNext, m, ld_n) + partials; }

// Matrices that the rest of the workspace and of a launch's workgroups hold.
inline int64_t muon_fit(int64_t bytes_left, int64_t bytes_each, int64_t blocks_used, int64_t blocks_each) {
    const int64_t fit = bytes_left / bytes_each, fit_blocks = (kMuonMostBlocks - blocks_used) / blocks_each;
    return fit < fit_blocks ? fit : fit_blocks;
}

}  // namespace
}  // namespace epk
