// Which tile shape each product of the experts' feed-forward takes (ep_ffn.hip).
// Host code of plain integers.  Not installed; callers use include/ep_layout.h.
#pragma once

#include <stdint.h>

namespace epk {

// The products.
enum FfnOp { kUp, kDown, kActGrad, kRowGrad, kWeightGrad };

// The tiles' shapes.  The widest, 256 x 256 with 8 waves and the register
// pipeline, moves the fewest bytes through L2, which bounds these products (of
// the shapes below, 32 experts of 2048 rows: gate and up 3.39 ms against 4.54
// with 128 x 128; with 4 waves it loads at two thirds of the rate).  It needs two
// rounds of tiles, or the last one leaves too many compute units idle: 1.3
// rounds of it took 77 and 133 us in two products where 128 x 128 took 67 and
// 106; of the weights' gradients, whose tiles are short, 3.4 rounds took 120
// against 112.
// Low, 64 x 128 with three tiles in LDS, is for rows that wait for the weights:
// 256 tokens over 64 experts of 7168 x 2048 take 992 us; 1054 with two tiles,
// 1007 at 64 x 256, 1079 at 32 x 128.  Small is Low for less than a round of
// tiles (8 experts of 256 x 512, 32 rows: 5.5-7.0 us a product against 6.6-11.2).
// Few, 16 high with four tiles: one token over 8 experts 121 us; 123-130 with 64
// columns, 126 with six tiles, 142 at 16 x 256.
enum FfnShape { kWide, kMiddle, kLow, kSmall, kFew };
struct FfnTile {
    int m, n;                   // rows and columns
};
constexpr FfnTile kFfnTiles[] = {{256, 256}, {128, 128}, {64, 128}, {64, 64}, {16, 128}};

// What the choice depends on.
struct FfnSizes {
    int32_t E;
    int64_t slots;              // num_tokens * top_k: bound on the rows
    int32_t M;                  // rows of a weight gradient
    int32_t N;                  // columns
    int32_t num_cu;
};

// Tiles that the product can need at most.  kUp: half of a tile's columns are
// the gate's, half the up's.
inline int64_t ffn_tile_count(FfnOp op, FfnTile t, const FfnSizes& s) {
    const int64_t used = s.slots < s.E ? s.slots : s.E;
    const int64_t rows = op == kWeightGrad ? (int64_t)s.E * ((s.M + t.m - 1) / t.m) : used + s.slots / t.m;
    const int cols = op == kUp ? t.n / 2 : t.n;
    return rows * ((s.N + cols - 1) / cols);
}

inline bool ffn_is_small(FfnOp op, const FfnSizes& s) {
    return s.slots <= (int64_t)48 * s.E && s.slots > (int64_t)16 * s.E && ffn_tile_count(op, kFfnTiles[kLow], s) < s.num_cu;
}

inline FfnShape ffn_rows_shape(FfnOp op, const FfnSizes& s) {
    const int64_t mean = (s.slots + s.E - 1) / s.E;
    if (mean > 128 && ffn_tile_count(op, kFfnTiles[kWide], s) >= 2 * s.num_cu) return kWide;
    if (mean > 48) return kMiddle;
    if (ffn_is_small(op, s)) return kSmall;
    return mean > 16 ? kLow : kFew;
}

inline FfnShape ffn_weight_grad_shape(const FfnSizes& s) {
    return ffn_tile_count(kWeightGrad, kFfnTiles[kWide], s) >= 4 * s.num_cu ? kWide : kMiddle;
}

// Whether the three products that follow the activation's gradient go in one launch.
inline bool ffn_after_in_one(const FfnSizes& rows, const FfnSizes& gate_up, const FfnSizes& down) {
    return ffn_is_small(kRowGrad, rows) && ffn_tile_count(kWeightGrad, kFfnTiles[kMiddle], gate_up) <= rows.num_cu &&
           ffn_tile_count(kWeightGrad, kFfnTiles[kMiddle], down) <= rows.num_cu;
}

}  // namespace epk
