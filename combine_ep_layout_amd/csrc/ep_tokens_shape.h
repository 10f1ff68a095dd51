// Which form of its kernels the layer for a few tokens takes (ep_tokens.hip).
// Host code of plain integers.  Not installed; callers use include/ep_layout.h.
#pragma once

#include <stdint.h>

namespace epk {

constexpr int kTokensRows = 16;             // rows of a matrix in a tile
constexpr int kTokensWaves = 8;             // of a workgroup
// Past so many tokens or experts the choice has a launch of its own: a workgroup
// would have to make more than its waves can at once.
constexpr int kRouteHereTokens = kTokensWaves;
constexpr int kRouteHereExperts = 256;
static_assert(kRouteHereTokens <= 16, "no expert has more");

// What the choice depends on.
struct TokensSizes {
    int32_t T, K, E, H, I;
    int32_t up_tiles;           // row tiles of a wave in the gate and up products, by the weights' form
    int32_t num_cu;
};

struct TokensShape {
    bool route_here;            // the choice of the experts is made in the gate and up kernel
    bool many;                  // an expert may have more than 16 tokens
    int up_tiles, up_groups;    // row tiles of a wave, and groups of waves with tiles of their own
    int down_tiles;             // row tiles of a workgroup in the down product
    int64_t up_items, down_items;
};

// Four row tiles a workgroup in the gate and up products where that leaves no more
// rounds of the compute units behind than two (32 tokens in 4 bits, 2048 x 1024: 93 us,
// 110); one row tile a wave where two would leave half of the compute units
// without work.
inline TokensShape tokens_shape(const TokensSizes& s) {
    const int64_t slots = (int64_t)s.T * s.K, used = slots < s.E ? slots : s.E;
    auto items = [](int rows, int r) { return (int64_t)((rows + r * kTokensRows - 1) / (r * kTokensRows)); };
    auto rounds = [&](int64_t n) { return (n + s.num_cu - 1) / s.num_cu; };
    TokensShape f;
    f.route_here = s.T <= kRouteHereTokens && s.E <= kRouteHereExperts;
    f.many = s.T > 16;
    const int64_t more = used * items(s.I, s.up_tiles), twice = used * items(s.I, 2 * s.up_tiles);
    f.up_tiles = s.up_tiles;
    f.up_groups = 1;
    f.up_items = more;
    if (more <= s.num_cu / 2) {
        f.up_tiles = 1;
        f.up_items = used * items(s.I, 1);
    } else if (s.up_tiles > 1 && 2 * rounds(twice) <= rounds(more)) {
        f.up_groups = 2;
        f.up_items = twice;
    }
    f.down_tiles = items(s.H, 2) > s.num_cu / 2 ? 2 : 1;
    f.down_items = items(s.H, f.down_tiles);
    return f;
}

}  // namespace epk
