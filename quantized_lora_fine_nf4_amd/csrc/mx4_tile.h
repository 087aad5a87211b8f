// mx4_tile.h -- what the tiled products share: the order of the output tiles and
// the split of the reduction.
#pragma once
#include "mx4_format.h"

namespace mx4k {

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

struct TileGrid {
    int mt, nt;       // output tiles along the tokens and the columns
    int parts;        // splits of the reduction
    int per_part;     // its steps per split
};

// Consecutive workgroups go to the eight XCDs in turn, each with an L2 of its
// own: every XCD takes a contiguous run of an order in which kBand row tiles at a
// time walk along the columns, so that the tiles that run together share rows of
// both operands.
constexpr int kBand = 8;

__device__ __forceinline__ void tile_of(const TileGrid& g, int b, int& tm, int& tn, int& part)
{
    const int total = g.mt * g.nt * g.parts, q = total / 8, r = total % 8, x = b % 8;
    int t = x * q + (x < r ? x : r) + b / 8;
    part = __builtin_amdgcn_readfirstlane(t % g.parts);
    t /= g.parts;
    const int band = t / (kBand * g.nt), left = g.mt - band * kBand, h = left < kBand ? left : kBand;
    const int in = t - band * kBand * g.nt;
    tm = __builtin_amdgcn_readfirstlane(band * kBand + in % h);
    tn = __builtin_amdgcn_readfirstlane(in / h);
}

}  // namespace mx4k
