// mx4_tile.h -- what the tiled products share: the order of the output tiles, the
// split of the reduction, the order of instructions in a sub-step and the way out.
// A workgroup is 2 x 2 waves of TM x TN tiles of 32 x 32.
#pragma once
#include <type_traits>

#include "mx4_format.h"
#include "mx4_sum.h"

namespace mx4k {

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

struct TileGrid {
    int mt, nt;       // output tiles along the tokens and the columns
    int parts;        // splits of the reduction
    int per_part;     // its steps per split
};

// How the output is cut: 256 x 256 tiles on the first 256 * big.nt columns, 128 x
// 128 tiles on the others (nt 0: none there).
struct TilePlan {
    TileGrid big, small;
};

constexpr int kCus = 256;

// Measured on this card, in us: a step of the reduction, and what a tile costs
// besides (its start and its stores), for a round of large tiles (one on each compute
// unit), for one of small tiles with one on each, and for one with two.
struct TileCosts {
    double big_step, big_tile, one_step, one_tile, two_step, two_tile;
};

// So many small tiles of so many steps: rounds of two on each compute unit and a rest.
// Between one and two on each it grows with their number, 0.4 of the way at once.
inline double small_us(int64_t tiles, int steps, const TileCosts& c)
{
    const double one = steps * c.one_step + c.one_tile, two = steps * c.two_step + c.two_tile;
    const int64_t rounds = tiles / (2 * kCus), rest = tiles % (2 * kCus);
    if (rest == 0) return rounds * two;
    if (rest <= kCus) return rounds * two + one;
    const double over = double(rest - kCus) / kCus;
    return rounds * two + one + (two - one) * (over > 0.4 ? over : 0.4);
}

// The small tiles of m x ncol outputs: into how many parts their reduction goes and
// what that costs, with 4.3 us for the sum and the partials' 8 bytes (written and read)
// at 6 TB/s (they stay in the caches).
inline TileGrid small_plan(int64_t m, int64_t ncol, int steps, const TileCosts& c, double* cost)
{
    TileGrid best = {(int)ceil_div(m, 128), (int)ceil_div(ncol, 128), 1, steps};
    const int64_t tiles = (int64_t)best.mt * best.nt;
    *cost = small_us(tiles, steps, c);
    for (int p = 2; p <= 16 && p <= steps; ++p) {
        const int per = (int)ceil_div(steps, p), parts = (int)ceil_div(steps, per);
        const double us = small_us(tiles * parts, per, c) + 4.3 + double(parts) * double(m) * double(ncol) * 8e-6 / 6.0;
        if (us < *cost) {
            *cost = us;
            best.parts = parts;
            best.per_part = per;
        }
    }
    return best;
}

// The cheapest of: small tiles only, big ones only, whole rounds of big ones and
// small ones on the columns that are left.
inline TilePlan tile_plan(int64_t m, int64_t ncol, int steps, const TileCosts& c, double* us = nullptr)
{
    TilePlan p = {};
    double least;
    p.small = small_plan(m, ncol, steps, c, &least);
    const int64_t mt = ceil_div(m, 256), nt = ceil_div(ncol, 256), rounds = mt * nt / kCus, fit = rounds * kCus / mt;
    const double round = steps * c.big_step + c.big_tile;
    if (ceil_div(mt * nt, kCus) * round < least) {
        least = ceil_div(mt * nt, kCus) * round;
        p = TilePlan{{(int)mt, (int)nt, 1, steps}, {}};
    }
    if (fit > 0 && fit < nt) {
        double rest;
        const TileGrid small = small_plan(m, ncol - 256 * fit, steps, c, &rest);
        if (rounds * round + rest < least) {
            least = rounds * round + rest;
            p = TilePlan{{(int)mt, (int)fit, 1, steps}, small};
        }
    }
    if (us) *us = least;
    return p;
}

// fp32 partials of the small tiles' columns, [parts][m][those columns].
inline size_t plan_ws(const TilePlan& p, int64_t m, int64_t ncol)
{
    return p.small.parts > 1 ? size_t(p.small.parts) * size_t(m) * size_t(ncol - 256 * p.big.nt) * sizeof(float) : 0;
}

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

typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kThreads = 256;
constexpr int kVmcnt0 = 0x0f70;   // s_waitcnt: vector memory only, none outstanding

// READS LDS reads, VALU vector instructions and LOADS loads spread over N matrix
// instructions, the reads over the first three quarters: the next sub-step begins
// with what they bring.  Four waves share the LDS and the address unit, and what is
// bunched waits there while the matrix cores are idle.
template <int N, int READS, int VALU, int LOADS, int I = 0>
__device__ __forceinline__ void spread()
{
    if constexpr (I < N) {
        constexpr int kOver = N * 3 / 4, kTo = I + 1 < kOver ? I + 1 : kOver, kFrom = I < kOver ? I : kOver;
        constexpr int kReads = kTo * READS / kOver - kFrom * READS / kOver;
        constexpr int kLoads = (I + 1) * LOADS / N - I * LOADS / N, kValu = (I + 1) * VALU / N - I * VALU / N;
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        if constexpr (kReads > 0) __builtin_amdgcn_sched_group_barrier(0x100, kReads, 0);
        if constexpr (kValu > 0) __builtin_amdgcn_sched_group_barrier(0x002, kValu, 0);
        if constexpr (kLoads > 0) __builtin_amdgcn_sched_group_barrier(0x020, kLoads, 0);
        spread<N, READS, VALU, LOADS, I + 1>();
    } else {
        __builtin_amdgcn_sched_barrier(0);
    }
}

template <int K>
using Kind = std::integral_constant<int, K>;

// What the neighbour lane (r ^ 1) has.
__device__ __forceinline__ uint32_t neighbour(uint32_t v) { return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xf, 0xf, true); }
__device__ __forceinline__ float neighbour(float v) { return __builtin_bit_cast(float, neighbour(__builtin_bit_cast(uint32_t, v))); }

// A wave's sums to out, or to its part's partial (with more than one).  The
// workgroup's tile begins at (m0, n0); wave (wm, wn), lane (r, h): columns TN r to
// TN r + TN - 1 of the wave's, rows 8 a + 4 h + b of each 32.  PAIRS (TN 4): lane
// r = 8 q + i has columns 32 q + 2 i, + 1, + 16, + 17 instead; an even lane gives its
// upper pair for its neighbour's lower one.  ncol: the columns of the call's region,
// and a partial's row pitch; ldo: out's.
template <int TM, int TN, bool PAIRS = false>
__device__ __forceinline__ void store_tile(f32x16 (&acc)[TM][TN], void* dst, float* partial, int dst_kind,
                                           const TileGrid& grid, int part, int64_t m, int64_t ncol, int64_t out_pitch,
                                           int64_t m0, int64_t n0, int wm, int wn, int r, int h)
{
    constexpr int kBM = 64 * TM;
    const bool split = grid.parts > 1;
    const int64_t ldo = split ? ncol : out_pitch;
    char* out = split ? (char*)(partial + (int64_t)part * m * ldo) : (char*)dst;
    const int kind = split ? (int)kOutFp32 : dst_kind;
    const int odd = r & 1;
    const int col = wn * (32 * TN) + (PAIRS ? 32 * (r >> 3) + 4 * ((r & 7) >> 1) + 16 * odd : TN * r);
    if (!PAIRS && n0 + col >= ncol) return;
    const bool in = n0 + col < ncol;   // with PAIRS the neighbour may need this lane
    auto put = [&](auto k, auto all) {
        constexpr int kBytes = k == kOutFp32 ? 4 : 2;
        char* base = out + ((m0 + wm * (32 * TM)) * ldo + n0) * kBytes;   // uniform
        const uint32_t at = (uint32_t)(4 * h * ldo + col) * kBytes;
        const int64_t pitch = ldo * kBytes;
        const int left = (int)(all || m - m0 > kBM ? kBM : m - m0) - wm * (32 * TM) - 4 * h;
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            // one row of tiles at a time out of the accumulation registers: moved all at once the sums spill
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int k2 = i; k2 < TM; ++k2)
#pragma unroll
                for (int j = 0; j < TN; ++j) __asm__ volatile("" : "+a"(acc[k2][j]));
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const int row = i * 32 + 8 * (e >> 2) + (e & 3);
                if constexpr (PAIRS) {
                    const float c0 = acc[i][0][e], c1 = acc[i][1][e], c2 = acc[i][2][e], c3 = acc[i][3][e];
                    const float w = odd ? c2 : c0, x = odd ? c3 : c1;
                    const float y = neighbour(odd ? c0 : c2), z = neighbour(odd ? c1 : c3);
                    if ((all || row < left) && in)
                        put4<k>((MX4_GLOBAL char*)base + row * pitch + at, odd ? f32x4{y, z, w, x} : f32x4{w, x, y, z});
                } else if (all || row < left) {
                    MX4_GLOBAL char* p = (MX4_GLOBAL char*)base + row * pitch;
                    if constexpr (TN == 4) put4<k>(p + at, f32x4{acc[i][0][e], acc[i][1][e], acc[i][2][e], acc[i][3][e]});
                    else put2<k>(p + at, f32x2{acc[i][0][e], acc[i][1][e]});
                }
            }
        }
    };
    auto of_kind = [&](auto all) {
        if (kind == kOutBf16) put(Kind<kOutBf16>{}, all);
        else if (kind == kOutFp16) put(Kind<kOutFp16>{}, all);
        else put(Kind<kOutFp32>{}, all);
    };
    if (m0 + kBM <= m) of_kind(std::true_type{});
    else of_kind(std::false_type{});
}

}  // namespace mx4k
