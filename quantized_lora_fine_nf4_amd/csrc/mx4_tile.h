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
// with what they bring.  Four waves share the LDS and the address unit, and what is bunched waits
// there while the matrix cores are idle.
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
// upper pair for its neighbour's lower one.  ncol: out's columns, ldo its row pitch
// (the partials' too).
template <int TM, int TN, bool PAIRS = false>
__device__ __forceinline__ void store_tile(f32x16 (&acc)[TM][TN], void* dst, float* partial, int dst_kind,
                                           const TileGrid& grid, int part, int64_t m, int64_t ncol, int64_t ldo,
                                           int64_t m0, int64_t n0, int wm, int wn, int r, int h)
{
    constexpr int kBM = 64 * TM;
    const bool split = grid.parts > 1;
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
