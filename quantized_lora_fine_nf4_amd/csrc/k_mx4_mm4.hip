// k_mx4_mm4.hip -- the product of two microscaled 4-bit operands on gfx950's
// scaled matrix instructions: out[t, n] = sum_k x[t, k] W[n, k].
//
// v_mfma_scale_f32_32x32x64 takes 32 codes (16 bytes, one group) and one scale
// byte a lane, as they lie in memory: nothing is converted.  It does four times
// the operations of the 16-bit instructions per cycle, so the operands' way to it
// counts: a 256 x 256 output tile by four waves of 128 x 128 (one per SIMD, 256
// accumulator registers each) reads 128 KB from LDS a step and 64 KB come into it, for
// 2,048 matrix cycles.  Eight waves of 128 x 64 would read half as much again.
//
// 8192 x 8192 x 8192 takes 263 to 288 us (3.8 to 4.2 PF), with operands of zeros 205 to
// 257.  A round of tiles through 5120 columns takes 47 to 49 us (zeros 41): 3.0 until the
// first step is there, 39 for the 20 steps, 3.5 for the stores and 1.3 until the next
// tile.  The steps' matrix instructions are 17 of the 39 at 2.4 GHz: with two buffers a
// wave waits at each step's barrier for all that it has asked for, and nothing else is
// on its SIMD.  That first, then a tile's ends, and power last are why 4096 tokens
// through 13824 x 5120 (3.4 rounds, 183 us) reach 3.2 PF.
//
// A step is 256 columns: 128 bytes of codes and 8 scales of each row.  The codes go
// straight to one of two LDS buffers (global_load_lds) while the other one is
// multiplied.  The 16-byte pieces of a row are permuted by half its index, so that
// a read's lanes touch all 64 banks (two rows).  Weight row TN r + c of a wave's
// columns is row r of its tile c: a lane ends with TN consecutive columns.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "mx4_format.h"
#include "mx4_launch.h"
#include "mx4_sum.h"
#include "mx4_tile.h"

namespace mx4k {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int kStep = 256;            // columns a step
constexpr int kRowBytes = kStep / 2;
constexpr int kGroups = kStep / kGroup;

// cols >= kStep.
struct Mm4Args {
    const uint8_t *codes, *scales, *xcodes, *xscales;
    void* out;
    float* part;   // parts > 1: fp32 [parts][m x rows]
    int64_t m, rows, ldo;   // ldo: out's row pitch
    int cols, kind;
    TileGrid grid;
};

template <int S>
__device__ __forceinline__ f32x16 mfma4(const u32x4& a, uint32_t sa, const u32x4& b, uint32_t sb, const f32x16& c)
{
    const i32x8 x = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
    const i32x8 y = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(x, y, c, 4, 4, S, (int)sa, S, (int)sb);
}

// A wave's tile: TM x TN tiles of 32 x 32; the workgroup's: 2 x 2 waves.
template <int TM, int TN>
struct Shape {
    static constexpr int kBM = 64 * TM, kBN = 64 * TN;
    static constexpr int kA = 2 * TM, kW = 2 * TN;   // 16-byte pieces of the operands per thread and step
};

template <int TM, int TN>
struct Buffer {
    u32x4 a[64 * TM * (kRowBytes / 16)], w[64 * TN * (kRowBytes / 16)];
    u32x2 as[64 * TM], ws[64 * TN];
};

template <int TM, int TN>
__global__ __launch_bounds__(kThreads, 1) void k_mm4(Mm4Args g)
{
    typedef Shape<TM, TN> S;
    __shared__ Buffer<TM, TN> b0, b1;   // two objects, so that reads of one need not wait for what comes into the other
    int tm, tn, part;
    tile_of(g.grid, blockIdx.x, tm, tn, part);
    const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6), r = lane & 31, h = lane >> 5;
    const int wm = wave >> 1, wn = wave & 1;
    const int64_t m0 = (int64_t)tm * S::kBM, n0 = (int64_t)tn * S::kBN;
    const uint32_t pitch = (uint32_t)g.cols / 2;
    const int spitch = g.cols / kGroup;
    const int steps_all = (g.cols + kStep - 1) / kStep, first = part * g.grid.per_part;
    const int last = first + g.grid.per_part < steps_all ? first + g.grid.per_part : steps_all;

    // the rows t / 8 + 32 i of both operands, as offsets from the tile's first row
    uint32_t ao[S::kA], wo[S::kW];
#pragma unroll
    for (int i = 0; i < S::kA; ++i) {
        int64_t row = m0 + 32 * i + (t >> 3);
        row = (row < g.m ? row : g.m - 1) - m0;
        ao[i] = (uint32_t)row * pitch;
    }
#pragma unroll
    for (int i = 0; i < S::kW; ++i) {
        int64_t row = n0 + (i / TN) * (32 * TN) + TN * (t >> 3) + i % TN;
        row = (row < g.rows ? row : g.rows - 1) - n0;
        wo[i] = (uint32_t)row * pitch;
    }
    // and scale rows t of both (LDS order)
    int64_t aso, wso;
    {
        int64_t row = m0 + t % S::kBM;
        aso = ((row < g.m ? row : g.m - 1) - m0) * spitch;
        const int l = t % S::kBN;
        row = n0 + (l / (32 * TN)) * (32 * TN) + TN * (l & 31) + (l >> 5) % TN;
        wso = ((row < g.rows ? row : g.rows - 1) - n0) * spitch;
    }
    const MX4_GLOBAL uint8_t* ap = (const MX4_GLOBAL uint8_t*)g.xcodes + m0 * pitch;
    const MX4_GLOBAL uint8_t* wp = (const MX4_GLOBAL uint8_t*)g.codes + n0 * pitch;
    const MX4_GLOBAL uint8_t* asp = (const MX4_GLOBAL uint8_t*)g.xscales + m0 * spitch + aso;
    const MX4_GLOBAL uint8_t* wsp = (const MX4_GLOBAL uint8_t*)g.scales + n0 * spitch + wso;

    // the codes of a step: wave instructions of eight rows each; piece p of row i lies at p ^ (i / 2 & 7), and this
    // thread fetches what belongs into slot t % 8 of rows t / 8 + 32 i
    const int slot = t & 7, piece = slot ^ ((t >> 4) & 7);
    auto fetch = [&](Buffer<TM, TN>& b, int step, auto from, auto to) {
        const int left = spitch - step * kGroups;
        // a piece past the row's end: the step's first one, under scales of 0
        const uint32_t at = (uint32_t)step * kRowBytes + (piece < left ? 16 * piece : 0);
#pragma unroll
        for (int i = 0; i < S::kA + S::kW; ++i) {
            if (i < from || i >= to) continue;
            const MX4_GLOBAL uint8_t* src = i < S::kA ? ap + (ao[i < S::kA ? i : 0] + at) : wp + (wo[i < S::kA ? 0 : i - S::kA] + at);
            u32x4* dst = (i < S::kA ? b.a + 256 * i : b.w + 256 * (i - S::kA)) + 64 * wave;
            __builtin_amdgcn_global_load_lds((const MX4_GLOBAL uint32_t*)src, (MX4_LDS uint32_t*)dst, 16, 0, 0);
        }
    };
    auto clamp = [&](int step) { return step < last ? step : last - 1; };
    uint64_t ras, rws;
    auto fetch_scales = [&](int step) {
        const int at = step * kGroups + kGroups <= spitch ? step * kGroups : spitch - kGroups;
        __builtin_memcpy(&ras, (const uint8_t*)asp + at, 8);
        __builtin_memcpy(&rws, (const uint8_t*)wsp + at, 8);
    };
    auto store_scales = [&](Buffer<TM, TN>& b, int step) {
        // past the row's end, and past the last step: scales 0, 2^-254 for the two, so that those products are 0 in
        // fp32 whatever the codes
        const int left = spitch - step * kGroups, shift = left >= kGroups || left <= 0 ? 0 : 8 * (kGroups - left);
        const uint64_t in = step < last ? ~0ull : 0ull;
        // threads past the tile's rows write the rows of others once more, to the same values
        b.as[t % S::kBM] = __builtin_bit_cast(u32x2, ras >> shift & in);
        b.ws[t % S::kBN] = __builtin_bit_cast(u32x2, rws >> shift & in);
    };
    typedef std::integral_constant<int, 0> Zero;
    typedef std::integral_constant<int, (S::kA + S::kW) / 3> Third;
    typedef std::integral_constant<int, 2 * (S::kA + S::kW) / 3> TwoThirds;
    typedef std::integral_constant<int, S::kA + S::kW> All;

    f32x16 acc[TM][TN] = {};
    u32x4 fa[2][TM], fw[2][TN];
    uint32_t sa[TM], sw[TN];
    const uint32_t pick = h ? 0x07050301u : 0x06040200u;   // this half's scales of the four sub-steps
    u32x2 na[TM], nw[TN];
    auto frags = [&](const Buffer<TM, TN>& b, int s, int to) {
        const int at = r * 8 + ((2 * s + h) ^ ((r >> 1) & 7));
        // in the order of their use
        fa[to][0] = b.a[wm * TM * 256 + at];
#pragma unroll
        for (int i = 0; i < TN; ++i) fw[to][i] = b.w[(wn * TN + i) * 256 + at];
#pragma unroll
        for (int i = 1; i < TM; ++i) fa[to][i] = b.a[(wm * TM + i) * 256 + at];
    };
    // the first sub-step's fragments and the scales of a step
    auto begin = [&](const Buffer<TM, TN>& b) {
        frags(b, 0, 0);
#pragma unroll
        for (int i = 0; i < TM; ++i) na[i] = b.as[(wm * TM + i) * 32 + r];
#pragma unroll
        for (int i = 0; i < TN; ++i) nw[i] = b.ws[(wn * TN + i) * 32 + r];
    };
#define MX4_MULTIPLY(SUB, FROM)                                                                            \
    _Pragma("unroll") for (int i = 0; i < TM; ++i)                                                         \
        _Pragma("unroll") for (int j = 0; j < TN; ++j)                                                     \
            acc[i][j] = mfma4<SUB>(fa[FROM][i], sa[i], fw[FROM][j], sw[j], acc[i][j])
    // One step out of `now`.  The codes of the step after it are on their way to `next` (their first third was asked for
    // in the step before).  Steps past the last one are the last one again, fetched and not used.
    auto body = [&](Buffer<TM, TN>& now, Buffer<TM, TN>& next, int step) {
#pragma unroll
        for (int i = 0; i < TM; ++i) sa[i] = __builtin_amdgcn_perm(na[i][1], na[i][0], pick);
#pragma unroll
        for (int j = 0; j < TN; ++j) sw[j] = __builtin_amdgcn_perm(nw[j][1], nw[j][0], pick);
        fetch(next, clamp(step + 1), Third{}, TwoThirds{});
        frags(now, 1, 1);
        MX4_MULTIPLY(0, 0);
        spread<TM * TN, TM + TN, 0, TwoThirds::value - Third::value>();
        fetch(next, clamp(step + 1), TwoThirds{}, All{});
        frags(now, 2, 0);
        MX4_MULTIPLY(1, 1);
        spread<TM * TN, TM + TN, 0, All::value - TwoThirds::value>();
        frags(now, 3, 1);
        MX4_MULTIPLY(2, 0);
        spread<TM * TN, TM + TN, 0, 0>();
        __builtin_amdgcn_s_waitcnt(kVmcnt0);
        store_scales(next, step + 1);
        __syncthreads();
        begin(next);
        fetch_scales(clamp(step + 2));
        fetch(now, clamp(step + 2), Zero{}, Third{});
        MX4_MULTIPLY(3, 1);
        spread<TM * TN, 2 * (TM + TN), 0, Third::value + 2>();
    };
    fetch_scales(first);
    fetch(b0, first, Zero{}, All{});
    __builtin_amdgcn_s_waitcnt(kVmcnt0);
    store_scales(b0, first);
    __syncthreads();
    begin(b0);
    fetch_scales(clamp(first + 1));
    fetch(b1, clamp(first + 1), Zero{}, Third{});
    // Pairs of steps, and an odd one by itself (600 tokens through 4232 x 544 6.8 us, with a fourth step 7.5).  The large
    // tile's sums leave no registers for another way out (4096 through 13824 x 5120 192 us for 186): there an odd one is
    // followed by one under scales of 0.
    constexpr bool kTail = TM < 4;
    for (int step = first; step + kTail < last; step += 2) {
        body(b0, b1, step);
        body(b1, b0, step + 1);
    }
    if constexpr (kTail) {
        if ((last - first) % 2) body(b0, b1, last - 1);
    }
    __builtin_amdgcn_s_waitcnt(kVmcnt0);   // nothing may come into LDS after the end
#undef MX4_MULTIPLY

    store_tile<TM, TN>(acc, g.out, g.part, g.kind, g.grid, part, g.m, g.rows, g.ldo, m0, n0, wm, wn, r, h);
}

template <int TM, int TN>
hipError_t mm4_go(Mm4Args a, hipStream_t s)
{
    const unsigned blocks = (unsigned)(a.grid.mt * a.grid.nt * a.grid.parts);
    k_mm4<TM, TN><<<blocks, kThreads, 0, s>>>(a);
    return hipGetLastError();
}

// 4096 tokens through 4096 x 1024 .. 13824 take 22.0 .. 113 us, 333 through 2048 x 8192 in 1, 2, 4, 8 parts 28.5, 20.6,
// 16.3 and 18.7.
constexpr TileCosts kCosts = {1.80, 14.0, 0.90, 3.2, 1.50, 7.0};

TilePlan mm4_plan(int64_t rows, int64_t cols, int64_t m) { return tile_plan(m, rows, (int)ceil_div(cols, kStep), kCosts); }

}  // namespace

double mm4_tiled_us(int64_t rows, int64_t cols, int64_t m)
{
    double us;
    tile_plan(m, rows, (int)ceil_div(cols, kStep), kCosts, &us);
    return us;
}

size_t mm4_tiled_ws(int64_t rows, int64_t cols, int64_t m)
{
    return plan_ws(mm4_plan(rows, cols, m), m, rows);
}

hipError_t launch_mm4_tiled(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols,
                            const uint8_t* xcodes, const uint8_t* xscales, int64_t m, void* out, int out_kind,
                            float* part, hipStream_t s)
{
    const TilePlan p = mm4_plan(rows, cols, m);
    Mm4Args a{codes, scales, xcodes, xscales, out, part, m, rows, rows, (int)cols, out_kind, p.big};
    if (p.big.nt > 0) {
        const int64_t done = 256 * (int64_t)p.big.nt;
        if (p.small.nt > 0) a.rows = done;
        const hipError_t e = mm4_go<4, 4>(a, s);
        if (e != hipSuccess || p.small.nt == 0) return e;
        a.codes += done * (cols / 2);
        a.scales += done * (cols / kGroup);
        a.out = (char*)out + done * (out_kind == kOutFp32 ? 4 : 2);
        a.rows = rows - done;
    }
    a.grid = p.small;
    const hipError_t e = mm4_go<2, 2>(a, s);
    if (e != hipSuccess || p.small.parts == 1) return e;
    return launch_split_sum(part, p.small.parts, m, a.rows, a.out, rows, out_kind, s);
}

}  // namespace mx4k
