// k_mx4_mm.hip -- the product of a 16-bit operand and a microscaled 4-bit weight
// on gfx950 matrix cores: out = x W^T (forward) or x W (backward).
//
// v_mfma_f32_32x32x16; a 256 x 256 output tile by four waves of 128 x 128, one per
// SIMD.  A step is 64 of the reduction: x's rows (128 bytes each) and the weight's
// codes go straight into one of three or four LDS buffers (one multiplied, one
// complete, the others on their way).  The codes leave LDS as codes: each wave
// converts the fragments it multiplies, two values an instruction, in the shadow of
// the matrix instructions; the weight is never written anywhere in 16 bits.
//
// A step has four sub-steps of 16.  While one is multiplied, the next one's weight
// is converted, its x read, and the codes of the one after it.  The barrier stands
// before the third, when the next step's buffer is first read.
//
// Forward: lane (r, h) reads row r's 16 bytes of block h of the step, one scale
// under which its four dwords become the fragments of the four sub-steps
// (reduction index 32 h + 8 f + j).  Weight row TN r + c of a wave's is row r of its
// tile c, so that a lane ends with TN consecutive columns.  The scales of twelve or
// sixteen steps are loaded at once and a round ahead, so that a step waits by count
// for what it reads and for no more: 7% of the large product, a quarter where a tile
// has the compute unit alone.
//
// Backward the reduction runs over the weight's rows, whose scales differ.  The
// transposing read gives lane (r, h) the bytes (two columns) of rows 32 h + 8 f + j,
// j = 0 .. 7, in one register pair; each byte is converted under its row's scale,
// and the halves of two rows are put together as pairs of the fragments.  Of a
// wave's 128 columns lane r = 8 q + i has 32 q + 2 i, + 1, + 16, + 17 (one scale
// group); neighbours exchange a pair at the end and hold four in a row.
//
// x's 16-byte pieces lie permuted by half their row's index, so that a read's lanes
// touch all 64 banks (two rows of 128 bytes), and forward the codes' by an eighth of
// it.  Reads alone run 1.9 times as fast as with a permutation by the index itself;
// the products, which other things bound, take the same time.  The transposing reads
// of the codes backward are not free of conflicts: 0.17 of the cycles that LDS is
// busy, where forward there are none.
//
// 4096 tokens through 13824 x 5120 in bf16 take 445 us forward and 459 backward (1.30
// and 1.26 PF; the library's product alone, of a weight in 16 bits, 487 and 628), 8192 x
// 8192 x 8192 780 to 790 each.  What is left is one wave a SIMD that waits at each
// step's barrier, a tile's ends (12 us a round), and power: with operands of zeros 8192
// x 8192 x 8192 takes 621 us of 781 forward, 641 of 788 backward.  Eight waves of 128 x
// 64 took 3% longer.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "mx4_format.h"
#include "mx4_launch.h"
#include "mx4_sum.h"
#include "mx4_tile.h"

namespace mx4k {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

constexpr int kStep = 64;             // of the reduction
constexpr uint32_t kFar = 0x80000000u;

struct MmArgs {
    const uint8_t *codes, *scales;    // W [rows x cols]
    const uint16_t* x;                // [m x kred]
    void* out;                        // [m x ncol], row pitch ldo
    float* part;                      // parts > 1: fp32 [parts][m x ncol]
    int64_t m, ncol, ldo;
    int cols, kred, kind;
    TileGrid grid;
};

template <int DT>
__device__ __forceinline__ f32x16 mfma16(const u32x4& a, const u32x4& b, const f32x16& c)
{
    if constexpr (DT == 0)
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// ---- forward

template <int TM, int TN>
struct Buffer {
    u32x4 a[64 * TM * 8];       // x: 64 TM rows of 128 bytes
    u32x4 w[64 * TN * 2];       // codes: 64 TN rows of 32 bytes
};

struct NoBuffer {};             // in the fourth one's place

// Scales come kQ steps at a time, through registers, while the steps before them are
// multiplied: one load a step would have to be waited for with the step's own.
template <int TN, int NB>
struct Scales {
    static constexpr int kQ = 4 * NB;                            // steps
    static constexpr int kPitch = 2 * kQ + 4;    // of a weight row, in bytes; 4 move the next one's banks
    uint32_t s[2][64 * TN * kPitch / 4];
};

// A barrier that waits for this wave's LDS instructions and not, as a fence would, for
// all that is on its way from memory into LDS: the caller has waited for as much of
// that as the others will read.
__device__ __forceinline__ void sync_lds()
{
    __asm__ volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xc07f);   // lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    __asm__ volatile("" ::: "memory");
}

template <int DT, int TM, int TN, int NB>
__global__ __launch_bounds__(kThreads, 1) void k_mm(MmArgs g)
{
    typedef Buffer<TM, TN> Buf;
    typedef Scales<TN, NB> Sc;
    __shared__ Buf b0, b1, b2;   // objects of their own, so that reads of one need not wait for what comes into another
    __shared__ std::conditional_t<NB == 4, Buf, NoBuffer> b3;
    __shared__ Sc sc;
    static_assert(NB * sizeof(Buf) + sizeof(Sc) < 160 * 1024, "a compute unit's LDS");
    constexpr int kBM = 64 * TM, kBN = 64 * TN;
    constexpr int kA = 2 * TM, kW = TN / 2;   // 16-byte pieces per thread and step
    int tm, tn, part;
    tile_of(g.grid, blockIdx.x, tm, tn, part);
    const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6), r = lane & 31, h = lane >> 5;
    const int wm = wave >> 1, wn = wave & 1;
    const int64_t m0 = (int64_t)tm * kBM, n0 = (int64_t)tn * kBN;
    const int steps_all = (g.kred + kStep - 1) / kStep, first = part * g.grid.per_part;
    const int last = first + g.grid.per_part < steps_all ? first + g.grid.per_part : steps_all;
    const uint32_t wpitch = (uint32_t)g.cols / 2;
    const int spitch = g.cols / kGroup;

    // x: this thread fetches slot t % 8 of rows t / 8 + 32 i, which holds piece (t % 8) ^ (row / 2 % 8)
    const uint32_t xpitch = (uint32_t)g.kred * 2;
    const int64_t xleft = (g.m - m0 < kBM ? g.m - m0 : kBM) * xpitch;
    const __amdgpu_buffer_rsrc_t xr =
        __builtin_amdgcn_make_buffer_rsrc((void*)(g.x + m0 * g.kred), 0, (int)xleft, 0x00027000);
    const int piece = (t & 7) ^ ((t >> 4) & 7);
    const uint32_t ao = (uint32_t)(t >> 3) * xpitch + 16 * piece;
    auto fetch_x = [&](Buf& b, int step, auto from, auto to) {
        const bool in = (step < last) & (step * kStep + 8 * piece < g.kred);
        const uint32_t at = in ? ao + (uint32_t)step * (2 * kStep) : kFar;
#pragma unroll
        for (int i = from; i < to; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(xr, (MX4_LDS uint32_t*)(b.a + 256 * i + 64 * wave), 16,
                                                     at + (uint32_t)i * (32 * xpitch), 0, 0, 0);
    };
    // codes: two pieces a row, LDS row t / 2 + 128 i, slot (t & 1) holds piece (t & 1) ^ (row / 8 & 1).
    const MX4_GLOBAL uint8_t* wp = (const MX4_GLOBAL uint8_t*)g.codes;
    int64_t wo[kW];
#pragma unroll
    for (int i = 0; i < kW; ++i) {
        const int l = (t >> 1) + 128 * i;
        const int64_t n = n0 + l / (32 * TN) * (32 * TN) + TN * (l % 32) + l / 32 % TN;
        wo[i] = (n < g.ncol ? n : g.ncol - 1) * wpitch;
    }
    auto fetch_w = [&](Buf& b, int step) {
        const int s = step < last ? step : last - 1;
#pragma unroll
        for (int i = 0; i < kW; ++i) {
            const int p = (t & 1) ^ ((t >> 4) & 1);   // past the row's end: the step's first piece, under scale 0
            const MX4_GLOBAL uint8_t* src = wp + wo[i] + (s * (kStep / 2) + (s * kStep + 32 * p < g.kred ? 16 * p : 0));
            __builtin_amdgcn_global_load_lds((const MX4_GLOBAL uint32_t*)src, (MX4_LDS uint32_t*)(b.w + 256 * i + 64 * wave), 16, 0, 0);
        }
    };
    const MX4_GLOBAL uint8_t* sp = (const MX4_GLOBAL uint8_t*)g.scales;
    constexpr int kQ = Sc::kQ;
    // kU eights of bytes a thread, four steps of a row each
    constexpr int kRowUnits = kQ / 4, kUnits = 64 * TN * kRowUnits, kU = (kUnits + kThreads - 1) / kThreads;
    typedef uint64_t Eights[kU];
    auto load_scales = [&](Eights& ls, int base) {
        const MX4_GLOBAL uint8_t* row[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int l = (t * kU + u) / kRowUnits;
            const int64_t n = n0 + l / (32 * TN) * (32 * TN) + TN * (l % 32) + l / 32 % TN;
            row[u] = sp + (n < g.ncol ? n : g.ncol - 1) * spitch;
        }
        if (spitch >= 8) {
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                const int o = 2 * base + 8 * ((t * kU + u) % kRowUnits);
                __builtin_memcpy(ls + u, (const uint8_t*)row[u] + (o + 8 <= spitch ? o : spitch - 8), 8);
            }
        } else {
            for (int u = 0; u < kU; ++u) {
                ls[u] = 0;
                for (int k = 0; k < spitch; ++k) ls[u] |= (uint64_t)row[u][k] << (8 * (8 - spitch + k));   // as the load above
            }
        }
    };
    // past the row's, the weight's or the part's end: 0 and not NaN, against zeros of x
    auto store_scales = [&](const Eights& ls, int base) {
        uint32_t* to = sc.s[(base - first) / kQ & 1];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int unit = (t * kU + u) % kRowUnits, left = spitch - (2 * base + 8 * unit), steps = last - (base + 4 * unit);
            uint64_t v = left >= 8 ? ls[u] : left <= 0 ? 0 : ls[u] >> (64 - 8 * left);
            v = steps >= 4 ? v : steps <= 0 ? 0 : v & ((1ull << (16 * steps)) - 1);
            uint32_t* p = to + ((t * kU + u) / kRowUnits) * (Sc::kPitch / 4) + 2 * unit;
            if (t * kU + u < kUnits) {
                p[0] = (uint32_t)v;
                p[1] = (uint32_t)(v >> 32);
            }
        }
    };
    // the bytes before a step's
    auto scales_of = [&](int step) {
        return ((step - first) / kQ & 1) * (int)(sizeof(sc) / 2) + 2 * ((step - first) % kQ);
    };

    f32x16 acc[TM][TN] = {};
    u32x4 fa[2][TM], fw[2][TN];
    auto frags = [&](const Buf& b, int f, int to) {
        const int at = r * 8 + ((4 * h + f) ^ ((r >> 1) & 7));
#pragma unroll
        for (int i = 0; i < TM; ++i) fa[to][i] = b.a[(wm * TM + i) * 256 + at];
    };
    // a step's codes and scales, now and next
    u32x4 code[2][TN];
    uint32_t scale[2][TN];
    auto read_step = [&](const Buf& b, int step) {
        const int at = scales_of(step) + h;
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            const int l = (wn * TN + j) * 32 + r;
            code[1][j] = b.w[l * 2 + (h ^ ((l >> 3) & 1))];
            scale[1][j] = ((const uint8_t*)&sc)[at + l * Sc::kPitch];
        }
    };
    auto decode = [&](int f, int which, int to) {   // sub-step f of step `which`
#pragma unroll
        for (int j = 0; j < TN; ++j) fw[to][j] = decode8<DT>(code[which][j][f], scale_arg(scale[which][j]));
    };
    auto multiply = [&](int from) {
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j) acc[i][j] = mfma16<DT>(fa[from][i], fw[from][j], acc[i][j]);
    };
    constexpr int kN = TM * TN, kReads = TM, kValu = 4 * TN;
    typedef std::integral_constant<int, 0> P0;
    // how much of x is asked for in each half of a step: all right after the barrier where that does not hold up LDS
    typedef std::integral_constant<int, (NB > 3) ? kA / 2 : kA / 4> P1;
    typedef std::integral_constant<int, (NB > 3) ? kA : kA * 5 / 8> P2;
    typedef std::integral_constant<int, kA> All;

    // One step out of `now`; `next` is on its way until the barrier, `then` (NB - 1 steps on) is asked for after it.
    // Steps past the last one are zeros under scales of 0.
    constexpr int kAhead = (NB - 3) * (kA + kW);   // loads of the steps after the next one
    auto body = [&](Buf& now, Buf& next, Buf& then, int step) {
        fetch_x(next, step + 1, P2{}, All{});
        frags(now, 1, 1);
        decode(1, 0, 1);
        multiply(0);
        spread<kN, kReads, kValu, kA - P2::value>();
        frags(now, 2, 0);
        decode(2, 0, 0);
        multiply(1);
        spread<kN, kReads, kValu, 0>();
        __builtin_amdgcn_s_waitcnt(kVmcnt0 | (kAhead & 15) | kAhead >> 4 << 14);
        sync_lds();
        fetch_w(then, step + NB - 1);
        fetch_x(then, step + NB - 1, P0{}, P1{});
        frags(now, 3, 1);
        decode(3, 0, 1);
        read_step(next, step + 1);
        multiply(0);
        spread<kN, TM + 2 * TN, kValu, kW + P1::value>();
        fetch_x(then, step + NB - 1, P1{}, P2{});
        frags(next, 0, 0);
        decode(0, 1, 0);
        multiply(1);
        spread<kN, kReads, kValu, P2::value - P1::value>();
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            code[0][j] = code[1][j];
            scale[0][j] = scale[1][j];
        }
    };

    // Steps left over by the buffers' turns come after the loop (600 tokens through 4232 x 544, nine steps: 9.0 us, with
    // twelve 10.2).  The large tile's sums leave no registers for a second way out of it (4096 tokens through 13824 x 5120
    // 515 us for 451): there they are followed by steps of zeros.
    constexpr bool kTail = TM < 4;
    Eights ls, ls0;
    load_scales(ls0, first);
    load_scales(ls, first + kQ);
    fetch_w(b0, first);
    fetch_x(b0, first, P0{}, All{});
    fetch_w(b1, first + 1);
    if constexpr (NB == 4) {
        fetch_x(b1, first + 1, P0{}, All{});
        fetch_w(b2, first + 2);
        fetch_x(b2, first + 2, P0{}, All{});
    } else {
        fetch_x(b1, first + 1, P0{}, P2{});
    }
    store_scales(ls0, first);
    constexpr int kFirst = kAhead + kW + P2::value;
    __builtin_amdgcn_s_waitcnt(kVmcnt0 | (kFirst & 15) | kFirst >> 4 << 14);
    sync_lds();
    frags(b0, 0, 0);
    read_step(b0, first);
#pragma unroll
    for (int j = 0; j < TN; ++j) {
        code[0][j] = code[1][j];
        scale[0][j] = scale[1][j];
    }
    decode(0, 0, 0);
    for (int base = first; base < last; base += kQ) {
        // into the place of the scales before this round's: none of those is read any more, and a barrier follows
        if (base + kQ < last) {
            store_scales(ls, base + kQ);
            load_scales(ls, base + 2 * kQ);
        }
        const int end = base + kQ < last ? base + kQ : last;
        for (int step = base; step + (kTail ? NB - 1 : 0) < end; step += NB) {
            if constexpr (NB == 4) {
                body(b0, b1, b3, step);
                body(b1, b2, b0, step + 1);
                body(b2, b3, b1, step + 2);
                body(b3, b0, b2, step + 3);
            } else {
                body(b0, b1, b2, step);
                body(b1, b2, b0, step + 1);
                body(b2, b0, b1, step + 2);
            }
        }
    }
    if constexpr (kTail) {
        const int left = (last - first) % NB, step = last - left;
        if (left > 0) {
            if constexpr (NB == 4) body(b0, b1, b3, step);
            else body(b0, b1, b2, step);
            if (left > 1) {
                body(b1, b2, b0, step + 1);
                if constexpr (NB == 4) {
                    if (left > 2) body(b2, b3, b1, step + 2);
                }
            }
        }
    }
    __builtin_amdgcn_s_waitcnt(kVmcnt0);   // nothing may come into LDS after the end
    store_tile<TM, TN>(acc, g.out, g.part, g.kind, g.grid, part, g.m, g.ncol, g.ldo, m0, n0, wm, wn, r, h);
}

// ---- backward

template <int TM, int TN>
struct BackBuffer {
    u32x4 a[64 * TM * 8];       // x: 64 TM rows of 128 bytes
    u32x4 w[64 * TN * 2];       // codes: 64 rows of 32 TN bytes
    uint8_t s[128 * TN];        // scales: [2 TN groups][64 rows]
};

__device__ __forceinline__ uint32_t low16(uint32_t a, uint32_t b) { return __builtin_amdgcn_perm(b, a, 0x05040100u); }
__device__ __forceinline__ uint32_t high16(uint32_t a, uint32_t b) { return __builtin_amdgcn_perm(b, a, 0x07060302u); }

template <int DT, int TM, int TN>
__global__ __launch_bounds__(kThreads, 1) void k_mm_back(MmArgs g)
{
    typedef BackBuffer<TM, TN> Buf;
    __shared__ Buf b0, b1, b2;   // objects of their own, so that reads of one need not wait for what comes into another
    constexpr int kBM = 64 * TM, kBN = 64 * TN;
    constexpr int kA = 2 * TM, kW = TN / 2;   // 16-byte pieces per thread and step
    int tm, tn, part;
    tile_of(g.grid, blockIdx.x, tm, tn, part);
    const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6), r = lane & 31, h = lane >> 5;
    const int wm = wave >> 1, wn = wave & 1;
    const int64_t m0 = (int64_t)tm * kBM, n0 = (int64_t)tn * kBN;
    const int steps_all = (g.kred + kStep - 1) / kStep, first = part * g.grid.per_part;
    const int last = first + g.grid.per_part < steps_all ? first + g.grid.per_part : steps_all;
    const uint32_t wpitch = (uint32_t)g.cols / 2;
    const int spitch = g.cols / kGroup;

    // x: this thread fetches slot t % 8 of rows t / 8 + 32 i, which holds piece (t % 8) ^ (row / 2 % 8)
    const uint32_t xpitch = (uint32_t)g.kred * 2;
    const int64_t xleft = (g.m - m0 < kBM ? g.m - m0 : kBM) * xpitch;
    const __amdgpu_buffer_rsrc_t xr =
        __builtin_amdgcn_make_buffer_rsrc((void*)(g.x + m0 * g.kred), 0, (int)xleft, 0x00027000);
    const int piece = (t & 7) ^ ((t >> 4) & 7);
    const uint32_t ao = (uint32_t)(t >> 3) * xpitch + 16 * piece;
    auto fetch_x = [&](Buf& b, int step, auto from, auto to) {
        const bool in = (step < last) & (step * kStep + 8 * piece < g.kred);
        const uint32_t at = in ? ao + (uint32_t)step * (2 * kStep) : kFar;
#pragma unroll
        for (int i = from; i < to; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(xr, (MX4_LDS uint32_t*)(b.a + 256 * i + 64 * wave), 16,
                                                     at + (uint32_t)i * (32 * xpitch), 0, 0, 0);
    };
    // codes: 2 TN pieces a row, row t / (2 TN) of the step (and 32 below with TN = 4), permuted by row % (2 TN).
    const MX4_GLOBAL uint8_t* wp = (const MX4_GLOBAL uint8_t*)g.codes;
    int64_t wo[kW];
#pragma unroll
    for (int i = 0; i < kW; ++i) {
        const int64_t c = n0 + 32 * ((t % (2 * TN)) ^ (t / (2 * TN) % (2 * TN)));
        wo[i] = (c < g.ncol ? c : n0) / 2;
    }
    auto fetch_w = [&](Buf& b, int step) {
        const int s = step < last ? step : last - 1;
#pragma unroll
        for (int i = 0; i < kW; ++i) {
            const int n = s * kStep + t / (2 * TN) + 32 * i;
            const MX4_GLOBAL uint8_t* src = wp + wo[i] + (int64_t)(n < g.kred ? n : g.kred - 1) * wpitch;
            __builtin_amdgcn_global_load_lds((const MX4_GLOBAL uint32_t*)src, (MX4_LDS uint32_t*)(b.w + 256 * i + 64 * wave), 16, 0, 0);
        }
    };
    // scales: group t % 4 + 4 i of row t / 4
    const MX4_GLOBAL uint8_t* sp = (const MX4_GLOBAL uint8_t*)g.scales;
    uint32_t rs[kW];
    auto fetch_s = [&](int step) {
        const int s = step < last ? step : last - 1;
#pragma unroll
        for (int i = 0; i < kW; ++i) {
            const int n = s * kStep + (t >> 2);
            const int64_t c = n0 / kGroup + (t & 3) + 4 * i;
            rs[i] = sp[(int64_t)(n < g.kred ? n : g.kred - 1) * spitch + (c < g.ncol / kGroup ? c : 0)];
        }
    };
    auto store_s = [&](Buf& b, int step) {
#pragma unroll
        for (int i = 0; i < kW; ++i) {
            // past the end: 0 and not NaN, against zeros of x
            const bool in = (step < last) & (step * kStep + (t >> 2) < g.kred);
            b.s[((t & 3) + 4 * i) * 64 + (t >> 2)] = (uint8_t)(in ? rs[i] : 0u);
        }
    };

    f32x16 acc[TM][TN] = {};
    u32x4 fa[2][TM], fw[2][TN];
    auto frags = [&](const Buf& b, int f, int to) {
        const int at = r * 8 + ((4 * h + f) ^ ((r >> 1) & 7));
#pragma unroll
        for (int i = 0; i < TM; ++i) fa[to][i] = b.a[(wm * TM + i) * 256 + at];
    };
    // the next sub-step's codes and scales, and those of the one after it
    u32x2 raw[2][TN / 2], rawscale[2];
    // the transposing read: of 16 lanes, lanes 2 j and 2 j + 1 give eight bytes each of row j, lane i takes byte i of all
    const int trow = (lane & 15) >> 1, thalf = lane & 1, tquad = (lane >> 4) & 1;
    auto read_sub = [&](const Buf& b, int f, int to) {
#pragma unroll
        for (int k = 0; k < TN / 2; ++k) {
            const int p = TN == 4 ? wn * 4 + 2 * tquad + thalf : wn * 2 + tquad, half = TN == 4 ? k : thalf;
            const int row = 32 * h + 8 * f + trow;
            const uint8_t* at = (const uint8_t*)b.w + row * (32 * TN) + 16 * (p ^ (row % (2 * TN))) + 8 * half;
            typedef int i32x2 __attribute__((ext_vector_type(2)));
            raw[to][k] = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr8_b64_v2i32((MX4_LDS i32x2*)at));
        }
        rawscale[to] = *(const u32x2*)(b.s + (wn * TN + r * TN / 32) * 64 + 32 * h + 8 * f);
    };
    auto decode = [&](int from, int to) {
        const uint32_t s0 = rawscale[from][0], s1 = rawscale[from][1];
#pragma unroll
        for (int k = 0; k < TN / 2; ++k) {
            const uint32_t c0 = raw[from][k][0], c1 = raw[from][k][1];
            const uint32_t v[8] = {decode2<DT, 0>(c0, byte_arg<0>(s0)), decode2<DT, 1>(c0, byte_arg<1>(s0)),
                                   decode2<DT, 2>(c0, byte_arg<2>(s0)), decode2<DT, 3>(c0, byte_arg<3>(s0)),
                                   decode2<DT, 0>(c1, byte_arg<0>(s1)), decode2<DT, 1>(c1, byte_arg<1>(s1)),
                                   decode2<DT, 2>(c1, byte_arg<2>(s1)), decode2<DT, 3>(c1, byte_arg<3>(s1))};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                fw[to][2 * k][j] = low16(v[2 * j], v[2 * j + 1]);
                fw[to][2 * k + 1][j] = high16(v[2 * j], v[2 * j + 1]);
            }
        }
    };
    auto multiply = [&](int from) {
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j) acc[i][j] = mfma16<DT>(fa[from][i], fw[from][j], acc[i][j]);
    };
    constexpr int kN = TM * TN, kReads = TM + TN / 2 + 1, kValu = 8 * TN + 8;
    typedef std::integral_constant<int, 0> P0;
    typedef std::integral_constant<int, kA / 4> P1;
    typedef std::integral_constant<int, kA * 5 / 8> P2;
    typedef std::integral_constant<int, kA> All;

    // One step out of `now`; `next` is on its way until the barrier, `then` is asked for after it.  Steps past the last
    // one are zeros under scales of 0.
    auto body = [&](Buf& now, Buf& next, Buf& then, int step) {
        fetch_x(next, step + 1, P2{}, All{});
        frags(now, 1, 1);
        read_sub(now, 2, 0);
        decode(1, 1);
        multiply(0);
        spread<kN, kReads, kValu, kA - P2::value>();
        frags(now, 2, 0);
        read_sub(now, 3, 1);
        decode(0, 0);
        multiply(1);
        spread<kN, kReads, kValu, 0>();
        __builtin_amdgcn_s_waitcnt(kVmcnt0);
        store_s(next, step + 1);
        __syncthreads();
        fetch_s(step + 2);
        fetch_w(then, step + 2);
        fetch_x(then, step + 2, P0{}, P1{});
        frags(now, 3, 1);
        read_sub(next, 0, 0);
        decode(1, 1);
        multiply(0);
        spread<kN, kReads, kValu, 2 * kW + P1::value>();
        fetch_x(then, step + 2, P1{}, P2{});
        frags(next, 0, 0);
        read_sub(next, 1, 1);
        decode(0, 0);
        multiply(1);
        spread<kN, kReads, kValu, P2::value - P1::value>();
    };

    fetch_s(first);
    fetch_w(b0, first);
    fetch_x(b0, first, P0{}, All{});
    __builtin_amdgcn_s_waitcnt(kVmcnt0);
    store_s(b0, first);
    __syncthreads();
    fetch_s(first + 1);
    fetch_w(b1, first + 1);
    fetch_x(b1, first + 1, P0{}, P2{});
    frags(b0, 0, 0);
    read_sub(b0, 0, 0);
    read_sub(b0, 1, 1);
    decode(0, 0);
    constexpr bool kTail = TM < 4;   // as forward (333 tokens through 8192 x 2048 25.6 us for 26.5)
    for (int step = first; step + (kTail ? 2 : 0) < last; step += 3) {
        body(b0, b1, b2, step);
        body(b1, b2, b0, step + 1);
        body(b2, b0, b1, step + 2);
    }
    if constexpr (kTail) {
        const int left = (last - first) % 3, step = last - left;
        if (left > 0) {
            body(b0, b1, b2, step);
            if (left > 1) body(b1, b2, b0, step + 1);
        }
    }
    __builtin_amdgcn_s_waitcnt(kVmcnt0);   // nothing may come into LDS after the end
    store_tile<TM, TN, TN == 4>(acc, g.out, g.part, g.kind, g.grid, part, g.m, g.ncol, g.ldo, m0, n0, wm, wn, r, h);
}

// NB: the forward kernel's buffers.
template <int TM, int TN, int NB>
hipError_t mm_go(int dtype, bool forward, const MmArgs& a, hipStream_t s)
{
    const unsigned blocks = (unsigned)(a.grid.mt * a.grid.nt * a.grid.parts);
    if (dtype == 0) {
        if (forward) k_mm<0, TM, TN, NB><<<blocks, kThreads, 0, s>>>(a);
        else k_mm_back<0, TM, TN><<<blocks, kThreads, 0, s>>>(a);
    } else {
        if (forward) k_mm<1, TM, TN, NB><<<blocks, kThreads, 0, s>>>(a);
        else k_mm_back<1, TM, TN><<<blocks, kThreads, 0, s>>>(a);
    }
    return hipGetLastError();
}

// Backward and forward.  Forward up to 256 small tiles have four buffers and a compute unit each, more of them three
// and share it in pairs (128 tokens through 32768 x 4096 in 256 tiles 34.6 us, with three buffers 42.8; 256 in 512
// tiles 61 in pairs, 66 one after another).  Backward there are three: the same change was measured while both forms filled
// the steps left over by the buffers' turns up with zeros (333 tokens through 8192 x 2048 24.5 us for 26.5; 300 through
// 5120 x 13824, which are more tiles than compute units, 72 for 64), and not since they no longer do (25.5 to 27.6 now).
constexpr TileCosts kCosts[2] = {{1.58, 12.0, 0.67, 3.2, 0.98, 7.0}, {1.44, 13.0, 0.45, 3.3, 0.85, 7.0}};

TilePlan mm_plan(int64_t kred, int64_t ncol, int64_t m, bool forward, double* us = nullptr)
{
    return tile_plan(m, ncol, (int)ceil_div(kred, kStep), kCosts[forward], us);
}

}  // namespace

double mm_tiled_us(int64_t kred, int64_t ncol, int64_t m, bool forward)
{
    double us;
    mm_plan(kred, ncol, m, forward, &us);
    return us;
}

size_t mm_tiled_ws(int64_t kred, int64_t ncol, int64_t m, bool forward)
{
    return plan_ws(mm_plan(kred, ncol, m, forward), m, ncol);
}

hipError_t launch_mm_tiled(int dtype, const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols,
                           bool forward, const void* x, int64_t m, void* out, int out_kind, float* part, hipStream_t s)
{
    const int64_t kred = forward ? cols : rows, ncol = forward ? rows : cols;
    const TilePlan p = mm_plan(kred, ncol, m, forward);
    MmArgs a{codes, scales, static_cast<const uint16_t*>(x), out, part, m, ncol, ncol, (int)cols, (int)kred, out_kind, p.big};
    if (p.big.nt > 0) {
        const int64_t done = 256 * (int64_t)p.big.nt;
        if (p.small.nt > 0) a.ncol = done;
        const hipError_t e = mm_go<4, 4, 3>(dtype, forward, a, s);
        if (e != hipSuccess || p.small.nt == 0) return e;
        // the other columns: the weight's rows from there on, or its columns
        a.codes += forward ? done * (cols / 2) : done / 2;
        a.scales += forward ? done * (cols / kGroup) : done / kGroup;
        a.out = (char*)out + done * (out_kind == kOutFp32 ? 4 : 2);
        a.ncol = ncol - done;
    }
    a.grid = p.small;
    const bool pairs = (int64_t)p.small.mt * p.small.nt * p.small.parts > kCus;
    const hipError_t e = pairs ? mm_go<2, 2, 3>(dtype, forward, a, s) : mm_go<2, 2, 4>(dtype, forward, a, s);
    if (e != hipSuccess || p.small.parts == 1) return e;
    return launch_split_sum(part, p.small.parts, m, a.ncol, a.out, ncol, out_kind, s);
}

}  // namespace mx4k
