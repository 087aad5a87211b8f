// k_mx4_few.hip -- the microscaled products at few tokens, on gfx950 matrix
// cores.  The weights' codes are read once, 16 bytes a lane, and that read bounds
// the call; nothing of them goes through LDS.
//
//   forward   out[t, n] = sum_k x[t, k] W[n, k]
//   backward  out[t, k] = sum_n x[t, n] W[n, k]
//
// Forward: a wave takes kRT x 16 weight rows and every kWaves-th run of 512
// columns.  Lane (r, g) holds four blocks of 32 of row r, block 4 g + j in the j-th
// of four steps: one load each and one for their four scales.  In 16 bits a block
// makes four fragments of v_mfma_f32_16x16x32 (x is read to match: any order of the
// reduction will do that is the same on both sides); with x in 4 bits too, it is the
// operand of v_mfma_scale_f32_16x16x128 as it is.  The waves' sums meet in LDS.
//
// Backward the reduction runs over the weight's rows, whose scales differ.  Lane
// (r, g) reads eight or sixteen columns of rows 8 g .. 8 g + 7 of a 32-row slab; a
// byte (two columns of one row) is converted under that row's scale, and the
// halves of two rows' results are put together as the fragments' pairs.  Column
// T r + c of a wave's 16 T is row r of tile c, so that a lane ends with T
// consecutive columns.
//
// One token through 13824 x 5120 in bf16 takes 9.0 us (4.2 TB/s of codes), backward
// 19.5 to 19.9: 15.6 the kernel and 4.5 the parts' sum.  320 workgroups come to 256
// compute units there; on those that have two, 18,000 vector instructions (4,500 a
// SIMD) take about 8 us, and half of a wave's time is waiting.
// With small weights these kernels need no second launch where the tiled ones split
// their reduction, and take many tokens too.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <cmath>
#include <type_traits>

#include "mx4_format.h"
#include "mx4_launch.h"
#include "mx4_sum.h"
#include "mx4_tile.h"

namespace mx4k {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr u32x4 kZero = {0, 0, 0, 0};

template <int DT>
__device__ __forceinline__ f32x4 mfma16(const u32x4& a, const u32x4& b, const f32x4& c)
{
    if constexpr (DT == 0)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

template <int S>
__device__ __forceinline__ f32x4 mfma4(const u32x4& a, uint32_t sa, const u32x4& b, uint32_t sb, const f32x4& c)
{
    const i32x8 x = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
    const i32x8 y = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, c, 4, 4, S, (int)sa, S, (int)sb);
}

struct FewArgs {
    const uint8_t *codes, *scales;   // W [rows x cols]
    const void* x;                   // [m x cols] (backward [m x rows]) in 16 bits, or codes
    const uint8_t* xscales;
    void* out;
    float* part;                     // backward with parts > 1: fp32 [parts][m x cols]
    int64_t m, rows, cols;
    int kind;                        // of out
    int parts;
    uint32_t token_tiles;            // workgroups along the tokens
};

__device__ __forceinline__ int64_t least(int64_t a, int64_t b) { return a < b ? a : b; }

constexpr int kWaves = 8;

// Four scales of a row in one dword; past its end zeros.
__device__ __forceinline__ uint32_t load_scales(const MX4_GLOBAL uint8_t* p, int have)
{
    uint32_t v = 0;
    if (have == 4) {
        __builtin_memcpy(&v, (const uint8_t*)p, 4);
    } else {
        for (int i = 0; i < have; ++i) v |= (uint32_t)p[i] << (8 * i);
    }
    return v;
}

// DT 0, 1: x in bf16, fp16; 2: in codes.
template <int DT, int kRT, int kMT, int kW>
__global__ __launch_bounds__(64 * kW) void k_few(FewArgs a)
{
    __shared__ f32x4 sums[kW > 1 ? kW : 1][kW > 1 ? kRT * kMT : 1][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, g = lane >> 4;
    const int64_t n0 = (int64_t)(blockIdx.x / a.token_tiles) * (16 * kRT), t0 = (int64_t)(blockIdx.x % a.token_tiles) * (16 * kMT);
    const int64_t blocks = a.cols / kGroup;
    const MX4_GLOBAL uint8_t *wc[kRT], *ws[kRT];
#pragma unroll
    for (int i = 0; i < kRT; ++i) {
        const int64_t n = least(n0 + 16 * i + r, a.rows - 1);
        wc[i] = (const MX4_GLOBAL uint8_t*)a.codes + n * (a.cols / 2);
        ws[i] = (const MX4_GLOBAL uint8_t*)a.scales + n * blocks;
    }
    const MX4_GLOBAL uint8_t* xc[kMT];   // the token's row, bytes
    const MX4_GLOBAL uint8_t* xs[kMT];
#pragma unroll
    for (int u = 0; u < kMT; ++u) {
        const int64_t t = least(t0 + 16 * u + r, a.m - 1);
        xc[u] = (const MX4_GLOBAL uint8_t*)a.x + t * (DT == 2 ? a.cols / 2 : a.cols * 2);
        xs[u] = (const MX4_GLOBAL uint8_t*)a.xscales + t * blocks;
    }
    // tokens past the last one: lanes that read nothing, columns that are not stored
    const int here = (int)least(a.m - t0, 16 * kMT);
    f32x4 acc[kRT][kMT] = {};
    u32x4 x[kMT][DT == 2 ? 1 : 4] = {};
    uint32_t e[kMT] = {};
    for (int64_t at = 16 * wave; at < blocks; at += 16 * kW) {
        const int64_t blk = at + 4 * g;                      // this lane's four
        const int have = (int)least(blocks - blk, 4);
        uint32_t s[kRT];
#pragma unroll
        for (int i = 0; i < kRT; ++i) s[i] = load_scales(ws[i] + blk, have);
        if constexpr (DT == 2) {
#pragma unroll
            for (int u = 0; u < kMT; ++u)
                if (16 * u + r < here) e[u] = load_scales(xs[u] + blk, have);
        }
        u32x4 c[4][kRT];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int i = 0; i < kRT; ++i) c[j][i] = j < have ? *(const MX4_GLOBAL u32x4*)(wc[i] + 16 * (blk + j)) : kZero;
        auto part = [&](auto which) {
            constexpr int j = which;
            const bool in = j < have;
#pragma unroll
            for (int u = 0; u < kMT; ++u) {
                if (16 * u + r < here) {
                    if constexpr (DT == 2) {
                        x[u][0] = in ? *(const MX4_GLOBAL u32x4*)(xc[u] + 16 * (blk + j)) : kZero;
                    } else {
#pragma unroll
                        for (int f = 0; f < 4; ++f)
                            x[u][f] = in ? *(const MX4_GLOBAL u32x4*)(xc[u] + 64 * (blk + j) + 16 * f) : kZero;
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < kRT; ++i) {
                if constexpr (DT == 2) {
#pragma unroll
                    for (int u = 0; u < kMT; ++u) acc[i][u] = mfma4<j>(c[j][i], s[i], x[u][0], e[u], acc[i][u]);
                } else {
                    const float arg = byte_arg<j>(s[i]);
#pragma unroll
                    for (int f = 0; f < 4; ++f) {
                        const u32x4 w = decode8<DT>(c[j][i][f], arg);
#pragma unroll
                        for (int u = 0; u < kMT; ++u) acc[i][u] = mfma16<DT>(w, x[u][f], acc[i][u]);
                    }
                }
            }
        };
        part(std::integral_constant<int, 0>{});
        part(std::integral_constant<int, 1>{});
        part(std::integral_constant<int, 2>{});
        part(std::integral_constant<int, 3>{});
    }
    // lane (r, g) of a tile: token r, weight rows 4 g .. 4 g + 3
    if constexpr (kW == 1) {
#pragma unroll
        for (int i = 0; i < kRT; ++i)
#pragma unroll
            for (int u = 0; u < kMT; ++u) {
                const int64_t t = t0 + 16 * u + r, n = n0 + 16 * i + 4 * g;
                if (t < a.m && n < a.rows) store4(a.out, a.kind, t * a.rows + n, acc[i][u]);
            }
    } else {
#pragma unroll
        for (int i = 0; i < kRT; ++i)
#pragma unroll
            for (int u = 0; u < kMT; ++u) sums[wave][i * kMT + u][lane] = acc[i][u];
        __syncthreads();
        for (int e = threadIdx.x; e < kRT * kMT * 64; e += 64 * kW) {
            const int tile = e >> 6, l = e & 63;
            f32x4 v = sums[0][tile][l];
#pragma unroll
            for (int w = 1; w < kW; ++w) v += sums[w][tile][l];
            const int64_t t = t0 + 16 * (tile % kMT) + (l & 15), n = n0 + 16 * (tile / kMT) + 4 * (l >> 4);
            if (t < a.m && n < a.rows) store4(a.out, a.kind, t * a.rows + n, v);
        }
    }
}

// Up to 16 tokens, forward.  The 16 rows of a matrix instruction's first operand are
// four weight rows times four neighbouring blocks b, those of the second four tokens
// times the same four blocks; of the products only those of equal b count, the
// diagonals, and the quad's four are added at the end.  So four neighbouring lanes
// read 64 bytes in a row, where k_few's sixteen rows cost a line for each lane.  A
// run is 512 columns (lane (a, b, g): row a, block 4 g + b); kRT x 4 rows and kTG x 4
// tokens a wave.  Seven tokens through 5120 x 13824, both operands in codes: 8.1 us,
// k_few 15.4; two through 13824 x 5120 in 16 bits 9.9, k_few 13.8.
template <int DT, int kRT, int kTG, int kThinWaves>
__global__ __launch_bounds__(64 * kThinWaves) void k_thin(FewArgs a)
{
    __shared__ float sums[kThinWaves][kRT][kTG][16];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, quad = (lane & 15) >> 2, b = lane & 3, g = lane >> 4;
    const int64_t n0 = (int64_t)blockIdx.x * (4 * kRT), blocks = a.cols / kGroup;
    const MX4_GLOBAL uint8_t *wc[kRT], *ws[kRT], *xc[kTG], *xs[kTG];
#pragma unroll
    for (int i = 0; i < kRT; ++i) {
        const int64_t n = least(n0 + 4 * i + quad, a.rows - 1);
        wc[i] = (const MX4_GLOBAL uint8_t*)a.codes + n * (a.cols / 2);
        ws[i] = (const MX4_GLOBAL uint8_t*)a.scales + n * blocks;
    }
#pragma unroll
    for (int u = 0; u < kTG; ++u) {
        const int64_t t = least(4 * u + quad, a.m - 1);
        xc[u] = (const MX4_GLOBAL uint8_t*)a.x + t * (DT == 2 ? a.cols / 2 : a.cols * 2);
        xs[u] = (const MX4_GLOBAL uint8_t*)a.xscales + t * blocks;
    }
    f32x4 acc[kRT][kTG] = {};
    for (int64_t at = 16 * wave; at < blocks; at += 16 * kThinWaves) {
        const bool in = at + 4 * g + b < blocks;
        const int64_t blk = in ? at + 4 * g + b : 0;
        u32x4 c[kRT];
        uint32_t s[kRT];
#pragma unroll
        for (int i = 0; i < kRT; ++i) {
            c[i] = *(const MX4_GLOBAL u32x4*)(wc[i] + 16 * blk);
            s[i] = ws[i][blk];
        }
        // blocks past the row's end: x 0 and the weight finite
#pragma unroll
        for (int i = 0; i < kRT; ++i) s[i] = in ? s[i] : 0u;
#pragma unroll
        for (int u = 0; u < kTG; ++u) {
            const bool mine = in && 4 * u + quad < a.m;
            if constexpr (DT == 2) {
                const u32x4 x = mine ? *(const MX4_GLOBAL u32x4*)(xc[u] + 16 * blk) : kZero;
                const uint32_t e = mine ? xs[u][blk] : 0u;
#pragma unroll
                for (int i = 0; i < kRT; ++i) acc[i][u] = mfma4<0>(c[i], s[i], x, e, acc[i][u]);
            } else {
#pragma unroll
                for (int f = 0; f < 4; ++f) {
                    const u32x4 x = mine ? *(const MX4_GLOBAL u32x4*)(xc[u] + 64 * blk + 16 * f) : kZero;
#pragma unroll
                    for (int i = 0; i < kRT; ++i)
                        acc[i][u] = mfma16<DT>(decode8<DT>(c[i][f], scale_arg(s[i])), x, acc[i][u]);
                }
            }
        }
    }
    // lane (r, g) of the result: row g, blocks 0 .. 3 in the four registers; column r = token quad, block b
#pragma unroll
    for (int i = 0; i < kRT; ++i)
#pragma unroll
        for (int u = 0; u < kTG; ++u) {
            const float c0 = acc[i][u][0], c1 = acc[i][u][1], c2 = acc[i][u][2], c3 = acc[i][u][3];
            float v = b == 0 ? c0 : b == 1 ? c1 : b == 2 ? c2 : c3;
            v += __shfl_xor(v, 1);
            v += __shfl_xor(v, 2);
            if (b == 0) sums[wave][i][u][4 * quad + g] = v;
        }
    __syncthreads();
    for (int e = threadIdx.x; e < kRT * kTG * 4; e += 64 * kThinWaves) {
        const int i = e % kRT, t = e / kRT;   // token t, rows n0 + 4 i ..
        f32x4 v = *(const f32x4*)&sums[0][i][t / 4][4 * (t % 4)];
#pragma unroll
        for (int w = 1; w < kThinWaves; ++w) v += *(const f32x4*)&sums[w][i][t / 4][4 * (t % 4)];
        if (t < a.m && n0 + 4 * i < a.rows) store4(a.out, a.kind, t * a.rows + n0 + 4 * i, v);
    }
}

// The low and the high halves of two dwords, put together.
__device__ __forceinline__ uint32_t low16(uint32_t a, uint32_t b) { return __builtin_amdgcn_perm(b, a, 0x05040100u); }
__device__ __forceinline__ uint32_t high16(uint32_t a, uint32_t b) { return __builtin_amdgcn_perm(b, a, 0x07060302u); }

// Two columns (byte B of each row's dword) of eight rows to two fragments.
template <int DT, int B>
__device__ __forceinline__ void decode_columns(const uint32_t (&c)[8], const float (&s)[8], u32x4& even, u32x4& odd)
{
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t p = decode2<DT, B>(c[2 * j], s[2 * j]), q = decode2<DT, B>(c[2 * j + 1], s[2 * j + 1]);
        even[j] = low16(p, q);
        odd[j] = high16(p, q);
    }
}

// 128 kWords columns a wave: kWords dwords of each of eight rows a lane.  The waves'
// sums meet in LDS, in kPhases parts that each take turns there.
template <int DT, int kMT, int kWords, int kPhases>
__global__ __launch_bounds__(64 * kWaves) void k_few_back(FewArgs a)
{
    constexpr int kTiles = 8 * kWords, kShare = kTiles * kMT / kPhases, kPairs = kShare / 2;
    static_assert(64 * kPairs * kPhases == 64 * kWaves, "a pair of tiles' lane for each thread");
    __shared__ f32x4 sums[kWaves][kShare][65];   // 65: lanes that read neighbouring tiles touch other banks
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, g = lane >> 4;
    const int64_t c0 = (int64_t)(blockIdx.x / a.token_tiles) * (16 * kTiles), t0 = (int64_t)(blockIdx.x % a.token_tiles) * (16 * kMT);
    const int64_t col = least(c0 + kTiles * r, a.cols - kTiles);
    const MX4_GLOBAL uint8_t* wc = (const MX4_GLOBAL uint8_t*)a.codes + col / 2;
    const MX4_GLOBAL uint8_t* ws = (const MX4_GLOBAL uint8_t*)a.scales + col / kGroup;
    const MX4_GLOBAL uint16_t* xr[kMT];
#pragma unroll
    for (int u = 0; u < kMT; ++u) xr[u] = (const MX4_GLOBAL uint16_t*)a.x + least(t0 + 16 * u + r, a.m - 1) * a.rows;
    const int here = (int)least(a.m - t0, 16 * kMT);
    f32x4 acc[kMT][kTiles] = {};
    u32x4 x[kMT] = {};
    const int64_t slabs = (a.rows + 31) / 32, stride = (int64_t)kWaves * a.parts;
    for (int64_t slab = wave + (int64_t)kWaves * blockIdx.y; slab < slabs; slab += stride) {
        const int64_t n = 32 * slab + 8 * g;
        const bool in = n < a.rows;   // rows come in eights
        uint32_t c[kWords][8], s[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const MX4_GLOBAL uint8_t* p = wc + (in ? n + j : 0) * (a.cols / 2);
            if constexpr (kWords == 2) {
                const u32x2 v = *(const MX4_GLOBAL u32x2*)p;
                c[0][j] = v[0];
                c[1][j] = v[1];
            } else {
                c[0][j] = *(const MX4_GLOBAL uint32_t*)p;
            }
            s[j] = ws[(in ? n + j : 0) * (a.cols / kGroup)];
        }
#pragma unroll
        for (int u = 0; u < kMT; ++u)
            if (16 * u + r < here) x[u] = in ? *(const MX4_GLOBAL u32x4*)(xr[u] + n) : kZero;
        float f[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = scale_arg(in ? s[j] : 0u);   // rows past the end: finite, against zeros of x
#pragma unroll
        for (int k = 0; k < kWords; ++k) {
            u32x4 w[8];
            decode_columns<DT, 0>(c[k], f, w[0], w[1]);
            decode_columns<DT, 1>(c[k], f, w[2], w[3]);
            decode_columns<DT, 2>(c[k], f, w[4], w[5]);
            decode_columns<DT, 3>(c[k], f, w[6], w[7]);
#pragma unroll
            for (int u = 0; u < kMT; ++u)
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[u][8 * k + i] = mfma16<DT>(x[u], w[i], acc[u][8 * k + i]);
        }
    }
    // a thread adds up two neighbouring tiles of one lane: two columns of four tokens
    const int phase = threadIdx.x / (64 * kPairs), pair = threadIdx.x % kPairs, from = threadIdx.x / kPairs % 64;
    f32x4 v0, v1;
#pragma unroll
    for (int ph = 0; ph < kPhases; ++ph) {
        if (ph > 0) __syncthreads();
#pragma unroll
        for (int i = 0; i < kShare; ++i) sums[wave][i][lane] = acc[(ph * kShare + i) / kTiles][(ph * kShare + i) % kTiles];
        __syncthreads();
        if (phase == ph) {
            v0 = sums[0][2 * pair][from];
            v1 = sums[0][2 * pair + 1][from];
#pragma unroll
            for (int w = 1; w < kWaves; ++w) {
                v0 += sums[w][2 * pair][from];
                v1 += sums[w][2 * pair + 1][from];
            }
        }
    }
    const int tile = phase * kShare + 2 * pair;
    const int64_t c = c0 + kTiles * (from & 15) + tile % kTiles;
    if (c >= a.cols) return;
    void* out = a.parts > 1 ? (void*)(a.part + (int64_t)blockIdx.y * a.m * a.cols) : a.out;
    const int kind = a.parts > 1 ? (int)kOutFp32 : a.kind;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t t = t0 + 16 * (tile / kTiles) + 4 * (from >> 4) + i;
        if (t < a.m) store2(out, kind, t * a.cols + c, f32x2{v0[i], v1[i]});
    }
}

__global__ __launch_bounds__(256) void k_split_sum(const float* part, int splits, int64_t n, int width8, void* out,
                                                   int64_t ldo, int kind)
{
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (8 * i >= n) return;
    const MX4_GLOBAL f32x4* p = (const MX4_GLOBAL f32x4*)(part + 8 * i);
    f32x4 a = {0, 0, 0, 0}, b = a;
    // four partials in flight: a call with few sums is bound by their latency
    for (int s = 0; s < splits; s += 4) {
        f32x4 v[4][2];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int64_t at = (s + k < splits ? s + k : s) * (n / 4);
            v[k][0] = p[at];
            v[k][1] = p[at + 1];
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (s + k < splits) {
                a += v[k][0];
                b += v[k][1];
            }
        }
    }
    const int64_t row = i / width8;
    store8(out, kind, row * ldo + 8 * (i - row * width8), a, b);
}

// k_few's time in us: for each round of a workgroup on every compute unit 1.5, 0.15 for
// each of a wave's tiles and 30 ns (22 with x in codes) for each load instruction of its
// waves (64 lanes on 64 lines).  kRT x kMT tiles of 16 x 16 a wave, the cheapest (4096 x
// 4096, 4 tokens: 1 x 1 5.7, 2 x 1 7.5; 13824 x 5120, 16 tokens: 4 x 1 16.1, 2 x 1 20.5,
// 1 x 1 29.6).
// Rows of one run need one wave, and many of those fit a compute unit at once.
constexpr int64_t kOneWave = 512;

struct FewPlan {
    int rt, mt;
    double us;
};

FewPlan few_plan(int64_t rows, int64_t cols, int64_t m, bool codes)
{
    FewPlan best = {};
    for (int rt = 4; rt; rt >>= 1)
        for (int mt = 4; mt; mt >>= 1) {
            if (mt > 1 && 8 * mt >= m) continue;   // half of it would be empty
            const double groups = double(ceil_div(rows, 16 * rt)) * double(ceil_div(m, 16 * mt));
            const double full = m < 16 ? m / 16.0 : 1.0;   // lanes of x that read
            const double loads = double(ceil_div(cols, 128)) * (2 * rt + (codes ? 2 : 4) * mt * full);
            const double each = 0.15 * rt * mt, load = loads * (codes ? 0.022 : 0.03);
            const double us = cols <= kOneWave ? 2.5 + each + (groups > kCus ? groups / kCus : 1.0) * load
                                               : 1.0 + std::ceil(groups / kCus) * (1.5 + each + load);
            if (best.rt == 0 || us < best.us) best = {rt, mt, us};
        }
    return best;
}

// k_thin's tokens: with x in 16 bits a token's values are four times those of its codes.
bool thin(int64_t m, bool codes) { return m <= (codes ? 16 : 8); }

// Backward: tiles of 16 tokens a workgroup takes, how many workgroups they make, and a wave's columns.
int token_tiles(int64_t m) { return m <= 16 ? 1 : 2; }
uint32_t token_groups(int64_t m) { return (uint32_t)ceil_div(m, 16 * token_tiles(m)); }
int back_columns(int64_t m) { return m <= 16 ? 256 : 128; }

// k_few_back's parts of the reduction and its time in us: the launch, 0.5 for each
// round's sums over the waves, 0.34 for each slab of a wave on a compute unit but 1.2
// for one after another of the same wave, and the split's sum.  One part, or as many
// as make about 1,024 workgroups with two slabs a wave at least.
struct BackPlan {
    int parts;
    double us;
};

BackPlan back_plan(int64_t rows, int64_t cols, int64_t m)
{
    const int64_t groups = ceil_div(cols, back_columns(m)) * token_groups(m), slabs = ceil_div(rows, 32);
    auto us = [&](int64_t parts) {
        const double one = 1.2 * double(ceil_div(slabs, kWaves * parts)), all = 0.34 * double(groups) * double(slabs) / kCus;
        return 2.5 + 0.5 * double(ceil_div(groups * parts, kCus)) + (one > all ? one : all) +
               (parts > 1 ? 3.0 + double(parts) * double(m) * double(cols) * 8e-6 / 6.0 : 0.0);
    };
    int64_t p = ceil_div(1024, groups);
    const int64_t most = ceil_div(slabs, 2 * kWaves);
    p = p > most ? most : p;
    p = p > 16 ? 16 : p;
    const double whole = us(1), split = us(p);
    return p < 2 || whole <= split ? BackPlan{1, whole} : BackPlan{(int)p, split};
}

// Whether these kernels take a product, or the tiled ones: by the estimates, up to as many tokens as their grids are
// made for (forward: 100 tokens through 1024 x 1024 4.6 us, tiled 10.4; 64 through 4096 x 4096 14.1 and 15.8, where
// the estimates are level and take the tiled one, through 13824 x 5120 32.2 and 25.6; backward 300 through 512 x 512 5.3
// and 7.0, 64 through 4096 x 4096 17.5 and 15.8; in codes 64 through 4096 x 4096 8.3 and 13.7, through 13824 x 5120 19.7
// and 17.0).  The tiled kernel of two
// operands in codes takes rows of 256 at least.
constexpr int64_t kFewTokens = 4096;

bool mm_few(int64_t rows, int64_t cols, int64_t m, bool forward)
{
    if (m > kFewTokens) return false;
    if (!forward) return m <= 16 || back_plan(rows, cols, m).us < mm_tiled_us(rows, cols, m, false);
    return thin(m, false) || few_plan(rows, cols, m, false).us < mm_tiled_us(cols, rows, m, true);
}
bool mm4_few(int64_t rows, int64_t cols, int64_t m)
{
    return cols < 256 || thin(m, true) || (m <= kFewTokens && few_plan(rows, cols, m, true).us < mm4_tiled_us(rows, cols, m));
}

template <int DT, int kRT, int kW>
hipError_t few_tokens(const FewArgs& a, int mt, hipStream_t s)
{
    const dim3 grid((unsigned)ceil_div(a.rows, 16 * kRT) * a.token_tiles);
    if (mt == 1) k_few<DT, kRT, 1, kW><<<grid, 64 * kW, 0, s>>>(a);
    else if (mt == 2) k_few<DT, kRT, 2, kW><<<grid, 64 * kW, 0, s>>>(a);
    else k_few<DT, kRT, 4, kW><<<grid, 64 * kW, 0, s>>>(a);
    return hipGetLastError();
}

template <int DT, int kW>
hipError_t few_rows(const FewArgs& a, const FewPlan& p, hipStream_t s)
{
    if (p.rt == 4) return few_tokens<DT, 4, kW>(a, p.mt, s);
    return p.rt == 2 ? few_tokens<DT, 2, kW>(a, p.mt, s) : few_tokens<DT, 1, kW>(a, p.mt, s);
}

template <int DT, int kRT, int kTG, int kThinWaves>
hipError_t thin_go(const FewArgs& a, hipStream_t s)
{
    k_thin<DT, kRT, kTG, kThinWaves><<<(unsigned)ceil_div(a.rows, 4 * kRT), 64 * kThinWaves, 0, s>>>(a);
    return hipGetLastError();
}

template <int DT>
hipError_t few_go(FewArgs a, hipStream_t s)
{
    if (thin(a.m, DT == 2)) {
        // few rows: four of them a workgroup and eight waves (a token through 64 x 6912 3.2 us, eight rows and four waves
        // 4.0; six tokens 4.2, sixteen rows and two 9.4; through 1024 x 4096 3.9 and 5.0, but through 4096 x 4096 6.5 and 5.7)
        if (a.rows <= 2048) {
            if (a.m <= 4) return thin_go<DT, 1, 1, 8>(a, s);
            if constexpr (DT == 2) return a.m <= 8 ? thin_go<DT, 1, 2, 8>(a, s) : thin_go<DT, 1, 4, 8>(a, s);
            return thin_go<DT, 1, 2, 8>(a, s);
        }
        const int64_t runs = ceil_div(a.cols, 512);
        if (a.m <= 4) return thin_go<DT, 2, 1, 4>(a, s);
        if constexpr (DT == 2) return a.m <= 8 ? thin_go<DT, 2, 2, 4>(a, s) : thin_go<DT, 2, 4, 4>(a, s);
        // 16 bits, five to eight tokens: two waves where four would share the runs unevenly (8 tokens through 13824 x
        // 5120, 10 runs: 13.6 us, with four 16.2; through 11008 x 4096, 8 runs: 11.0 and 8.9)
        if (10 * ceil_div(runs, 4) * 4 > 11 * runs) return thin_go<DT, 4, 2, 2>(a, s);
        return thin_go<DT, 4, 2, 4>(a, s);
    }
    const FewPlan p = few_plan(a.rows, a.cols, a.m, DT == 2);
    a.token_tiles = (uint32_t)ceil_div(a.m, 16 * p.mt);
    return a.cols <= kOneWave ? few_rows<DT, 1>(a, p, s) : few_rows<DT, kWaves>(a, p, s);
}

template <int DT>
hipError_t few_back_go(const FewArgs& a, hipStream_t s)
{
    const int mt = token_tiles(a.m);
    const dim3 grid((unsigned)ceil_div(a.cols, back_columns(a.m)) * a.token_tiles, (unsigned)a.parts);
    // in one phase the sums take most of a compute unit's LDS
    const bool alone = (int64_t)grid.x * grid.y <= kCus;
    if (mt == 1 && alone) k_few_back<DT, 1, 2, 1><<<grid, 64 * kWaves, 0, s>>>(a);
    else if (mt == 1) k_few_back<DT, 1, 2, 2><<<grid, 64 * kWaves, 0, s>>>(a);
    else if (alone) k_few_back<DT, 2, 1, 1><<<grid, 64 * kWaves, 0, s>>>(a);
    else k_few_back<DT, 2, 1, 2><<<grid, 64 * kWaves, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_split_sum(const float* part, int splits, int64_t m, int64_t ncol, void* out, int64_t ldo, int out_kind,
                            hipStream_t s)
{
    const int64_t n = m * ncol;
    k_split_sum<<<(unsigned)ceil_div(n, 2048), 256, 0, s>>>(part, splits, n, (int)(ncol / 8), out, ldo, out_kind);
    return hipGetLastError();
}

size_t matmul_ws(int64_t rows, int64_t cols, bool forward, int64_t m)
{
    if (!mm_few(rows, cols, m, forward)) return forward ? mm_tiled_ws(cols, rows, m, true) : mm_tiled_ws(rows, cols, m, false);
    if (forward) return 0;
    const int parts = back_plan(rows, cols, m).parts;
    return parts > 1 ? size_t(parts) * size_t(m) * size_t(cols) * sizeof(float) : 0;
}

hipError_t launch_matmul(int dtype, const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols,
                         bool forward, const void* x, int64_t m, void* out, int out_kind, float* part, hipStream_t s)
{
    if (!mm_few(rows, cols, m, forward)) return launch_mm_tiled(dtype, codes, scales, rows, cols, forward, x, m, out, out_kind, part, s);
    FewArgs a{codes, scales, x, nullptr, out, part, m, rows, cols, out_kind, 1, token_groups(m)};
    if (forward) return dtype == 0 ? few_go<0>(a, s) : few_go<1>(a, s);
    a.parts = back_plan(rows, cols, m).parts;
    const hipError_t e = dtype == 0 ? few_back_go<0>(a, s) : few_back_go<1>(a, s);
    if (e != hipSuccess || a.parts == 1) return e;
    return launch_split_sum(part, a.parts, m, cols, out, cols, out_kind, s);
}

size_t matmul4_ws(int64_t rows, int64_t cols, int64_t m) { return mm4_few(rows, cols, m) ? 0 : mm4_tiled_ws(rows, cols, m); }

hipError_t launch_matmul4(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols,
                          const uint8_t* xcodes, const uint8_t* xscales, int64_t m, void* out, int out_kind,
                          float* part, hipStream_t s)
{
    if (!mm4_few(rows, cols, m))
        return launch_mm4_tiled(codes, scales, rows, cols, xcodes, xscales, m, out, out_kind, part, s);
    // narrow weights come here with any number of tokens: what keeps a launch under 2^32 threads at once
    const int64_t most = (int64_t(1) << 34) / rows;
    for (int64_t t = 0; t < m; t += most) {
        const FewArgs a{codes, scales, xcodes + t * (cols / 2), xscales + t * (cols / kGroup),
                        (char*)out + t * rows * (out_kind == kOutFp32 ? 4 : 2), nullptr, m - t < most ? m - t : most,
                        rows, cols, out_kind, 1, 1};
        const hipError_t e = few_go<2>(a, s);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace mx4k
