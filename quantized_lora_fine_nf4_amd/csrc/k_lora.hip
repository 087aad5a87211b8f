// k_lora.hip -- the small operators of an adapted NF4 layer on gfx950: dropout
// from a counter-based mask, the gradient of the matmul's epilogue, and the
// low-rank adapter's products ("QLoRA" paper summary page, How It Works: the
// 4-bit weight stays frozen and low-rank adapters are trained on top of it).
//
//   dropout   y = keep ? c x : 0
//   act_grad  dz = dy act'(z), dbias = sum over tokens of dz
//   project   h = s c (keep . x) A^T      (forward;  x m x k, A rank x k)
//             h = s x B                   (backward; x m x k, B k x rank)
//   grad      dA = c u^T (keep . x), dB = x^T u   (x m x n, u m x rank)
//
// All sums are fp32, in an order fixed by the shape, so every result is bitwise
// reproducible; 16-bit results are rounded once, at the store.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "nf4_act.h"
#include "nf4_launch.h"
#include "nf4_philox.h"

namespace nf4k {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

#define GLOBAL __attribute__((address_space(1)))

template <int DT> struct Frag { typedef bf16x8 T; };
template <> struct Frag<1> { typedef f16x8 T; };

template <int DT>
__device__ __forceinline__ f32x4 mfma(const u32x4& a, const u32x4& b, const f32x4& c)
{
    typedef typename Frag<DT>::T F;
    if constexpr (DT == 0)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(F, a), __builtin_bit_cast(F, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(F, a), __builtin_bit_cast(F, b), c, 0, 0, 0);
}

// Two packed 16-bit values to fp32 and back (nearest, ties to even).
template <int DT>
__device__ __forceinline__ f32x2 unpack2(uint32_t v)
{
    if constexpr (DT == 0)
        return f32x2{__builtin_bit_cast(float, v << 16), __builtin_bit_cast(float, v & 0xffff0000u)};
    else return __builtin_convertvector(__builtin_bit_cast(f16x2, v), f32x2);
}

template <int DT>
__device__ __forceinline__ uint32_t pack2(float a, float b)
{
    const f32x2 in = {a, b};
    if constexpr (DT == 0) return __builtin_bit_cast(uint32_t, __builtin_convertvector(in, bf16x2));
    else return __builtin_bit_cast(uint32_t, __builtin_convertvector(in, f16x2));
}

template <int DT>
__device__ __forceinline__ uint16_t pack1(float a) { return (uint16_t)pack2<DT>(a, 0.0f); }

// ---- dropout
//
// Bound by memory: 4 bytes per element and no more (counted); 8192 x 13824 in 78
// us, 5.8 TB/s.  The generator, the masks and the conversions are 80 vector
// instructions per eight elements (counted), hidden but for 2 us: with
// probability 0 the call takes 76.7.  One mask group (eight elements, 16 bytes)
// per thread and step, four loads in flight.
constexpr int kDropGroups = 4;   // groups per thread

template <int DT>
__device__ __forceinline__ u32x4 drop8(const u32x4& x, const Bits128& b, uint32_t thr, float keep)
{
    u32x4 r;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const f32x2 v = unpack2<DT>(x[j]);
        r[j] = keep2(pack2<DT>(v.x * keep, v.y * keep), b.w[j], thr);
    }
    return r;
}

// Results past what the caches hold for the next kernel go around them (stream):
// at 113 MB dropout takes 39.6 us instead of 42.2, act_grad 69.8 instead of 73.1;
// below that the next kernel reads them from the caches (act_grad, project and
// grad over 28 MB: 48.6 us, 53.2 with streamed stores; over 113 MB 121 both ways).
constexpr int64_t kStreamBytes = int64_t(64) << 20;

template <bool STREAM>
__device__ __forceinline__ void store_result(const u32x4& v, GLOBAL u32x4* p)
{
    if constexpr (STREAM) __builtin_nontemporal_store(v, p);
    else *p = v;
}

// DROP false (probability 0, no rng): a copy.
template <int DT, bool DROP, bool STREAM>
__global__ __launch_bounds__(256) void k_dropout(const uint16_t* x, int64_t n, DropArgs d, uint16_t* out)
{
    PhiloxKey key = {};
    if constexpr (DROP) key = philox_key(d.rng);
    const int64_t groups = n >> 3, g0 = (int64_t)blockIdx.x * (256 * kDropGroups) + threadIdx.x;
    u32x4 v[kDropGroups];
#pragma unroll
    for (int i = 0; i < kDropGroups; ++i) {
        const int64_t g = g0 + 256 * i;
        if (g < groups) v[i] = ((const GLOBAL u32x4*)x)[g];
    }
#pragma unroll
    for (int i = 0; i < kDropGroups; ++i) {
        const int64_t g = g0 + 256 * i;
        if (g >= groups) continue;
        if constexpr (DROP) v[i] = drop8<DT>(v[i], philox7(key, (uint64_t)g), d.thr, d.keep);
        store_result<STREAM>(v[i], (GLOBAL u32x4*)out + g);
    }
    // the last partial group, element by element
    if (blockIdx.x == 0 && threadIdx.x == 0 && (n & 7)) {
        uint32_t bits = 255;
        if constexpr (DROP) bits = keep_bits8(philox7(key, (uint64_t)groups), d.thr);
        for (int i = 0; i < (int)(n & 7); ++i) {
            const f32x2 v1 = unpack2<DT>(x[8 * groups + i]);
            out[8 * groups + i] = (bits >> i & 1) ? pack1<DT>(v1.x * d.keep) : (uint16_t)0;
        }
    }
}

template <int DT, bool STREAM>
hipError_t dropout_go(const uint16_t* x, int64_t n, DropArgs d, uint16_t* out, unsigned blocks, hipStream_t s)
{
    if (d.thr) hipLaunchKernelGGL((k_dropout<DT, true, STREAM>), dim3(blocks), dim3(256), 0, s, x, n, d, out);
    else hipLaunchKernelGGL((k_dropout<DT, false, STREAM>), dim3(blocks), dim3(256), 0, s, x, n, d, out);
    return hipGetLastError();
}

// ---- gradient of the epilogue
//
// Bound by memory: 6 bytes per element; 4096 x 13824 (silu, with the bias
// gradient) in 69.8 us with the sum of the partials, 4.9 TB/s.  A workgroup
// takes 8 L columns (L lanes
// of eight, a power of two up to 64) and `rows` rows per lane; the column
// sums are kept per lane over its rows, added over the workgroup's rows in
// LDS and stored as one partial row per row block, added in block order by
// k_sum_parts.
struct ActArgs {
    const uint16_t* dy;
    const uint16_t* z;
    uint16_t* dz;      // null: no dz (activation none)
    float* part;       // fp32 partials [row blocks][n], or dbias itself with one block; null: no bias gradient
    int64_t m, n;
    int act, lshift;   // L = 1 << lshift
    int64_t rows;      // rows per lane
};

template <int DT, bool STREAM>
__global__ __launch_bounds__(256) void k_act_grad(ActArgs g)
{
    __shared__ __attribute__((aligned(16))) float s_sum[256 * 8];
    const int t = threadIdx.x, L = 1 << g.lshift, lane = t & (L - 1), row0 = t >> g.lshift, nrow = 256 >> g.lshift;
    const int64_t col = ((int64_t)blockIdx.x * L + lane) * 8;
    const int64_t m0 = (int64_t)blockIdx.y * nrow * g.rows + row0;
    float sum[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[i] = 0.0f;
    if (col < g.n) {
        // two rows' loads in flight (the last row of an odd count twice, once used)
        for (int64_t r = 0; r < g.rows; r += 2) {
            const int64_t row[2] = {m0 + r * nrow, m0 + (r + 1) * nrow};
            const bool in[2] = {row[0] < g.m, r + 1 < g.rows && row[1] < g.m};
            if (!in[0]) break;
            u32x4 dy[2], zv[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int64_t at = (in[k] ? row[k] : row[0]) * g.n + col;
                dy[k] = *(const GLOBAL u32x4*)(g.dy + at);
                zv[k] = u32x4{0, 0, 0, 0};
                if (g.act != ACT_NONE) zv[k] = *(const GLOBAL u32x4*)(g.z + at);
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                if (!in[k]) continue;
                u32x4 o;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    f32x2 v = unpack2<DT>(dy[k][j]);
                    const f32x2 z = unpack2<DT>(zv[k][j]);
                    v.x *= act_slope(z.x, g.act);
                    v.y *= act_slope(z.y, g.act);
                    sum[2 * j] += v.x;
                    sum[2 * j + 1] += v.y;
                    o[j] = pack2<DT>(v.x, v.y);
                }
                if (g.dz) store_result<STREAM>(o, (GLOBAL u32x4*)(g.dz + row[k] * g.n + col));
            }
        }
    }
    if (!g.part) return;   // uniform
#pragma unroll
    for (int i = 0; i < 8; ++i) s_sum[t * 8 + i] = sum[i];
    __syncthreads();
    // column c of the workgroup: the rows' sums in row order
    for (int c = t; c < 8 * L; c += 256) {
        float a = 0.0f;
        for (int r = 0; r < nrow; ++r) a += s_sum[(r << g.lshift) * 8 + c];
        const int64_t cc = (int64_t)blockIdx.x * L * 8 + c;
        if (cc < g.n) ((GLOBAL float*)g.part)[(int64_t)blockIdx.y * g.n + cc] = a;
    }
}

// out[i] = scale * (part[0][i] + part[1][i] + ...); n a multiple of 4.  Bound by
// latency (128 parts of 13,824: 33 us with one thread per four columns, 4.6 us
// with 16).  A workgroup takes 256 >> glog columns of four values; its 1 << glog groups of
// threads add every (1 << glog)-th part, and the groups' sums are added in
// group order: a fixed order for a given part count.
__global__ __launch_bounds__(256) void k_sum_parts(const float* part, int nparts, int glog, int64_t n, float scale,
                                                   float* out)
{
    __shared__ __attribute__((aligned(16))) f32x4 s_sum[256];
    const int t = threadIdx.x, per = 256 >> glog, c = t & (per - 1), g = t >> (8 - glog), ng = 1 << glog;
    const int64_t i = ((int64_t)blockIdx.x * per + c) * 4;
    f32x4 a = {0.0f, 0.0f, 0.0f, 0.0f};
    if (i < n) {
#pragma unroll 4
        for (int p = g; p < nparts; p += ng) a += *(const GLOBAL f32x4*)(part + (int64_t)p * n + i);
    }
    if (glog > 0) {
        s_sum[t] = a;
        __syncthreads();
        if (g > 0) return;
        for (int k = 1; k < ng; ++k) a += s_sum[k * per + c];
    }
    if (i < n) *(GLOBAL f32x4*)(out + i) = a * scale;
}

// ---- 16-rank operand tiles
//
// The reduction index of a [k x rank] matrix is its slow index, while an MFMA
// fragment wants eight consecutive k of one rank.  With the rank a multiple of
// V = 8 or 4 a wave copies a 32 x 16 RT tile to LDS (16 or 8 bytes a piece, rank
// contiguous) and reads it back with the transposing 64-bit read: in each group
// of 16 lanes, lane i receives element i % 4 of the pieces read by lanes 4 j +
// i / 4, so lanes reading rows r .. r + 3 at columns C + 4 (i % 4) get column
// C + i of those rows.  Otherwise each lane gathers its eight values from memory
// (4096 x 5120 backward at rank 4: 26 us gathered, 9.9 us in pieces).

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// Orders a wave's LDS writes before its lanes' later reads (and the reverse);
// LDS executes one wave's accesses in order.
__device__ __forceinline__ void wave_sync()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

__device__ __forceinline__ u32x4 ld16(const uint16_t* base, uint32_t off)
{
    return *(const GLOBAL u32x4*)((const GLOBAL uint8_t*)base + off);
}

// Rows k0 .. k0 + 31 (past `rows` the last row again), ranks r0 .. r0 + 16 RT
// - 1 of p [rows x rank], rank a multiple of V: piece t * 64 + lane of V values.
template <int RT, int V>
__device__ __forceinline__ void load_tile(const uint16_t* p, int64_t rows, int rank, int64_t k0, int r0, u32x4 (&d)[RT])
{
    constexpr int kRow = 16 * RT / V;   // pieces per row
    const int lane = threadIdx.x & 63;
    const uint16_t* base = p + k0 * rank;
    const int left = k0 + 32 <= rows ? 31 : (int)(rows - 1 - k0);
    auto off = [&](int t) {
        const int item = t * 64 + lane, r = r0 + V * (item % kRow), k = item / kRow;
        return (uint32_t)((k < left ? k : left) * rank + (r < rank ? r : rank - V)) * 2;
    };
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        if constexpr (V == 8) d[t] = ld16(base, off(t));
        else {
            const u32x2 a = *(const GLOBAL u32x2*)((const GLOBAL uint8_t*)base + off(2 * t));
            const u32x2 b = *(const GLOBAL u32x2*)((const GLOBAL uint8_t*)base + off(2 * t + 1));
            d[t] = u32x4{a.x, a.y, b.x, b.y};
        }
    }
}

// Through LDS (32 x 16 RT values of the wave's own) to the fragments of the RT
// rank tiles.
template <int RT, int V>
__device__ __forceinline__ void transpose_tile(const u32x4 (&d)[RT], uint16_t* lds, u32x4 (&f)[RT])
{
    const int lane = threadIdx.x & 63, q = lane & 15, kg = lane >> 4;
    wave_sync();
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        if constexpr (V == 8) *(u32x4*)(lds + (t * 64 + lane) * 8) = d[t];
        else {
            *(u32x2*)(lds + (2 * t * 64 + lane) * 4) = u32x2{d[t].x, d[t].y};
            *(u32x2*)(lds + ((2 * t + 1) * 64 + lane) * 4) = u32x2{d[t].z, d[t].w};
        }
    }
    wave_sync();
#pragma unroll
    for (int j = 0; j < RT; ++j) {
        u32x2 h[2];
#pragma unroll
        for (int u = 0; u < 2; ++u)
            h[u] = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (__attribute__((address_space(3))) s16x4*)(lds + (8 * kg + 4 * u + (q >> 2)) * (16 * RT) + 16 * j +
                                                            4 * (q & 3))));
        f[j] = u32x4{h[0].x, h[0].y, h[1].x, h[1].y};
    }
}

// The same fragments gathered from memory, any rank.
template <int RT>
__device__ __forceinline__ void gather_tile(const uint16_t* p, int64_t rows, int rank, int64_t k0, int r0, u32x4 (&f)[RT])
{
    const int lane = threadIdx.x & 63, q = lane & 15, kg = lane >> 4;
#pragma unroll
    for (int j = 0; j < RT; ++j) {
        const int r = r0 + 16 * j + q;
        const GLOBAL uint16_t* col = (const GLOBAL uint16_t*)p + (r < rank ? r : rank - 1);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t k = k0 + 8 * kg + 2 * i;
            const uint32_t lo = col[(k < rows ? k : rows - 1) * rank], hi = col[(k + 1 < rows ? k + 1 : rows - 1) * rank];
            f[j][i] = lo | (hi << 16);
        }
    }
}

// ---- the adapter's down product
//
// h[m x rank] = alpha (keep . x) W, reduction over k.  A workgroup takes
// 16 MB rows of x and 16 RT ranks; its waves share the reduction in chunks of
// 64 k (two 16 x 16 x 32 MFMA steps; lane l holds x row l % 16, k 8 (l / 16)
// .. + 7 of a step), the next chunk loaded while this one multiplies, and their
// sums are added pairwise in LDS.  x goes straight to fragments; W goes through
// LDS, so that memory is read in whole 128-byte lines (fragments read straight
// from its rows, 64 bytes each, took 1.5 times as long at rank 64).  Bound by
// x's bytes at rank 16 (4096 x 5120 in 10 us, 4.2 TB/s; 4096 x 13824 backward in
// 26 us, 4.5 TB/s, its waves waiting 80% of their time).  Above, by the reads of
// W from the L2, which every 16 or 32 rows read whole (8192 x 5120 rank 64: 168 MB
// beside x's 84, 22 us; the mask's work is hidden, 22.5 us with dropout).  Ranks
// over 64 are two groups that read x twice (4096 x 13824 rank 128: 57 us).
enum ProjMode { PROJ_FWD, PROJ_DROP, PROJ_BACK8, PROJ_BACK4, PROJ_BACK_ANY };   // backward: pieces of W, or gathered

struct ProjArgs {
    const uint16_t* x;    // [m x k]
    const uint16_t* w;    // forward [rank x k], backward [k x rank]
    uint16_t* h;          // [m x rank]
    int64_t m, k;
    int rank;
    float alpha;          // scale (times the dropout factor)
    DropArgs drop;
};

constexpr int kProjWaves = 8;    // 256 registers a wave: the next chunk of x and W fits (16 waves: 10-15% slower)
constexpr int kProjPitch = 72;   // staged W row of 64 k (144 B: conflict-free 16-byte reads)

template <int DT, int MODE, int MB, int RT>
__global__ __launch_bounds__(64 * kProjWaves) void k_lora_project(ProjArgs g)
{
    constexpr int W = kProjWaves;
    constexpr bool DROP = MODE == PROJ_DROP;
    // the waves' operand tiles, then the sums
    constexpr bool FWD = MODE == PROJ_FWD || MODE == PROJ_DROP;
    constexpr bool TILE = MODE == PROJ_BACK8 || MODE == PROJ_BACK4;
    constexpr int V = MODE == PROJ_BACK4 ? 4 : 8;
    constexpr int kWave = FWD ? 16 * RT * kProjPitch * 2 : TILE ? RT * 1024 : 0;
    constexpr int kTile = W * kWave, kSums = W / 2 * MB * RT * 1024;
    __shared__ __attribute__((aligned(16))) uint8_t s_mem[kTile > kSums ? kTile : kSums > 0 ? kSums : 16];
    const int t = threadIdx.x, lane = t & 63, wv = t >> 6;
    const int q = lane & 15, kg = lane >> 4;
    const int64_t m0 = (int64_t)blockIdx.x * (16 * MB);
    const int r0 = blockIdx.y * (16 * RT);
    PhiloxKey key = {};
    if constexpr (DROP) key = philox_key(g.drop.rng);
    // Loads address a uniform base, advanced per chunk, plus a 32-bit lane
    // offset (k is below 2^26).  Rows and ranks past the end repeat the last
    // one: they feed only results that are not stored.
    uint32_t xo[MB];
    uint64_t grp[MB];   // mask group of this lane's k in the row, chunk at 0
#pragma unroll
    for (int b = 0; b < MB; ++b) {
        const int64_t left = g.m - 1 - m0;
        const uint32_t r = 16 * b + q < left ? 16 * b + q : (uint32_t)left;
        xo[b] = (uint32_t)(r * g.k + 8 * kg) * 2;
        if constexpr (DROP) grp[b] = (uint64_t)((m0 + r) * g.k + 8 * kg) >> 3;
    }
    f32x4 acc[MB][RT];
#pragma unroll
    for (int b = 0; b < MB; ++b)
#pragma unroll
        for (int j = 0; j < RT; ++j) acc[b][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    const uint16_t* xb = g.x + m0 * g.k;
    uint16_t* tile = (uint16_t*)(s_mem + wv * kWave);
    // W of the 64 k at k0 (over: how far they run past the end): forward rows 8 t
    // + lane / 8 of the rank tile, 16-byte piece lane % 8; backward one 32-row
    // tile or fragment set per step
    auto load_w = [&](int64_t k0, int over, u32x4 (&w)[2 * RT]) {
        if constexpr (FWD) {
            const int piece = lane & 7, last = 7 - over / 8;
#pragma unroll
            for (int t = 0; t < 2 * RT; ++t) {
                const int rb = r0 + 8 * t < g.rank ? r0 + 8 * t : r0, left = g.rank - 1 - rb, r = lane >> 3;
                const int64_t at = (r < left ? r : left) * g.k + 8 * (piece < last ? piece : last);
                w[t] = ld16(g.w + rb * g.k + k0, (uint32_t)at * 2);
            }
        } else {
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                if (32 * s >= 64 - over) break;   // no step there (uniform)
                u32x4 d[RT];
                if constexpr (TILE) load_tile<RT, V>(g.w, g.k, g.rank, k0 + 32 * s, r0, d);
                else gather_tile<RT>(g.w, g.k, g.rank, k0 + 32 * s, r0, d);
#pragma unroll
                for (int j = 0; j < RT; ++j) w[s * RT + j] = d[j];
            }
        }
    };
    auto load_x = [&](int64_t k0, int over, u32x4 (&x)[2][MB]) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            if (over && 32 * s >= 64 - over) break;   // no step there (uniform)
            // lanes past the end load the step's last eight k (past <= 8 kg: never before the row)
            const int past = 32 * s + 8 * kg + 8 - (64 - over);
            const int32_t back = over && past > 0 ? -2 * past : 0;
#pragma unroll
            for (int b = 0; b < MB; ++b) x[s][b] = ld16(xb + k0 + 32 * s, xo[b] + back);
        }
    };
    auto multiply = [&](int64_t k0, int over, u32x4 (&x)[2][MB], u32x4 (&w)[2 * RT]) {
        if constexpr (FWD) {
            wave_sync();
#pragma unroll
            for (int t = 0; t < 2 * RT; ++t) *(u32x4*)(tile + (8 * t + (lane >> 3)) * kProjPitch + 8 * (lane & 7)) = w[t];
            wave_sync();
        }
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            if (over && 32 * s >= 64 - over) break;
            u32x4 f[RT];
            if constexpr (FWD) {
#pragma unroll
                for (int j = 0; j < RT; ++j) f[j] = *(const u32x4*)(tile + (16 * j + q) * kProjPitch + 32 * s + 8 * kg);
            } else {
                u32x4 d[RT];
#pragma unroll
                for (int j = 0; j < RT; ++j) d[j] = f[j] = w[s * RT + j];
                if constexpr (TILE) transpose_tile<RT, V>(d, tile, f);
            }
            // k past the end: zeros on both sides (an infinite last weight times zero would be NaN)
            const bool past = over && 32 * s + 8 * kg >= 64 - over;
#pragma unroll
            for (int j = 0; j < RT; ++j)
                if (past) f[j] = u32x4{0, 0, 0, 0};
#pragma unroll
            for (int b = 0; b < MB; ++b) {
                u32x4 a = x[s][b];
                if constexpr (DROP) {
                    const Bits128 bits = philox7(key, grp[b] + (uint64_t)((k0 + 32 * s) >> 3));
#pragma unroll
                    for (int j = 0; j < 4; ++j) a[j] = keep2(a[j], bits.w[j], g.drop.thr);
                }
                if (past) a = u32x4{0, 0, 0, 0};
#pragma unroll
                for (int j = 0; j < RT; ++j) acc[b][j] = mfma<DT>(a, f[j], acc[b][j]);
            }
        }
    };
    // whole chunks, the next one in flight (at the end the same one again, unused)
    u32x4 x[2][MB], w[2 * RT];
    int64_t k0 = (int64_t)wv * 64;
    if (k0 + 64 <= g.k) {
        load_x(k0, 0, x);
        load_w(k0, 0, w);
    }
    for (; k0 + 64 <= g.k; k0 += 64 * W) {
        const int64_t kn = k0 + 64 * W + 64 <= g.k ? k0 + 64 * W : k0;
        u32x4 xc[2][MB], wc[2 * RT];
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int b = 0; b < MB; ++b) xc[s][b] = x[s][b];
#pragma unroll
        for (int t = 0; t < 2 * RT; ++t) wc[t] = w[t];
        load_x(kn, 0, x);
        load_w(kn, 0, w);
        multiply(k0, 0, xc, wc);
    }
    if (k0 < g.k) {   // the last partial chunk, of one wave
        const int over = (int)(k0 + 64 - g.k);
        load_x(k0, over, x);
        load_w(k0, over, w);
        multiply(k0, over, x, w);
    }
    if constexpr (kTile > 0) __syncthreads();   // every wave done with its tile
    float* s_acc = (float*)s_mem;
#pragma unroll
    for (int half = W / 2; half > 0; half >>= 1) {
        if (wv >= half && wv < 2 * half) {
#pragma unroll
            for (int b = 0; b < MB; ++b)
#pragma unroll
                for (int j = 0; j < RT; ++j)
                    *(f32x4*)(s_acc + (((wv - half) * MB * RT + b * RT + j) * 64 + lane) * 4) = acc[b][j];
        }
        __syncthreads();
        if (wv < half) {
#pragma unroll
            for (int b = 0; b < MB; ++b)
#pragma unroll
                for (int j = 0; j < RT; ++j)
                    acc[b][j] += *(const f32x4*)(s_acc + ((wv * MB * RT + b * RT + j) * 64 + lane) * 4);
        }
        __syncthreads();
    }
    if (wv != 0) return;
    // lane l, value i: row 4 (l / 16) + i, rank l % 16
#pragma unroll
    for (int b = 0; b < MB; ++b)
#pragma unroll
        for (int j = 0; j < RT; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t row = m0 + 16 * b + 4 * kg + i;
                const int r = r0 + 16 * j + q;
                if (row < g.m && r < g.rank)
                    ((GLOBAL uint16_t*)g.h)[row * g.rank + r] = pack1<DT>(acc[b][j][i] * g.alpha);
            }
}

// ---- the adapter's gradients
//
// G[rank x n] = u^T (keep . x), reduction over the m tokens, which are the
// slow index of both operands.  Lane l loads eight consecutive columns
// n0 + 8 (l % 16) of the eight rows m0 + 8 (l / 16) + i (16 bytes each) and
// transposes the 8 x 8 block in registers with byte permutes: column c of the
// block is the lane's fragment of MFMA c (16 x 16 x 32), whose 16 columns are
// n0 + 8 q + c, q = 0 .. 15.  A wave covers 128 columns and 16 RT ranks, the
// W waves of a workgroup share its rows, and their sums are added in LDS.
// Bound by x's bytes where the tokens are many (4096 x 13824 rank 8: 25 us with
// the sum of the splits, 4.5 TB/s).  Where they are few a wave has two to four
// rounds of loads, none of them ahead, and waits half its time and more, and the
// splits' partials count beside x (4096 x 5120 rank 16: 12.4 us; 1999 x 8192 rank
// 64 13 us, 12.6 MB of partials written and read beside 35 MB).  Loading the next
// rows ahead, in fewer waves, took 4 to 10% longer.
struct GradArgs {
    const uint16_t* u;     // [m x rank]
    const uint16_t* x;     // [m x n]
    float* out;            // the result, or fp32 partials [splits][result]
    int64_t m, n;
    int rank;
    bool by_col;           // result layout: [n x rank] instead of [rank x n]
    int64_t rows_split;    // rows per split, a multiple of 32
    float scale;           // applied here when there is one split
    DropArgs drop;
};

// Waves of a workgroup: as many as the accumulators (32 RT registers) leave
// room for on a CU.
template <int RT> constexpr int kGradWaves = RT == 1 ? 16 : 8;

template <int DT, bool DROP, int V, int RT>
__global__ __launch_bounds__(64 * kGradWaves<RT>) void k_lora_grad(GradArgs g)
{
    constexpr int W = kGradWaves<RT>;
    constexpr bool VEC = V > 1;   // pieces of u; gathered otherwise
    // the waves' tiles of u, then the sums
    constexpr int kTile = VEC ? W * RT * 1024 : 0, kSums = W / 2 * 8 * RT * 1024;
    __shared__ __attribute__((aligned(16))) uint8_t s_mem[kTile > kSums ? kTile : kSums];
    const int t = threadIdx.x, lane = t & 63, wv = t >> 6, q = lane & 15, mg = lane >> 4;
    const int64_t n0 = (int64_t)blockIdx.x * 128 + 8 * q;
    const int64_t nc = n0 < g.n ? n0 : g.n - 8;
    const int r0 = blockIdx.z * (16 * RT);
    const int64_t s0 = (int64_t)blockIdx.y * g.rows_split;
    const int64_t s1 = s0 + g.rows_split < g.m ? s0 + g.rows_split : g.m;
    PhiloxKey key = {};
    if constexpr (DROP) key = philox_key(g.drop.rng);
    f32x4 acc[RT][8];
#pragma unroll
    for (int j = 0; j < RT; ++j)
#pragma unroll
        for (int c = 0; c < 8; ++c) acc[j][c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int64_t m0 = s0 + 32 * wv; m0 < s1; m0 += 32 * W) {
        u32x4 x[8], a[RT];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int64_t row = m0 + 8 * mg + i;
            x[i] = *(const GLOBAL u32x4*)(g.x + (row < s1 ? row : s1 - 1) * g.n + nc);
        }
        if constexpr (VEC) {
            u32x4 d[RT];
            load_tile<RT, V>(g.u, s1, g.rank, m0, r0, d);
            transpose_tile<RT, V>(d, (uint16_t*)(s_mem + wv * RT * 1024), a);
        } else {
            gather_tile<RT>(g.u, s1, g.rank, m0, r0, a);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int64_t row = m0 + 8 * mg + i;
            if constexpr (DROP) {
                const Bits128 bits = philox7(key, (uint64_t)(row * g.n + nc) >> 3);
#pragma unroll
                for (int j = 0; j < 4; ++j) x[i][j] = keep2(x[i][j], bits.w[j], g.drop.thr);
                // two generator calls at a time: more of them interleaved spill beside 64 ranks of sums
                if (RT == 4 && (i & 1)) __builtin_amdgcn_sched_barrier(0);
            }
        }
        // rows past the end: zeros on both sides (an infinite last u times zero would be NaN)
        if (m0 + 32 > s1) {
            const int left = (int)(s1 - m0) - 8 * mg;   // of this lane's eight rows
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i >= left) x[i] = u32x4{0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t keep = left > 2 * i + 1 ? 0xffffffffu : left > 2 * i ? 0xffffu : 0u;
#pragma unroll
                for (int j = 0; j < RT; ++j) a[j][i] &= keep;
            }
        }
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const uint32_t sel = (c & 1) ? 0x07060302u : 0x05040100u;
            u32x4 b;
#pragma unroll
            for (int i = 0; i < 4; ++i) b[i] = __builtin_amdgcn_perm(x[2 * i + 1][c >> 1], x[2 * i][c >> 1], sel);
#pragma unroll
            for (int j = 0; j < RT; ++j) acc[j][c] = mfma<DT>(a[j], b, acc[j][c]);
        }
    }
    if constexpr (kTile > 0) __syncthreads();   // every wave done with its tile
    f32x4* s_acc = (f32x4*)s_mem;
#pragma unroll
    for (int half = W / 2; half > 0; half >>= 1) {
        if (wv >= half && wv < 2 * half) {
#pragma unroll
            for (int j = 0; j < RT; ++j)
#pragma unroll
                for (int c = 0; c < 8; ++c) s_acc[((wv - half) * RT * 8 + j * 8 + c) * 64 + lane] = acc[j][c];
        }
        __syncthreads();
        if (wv < half) {
#pragma unroll
            for (int j = 0; j < RT; ++j)
#pragma unroll
                for (int c = 0; c < 8; ++c) acc[j][c] += s_acc[(wv * RT * 8 + j * 8 + c) * 64 + lane];
        }
        __syncthreads();
    }
    if (wv != 0 || n0 >= g.n) return;
    // lane l, value i of acc[j][c]: rank r0 + 16 j + 4 (l / 16) + i, column n0 + c
    GLOBAL float* out = (GLOBAL float*)g.out + (int64_t)blockIdx.y * g.rank * g.n;
#pragma unroll
    for (int j = 0; j < RT; ++j) {
        const int rb = r0 + 16 * j + 4 * mg;
        if (g.by_col && (g.rank & 3) == 0) {
            if (rb < g.rank) {
#pragma unroll
                for (int c = 0; c < 8; ++c) *(GLOBAL f32x4*)(out + (n0 + c) * g.rank + rb) = acc[j][c] * g.scale;
            }
            continue;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = rb + i;
            if (r >= g.rank) continue;
            if (g.by_col) {
#pragma unroll
                for (int c = 0; c < 8; ++c) out[(n0 + c) * g.rank + r] = acc[j][c][i] * g.scale;
            } else {
#pragma unroll
                for (int c = 0; c < 8; c += 4)
                    *(GLOBAL f32x4*)(out + (int64_t)r * g.n + n0 + c) =
                        f32x4{acc[j][c][i], acc[j][c + 1][i], acc[j][c + 2][i], acc[j][c + 3][i]} * g.scale;
            }
        }
    }
}

constexpr int64_t kMaxGrid = (int64_t(1) << 32) / 256 - 1;

hipError_t sum_parts(const float* part, int nparts, int64_t n, float scale, float* out, hipStream_t s)
{
    const int glog = nparts >= 16 ? 4 : nparts >= 4 ? 2 : 0;
    const int64_t per = (256 >> glog) * 4, blocks = (n + per - 1) / per;
    if (blocks > kMaxGrid) return hipErrorInvalidValue;
    hipLaunchKernelGGL(k_sum_parts, dim3((unsigned)blocks), dim3(256), 0, s, part, nparts, glog, n, scale, out);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_dropout(int dtype, const void* x, int64_t n, DropArgs d, void* out, hipStream_t s)
{
    const int64_t per = 8 * 256 * kDropGroups, blocks = (n + per - 1) / per;
    if (blocks > kMaxGrid) return hipErrorInvalidValue;
    const uint16_t* xi = static_cast<const uint16_t*>(x);
    uint16_t* o = static_cast<uint16_t*>(out);
    const unsigned b = (unsigned)blocks;
    if (2 * n > kStreamBytes)
        return dtype == 0 ? dropout_go<0, true>(xi, n, d, o, b, s) : dropout_go<1, true>(xi, n, d, o, b, s);
    return dtype == 0 ? dropout_go<0, false>(xi, n, d, o, b, s) : dropout_go<1, false>(xi, n, d, o, b, s);
}

namespace {

// Lanes of eight columns per row: the power of two that covers n, at most 64.
int act_lshift(int64_t n)
{
    int l = 0;
    while (l < 6 && (int64_t(8) << l) < n) ++l;
    return l;
}

// Rows per lane: eight (32 rows and a 4% partial per workgroup at 64 lanes),
// more where that would make over 4,096 workgroups, four or two where it would
// make fewer than 1,024 and there is more than one block of tokens anyway (333 x
// 8192: two 9.2 us, eight 14.1; 17 x 5120 in one block 6.5 us, in three 9.4).
int64_t act_rows(int64_t m, int64_t n)
{
    const int ls = act_lshift(n);
    const int64_t cols = int64_t(8) << ls, gx = (n + cols - 1) / cols, lrows = (m + (256 >> ls) - 1) / (256 >> ls);
    if (lrows <= 8) return lrows;
    const int64_t target = 4096 / gx > 1 ? 4096 / gx : 1, rows = (lrows + target - 1) / target;
    if (rows > 8) return rows;
    const int64_t fill = lrows * gx / 1024;
    return fill >= 8 ? 8 : fill >= 4 ? 4 : 2;
}

}  // namespace

int64_t act_grad_blocks(int64_t m, int64_t n)
{
    const int64_t rows = (int64_t)(256 >> act_lshift(n)) * act_rows(m, n);
    return (m + rows - 1) / rows;
}

hipError_t launch_act_grad(int dtype, const void* dy, const void* z, int act, int64_t m, int64_t n, void* dz,
                           float* dbias, float* part, hipStream_t s)
{
    const int64_t blocks = act_grad_blocks(m, n);
    ActArgs g;
    g.dy = static_cast<const uint16_t*>(dy);
    g.z = static_cast<const uint16_t*>(z);
    g.dz = static_cast<uint16_t*>(dz);
    g.part = dbias ? (blocks > 1 ? part : dbias) : nullptr;
    g.m = m;
    g.n = n;
    g.act = act;
    g.lshift = act_lshift(n);
    g.rows = act_rows(m, n);
    const int64_t cols = int64_t(8) << g.lshift, gx = (n + cols - 1) / cols;
    if (gx > kMaxGrid || blocks > 65535) return hipErrorInvalidValue;
    const dim3 grid((unsigned)gx, (unsigned)blocks);
    if (2 * m * n > kStreamBytes) {
        if (dtype == 0) hipLaunchKernelGGL((k_act_grad<0, true>), grid, dim3(256), 0, s, g);
        else hipLaunchKernelGGL((k_act_grad<1, true>), grid, dim3(256), 0, s, g);
    } else {
        if (dtype == 0) hipLaunchKernelGGL((k_act_grad<0, false>), grid, dim3(256), 0, s, g);
        else hipLaunchKernelGGL((k_act_grad<1, false>), grid, dim3(256), 0, s, g);
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !dbias || blocks <= 1) return e;
    return sum_parts(part, (int)blocks, n, 1.0f, dbias, s);
}

namespace {

template <int DT, int MODE, int MB, int RT>
hipError_t project_go(const ProjArgs& g, hipStream_t s)
{
    const dim3 grid((unsigned)((g.m + 16 * MB - 1) / (16 * MB)), (unsigned)((g.rank + 16 * RT - 1) / (16 * RT)));
    hipLaunchKernelGGL((k_lora_project<DT, MODE, MB, RT>), grid, dim3(64 * kProjWaves), 0, s, g);
    return hipGetLastError();
}

// The fewest ranks per workgroup (16, 32, 64) that still make one round of the
// 256 CUs: few rows get a workgroup per rank tile, many rows read x (and compute
// its mask) once; past one round 32 rows at a time, so that W is read half as
// often.  At 5120 k, rank 64 with 16 / 32 / 64 ranks at a time: 1000 rows 9.6 /
// 10.7 / 15.0 us, 2048 rows 16.1 / 11.1 / 15.4, 3000 rows 23.1 / 20.4 / 15.8;
// 64 ranks and 16 / 32 rows at a time: 6000 rows 32.2 / 26.1, 8192 rows 39.3 /
// 28.5.
template <int DT, int MODE>
hipError_t project_shape(const ProjArgs& g, hipStream_t s)
{
    const int64_t tiles = (g.m + 15) / 16;
    const int cover = g.rank <= 16 ? 1 : g.rank <= 32 ? 2 : 4;
    auto groups = [&](int rt) { return tiles * ((g.rank + 16 * rt - 1) / (16 * rt)); };
    int rt = 1;
    while (rt < cover && groups(rt) > 256) rt *= 2;
    const bool two = groups(rt) > 256;
    if (rt == 1) return two ? project_go<DT, MODE, 2, 1>(g, s) : project_go<DT, MODE, 1, 1>(g, s);
    if (rt == 2) return two ? project_go<DT, MODE, 2, 2>(g, s) : project_go<DT, MODE, 1, 2>(g, s);
    return two ? project_go<DT, MODE, 2, 4>(g, s) : project_go<DT, MODE, 1, 4>(g, s);
}

template <int DT>
hipError_t project_dt(const ProjArgs& g, bool backward, hipStream_t s)
{
    if (backward) {
        if (g.rank % 8 == 0) return project_shape<DT, PROJ_BACK8>(g, s);
        return g.rank % 4 == 0 ? project_shape<DT, PROJ_BACK4>(g, s) : project_shape<DT, PROJ_BACK_ANY>(g, s);
    }
    return g.drop.thr ? project_shape<DT, PROJ_DROP>(g, s) : project_shape<DT, PROJ_FWD>(g, s);
}

}  // namespace

hipError_t launch_lora_project(int dtype, const void* x, int64_t m, int64_t k, const void* w, int rank, bool backward,
                               float scale, DropArgs drop, void* h, hipStream_t s)
{
    ProjArgs g;
    g.x = static_cast<const uint16_t*>(x);
    g.w = static_cast<const uint16_t*>(w);
    g.h = static_cast<uint16_t*>(h);
    g.m = m;
    g.k = k;
    g.rank = rank;
    g.alpha = drop.thr ? scale * drop.keep : scale;
    g.drop = drop;
    if ((m + 15) / 16 >= kMaxGrid / 4) return hipErrorInvalidValue;   // up to 1,024 threads each
    return dtype == 0 ? project_dt<0>(g, backward, s) : project_dt<1>(g, backward, s);
}

namespace {

// Ranks per workgroup in 16-rank tiles.
int grad_rt(int rank) { return rank <= 16 ? 1 : rank <= 32 ? 2 : 4; }

}  // namespace

// Splits of the token axis: a workgroup per CU, each split at least 128 rows
// and at least eight rows per rank (a split's fp32 partial is written and read
// back, 8 rank n bytes against the 2 rows n bytes of x that it reads).
int lora_grad_splits(int64_t m, int64_t n, int rank)
{
    const int rt = grad_rt(rank);
    const int64_t blocks = ((n + 127) / 128) * ((rank + 16 * rt - 1) / (16 * rt));
    const int64_t least = rank > 16 ? (int64_t)8 * rank : 128;
    int64_t sp = 256 / blocks;
    if (sp > m / least) sp = m / least;
    if (sp < 1) sp = 1;
    const int64_t rows = ((m + sp - 1) / sp + 31) / 32 * 32;
    return (int)((m + rows - 1) / rows);
}

namespace {

template <int DT, bool DROP, int V>
hipError_t grad_go(const GradArgs& g, int splits, hipStream_t s)
{
    const int rt = grad_rt(g.rank);
    const int64_t gx = (g.n + 127) / 128;
    if (gx > kMaxGrid || splits > 65535) return hipErrorInvalidValue;
    const dim3 grid((unsigned)gx, (unsigned)splits, (unsigned)((g.rank + 16 * rt - 1) / (16 * rt)));
    if (rt == 1) hipLaunchKernelGGL((k_lora_grad<DT, DROP, V, 1>), grid, dim3(64 * kGradWaves<1>), 0, s, g);
    else if (rt == 2) hipLaunchKernelGGL((k_lora_grad<DT, DROP, V, 2>), grid, dim3(64 * kGradWaves<2>), 0, s, g);
    else hipLaunchKernelGGL((k_lora_grad<DT, DROP, V, 4>), grid, dim3(64 * kGradWaves<4>), 0, s, g);
    return hipGetLastError();
}

template <int DT, bool DROP>
hipError_t grad_rank(const GradArgs& g, int splits, hipStream_t s)
{
    if (g.rank % 8 == 0) return grad_go<DT, DROP, 8>(g, splits, s);
    return g.rank % 4 == 0 ? grad_go<DT, DROP, 4>(g, splits, s) : grad_go<DT, DROP, 1>(g, splits, s);
}

template <int DT>
hipError_t grad_dt(const GradArgs& g, int splits, hipStream_t s)
{
    return g.drop.thr ? grad_rank<DT, true>(g, splits, s) : grad_rank<DT, false>(g, splits, s);
}

}  // namespace

hipError_t launch_lora_grad(int dtype, const void* u, const void* x, int64_t m, int64_t n, int rank, bool by_col,
                            DropArgs drop, float* grad, float* part, hipStream_t s)
{
    const int splits = lora_grad_splits(m, n, rank);
    const float scale = drop.thr ? drop.keep : 1.0f;
    GradArgs g;
    g.u = static_cast<const uint16_t*>(u);
    g.x = static_cast<const uint16_t*>(x);
    g.out = splits > 1 ? part : grad;
    g.m = m;
    g.n = n;
    g.rank = rank;
    g.by_col = by_col;
    g.rows_split = ((m + splits - 1) / splits + 31) / 32 * 32;
    g.scale = splits > 1 ? 1.0f : scale;
    g.drop = drop;
    const hipError_t e = dtype == 0 ? grad_dt<0>(g, splits, s) : grad_dt<1>(g, splits, s);
    if (e != hipSuccess || splits == 1) return e;
    return sum_parts(part, splits, n * rank, scale, grad, s);
}

}  // namespace nf4k
