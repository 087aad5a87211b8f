// k_norm.hip -- layer norm and its gradient on gfx950.
//
//   h = x + residual (rounded to 16 bits),  mean, r = 1 / sqrt(var + eps) per row
//   out = (h - mean) r weight + bias
//   g = dy weight,  c = (h - mean) r
//   dx = r (g - mean(g) - c mean(g c)) + residual
//   dweight = sum over rows of dy c,  dbias = sum over rows of dy
//
// Both are bound by memory.  A row lives in registers from its one read to its
// write: kLanes threads own eight-element pieces of it and keep their pieces of
// weight (and bias) over all rows that they take, and the next row's loads are
// issued before the current one is summed.  The variance is summed from the
// differences to the mean.  Sums are fp32, in an order fixed by the shape: within
// a lane, over the lanes of a wave, over the waves in wave order.  Rows past what
// registers hold are read again instead (k_norm_long, k_norm_grad_long).
//
// 8192 x 5120 in bf16 with a residual: 62 us, 5.4 TB/s; the gradient 65 us, 5.2 TB/s,
// and 5 us for the sum of the 256 workgroups' column sums (a copy reaches 5.2 TB/s).
// 17 x 5120 3.3 us, what any launch of this size takes.  Rows past the registers, 1024 x
// 24584 with a residual: 52 us (3.8 TB/s of what has to be read and written), the
// gradient 74 (2.7): 44 for dx, 25 for the column sums, 5 for the sum of their blocks.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "nf4_launch.h"
#include "nf4_pack16.h"

namespace nf4k {
using namespace pack16;
namespace {

#define GLOBAL __attribute__((address_space(1)))

// Sum over the 64 lanes, the same value in all of them.
__device__ __forceinline__ float wave_sum(float v)
{
    auto add = [](float a, int moved) { return a + __builtin_bit_cast(float, moved); };
    auto bits = [](float a) { return __builtin_bit_cast(int, a); };
    v = add(v, __builtin_amdgcn_update_dpp(0, bits(v), 0xB1, 0xf, 0xf, true));    // quads: lanes 1 0 3 2
    v = add(v, __builtin_amdgcn_update_dpp(0, bits(v), 0x4E, 0xf, 0xf, true));    // quads: lanes 2 3 0 1
    v = add(v, __builtin_amdgcn_update_dpp(0, bits(v), 0x141, 0xf, 0xf, true));   // mirrored within 8
    v = add(v, __builtin_amdgcn_update_dpp(0, bits(v), 0x140, 0xf, 0xf, true));   // mirrored within 16
    v = add(v, __builtin_amdgcn_update_dpp(0, bits(v), 0x142, 0xa, 0xf, true));   // row 0 into 1, 2 into 3
    v = add(v, __builtin_amdgcn_update_dpp(0, bits(v), 0x143, 0xc, 0xf, true));   // lane 31 into rows 2, 3
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(bits(v), 63));
}

// Sum over the kLanes threads of a row; buf: one slot per wave of the workgroup,
// not used by the reduction before this one.
template <int kLanes>
__device__ __forceinline__ float row_sum(float v, float* buf)
{
    v = wave_sum(v);
    if constexpr (kLanes > 64) {
        const int w = threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0) buf[w] = v;
        __syncthreads();
        constexpr int kWaves = kLanes / 64;
        const float* b = buf + (w & ~(kWaves - 1));
        v = b[0];
#pragma unroll
        for (int i = 1; i < kWaves; ++i) v += b[i];
    }
    return v;
}

__device__ __forceinline__ u32x4 load16(const uint16_t* p, int64_t at)
{
    return *((const GLOBAL u32x4*)(p + at));
}

template <int DT>
__device__ __forceinline__ void unpack8(const u32x4& v, float (&f)[8])
{
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const f32x2 p = unpack2<DT>(v[j]);
        f[2 * j] = p.x;
        f[2 * j + 1] = p.y;
    }
}

template <int DT>
__device__ __forceinline__ u32x4 pack8(const float (&f)[8])
{
    return u32x4{pack2<DT>(f[0], f[1]), pack2<DT>(f[2], f[3]), pack2<DT>(f[4], f[5]), pack2<DT>(f[6], f[7])};
}

// h = x + residual in fp32, rounded to the 16-bit type.
template <int DT>
__device__ __forceinline__ u32x4 add8(const u32x4& a, const u32x4& b)
{
    u32x4 r;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const f32x2 p = unpack2<DT>(a[j]), q = unpack2<DT>(b[j]);
        r[j] = pack2<DT>(p.x + q.x, p.y + q.y);
    }
    return r;
}

constexpr u32x4 kZero = {0, 0, 0, 0};

// kThreads / kLanes rows at a time, kPieces eight-element pieces a thread.
template <int DT, bool RES, int kLanes, int kPieces>
__global__ __launch_bounds__(kLanes < 256 ? 256 : kLanes) void k_norm(NormArgs a)
{
    constexpr int kThreads = kLanes < 256 ? 256 : kLanes, kRows = kThreads / kLanes;
    __shared__ float buf[2][kThreads / 64];
    const int lane = threadIdx.x % kLanes, n8 = a.n >> 3;
    const int64_t step = (int64_t)gridDim.x * kRows;
    int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / kLanes;
    u32x4 w[kPieces], b[kPieces], x[kPieces], r[kPieces];
    auto fetch = [&](int64_t at) {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int p = lane + i * kLanes;
            const bool in = p < n8 && at < a.m;
            x[i] = in ? load16(a.x, at * a.n + 8 * p) : kZero;
            if constexpr (RES) r[i] = in ? load16(a.residual, at * a.n + 8 * p) : kZero;
        }
    };
    fetch(row);
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
        const int p = lane + i * kLanes;
        w[i] = p < n8 ? load16(a.weight, 8 * p) : kZero;
        b[i] = p < n8 ? load16(a.bias, 8 * p) : kZero;
    }
    const float inv = 1.0f / (float)a.n;
    // the same number of rounds for all threads of the workgroup
    for (int64_t first = (int64_t)blockIdx.x * kRows; first < a.m; first += step, row += step) {
        u32x4 h[kPieces];
        float sum = 0;
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int p = lane + i * kLanes;
            h[i] = x[i];
            if constexpr (RES) {
                h[i] = add8<DT>(x[i], r[i]);
                if (p < n8 && row < a.m) *((GLOBAL u32x4*)(a.total + row * a.n + 8 * p)) = h[i];
            }
            float f[8];
            unpack8<DT>(h[i], f);
            sum += ((f[0] + f[1]) + (f[2] + f[3])) + ((f[4] + f[5]) + (f[6] + f[7]));
        }
        fetch(row + step);
        const float mean = row_sum<kLanes>(sum, buf[0]) * inv;
        float sq = 0;
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            if (lane + i * kLanes < n8) {
                float f[8];
                unpack8<DT>(h[i], f);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    f[j] -= mean;
                    sq = __builtin_fmaf(f[j], f[j], sq);
                }
            }
        }
        const float rstd = 1.0f / __builtin_sqrtf(row_sum<kLanes>(sq, buf[1]) * inv + a.eps);
        if (row < a.m) {
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                const int p = lane + i * kLanes;
                if (p < n8) {
                    float f[8], g[8], c[8];
                    unpack8<DT>(h[i], f);
                    unpack8<DT>(w[i], g);
                    unpack8<DT>(b[i], c);
#pragma unroll
                    for (int j = 0; j < 8; ++j) f[j] = __builtin_fmaf((f[j] - mean) * rstd, g[j], c[j]);
                    *((GLOBAL u32x4*)(a.out + row * a.n + 8 * p)) = pack8<DT>(f);
                }
            }
            if (lane == 0) *((GLOBAL f32x2*)(a.stats + 2 * row)) = f32x2{mean, rstd};
        }
    }
}

// Rows longer than the registers: three passes over the row.
template <int DT, bool RES>
__global__ __launch_bounds__(1024) void k_norm_long(NormArgs a)
{
    __shared__ float buf[2][16];
    const int n8 = a.n >> 3;
    const float inv = 1.0f / (float)a.n;
    // with a residual the sum is written first and read back by the same thread
    const uint16_t* h = RES ? a.total : a.x;
    for (int64_t row = blockIdx.x; row < a.m; row += gridDim.x) {
        float sum = 0;
        for (int p = threadIdx.x; p < n8; p += 1024) {
            u32x4 v = load16(a.x, row * a.n + 8 * (int64_t)p);
            if constexpr (RES) {
                v = add8<DT>(v, load16(a.residual, row * a.n + 8 * (int64_t)p));
                *((GLOBAL u32x4*)(a.total + row * a.n + 8 * (int64_t)p)) = v;
            }
            float f[8];
            unpack8<DT>(v, f);
            sum += ((f[0] + f[1]) + (f[2] + f[3])) + ((f[4] + f[5]) + (f[6] + f[7]));
        }
        const float mean = row_sum<1024>(sum, buf[0]) * inv;
        float sq = 0;
        for (int p = threadIdx.x; p < n8; p += 1024) {
            float f[8];
            unpack8<DT>(load16(h, row * a.n + 8 * (int64_t)p), f);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                f[j] -= mean;
                sq = __builtin_fmaf(f[j], f[j], sq);
            }
        }
        const float rstd = 1.0f / __builtin_sqrtf(row_sum<1024>(sq, buf[1]) * inv + a.eps);
        for (int p = threadIdx.x; p < n8; p += 1024) {
            float f[8], g[8], c[8];
            unpack8<DT>(load16(h, row * a.n + 8 * (int64_t)p), f);
            unpack8<DT>(load16(a.weight, 8 * (int64_t)p), g);
            unpack8<DT>(load16(a.bias, 8 * (int64_t)p), c);
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = __builtin_fmaf((f[j] - mean) * rstd, g[j], c[j]);
            *((GLOBAL u32x4*)(a.out + row * a.n + 8 * (int64_t)p)) = pack8<DT>(f);
        }
        if (threadIdx.x == 0) *((GLOBAL f32x2*)(a.stats + 2 * row)) = f32x2{mean, rstd};
    }
}

// ---- gradient

// kThreads / kLanes rows at a time; each thread sums its columns of dweight and
// dbias over the rows that it takes, the row groups' sums meet in LDS and are added
// in group order, and the workgroup writes one partial.
template <int DT, bool RES, int kLanes, int kPieces>
__global__ __launch_bounds__(512) void k_norm_grad(NormGradArgs a)
{
    constexpr int kThreads = 512, kRows = kThreads / kLanes;
    __shared__ float buf[4][kThreads / 64];
    __shared__ f32x4 acc[kRows > 1 ? kRows : 1][2][kRows > 1 ? 2 * kLanes * kPieces : 1];
    const int lane = threadIdx.x % kLanes, group = threadIdx.x / kLanes, n8 = a.n >> 3;
    const int64_t step = (int64_t)gridDim.x * kRows;
    int64_t row = (int64_t)blockIdx.x * kRows + group;
    u32x4 w[kPieces], x[kPieces], d[kPieces], r[kPieces];
    f32x2 st = {0, 0};
    auto fetch = [&](int64_t at) {
        if (at < a.m) st = *((const GLOBAL f32x2*)(a.stats + 2 * at));
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int p = lane + i * kLanes;
            const bool in = p < n8 && at < a.m;
            x[i] = in ? load16(a.x, at * a.n + 8 * p) : kZero;
            d[i] = in ? load16(a.dy, at * a.n + 8 * p) : kZero;
            if constexpr (RES) r[i] = in ? load16(a.residual, at * a.n + 8 * p) : kZero;
        }
    };
    fetch(row);
    float dw[kPieces][8] = {}, db[kPieces][8] = {};
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
        const int p = lane + i * kLanes;
        w[i] = p < n8 ? load16(a.weight, 8 * p) : kZero;
    }
    const float inv = 1.0f / (float)a.n;
    int slot = 0;
    for (int64_t first = (int64_t)blockIdx.x * kRows; first < a.m; first += step, row += step, slot ^= 2) {
        const float mean = st.x, rstd = st.y;
        u32x4 cx[kPieces], cd[kPieces], cr[kPieces];
        float s0 = 0, s1 = 0;
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            cx[i] = x[i];
            cd[i] = d[i];
            if constexpr (RES) cr[i] = r[i];
        }
        fetch(row + step);
        // rows and columns past the end have dy = 0; their c must not reach the sums as NaN
        if (row < a.m) {
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                if (lane + i * kLanes < n8) {
                    float f[8], e[8], g[8];
                    unpack8<DT>(cx[i], f);
                    unpack8<DT>(cd[i], e);
                    unpack8<DT>(w[i], g);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float c = (f[j] - mean) * rstd, t = e[j] * g[j];
                        dw[i][j] = __builtin_fmaf(e[j], c, dw[i][j]);
                        db[i][j] += e[j];
                        s0 += t;
                        s1 = __builtin_fmaf(t, c, s1);
                    }
                }
            }
        }
        const float m0 = row_sum<kLanes>(s0, buf[slot]) * inv, m1 = row_sum<kLanes>(s1, buf[slot + 1]) * inv;
        if (row < a.m) {
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                const int p = lane + i * kLanes;
                if (p < n8) {
                    float f[8], e[8], g[8], q[8];
                    unpack8<DT>(cx[i], f);
                    unpack8<DT>(cd[i], e);
                    unpack8<DT>(w[i], g);
                    if constexpr (RES) unpack8<DT>(cr[i], q);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float c = (f[j] - mean) * rstd, t = e[j] * g[j];
                        f[j] = (t - m0 - c * m1) * rstd;
                        if constexpr (RES) f[j] += q[j];
                    }
                    *((GLOBAL u32x4*)(a.dx + row * a.n + 8 * p)) = pack8<DT>(f);
                }
            }
        }
    }
    const bool direct = gridDim.x == 1;
    float* to_w = direct ? a.dweight : a.part + (int64_t)blockIdx.x * 2 * a.n;
    float* to_b = direct ? a.dbias : to_w + a.n;
    if constexpr (kRows == 1) {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int p = lane + i * kLanes;
            if (p < n8) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    *((GLOBAL f32x4*)(to_w + 8 * p + 4 * h)) =
                        f32x4{dw[i][4 * h], dw[i][4 * h + 1], dw[i][4 * h + 2], dw[i][4 * h + 3]};
                    *((GLOBAL f32x4*)(to_b + 8 * p + 4 * h)) =
                        f32x4{db[i][4 * h], db[i][4 * h + 1], db[i][4 * h + 2], db[i][4 * h + 3]};
                }
            }
        }
    } else {
        // quads of a group's 2 x 8 kLanes kPieces sums, a lane's four kLanes apart: no bank conflicts
#pragma unroll
        for (int i = 0; i < kPieces; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                acc[group][0][(2 * i + h) * kLanes + lane] =
                    f32x4{dw[i][4 * h], dw[i][4 * h + 1], dw[i][4 * h + 2], dw[i][4 * h + 3]};
                acc[group][1][(2 * i + h) * kLanes + lane] =
                    f32x4{db[i][4 * h], db[i][4 * h + 1], db[i][4 * h + 2], db[i][4 * h + 3]};
            }
        __syncthreads();
        for (int e = threadIdx.x; e < 4 * kLanes * kPieces; e += kThreads) {
            const int which = e / (2 * kLanes * kPieces), at = e % (2 * kLanes * kPieces), l = at % kLanes;
            const int p = l + at / (2 * kLanes) * kLanes, h = at / kLanes % 2;
            f32x4 t = acc[0][which][at];
#pragma unroll
            for (int k = 1; k < kRows; ++k) t += acc[k][which][at];
            if (p < n8) *((GLOBAL f32x4*)((which ? to_b : to_w) + 8 * p + 4 * h)) = t;
        }
    }
}

// Rows longer than the registers: dx by two passes over the row ...
template <int DT, bool RES>
__global__ __launch_bounds__(1024) void k_norm_grad_long(NormGradArgs a)
{
    __shared__ float buf[2][16];
    const int n8 = a.n >> 3;
    const float inv = 1.0f / (float)a.n;
    for (int64_t row = blockIdx.x; row < a.m; row += gridDim.x) {
        const int64_t at = row * a.n;
        const f32x2 st = *((const GLOBAL f32x2*)(a.stats + 2 * row));
        const float mean = st.x, rstd = st.y;
        float s0 = 0, s1 = 0;
        for (int p = threadIdx.x; p < n8; p += 1024) {
            float f[8], e[8], g[8];
            unpack8<DT>(load16(a.x, at + 8 * (int64_t)p), f);
            unpack8<DT>(load16(a.dy, at + 8 * (int64_t)p), e);
            unpack8<DT>(load16(a.weight, 8 * (int64_t)p), g);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float t = e[j] * g[j];
                s0 += t;
                s1 = __builtin_fmaf(t, (f[j] - mean) * rstd, s1);
            }
        }
        const float m0 = row_sum<1024>(s0, buf[0]) * inv, m1 = row_sum<1024>(s1, buf[1]) * inv;
        for (int p = threadIdx.x; p < n8; p += 1024) {
            float f[8], e[8], g[8], q[8];
            unpack8<DT>(load16(a.x, at + 8 * (int64_t)p), f);
            unpack8<DT>(load16(a.dy, at + 8 * (int64_t)p), e);
            unpack8<DT>(load16(a.weight, 8 * (int64_t)p), g);
            if constexpr (RES) unpack8<DT>(load16(a.residual, at + 8 * (int64_t)p), q);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                f[j] = (e[j] * g[j] - m0 - (f[j] - mean) * rstd * m1) * rstd;
                if constexpr (RES) f[j] += q[j];
            }
            *((GLOBAL u32x4*)(a.dx + at + 8 * (int64_t)p)) = pack8<DT>(f);
        }
    }
}

// ... and the column sums by a thread per piece over a block of rows.  Runs
// before k_norm_grad_long, so that dx may be dy or x.
template <int DT>
__global__ __launch_bounds__(256) void k_norm_columns(NormGradArgs a)
{
    const int p = blockIdx.x * 256 + threadIdx.x;
    if (p >= a.n >> 3) return;
    float dw[8] = {}, db[8] = {};
    for (int64_t row = blockIdx.y; row < a.m; row += gridDim.y) {
        const f32x2 st = *((const GLOBAL f32x2*)(a.stats + 2 * row));
        float f[8], e[8];
        unpack8<DT>(load16(a.x, row * a.n + 8 * (int64_t)p), f);
        unpack8<DT>(load16(a.dy, row * a.n + 8 * (int64_t)p), e);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            dw[j] = __builtin_fmaf(e[j], (f[j] - st.x) * st.y, dw[j]);
            db[j] += e[j];
        }
    }
    float* to_w = gridDim.y == 1 ? a.dweight : a.part + (int64_t)blockIdx.y * 2 * a.n;
    float* to_b = gridDim.y == 1 ? a.dbias : to_w + a.n;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        *((GLOBAL f32x4*)(to_w + 8 * (int64_t)p + 4 * h)) = f32x4{dw[4 * h], dw[4 * h + 1], dw[4 * h + 2], dw[4 * h + 3]};
        *((GLOBAL f32x4*)(to_b + 8 * (int64_t)p + 4 * h)) = f32x4{db[4 * h], db[4 * h + 1], db[4 * h + 2], db[4 * h + 3]};
    }
}

// The partials [blocks][2][n] summed over the blocks: 64 columns a workgroup, 32
// groups of 16 lanes that each take every 32nd block, then the groups in order.
__global__ __launch_bounds__(512) void k_norm_sum(const float* part, int blocks, int n, float* dweight, float* dbias)
{
    __shared__ f32x4 s[32][16];
    const int lane = threadIdx.x & 15, group = threadIdx.x >> 4;
    const int64_t at = (int64_t)blockIdx.x * 64 + 4 * lane, width = 2 * (int64_t)n;
    f32x4 t = {0, 0, 0, 0};
    if (at < width) {
        // four loads on their way: a few of them one after another is all a small sum's time
        for (int b = group; b < blocks; b += 128) {
            f32x4 v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = *((const GLOBAL f32x4*)(part + (b + 32 * k < blocks ? b + 32 * k : b) * width + at));
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (b + 32 * k < blocks) t += v[k];
        }
    }
    s[group][lane] = t;
    __syncthreads();
    if (group == 0 && at < width) {
        t = s[0][lane];
        for (int g = 1; g < 32; ++g) t += s[g][lane];
        *((GLOBAL f32x4*)(at < n ? dweight + at : dbias + (at - n))) = t;
    }
}

// Rows up to this many values stay in registers (forward, gradient).
constexpr int kMaxNorm = 24576, kMaxGrad = 16384;

// Workgroups of the kernels for longer ones: a row each, up to a grid's limit.
unsigned long_blocks(int64_t m) { return (unsigned)(m < 65536 ? m : 65536); }

template <int DT, bool RES, int kLanes, int kPieces>
hipError_t norm_go(const NormArgs& a, hipStream_t s)
{
    constexpr int kThreads = kLanes < 256 ? 256 : kLanes, kRows = kThreads / kLanes;
    const int64_t need = (a.m + kRows - 1) / kRows, most = 2048;
    k_norm<DT, RES, kLanes, kPieces><<<(unsigned)(need < most ? need : most), kThreads, 0, s>>>(a);
    return hipGetLastError();
}

template <int DT, bool RES, int kLanes>
hipError_t norm_pieces(const NormArgs& a, hipStream_t s)
{
    const int pieces = (a.n / 8 + kLanes - 1) / kLanes;
    if (pieces == 1) return norm_go<DT, RES, kLanes, 1>(a, s);
    if (pieces == 2) return norm_go<DT, RES, kLanes, 2>(a, s);
    if constexpr (kLanes == 1024) return norm_go<DT, RES, kLanes, 3>(a, s);   // four pieces do not fit 128 registers
    else return pieces == 3 ? norm_go<DT, RES, kLanes, 3>(a, s) : norm_go<DT, RES, kLanes, 4>(a, s);
}

template <int DT, bool RES>
hipError_t norm_any(const NormArgs& a, hipStream_t s)
{
    if (a.n <= 2048) return norm_pieces<DT, RES, 64>(a, s);
    if (a.n <= 8192) return norm_pieces<DT, RES, 256>(a, s);
    if (a.n <= kMaxNorm) return norm_pieces<DT, RES, 1024>(a, s);
    k_norm_long<DT, RES><<<long_blocks(a.m), 1024, 0, s>>>(a);
    return hipGetLastError();
}

// Threads of a row, by its length: one wave up to three pieces a thread (8192 x 1536 19.8 us, with 256 threads 22.9; 2000 x
// 2048 13.3 and 12.2).
int grad_lanes(int64_t n) { return n <= 1536 ? 64 : n <= 8192 ? 256 : 512; }

template <int DT, bool RES, int kLanes, int kPieces>
hipError_t grad_go(const NormGradArgs& a, int blocks, hipStream_t s)
{
    k_norm_grad<DT, RES, kLanes, kPieces><<<blocks, 512, 0, s>>>(a);
    return hipGetLastError();
}

template <int DT, bool RES, int kLanes>
hipError_t grad_pieces(const NormGradArgs& a, int blocks, hipStream_t s)
{
    const int pieces = (a.n / 8 + kLanes - 1) / kLanes;
    if (pieces == 1) return grad_go<DT, RES, kLanes, 1>(a, blocks, s);
    if (pieces == 2) return grad_go<DT, RES, kLanes, 2>(a, blocks, s);
    if constexpr (kLanes == 64) return grad_go<DT, RES, kLanes, 3>(a, blocks, s);
    else return pieces == 3 ? grad_go<DT, RES, kLanes, 3>(a, blocks, s) : grad_go<DT, RES, kLanes, 4>(a, blocks, s);
}

template <int DT, bool RES>
hipError_t grad_any(const NormGradArgs& a, hipStream_t s)
{
    const int blocks = norm_grad_blocks(a.m, a.n);
    hipError_t e;
    if (a.n > kMaxGrad) {
        k_norm_columns<DT><<<dim3((unsigned)((a.n / 8 + 255) / 256), (unsigned)blocks), 256, 0, s>>>(a);
        if ((e = hipGetLastError()) != hipSuccess) return e;
        k_norm_grad_long<DT, RES><<<long_blocks(a.m), 1024, 0, s>>>(a);
        e = hipGetLastError();
    } else if (a.n <= 1536) {
        e = grad_pieces<DT, RES, 64>(a, blocks, s);
    } else if (a.n <= 8192) {
        e = grad_pieces<DT, RES, 256>(a, blocks, s);
    } else {
        e = grad_pieces<DT, RES, 512>(a, blocks, s);
    }
    if (e != hipSuccess || blocks == 1) return e;
    k_norm_sum<<<(unsigned)((2 * (int64_t)a.n + 63) / 64), 512, 0, s>>>(a.part, blocks, a.n, a.dweight, a.dbias);
    return hipGetLastError();
}

}  // namespace

int norm_grad_blocks(int64_t m, int64_t n)
{
    if (n > kMaxGrad) {
        const int64_t b = (m + 15) / 16;   // at least 16 rows a block
        return (int)(b < 64 ? b : 64);
    }
    const int lanes = grad_lanes(n), rows = 512 / lanes;
    const int64_t b = (m + rows - 1) / rows, pieces = (n / 8 + lanes - 1) / lanes;
    // one workgroup's rounds take about half a us for each piece of a thread's; more workgroups need the sums' launch (8
    // rows of 2048 5.5 us in four rounds, 7.6 with a workgroup for every two; 32 rows of 512 4.9 in four and 64 7.3 in
    // eight, with a workgroup for every eight 6.0)
    if (b <= 5 && b * pieces <= 8) return 1;
    // past 64 two rounds each and half the partials (333 x 2048 7.9 us, with one round 8.5; 300 x 16384 18.2 and 21.5)
    const int64_t half = (b + 1) / 2;
    if (b > 64) return (int)(half < 64 ? 64 : half < 256 ? half : 256);
    return (int)b;
}

hipError_t launch_layer_norm(int dtype, const NormArgs& a, hipStream_t s)
{
    if (dtype == 0) return a.residual ? norm_any<0, true>(a, s) : norm_any<0, false>(a, s);
    return a.residual ? norm_any<1, true>(a, s) : norm_any<1, false>(a, s);
}

hipError_t launch_layer_norm_grad(int dtype, const NormGradArgs& a, hipStream_t s)
{
    if (dtype == 0) return a.residual ? grad_any<0, true>(a, s) : grad_any<0, false>(a, s);
    return a.residual ? grad_any<1, true>(a, s) : grad_any<1, false>(a, s);
}

}  // namespace nf4k
