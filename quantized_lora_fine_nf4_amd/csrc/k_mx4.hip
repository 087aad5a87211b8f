// k_mx4.hip -- microscaled 4-bit codes from 16-bit values and back, on gfx950.
//
//   e    = clamp(floor(log2(largest |x| of 32)) - 2, -127, 127), s = e + 127
//   code = nearest of x / 2^e (ties to even, 6 beyond)
//   err  = sum of (x - value)^2 over the matrix
//
// Rows are whole groups of 32, so a matrix is one run of elements.  A lane takes
// eight of them (16 bytes) and four lanes a group; the largest magnitude is an
// unsigned maximum over the bits without the sign, first in packed 16-bit halves
// and then over the four lanes, and s is its fp32 exponent field less 2.
//
// Both directions are one pass and bound by memory.  13824 x 5120 in bf16: codes,
// scales and error 34.4 us, 5.2 TB/s read and written, and the error's sum 5; back to
// 16 bits 27.5 us, 6.5 TB/s (a copy of 1 GiB reaches 5.2).  The error needs a fixed
// order: a workgroup's partial each, at most 2,048, and one workgroup for their sum.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mx4_format.h"
#include "mx4_launch.h"

namespace mx4k {
namespace {

typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

constexpr int kThreads = 256;
constexpr int kUnroll = 4;                               // 16-byte pieces in flight per lane
constexpr int64_t kPerBlock = 8 * kThreads * kUnroll;    // elements per workgroup and step
constexpr int64_t kMaxErrBlocks = 2048;

__device__ __forceinline__ uint32_t max16(uint32_t a, uint32_t b)
{
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a),
                                                                  __builtin_bit_cast(u16x2, b)));
}

// Largest magnitude of a group over its four lanes, as the 16-bit type's bits.
__device__ __forceinline__ uint32_t group_top(const u32x4& x)
{
    constexpr uint32_t kAbs = 0x7fff7fffu;
    uint32_t t = max16(max16(x[0] & kAbs, x[1] & kAbs), max16(x[2] & kAbs, x[3] & kAbs));
    t = max16(t, (uint32_t)__builtin_amdgcn_mov_dpp((int)t, 0xB1, 0xf, 0xf, true));   // lanes 1 0 3 2
    t = max16(t, (uint32_t)__builtin_amdgcn_mov_dpp((int)t, 0x4E, 0xf, 0xf, true));   // lanes 2 3 0 1
    const uint32_t lo = t & 0xffffu, hi = t >> 16;
    return lo > hi ? lo : hi;
}

template <int DT>
__device__ __forceinline__ uint32_t group_scale(uint32_t top)
{
    const uint32_t bits = __builtin_bit_cast(uint32_t, unpack2<DT>(top).x);
    const uint32_t f = bits >> 23;
    return f == 255 ? 255u : (f > 2 ? f - 2 : 0u);
}

// The squared error of eight values in fp64.  The fp32 difference is exact: for
// code 0 it is x; else |x| >= 2^(e - 2), both are multiples of x's last place
// (2^(e - 9) or more in bf16, 2^(e - 12) in fp16) and they differ by less than
// 2^(e + 1).
template <int DT>
__device__ __forceinline__ double err8(const u32x4& x, uint32_t codes, float scale)
{
    double e = 0;
    const f32x2 y[4] = {__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, scale, 0),
                        __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, scale, 1),
                        __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, scale, 2),
                        __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, scale, 3)};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const f32x2 v = unpack2<DT>(x[j]);
        const double a = (double)(v.x - y[j].x), b = (double)(v.y - y[j].y);
        e = __builtin_fma(a, a, e);
        e = __builtin_fma(b, b, e);
    }
    return e;
}

__device__ __forceinline__ double wave_sum(double v)
{
#pragma unroll
    for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
    return v;
}

template <int DT, bool ERR>
__global__ __launch_bounds__(kThreads) void k_quantize(const uint16_t* x, int64_t n, uint8_t* codes, uint8_t* scales,
                                                       double* part)
{
    const int64_t pieces = n >> 3;
    double err = 0;
    for (int64_t p0 = (int64_t)blockIdx.x * (kThreads * kUnroll) + threadIdx.x; p0 - threadIdx.x < pieces;
         p0 += (int64_t)gridDim.x * (kThreads * kUnroll)) {
        u32x4 v[kUnroll];
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            const int64_t p = p0 + i * kThreads;
            // past the end: zeros (the four lanes of a group are in or out together)
            v[i] = p < pieces ? __builtin_nontemporal_load((const MX4_GLOBAL u32x4*)x + p) : u32x4{0, 0, 0, 0};
        }
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            const int64_t p = p0 + i * kThreads;
            const uint32_t s = group_scale<DT>(group_top(v[i]));
            const float arg = scale_arg(s);
            const uint32_t c = encode8<DT>(v[i], arg);
            if (p < pieces) {
                ((MX4_GLOBAL uint32_t*)codes)[p] = c;
                if ((p & 3) == 0) ((MX4_GLOBAL uint8_t*)scales)[p >> 2] = (uint8_t)s;
            }
            if constexpr (ERR) err += err8<DT>(v[i], c, arg);
        }
    }
    if constexpr (ERR) {
        __shared__ double w[kThreads / 64];
        err = wave_sum(err);
        if ((threadIdx.x & 63) == 0) w[threadIdx.x >> 6] = err;
        __syncthreads();
        if (threadIdx.x == 0) {
            double t = w[0];
            for (int i = 1; i < kThreads / 64; ++i) t += w[i];
            part[blockIdx.x] = t;
        }
    }
}

__global__ __launch_bounds__(kThreads) void k_sum_err(const double* part, int blocks, double* err)
{
    __shared__ double w[kThreads / 64];
    double t = 0;
    for (int i = threadIdx.x; i < blocks; i += kThreads) t += part[i];
    t = wave_sum(t);
    if ((threadIdx.x & 63) == 0) w[threadIdx.x >> 6] = t;
    __syncthreads();
    if (threadIdx.x == 0) *err = ((w[0] + w[1]) + w[2]) + w[3];
}

template <int DT>
__global__ __launch_bounds__(kThreads) void k_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t n,
                                                         uint16_t* out)
{
    const int64_t pieces = n >> 3, p0 = (int64_t)blockIdx.x * (kThreads * kUnroll) + threadIdx.x;
    uint32_t c[kUnroll], s[kUnroll];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
        const int64_t p = p0 + i * kThreads;
        c[i] = p < pieces ? ((const MX4_GLOBAL uint32_t*)codes)[p] : 0u;
        s[i] = p < pieces ? ((const MX4_GLOBAL uint8_t*)scales)[p >> 2] : 0u;
    }
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
        const int64_t p = p0 + i * kThreads;
        if (p < pieces) ((MX4_GLOBAL u32x4*)out)[p] = decode8<DT>(c[i], scale_arg(s[i]));
    }
}

int64_t blocks_of(int64_t n) { return (n + kPerBlock - 1) / kPerBlock; }

}  // namespace

int64_t quantize_blocks(int64_t n)
{
    const int64_t b = blocks_of(n);
    // more than one need the sums' launch (24,576 values and back, in three steps of one 7.9 us a pass, in three of them
    // 10.2; in a graph 7.8 and 6.9)
    if (b <= 3) return 1;
    return b < kMaxErrBlocks ? b : kMaxErrBlocks;
}

hipError_t launch_quantize(int dtype, const void* x, int64_t n, uint8_t* codes, uint8_t* scales, double* err,
                           double* part, hipStream_t s)
{
    const uint16_t* xi = static_cast<const uint16_t*>(x);
    if (!err) {
        const dim3 grid((unsigned)blocks_of(n));
        if (dtype == 0) k_quantize<0, false><<<grid, kThreads, 0, s>>>(xi, n, codes, scales, nullptr);
        else k_quantize<1, false><<<grid, kThreads, 0, s>>>(xi, n, codes, scales, nullptr);
        return hipGetLastError();
    }
    const int64_t blocks = quantize_blocks(n);
    double* to = blocks == 1 ? err : part;
    if (dtype == 0) k_quantize<0, true><<<dim3((unsigned)blocks), kThreads, 0, s>>>(xi, n, codes, scales, to);
    else k_quantize<1, true><<<dim3((unsigned)blocks), kThreads, 0, s>>>(xi, n, codes, scales, to);
    if (blocks > 1) k_sum_err<<<1, kThreads, 0, s>>>(part, (int)blocks, err);
    return hipGetLastError();
}

hipError_t launch_dequantize(int dtype, const uint8_t* codes, const uint8_t* scales, int64_t n, void* out,
                             hipStream_t s)
{
    const dim3 grid((unsigned)blocks_of(n));
    uint16_t* o = static_cast<uint16_t*>(out);
    if (dtype == 0) k_dequantize<0><<<grid, kThreads, 0, s>>>(codes, scales, n, o);
    else k_dequantize<1><<<grid, kThreads, 0, s>>>(codes, scales, n, o);
    return hipGetLastError();
}

}  // namespace mx4k
