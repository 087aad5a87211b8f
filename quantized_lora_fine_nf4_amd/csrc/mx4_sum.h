// mx4_sum.h -- the output types of the microscaled products, and the sum of a
// split reduction's partials.
#pragma once
#include "mx4_format.h"

namespace mx4k {

enum OutKind { kOutBf16 = 0, kOutFp16 = 1, kOutFp32 = 2 };

// Two, four or eight consecutive fp32 sums to a place of the output type KIND
// (aligned to their size there).
template <int KIND>
__device__ __forceinline__ uint32_t pack_out(float a, float b)
{
    return KIND == kOutBf16 ? pack2<0>(a, b) : pack2<1>(a, b);
}

template <int KIND>
__device__ __forceinline__ void put2(MX4_GLOBAL char* p, const f32x2& v)
{
    if constexpr (KIND == kOutFp32) *(MX4_GLOBAL f32x2*)p = v;
    else *(MX4_GLOBAL uint32_t*)p = pack_out<KIND>(v.x, v.y);
}

template <int KIND>
__device__ __forceinline__ void put4(MX4_GLOBAL char* p, const f32x4& v)
{
    if constexpr (KIND == kOutFp32) *(MX4_GLOBAL f32x4*)p = v;
    else *(MX4_GLOBAL u32x2*)p = u32x2{pack_out<KIND>(v[0], v[1]), pack_out<KIND>(v[2], v[3])};
}

template <int KIND>
__device__ __forceinline__ void put8(MX4_GLOBAL char* p, const f32x4& a, const f32x4& b)
{
    if constexpr (KIND == kOutFp32) {
        *(MX4_GLOBAL f32x4*)p = a;
        *(MX4_GLOBAL f32x4*)(p + 16) = b;
    } else {
        *(MX4_GLOBAL u32x4*)p = u32x4{pack_out<KIND>(a[0], a[1]), pack_out<KIND>(a[2], a[3]), pack_out<KIND>(b[0], b[1]),
                                      pack_out<KIND>(b[2], b[3])};
    }
}

// The same with the type known at run time only, at element `at` of out.
__device__ __forceinline__ void store2(void* out, int kind, int64_t at, const f32x2& v)
{
    MX4_GLOBAL char* p = (MX4_GLOBAL char*)out;
    if (kind == kOutFp32) put2<kOutFp32>(p + 4 * at, v);
    else if (kind == kOutBf16) put2<kOutBf16>(p + 2 * at, v);
    else put2<kOutFp16>(p + 2 * at, v);
}

__device__ __forceinline__ void store4(void* out, int kind, int64_t at, const f32x4& v)
{
    MX4_GLOBAL char* p = (MX4_GLOBAL char*)out;
    if (kind == kOutFp32) put4<kOutFp32>(p + 4 * at, v);
    else if (kind == kOutBf16) put4<kOutBf16>(p + 2 * at, v);
    else put4<kOutFp16>(p + 2 * at, v);
}

__device__ __forceinline__ void store8(void* out, int kind, int64_t at, const f32x4& a, const f32x4& b)
{
    MX4_GLOBAL char* p = (MX4_GLOBAL char*)out;
    if (kind == kOutFp32) put8<kOutFp32>(p + 4 * at, a, b);
    else if (kind == kOutBf16) put8<kOutBf16>(p + 2 * at, a, b);
    else put8<kOutFp16>(p + 2 * at, a, b);
}

}  // namespace mx4k
