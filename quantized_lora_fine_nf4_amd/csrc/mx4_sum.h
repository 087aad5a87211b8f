// mx4_sum.h -- the output types of the microscaled products, and the sum of a
// split reduction's partials.
#pragma once
#include "mx4_format.h"

namespace mx4k {

enum OutKind { kOutBf16 = 0, kOutFp16 = 1, kOutFp32 = 2 };

// Two, four or eight consecutive fp32 sums to the output type at element `at`
// (a multiple of their number; 16-byte aligned buffer).
__device__ __forceinline__ void store2(void* out, int kind, int64_t at, const f32x2& v)
{
    if (kind == kOutFp32) *((MX4_GLOBAL f32x2*)((float*)out + at)) = v;
    else *((MX4_GLOBAL uint32_t*)((uint16_t*)out + at)) = kind == kOutBf16 ? pack2<0>(v.x, v.y) : pack2<1>(v.x, v.y);
}

__device__ __forceinline__ void store4(void* out, int kind, int64_t at, const f32x4& v)
{
    if (kind == kOutFp32) *((MX4_GLOBAL f32x4*)((float*)out + at)) = v;
    else if (kind == kOutBf16) *((MX4_GLOBAL u32x2*)((uint16_t*)out + at)) = u32x2{pack2<0>(v[0], v[1]), pack2<0>(v[2], v[3])};
    else *((MX4_GLOBAL u32x2*)((uint16_t*)out + at)) = u32x2{pack2<1>(v[0], v[1]), pack2<1>(v[2], v[3])};
}

__device__ __forceinline__ void store8(void* out, int kind, int64_t at, const f32x4& a, const f32x4& b)
{
    if (kind == kOutFp32) {
        *((MX4_GLOBAL f32x4*)((float*)out + at)) = a;
        *((MX4_GLOBAL f32x4*)((float*)out + at + 4)) = b;
    } else if (kind == kOutBf16) {
        *((MX4_GLOBAL u32x4*)((uint16_t*)out + at)) =
            u32x4{pack2<0>(a[0], a[1]), pack2<0>(a[2], a[3]), pack2<0>(b[0], b[1]), pack2<0>(b[2], b[3])};
    } else {
        *((MX4_GLOBAL u32x4*)((uint16_t*)out + at)) =
            u32x4{pack2<1>(a[0], a[1]), pack2<1>(a[2], a[3]), pack2<1>(b[0], b[1]), pack2<1>(b[2], b[3])};
    }
}

}  // namespace mx4k
