// mx4_format.h -- the microscaled 4-bit format on the device: E2M1 codes (0, 0.5, 1,
// 1.5, 2, 3, 4, 6 and their negatives), two to a byte, low nibble first, and one
// E8M0 scale (2^(s - 127), 255 is NaN) per 32 consecutive elements of a row
// (OCP Microscaling Formats specification 1.0).
//
// gfx950 converts from and to these codes itself: the conversions take the
// scale as an fp32 whose exponent field is s.  Every finite 16-bit input under 15
// scales from 0 to 254 and every code under every scale was compared with the
// definition: equal, ties to even, 6 beyond the range, s = 0 as 2^-127, 255 as NaN;
// sign and mantissa of the scale's fp32 do not matter.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "nf4_pack16.h"

namespace mx4k {

using namespace nf4k::pack16;

constexpr int kGroup = 32;   // elements per scale

// The fp32 that the conversions read as scale s.
__device__ __forceinline__ float scale_arg(uint32_t s) { return __builtin_bit_cast(float, s << 23); }

// The same from byte B of four packed scales: the conversions look at the exponent
// field alone, so a shift will do and no mask is needed.
template <int B>
__device__ __forceinline__ float byte_arg(uint32_t s)
{
    return __builtin_bit_cast(float, B == 3 ? s >> 1 : s << (23 - 8 * B));
}

// The two codes of byte `B` of a dword to two 16-bit values of type DT (0 bf16,
// 1 fp16), each code's value times 2^(s - 127) rounded once.
template <int DT, int B>
__device__ __forceinline__ uint32_t decode2(uint32_t codes, float scale)
{
    if constexpr (DT == 0) return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, B));
    else return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, scale, B));
}

// Eight codes (one dword) to eight 16-bit values.
template <int DT>
__device__ __forceinline__ u32x4 decode8(uint32_t codes, float scale)
{
    return u32x4{decode2<DT, 0>(codes, scale), decode2<DT, 1>(codes, scale), decode2<DT, 2>(codes, scale),
                 decode2<DT, 3>(codes, scale)};
}

// Two 16-bit values over 2^(s - 127) to their nearest codes, into byte B of `codes`.
template <int DT, int B>
__device__ __forceinline__ uint32_t encode2(uint32_t codes, uint32_t x, float scale)
{
    if constexpr (DT == 0) return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(codes, __builtin_bit_cast(bf16x2, x), scale, B);
    else return __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(codes, __builtin_bit_cast(f16x2, x), scale, B);
}

// Eight of them.
template <int DT>
__device__ __forceinline__ uint32_t encode8(const u32x4& x, float scale)
{
    uint32_t c = encode2<DT, 0>(0, x[0], scale);
    c = encode2<DT, 1>(c, x[1], scale);
    c = encode2<DT, 2>(c, x[2], scale);
    return encode2<DT, 3>(c, x[3], scale);
}

}  // namespace mx4k
