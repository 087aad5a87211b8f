// nf4_pack16.h -- vector types and the packing of two 16-bit values (DT 0 bf16, 1
// fp16) that the microscaled and the layer norm kernels share.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#define MX4_GLOBAL __attribute__((address_space(1)))
#define MX4_LDS __attribute__((address_space(3)))

namespace nf4k {
namespace pack16 {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

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

}  // namespace pack16
}  // namespace nf4k
