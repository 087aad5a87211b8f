// nf4_philox.h -- the counter-based dropout mask shared by the kernels that
// drop: a function of (seed, offset, element index) only, so every call
// recomputes it and none stores it.
//
// Generator: Philox4x32 with 7 rounds (Salmon, Moraes, Dror and Shaw,
// "Parallel random numbers: as easy as 1, 2, 3", 2011; the paper's tests find
// no failure from 7 rounds on).  One call gives 128 bits = eight 16-bit lanes,
// one per element of a group of eight consecutive elements; an element is kept
// iff its lane >= thr, so the drop probability is thr / 65536 exactly.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "nf4_launch.h"

namespace nf4k {

struct PhiloxKey {
    uint32_t k0, k1, o0, o1;
};

__device__ __forceinline__ PhiloxKey philox_key(const uint64_t* rng)
{
    const uint64_t seed = rng[0], off = rng[1];
    return PhiloxKey{(uint32_t)seed, (uint32_t)(seed >> 32), (uint32_t)off, (uint32_t)(off >> 32)};
}

struct Bits128 {
    uint32_t w[4];
};

// The 128 bits of group `group`: lane i of the eight is the low (i even) or
// high (i odd) half of w[i / 2].
__device__ __forceinline__ Bits128 philox7(const PhiloxKey& key, uint64_t group)
{
    uint32_t c0 = (uint32_t)group, c1 = (uint32_t)(group >> 32), c2 = key.o0, c3 = key.o1;
    uint32_t k0 = key.k0, k1 = key.k1;
#pragma unroll
    for (int i = 0; i < 7; ++i) {
        const uint64_t p0 = (uint64_t)0xD2511F53u * c0, p1 = (uint64_t)0xCD9E8D57u * c2;
        // the three-input exclusive or in one instruction (truth table 0x96)
        c0 = __builtin_amdgcn_bitop3_b32((uint32_t)(p1 >> 32), c1, k0, 0x96);
        c1 = (uint32_t)p1;
        c2 = __builtin_amdgcn_bitop3_b32((uint32_t)(p0 >> 32), c3, k1, 0x96);
        c3 = (uint32_t)p0;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return Bits128{{c0, c1, c2, c3}};
}

// x with the half whose 16-bit lane of w is below thr (thr >= 1) set to zero:
// the lanes as signed values around thr (both less 2^15), their saturated
// difference, its sign spread over the half.
__device__ __forceinline__ uint32_t keep2(uint32_t x, uint32_t w, uint32_t thr)
{
    typedef int16_t s16x2 __attribute__((ext_vector_type(2)));
    const int16_t t = (int16_t)(thr ^ 0x8000u);
    const s16x2 d = __builtin_elementwise_sub_sat(__builtin_bit_cast(s16x2, w ^ 0x80008000u), s16x2{t, t});
    return x & ~__builtin_bit_cast(uint32_t, d >> 15);
}

// Bit i set iff element i of the group is kept.
__device__ __forceinline__ uint32_t keep_bits8(const Bits128& b, uint32_t thr)
{
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        m |= (b.w[j] & 0xffffu) >= thr ? 1u << (2 * j) : 0u;
        m |= (b.w[j] >> 16) >= thr ? 2u << (2 * j) : 0u;
    }
    return m;
}

}  // namespace nf4k
