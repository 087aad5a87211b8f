// nf4_act.h -- the activations of the matmul epilogue and their slopes, in
// fp32, shared by the forward epilogue and its gradient.
//
// With S the logistic function and P the normal distribution function:
//   relu       max(z, 0)                 slope z > 0
//   silu       z S(z)                    slope S(z) (1 + z (1 - S(z)))
//   gelu       z P(z)                    slope P(z) + z exp(-z^2/2) / sqrt(2 pi)
//   gelu_tanh  z S(2 t(z)),  t = sqrt(2/pi) (z + 0.044715 z^3)
//                                        slope S + z S (1 - S) 2 t'(z)
// The slopes are taken at z limited to +-100, beyond which every one of them
// has reached its limit in fp32, so an infinite z (a 16-bit preactivation that
// overflowed) gives the limit and not inf * 0.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace nf4k {

enum Act : int { ACT_NONE = 0, ACT_RELU = 1, ACT_SILU = 2, ACT_GELU = 3, ACT_GELU_TANH = 4 };

// e^x in about 2 units of the last place: the hardware 2^t with the rounding
// error of t = x log2(e) carried along (2^(t + d) = 2^t (1 + d ln 2)).
__device__ __forceinline__ float act_exp(float x)
{
    const float l2e = 1.44269504088896341f, l2e_lo = 1.92596299e-8f, ln2 = 0.69314718056f;
    const float t = x * l2e;
    const float d = fmaf(x, l2e_lo, fmaf(x, l2e, -t));
    const float e = __builtin_amdgcn_exp2f(t);
    return fmaf(e, d * ln2, e);
}

__device__ __forceinline__ float act_limit(float z) { return __builtin_amdgcn_fmed3f(z, -100.0f, 100.0f); }

// S(x); exp overflows to inf below -88.7 and the reciprocal gives 0.
__device__ __forceinline__ float act_sigmoid(float x)
{
    return __builtin_amdgcn_rcpf(1.0f + act_exp(-__builtin_amdgcn_fmed3f(x, -88.0f, 88.0f)));
}

constexpr float kTanhK = 1.59576912160573081f;   // 2 sqrt(2/pi)

__device__ __forceinline__ float act_value(float z, int act)
{
    switch (act) {
        case ACT_RELU: return z > 0.0f ? z : 0.0f;
        case ACT_SILU: return z * act_sigmoid(z);
        case ACT_GELU: return 0.5f * z * erfcf(z * -0.70710678118654752f);
        case ACT_GELU_TANH: {
            const float c = act_limit(z);
            return z * act_sigmoid(kTanhK * fmaf(0.044715f * c, c * c, c));
        }
        default: return z;
    }
}

__device__ __forceinline__ float act_slope(float zin, int act)
{
    const float z = act_limit(zin);
    switch (act) {
        case ACT_RELU: return z > 0.0f ? 1.0f : 0.0f;
        case ACT_SILU: {
            const float s = act_sigmoid(z);
            return s * fmaf(z, 1.0f - s, 1.0f);
        }
        case ACT_GELU:
            return fmaf(z * 0.39894228040143268f, act_exp(-0.5f * z * z), 0.5f * erfcf(z * -0.70710678118654752f));
        case ACT_GELU_TANH: {
            const float s = act_sigmoid(kTanhK * fmaf(0.044715f * z, z * z, z));
            return fmaf(z * s * (1.0f - s), kTanhK * fmaf(0.134145f * z, z, 1.0f), s);
        }
        default: return 1.0f;
    }
}

}  // namespace nf4k
