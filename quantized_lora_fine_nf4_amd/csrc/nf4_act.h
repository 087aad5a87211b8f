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
// overflowed) gives the limit and not inf * 0; the values do so too.  A NaN stays NaN in every value
// and slope, so that a run that has diverged shows it.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace nf4k {

enum Act : int { ACT_NONE = 0, ACT_RELU = 1, ACT_SILU = 2, ACT_GELU = 3, ACT_GELU_TANH = 4 };

// e^x: 2^t is within a step, t = x log2(e) within a step of |t| (log2(e) rounded,
// then the product), so the relative error is about |x| 2^-23; 0 below 2^-126,
// infinite past the largest fp32.
__device__ __forceinline__ float act_exp(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504088896341f); }

// +-100 at most.  The maximum and minimum that keep a NaN: the three-way median
// of one is its lower limit.
__device__ __forceinline__ float act_limit(float z)
{
    return __builtin_elementwise_minimum(__builtin_elementwise_maximum(z, -100.0f), 100.0f);
}

// S(x): 0 below -88.7, where exp overflows, and 1 at +infinity.  Below -87.3 S is
// less than the least normal fp32 and the reciprocal gives 0 as well.
__device__ __forceinline__ float act_sigmoid(float x) { return __builtin_amdgcn_rcpf(1.0f + act_exp(-x)); }

// The z that a value's factor S or P multiplies: both are 0 at -100, so the value
// reaches its limit 0 at -infinity and not inf * 0.
__device__ __forceinline__ float act_floor(float z) { return __builtin_elementwise_maximum(z, -100.0f); }

// P(z) and e = exp(-z^2/2): for z < 0, P(z) = e Q(t) / 2 with t = 1 / (1 + p
// |z| / sqrt 2), Q(t) = erfc(x) exp(x^2) at x = |z| / sqrt 2 as a polynomial
// without constant term (the form of Abramowitz and Stegun, Handbook of
// Mathematical Functions, 7.1.26): degree 9 and p = 0.38 from a least-maximum fit
// of the relative error over 0 <= x <= 14.2 (2.6e-8; 3.6e-7 as evaluated in fp32).
__device__ __forceinline__ float act_normal(float z, float& e)
{
    e = act_exp(-0.5f * z * z);
    const float t = __builtin_amdgcn_rcpf(fmaf(__builtin_fabsf(z), 0.38f * 0.70710678118654752f, 1.0f));
    float q = 0.05828981101512909f;
    q = fmaf(q, t, -0.2592635452747345f);
    q = fmaf(q, t, 0.3581995666027069f);
    q = fmaf(q, t, -0.15564434230327606f);
    q = fmaf(q, t, 0.2264687418937683f);
    q = fmaf(q, t, 0.13996803760528564f);
    q = fmaf(q, t, 0.20361974835395813f);
    q = fmaf(q, t, 0.21395252645015717f);
    q = fmaf(q, t, 0.21440942585468292f);
    const float tail = 0.5f * e * (q * t);
    return z < 0.0f ? tail : 1.0f - tail;
}

constexpr float kTanhK = 1.59576912160573081f;   // 2 sqrt(2/pi)

__device__ __forceinline__ float act_value(float z, int act)
{
    switch (act) {
        case ACT_RELU: return __builtin_elementwise_maximum(z, 0.0f);
        case ACT_SILU: return act_floor(z) * act_sigmoid(z);
        case ACT_GELU: {
            float e;
            return act_floor(z) * act_normal(z, e);
        }
        case ACT_GELU_TANH: {
            const float c = act_floor(z);
            return c * act_sigmoid(kTanhK * fmaf(0.044715f * c, c * c, c));
        }
        default: return z;
    }
}

__device__ __forceinline__ float act_slope(float zin, int act)
{
    if (act == ACT_RELU) return zin > 0.0f ? 1.0f : zin != zin ? zin : 0.0f;
    const float z = act_limit(zin);
    switch (act) {
        case ACT_SILU: {
            const float s = act_sigmoid(z);
            return s * fmaf(z, 1.0f - s, 1.0f);
        }
        case ACT_GELU: {
            float e;
            const float n = act_normal(z, e);
            return fmaf(z * 0.39894228040143268f, e, n);
        }
        case ACT_GELU_TANH: {
            const float s = act_sigmoid(kTanhK * fmaf(0.044715f * z, z * z, z));
            return fmaf(z * s * (1.0f - s), kTanhK * fmaf(0.134145f * z, z, 1.0f), s);
        }
        default: return 1.0f;
    }
}

}  // namespace nf4k
