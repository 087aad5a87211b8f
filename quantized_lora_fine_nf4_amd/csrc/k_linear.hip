// k_linear.hip -- nf4_linear, forward: the kernels of nf4_gemm.h with the epilogue
// of an adapted layer (low-rank term, bias, activation, preactivation, residual).
// The kernels, tiles and splits are nf4_matmul_ws's for the same shape.
#include "nf4_gemm.h"

namespace nf4k {

hipError_t launch_nf4_linear_gemv(int dtype, const uint8_t* codes, const int8_t* qabsmax, const float* scale2,
                                  const float* absmax, int64_t rows, int64_t cols, const void* x, int64_t m, void* out,
                                  bool out_f32, float* part, int parts, const EpiArgs& epi, hipStream_t s)
{
    GemvArgs g;
    if (!gemv_args(g, codes, qabsmax, scale2, absmax, rows, cols, x, m, part, parts)) return hipErrorInvalidValue;
    return gemv_any(dtype, qabsmax != nullptr, out_f32, g, WithEpi{epi}, parts, out, s);
}

hipError_t launch_nf4_linear(int dtype, const uint8_t* codes, const int8_t* qabsmax, const float* scale2,
                             const float* absmax, int64_t rows, int64_t cols, const void* x, int64_t m, void* out,
                             bool out_f32, float* part, int nsplit, int tail_split, const EpiArgs& epi, hipStream_t s)
{
    const GemmArgs g = gemm_args(codes, qabsmax, scale2, absmax, rows, cols, true, x, m, out, part, nsplit, tail_split);
    return gemm_any<true>(dtype, qabsmax != nullptr, out_f32, g, WithEpi{epi}, s);
}

}  // namespace nf4k
