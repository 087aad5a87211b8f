// k_linear_back.hip -- nf4_linear, backward: the kernels of nf4_gemm.h with the
// epilogue of an adapted layer's input gradient (low-rank term, under dropout or
// not, and the gradient that it is added to).  The kernels, tiles and splits are
// nf4_matmul_ws's for the same shape.
#include "nf4_gemm.h"

namespace nf4k {

hipError_t launch_nf4_linear_back(int dtype, const uint8_t* codes, const int8_t* qabsmax, const float* scale2,
                                  const float* absmax, int64_t rows, int64_t cols, const void* x, int64_t m, void* out,
                                  bool out_f32, float* part, int nsplit, int tail_split, const EpiArgs& epi,
                                  hipStream_t s)
{
    const GemmArgs g = gemm_args(codes, qabsmax, scale2, absmax, rows, cols, false, x, m, out, part, nsplit, tail_split);
    const bool dq = qabsmax != nullptr;
    return epi.drop.thr ? gemm_any<false>(dtype, dq, out_f32, g, WithDrop{epi}, s)
                        : gemm_any<false>(dtype, dq, out_f32, g, WithEpi{epi}, s);
}

}  // namespace nf4k
