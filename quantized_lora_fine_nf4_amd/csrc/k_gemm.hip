// k_gemm.hip -- nf4_matmul and nf4_matmul_ws: the kernels of nf4_gemm.h without
// an epilogue, and the choice of kernel and split for a shape.
#include "nf4_gemm.h"

namespace nf4k {

int nf4_matmul_splits(int64_t rows, int64_t cols, bool forward, int64_t m)
{
    // More than 128 rows of x and too few 256 x 256 tiles for a round: the
    // large-tile kernels with their reduction split (big_splits).
    // Where the large-tile kernels take the call whole (use_big): no split.
    // Otherwise the 128 x 128 kernel: with fewer output tiles than the chip
    // has CUs, each workgroup walks the whole reduction one dependent k-step
    // after another and the call is bound by that latency (0.083 ms for any
    // m <= 256 on a 13824 x 5120 weight); then aim at about 1,024 (tile,
    // split) workgroups, at most 16 splits of whole k-steps.  Measured on
    // that weight: split at m <= 128 0.038-0.051 ms forward (dequantise +
    // library GEMM 0.060-0.075), 0.063-0.070 backward (0.087-0.131); at 432
    // output tiles and 80 k-steps (m = 512 forward) a 3-way split was slower
    // than none: shapes are split below 256 tiles, or below 512 when the
    // reduction has 128 k-steps or more.
    const int64_t kred = forward ? cols : rows, ncol = forward ? rows : cols;
    const int bsp = big_splits(forward, m, ncol, kred);
    if (bsp > 0) return bsp;   // the 256 x 256 kernels, split
    if (use_big(forward, m, ncol, kred)) return 1;   // the 256 x 256 kernels, whole
    const int64_t tiles = ((m + kBM - 1) / kBM) * (ncol / kBN);
    const int64_t ksteps = kred / kBK;
    if (ksteps < 2 || tiles >= 512 || (tiles >= 256 && ksteps < 128)) return 1;
    int64_t sp = (1024 + tiles - 1) / tiles;
    if (sp > 16) sp = 16;
    if (sp > ksteps) sp = ksteps;
    const int64_t per = (ksteps + sp - 1) / sp;
    return (int)((ksteps + per - 1) / per);
}

int nf4_matmul_tail_splits(int64_t rows, int64_t cols, bool forward, int64_t m, int64_t* rem_out)
{
    // only where the 256 x 256 kernels take the call whole (no split planned)
    const int64_t kred = forward ? cols : rows, ncol = forward ? rows : cols;
    if (nf4_matmul_splits(rows, cols, forward, m) != 1) return 0;
    int64_t full = 0, rem = 0;
    const int sp = big_tail_splits(forward, m, ncol, kred, full, rem);
    if (sp > 0 && rem_out) *rem_out = rem;
    return sp;
}

int nf4_gemv_parts(int64_t rows, int64_t cols, bool forward, int64_t m)
{
    if (!forward || m > 32) return 0;
    const int64_t sc = gemv_part_sc(rows, cols, gemv_blocks(m)), nsc = cols / 128;
    return (int)((nsc + sc - 1) / sc);
}

hipError_t launch_nf4_gemv(int dtype, const uint8_t* codes, const int8_t* qabsmax, const float* scale2,
                           const float* absmax, int64_t rows, int64_t cols, const void* x, int64_t m,
                           void* out, bool out_f32, float* part, int parts, hipStream_t s)
{
    GemvArgs g;
    if (!gemv_args(g, codes, qabsmax, scale2, absmax, rows, cols, x, m, part, parts)) return hipErrorInvalidValue;
    return gemv_any(dtype, qabsmax != nullptr, out_f32, g, NoEpi{}, parts, out, s);
}

hipError_t launch_nf4_matmul(int dtype, const uint8_t* codes, const int8_t* qabsmax, const float* scale2,
                             const float* absmax, int64_t rows, int64_t cols, bool forward,
                             const void* x, int64_t m, void* out, bool out_f32, float* part, int nsplit,
                             int tail_split, hipStream_t s)
{
    const GemmArgs g = gemm_args(codes, qabsmax, scale2, absmax, rows, cols, forward, x, m, out, part, nsplit,
                                 tail_split);
    return forward ? gemm_any<true>(dtype, qabsmax != nullptr, out_f32, g, NoEpi{}, s)
                   : gemm_any<false>(dtype, qabsmax != nullptr, out_f32, g, NoEpi{}, s);
}

}  // namespace nf4k
