/*
 * mx4.h -- C ABI of the microscaled 4-bit codec and products on MI355X
 * (gfx950), next to the NF4 codec of nf4.h in the same library.
 *
 * The format (MXFP4 of the OCP Microscaling Formats specification 1.0) is the
 * 4-bit one that the matrix cores read themselves: a matrix [rows x cols],
 * row-major, cols a multiple of 32, has
 *   codes   uint8 [rows x cols/2]: E2M1, the magnitudes 0, 0.5, 1, 1.5, 2, 3,
 *           4, 6 in code order and the sign in bit 3; element 2j in the low
 *           nibble of byte j;
 *   scales  uint8 [rows x cols/32]: E8M0, one per 32 consecutive elements of a
 *           row; s stands for 2^(s - 127), 255 for NaN.
 * An element's value is its code's times its scale.
 *
 * Quantisation: e = floor(log2(largest |x| of the 32)) - 2, clamped to -127 ..
 * 127 (-127 where all are zero), s = e + 127; the code nearest to x / 2^e,
 * ties to the even code, 6 beyond, the sign of x kept (a zero's too).  A group
 * that holds an infinity or a NaN gets s = 255 and codes that say nothing: all
 * its values read back as NaN.
 *
 * Conventions as in nf4.h: device buffers are the caller's, arguments are
 * checked on the host before anything is enqueued, calls only enqueue on
 * `stream`, nothing is kept between calls, results are the same from run to
 * run, and every call can be captured into a graph.  Calls that share no
 * buffer (workspaces among them) may overlap.
 */
#ifndef MX4_H
#define MX4_H

#include "nf4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Codes and scales of x [rows x cols] (dtype NF4_BF16 or NF4_FP16), and with
 * err (device fp64[1], else NULL) the matrix's reconstruction error, the sum
 * of (x - value)^2 in fp64: the score that aqlora_select takes.  1 <= rows, 1
 * <= cols, rows * cols < 2^40; cols not a multiple of 32: NF4_E_UNSUPPORTED.
 * x 16-byte, codes 16-byte, err 8-byte aligned.  ws:
 * mx4_quantize_workspace_bytes(rows, cols) with err, may be NULL where that is
 * 0; else unused. */
nf4_status mx4_quantize(const void* x, int64_t rows, int64_t cols, int32_t dtype, uint8_t* codes,
                        uint8_t* scales, double* err, void* ws, size_t ws_bytes, hipStream_t stream);

/* The values of codes and scales in dtype, each rounded once (infinity beyond its
 * range: fp16's, and in bf16 4 and 6 under scale 2^126, 2 to 6 under 2^127).  codes
 * and out 16-byte aligned. */
nf4_status mx4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols,
                          int32_t dtype, void* out, hipStream_t stream);

/* The product with a weight W [rows x cols] in this form and x in 16 bits:
 *   backward 0: out[m x rows] = x[m x cols] W^T
 *   backward 1: out[m x cols] = x[m x rows] W       (the input gradient)
 * x row-major in dtype, W's values rounded to dtype (as mx4_dequantize), sums
 * fp32 on the matrix cores; out row-major, fp32 (out_fp32 = 1) or dtype rounded
 * once.  rows a multiple of 8 and cols of 32 (else NF4_E_UNSUPPORTED), each
 * below 2^22 and their product below 2^40; 1 <= m <= 2^25; m times the larger side
 * at most 2^38.  x, codes and out 16-byte aligned; out must not overlap the
 * operands.  ws: mx4_matmul_workspace_bytes(rows, cols, backward, m), 256-byte
 * aligned, may be NULL where that is 0.  With few output tiles the reduction is split and the
 * parts are added in a fixed order.  A value that is not finite acts as in fp32
 * arithmetic, in its own row and column of the result only. */
nf4_status mx4_matmul(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols,
                      int32_t dtype, int32_t backward, const void* x, int64_t m, void* out,
                      int32_t out_fp32, void* ws, size_t ws_bytes, hipStream_t stream);

/* The forward product with both operands in this form: out[m x rows] = x W^T,
 * x [m x cols] as xcodes and xscales.  Sums are fp32 on the matrix cores.  The
 * product of two values, scales included, comes into them unrounded within fp32's
 * range, subnormal numbers among it; what is far below the smallest of those counts
 * as 0, what is past the largest number as an infinity.  A value past the range (6
 * under scale 254) times 0 is 0.  out: fp32 (out_fp32 = 1) or dtype rounded once.
 * Limits and alignment as for mx4_matmul, xcodes 16-byte aligned too.  ws:
 * mx4_matmul4_workspace_bytes(rows, cols, m). */
nf4_status mx4_matmul4(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols,
                       const uint8_t* xcodes, const uint8_t* xscales, int64_t m, int32_t dtype,
                       void* out, int32_t out_fp32, void* ws, size_t ws_bytes, hipStream_t stream);

/* ---- host-only helpers (pure; no HIP calls); 0 also on bad input ---- */
size_t mx4_quantize_workspace_bytes(int64_t rows, int64_t cols);
size_t mx4_matmul_workspace_bytes(int64_t rows, int64_t cols, int32_t backward, int64_t m);
size_t mx4_matmul4_workspace_bytes(int64_t rows, int64_t cols, int64_t m);
/* rows * cols / 2 + rows * cols / 32; -1 on bad input. */
int64_t mx4_storage_bytes(int64_t rows, int64_t cols);

#ifdef __cplusplus
}
#endif
#endif /* MX4_H */
