// mx4_launch.h -- the kernel launchers behind include/mx4.h, called by mx4_api.cpp after it has validated the arguments (not part of the
// public ABI).  dtype: 0 bf16, 1 fp16.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mx4k {

// n elements (a multiple of 32, consecutive) to codes and scales.  With err
// their squared error in fp64, through quantize_blocks(n) fp64 partials at part
// (one block: straight to err).
int64_t quantize_blocks(int64_t n);
hipError_t launch_quantize(int dtype, const void* x, int64_t n, uint8_t* codes, uint8_t* scales, double* err,
                           double* part, hipStream_t s);
hipError_t launch_dequantize(int dtype, const uint8_t* codes, const uint8_t* scales, int64_t n, void* out,
                             hipStream_t s);

// out[m x rows] = x W^T (forward) or out[m x cols] = x W, W [rows x cols] given
// by codes and scales, x of dtype; out_kind 0 bf16, 1 fp16, 2 fp32.  matmul_ws
// bytes of partials at part (0: unused), a function of the shape only.
size_t matmul_ws(int64_t rows, int64_t cols, bool forward, int64_t m);
hipError_t launch_matmul(int dtype, const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols,
                         bool forward, const void* x, int64_t m, void* out, int out_kind, float* part, hipStream_t s);

// Their tiled kernels (k_mx4_mm.hip), for all but few tokens; a function of the
// reduction's length and the output's columns.
size_t mm_tiled_ws(int64_t kred, int64_t ncol, int64_t m, bool forward);
double mm_tiled_us(int64_t kred, int64_t ncol, int64_t m, bool forward);   // about how long they take
hipError_t launch_mm_tiled(int dtype, const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols,
                           bool forward, const void* x, int64_t m, void* out, int out_kind, float* part, hipStream_t s);

// The same forward with x [m x cols] in the microscaled form too.
size_t matmul4_ws(int64_t rows, int64_t cols, int64_t m);
hipError_t launch_matmul4(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols,
                          const uint8_t* xcodes, const uint8_t* xscales, int64_t m, void* out, int out_kind,
                          float* part, hipStream_t s);

// Its tiled kernels (k_mx4_mm4.hip), for all but few tokens.
size_t mm4_tiled_ws(int64_t rows, int64_t cols, int64_t m);
double mm4_tiled_us(int64_t rows, int64_t cols, int64_t m);
hipError_t launch_mm4_tiled(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols,
                            const uint8_t* xcodes, const uint8_t* xscales, int64_t m, void* out, int out_kind,
                            float* part, hipStream_t s);

// The sum of `splits` fp32 partials [m x ncol] (ncol a multiple of 8) in split
// order, to out with row pitch ldo.
hipError_t launch_split_sum(const float* part, int splits, int64_t m, int64_t ncol, void* out, int64_t ldo, int out_kind,
                            hipStream_t s);

}  // namespace mx4k
