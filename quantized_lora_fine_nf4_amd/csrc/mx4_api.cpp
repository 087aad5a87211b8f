// mx4_api.cpp -- the C entry points of include/mx4.h: argument validation on the
// host, then the launch.
#include "mx4.h"

#include <hip/hip_runtime.h>

#include "mx4_launch.h"
#include "nf4_launch.h"

namespace {

constexpr int64_t kMaxN = int64_t(1) << 40, kMaxSide = int64_t(1) << 22, kMaxTokens = int64_t(1) << 25, kMaxOut = int64_t(1) << 38;

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

nf4_status check_codec(int64_t rows, int64_t cols, int32_t dtype)
{
    if (dtype != NF4_BF16 && dtype != NF4_FP16) return NF4_E_UNSUPPORTED;
    if (rows <= 0 || cols <= 0 || rows > (kMaxN - 1) / cols) return NF4_E_ARG;
    return cols % 32 ? NF4_E_UNSUPPORTED : NF4_OK;
}

nf4_status check_product(int64_t rows, int64_t cols, int64_t m, int32_t dtype, int32_t out_fp32)
{
    if (dtype != NF4_BF16 && dtype != NF4_FP16) return NF4_E_UNSUPPORTED;
    if (rows <= 0 || rows >= kMaxSide || cols <= 0 || cols >= kMaxSide || m <= 0 || m > kMaxTokens) return NF4_E_ARG;
    // more outputs than memory holds; the grids count their tiles in 32 bits
    if (m * (rows > cols ? rows : cols) > kMaxOut) return NF4_E_ARG;
    if (rows > (kMaxN - 1) / cols || (out_fp32 != 0 && out_fp32 != 1)) return NF4_E_ARG;
    return rows % 8 || cols % 32 ? NF4_E_UNSUPPORTED : NF4_OK;
}

nf4_status check_ws(const void* ws, size_t ws_bytes, size_t need)
{
    return need == 0 || (ws && aligned(ws, 256) && ws_bytes >= need) ? NF4_OK : NF4_E_WORKSPACE;
}

int out_kind(int32_t dtype, int32_t out_fp32) { return out_fp32 ? 2 : dtype == NF4_BF16 ? 0 : 1; }

nf4_status done(hipError_t e) { return e == hipSuccess ? NF4_OK : static_cast<nf4_status>(nf4k::hip_failed(e)); }

}  // namespace

extern "C" {

size_t mx4_quantize_workspace_bytes(int64_t rows, int64_t cols)
{
    if (check_codec(rows, cols, NF4_BF16) != NF4_OK) return 0;
    const int64_t blocks = mx4k::quantize_blocks(rows * cols);
    return blocks > 1 ? align256(size_t(blocks) * sizeof(double)) : 0;
}

nf4_status mx4_quantize(const void* x, int64_t rows, int64_t cols, int32_t dtype, uint8_t* codes, uint8_t* scales,
                        double* err, void* ws, size_t ws_bytes, hipStream_t stream)
{
    nf4_status st = check_codec(rows, cols, dtype);
    if (st != NF4_OK) return st;
    if (!x || !codes || !scales) return NF4_E_ARG;
    if (!aligned(x, 16) || !aligned(codes, 16) || !aligned(err, 8)) return NF4_E_ALIGN;
    if (err && (st = check_ws(ws, ws_bytes, mx4_quantize_workspace_bytes(rows, cols))) != NF4_OK) return st;
    return done(mx4k::launch_quantize(dtype, x, rows * cols, codes, scales, err, static_cast<double*>(ws), stream));
}

nf4_status mx4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, int32_t dtype,
                          void* out, hipStream_t stream)
{
    const nf4_status st = check_codec(rows, cols, dtype);
    if (st != NF4_OK) return st;
    if (!codes || !scales || !out) return NF4_E_ARG;
    if (!aligned(codes, 16) || !aligned(out, 16)) return NF4_E_ALIGN;
    return done(mx4k::launch_dequantize(dtype, codes, scales, rows * cols, out, stream));
}

size_t mx4_matmul_workspace_bytes(int64_t rows, int64_t cols, int32_t backward, int64_t m)
{
    if (check_product(rows, cols, m, NF4_BF16, 0) != NF4_OK || (backward != 0 && backward != 1)) return 0;
    return align256(mx4k::matmul_ws(rows, cols, backward == 0, m));
}

nf4_status mx4_matmul(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, int32_t dtype,
                      int32_t backward, const void* x, int64_t m, void* out, int32_t out_fp32, void* ws,
                      size_t ws_bytes, hipStream_t stream)
{
    nf4_status st = check_product(rows, cols, m, dtype, out_fp32);
    if (st != NF4_OK) return st;
    if (!codes || !scales || !x || !out || (backward != 0 && backward != 1)) return NF4_E_ARG;
    if (!aligned(codes, 16) || !aligned(x, 16) || !aligned(out, 16)) return NF4_E_ALIGN;
    if ((st = check_ws(ws, ws_bytes, mx4_matmul_workspace_bytes(rows, cols, backward, m))) != NF4_OK) return st;
    return done(mx4k::launch_matmul(dtype, codes, scales, rows, cols, backward == 0, x, m, out,
                                    out_kind(dtype, out_fp32), static_cast<float*>(ws), stream));
}

size_t mx4_matmul4_workspace_bytes(int64_t rows, int64_t cols, int64_t m)
{
    if (check_product(rows, cols, m, NF4_BF16, 0) != NF4_OK) return 0;
    return align256(mx4k::matmul4_ws(rows, cols, m));
}

nf4_status mx4_matmul4(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, const uint8_t* xcodes,
                       const uint8_t* xscales, int64_t m, int32_t dtype, void* out, int32_t out_fp32, void* ws,
                       size_t ws_bytes, hipStream_t stream)
{
    nf4_status st = check_product(rows, cols, m, dtype, out_fp32);
    if (st != NF4_OK) return st;
    if (!codes || !scales || !xcodes || !xscales || !out) return NF4_E_ARG;
    if (!aligned(codes, 16) || !aligned(xcodes, 16) || !aligned(out, 16)) return NF4_E_ALIGN;
    if ((st = check_ws(ws, ws_bytes, mx4_matmul4_workspace_bytes(rows, cols, m))) != NF4_OK) return st;
    return done(mx4k::launch_matmul4(codes, scales, rows, cols, xcodes, xscales, m, out, out_kind(dtype, out_fp32),
                                     static_cast<float*>(ws), stream));
}

int64_t mx4_storage_bytes(int64_t rows, int64_t cols)
{
    return check_codec(rows, cols, NF4_BF16) == NF4_OK ? rows * (cols / 2) + rows * (cols / 32) : -1;
}

}  // extern "C"
