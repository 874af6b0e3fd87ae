// int8.h -- internal launchers of the int8 (W8A8) operators (host side).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ffn {

// Rows to int8 (int8_rows.hip). Types are those of ffn_int8_dtype.
struct Int8RowsArgs {
    const void *x;         // [rows, cols]
    const void *residual;  // [rows, cols] or null
    const void *weight;    // norm weight [cols], or null: no norm
    int rows, cols;
    float eps, weight_offset;
    int8_t *codes;   // [rows, cols]
    float *scales;   // [rows]
    void *sum_out;   // [rows, cols] or null
    void *y_out;     // [rows, cols] or null
};
hipError_t launch_int8_rmsnorm(const Int8RowsArgs &a, int dtype, int weight_dtype, hipStream_t stream);
hipError_t launch_int8_quantize(const Int8RowsArgs &a, int dtype, hipStream_t stream);
// NVFP4 codes and scales [rows, cols] -> int8 rows, scales times scale2.
hipError_t launch_int8_requant(const uint8_t *codes, const uint8_t *scales, float scale2, int rows, int cols,
                               int8_t *q, float *qs, hipStream_t stream);

// What a product's sums are turned into.
enum Int8Out : int {
    I8_BF16 = 0,    // out [M, N]: xs * s0 * sum (+ bias), rounded to the type
    I8_F16 = 1,
    I8_F32 = 2,
    I8_H_SILU = 3,  // two weights: out [M, N] fp32 = act(xs s0 sum0) * (xs s1 sum1)
    I8_H_GELU = 4,
};

// The longest row that a product takes as reals (96 registers of a thread hold
// its share, and its codes fit LDS behind every ring).
constexpr int kInt8RowMost = 24576;

struct Int8GemmArgs {
    const int8_t *x;            // [M, K]
    const float *xs;            // [M]
    const float *row;           // or, for M = 1 and K <= kInt8RowMost and one weight, x as reals [K], 16-byte aligned
    const int8_t *w0, *w1;      // [N, K]; w1 null for one weight
    const float *s0, *s1;       // [N]
    const float *bias;          // [N] or null
    void *out;
    int M, K, N;
    int cus;                    // compute units of the device (device_cu_count())
};

constexpr bool int8_two_weights(int out)
{
    return out == I8_H_SILU || out == I8_H_GELU;
}

// The product (int8_tile.hip). `workspace` holds int8_gemm_workspace(...) bytes
// (any contents): what workgroups that share a tile exchange.
hipError_t launch_int8_gemm(const Int8GemmArgs &a, Int8Out out, void *workspace, hipStream_t stream);
size_t int8_gemm_workspace(int M, int K, int N, Int8Out out, int cus);

}  // namespace ffn
