// moe.h -- internal launchers of the sparse FFN's operators (host side).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace ffn {

// Types are those of ffn_moe_dtype.
constexpr int kMoeBf16 = 0, kMoeF16 = 1, kMoeF32 = 2;

// The router's choice (moe_route.hip).
struct MoeRouteArgs {
    const void *logits;  // [T, E]
    const float *bias;   // [E] or null
    int T, E, top_k;
    bool sigmoid, normalize;
    float scale;
    int32_t *ids;    // [T, top_k]
    float *weights;  // [T, top_k]
};
hipError_t launch_moe_route(const MoeRouteArgs &a, int dtype, hipStream_t stream);

// Expert order of R chosen experts (moe_plan.hip). `workspace`:
// moe_plan_workspace(R, E) bytes.
size_t moe_plan_workspace(int R, int E);
hipError_t launch_moe_plan(const int32_t *ids, int R, int E, int32_t *rows, int32_t *offsets, int32_t *places,
                           void *workspace, hipStream_t stream);

// out[t] = sum_j weights[t, j] * y[places[t, j]] (moe_combine.hip), y in fp32 and
// out of `dtype` with K columns, K a multiple of 8; places outside 0 .. R - 1 are
// skipped. With `ids` in place of places, y has a row for each slot; slots with
// ids outside 0 .. E - 1 are skipped.
hipError_t launch_moe_combine(const float *y, const int32_t *places, const int32_t *ids, const float *weights, int T,
                              int top_k, int R, int E, int K, int dtype, void *out, hipStream_t stream);

struct MoeWeightArg {
    const uint8_t *codes;   // [E, rows, cols/2]
    const uint8_t *scales;  // [E, rows, cols/16]
    const float *scale2;    // [E]
};

// What a grouped product's sums are turned into.
enum MoeOut : int {
    MOE_SAME = 0,    // scale2 * sum in x's type
    MOE_F32 = 1,     // scale2 * sum
    MOE_H_SILU = 2,  // two weights: act(s0 sum0) * (s1 sum1) in x's type
    MOE_H_GELU = 3,
};

constexpr bool moe_two_weights(int out)
{
    return out == MOE_H_SILU || out == MOE_H_GELU;
}

// The product grouped by expert (moe_gemm.hip).
struct MoeGemmArgs {
    const void *x;           // [x_rows, K]
    const int32_t *rows;     // [R] or null: row i of the product is x[rows[i] / top_k]
    const int32_t *offsets;  // [E + 1]
    const int32_t *ids;      // or, without a plan, the experts of the R slots: row s is of x[s / top_k]
    MoeWeightArg w0, w1;     // [E, N, K]; w1 for two weights
    void *out;               // [R, N]
    int x_rows, top_k, R, E, K, N;
};
// Whether products of R slots over [N, K] and [K, N] may go without a plan.
bool moe_by_slots(int R, int E, int K, int N);
hipError_t launch_moe_gemm(const MoeGemmArgs &a, int dtype, MoeOut out, hipStream_t stream);

}  // namespace ffn
