/*
 * ffn_moe.h -- C ABI of the sparse (mixture of experts) gated FFN of
 * libffn_nvfp4: the router's choice of experts, the plan that puts the chosen
 * (token, expert) pairs in expert order, the product grouped by expert over
 * NVFP4 weights, and the whole sparse FFN.
 *
 * A layer has E experts, each a gated FFN of its own with NVFP4 weights; a
 * token t goes through the top_k experts ids[t, 0 .. top_k - 1]:
 *     out[t] = sum_j weights[t, j] * W_d,e (act(W_g,e x[t]) * (W_u,e x[t])),
 *     e = ids[t, j],
 * products with fp32 accumulation, gate and up in fp32.
 *
 * The pair (t, j) is slot t * top_k + j. An id outside 0 .. E - 1 (-1, say)
 * is no expert: its slot adds nothing and no weight is read for it. That is
 * how padding tokens, and experts that live on another device, are left out. A
 * token may name an expert twice; it then counts twice.
 *
 * Expert order: the slots of expert 0, then those of expert 1 and so on, the
 * slots of one expert ascending. rows[i] is the slot at place i (-1 behind the
 * last expert's), offsets[e] the place where expert e begins (offsets[E]: where
 * the last one ends), places[s] the place of slot s (-1 for none).
 *
 * Conventions are those of ffn_nvfp4.h: device pointers owned by the caller,
 * row-major dense matrices, asynchronous on `stream`, host-side validation
 * before anything is enqueued, deterministic results, T = 0 a validated empty
 * call, status codes FFN_NVFP4_*, activations ffn_nvfp4_act. All of it can be
 * recorded in a graph.
 *   - T: 0 .. 65536; top_k: 1 .. 32 (else FFN_NVFP4_ERR_BATCH)
 *   - E: 1 .. 1024 (else FFN_NVFP4_ERR_SHAPE)
 *   - K, N: positive multiples of 32, at most 65536, unless an entry says
 *     otherwise (else FFN_NVFP4_ERR_SHAPE)
 *   - matrices of values or codes and workspaces are 16-byte aligned, block
 *     scales 2-byte, fp32 and int32 vectors 4-byte (else FFN_NVFP4_ERR_ALIGN)
 *   - an unknown type, activation or score is FFN_NVFP4_ERR_ACT
 *   - outputs and workspaces overlap no other buffer of the call, unless an
 *     entry says otherwise (else FFN_NVFP4_ERR_ALIAS)
 * What the device memory of a call holds cannot make it read or write outside
 * its buffers: ids, rows and offsets out of range are left out or taken as the
 * nearest in range.
 */
#ifndef FFN_MOE_H
#define FFN_MOE_H

#include <stddef.h>
#include <stdint.h>
#include <hip/hip_runtime_api.h>

#include "ffn_nvfp4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Types of real-valued inputs and outputs. */
typedef enum ffn_moe_dtype {
    FFN_MOE_BF16 = 0,
    FFN_MOE_F16 = 1,
    FFN_MOE_F32 = 2
} ffn_moe_dtype;

/* How a router's logits l[e] become scores. */
typedef enum ffn_moe_score {
    FFN_MOE_SOFTMAX = 0, /* exp(l[e]) / sum over all experts of exp(l) */
    FFN_MOE_SIGMOID = 1  /* 1 / (1 + exp(-l[e])) */
} ffn_moe_score;

/* NVFP4 weights [rows, cols] of E experts, one behind another: codes device
 * [E, rows, cols / 2], scales device E4M3 [E, rows, cols / 16], scale2 device
 * fp32 [E]. */
typedef struct ffn_moe_weight {
    const uint8_t *codes;
    const uint8_t *scales;
    const float *scale2;
} ffn_moe_weight;

/* The choice of experts: for each token the top_k experts of the largest keys,
 * the largest first, ties to the lower expert. The key is the logit itself, or
 * with a bias score + bias (in 64 bits, so that which of two close experts is
 * chosen does not hang on a rounding). weights = scale * score, or with
 * `normalize` scale * score / (sum of the chosen scores), 0 where that sum is 0.
 *   - An expert whose logit or key is -infinity is not available. Where
 *     fewer than top_k are, the ids behind them are -1, their weights 0.
 *   - A NaN logit ranks below every number but is available; weights are what
 *     the formula gives.
 *   - That holds where the scores alone are out of range too: logits of -88 and
 *     -89, or -1000 and -1001, have normalised sigmoid weights of 0.73 and 0.27.
 *     Only the sigmoid of the type's lowest finite value, which masks put in,
 *     counts as 0.
 *   logits   device [T, E] of `dtype`
 *   bias     device fp32 [E], or NULL
 *   scale    finite (else FFN_NVFP4_ERR_SCALE2)
 *   ids      device int32 [T, top_k] (written); weights: device fp32 (written)
 * top_k at most E (else FFN_NVFP4_ERR_BATCH). */
int ffn_moe_route(const void *logits, int T, int E, int dtype, const float *bias, int top_k, int score,
                  int normalize, float scale, int32_t *ids, float *weights, hipStream_t stream);

/* Bytes of device workspace ffn_moe_plan needs; 0 where it needs none, T = 0
 * or the shape is unsupported. Contents need no initialisation; calls that
 * share a workspace must not overlap. */
size_t ffn_moe_plan_workspace_bytes(int T, int top_k, int E);

/* Expert order of chosen experts (defined above).
 *   ids       device int32 [T, top_k]
 *   rows      device int32 [T * top_k] (written)
 *   offsets   device int32 [E + 1] (written, for T = 0 too)
 *   places    device int32 [T, top_k] (written)
 *   workspace device, >= ffn_moe_plan_workspace_bytes(T, top_k, E) bytes (may
 *             be NULL where that is 0) */
int ffn_moe_plan(const int32_t *ids, int T, int top_k, int E, int32_t *rows, int32_t *offsets, int32_t *places,
                 void *workspace, size_t workspace_bytes, hipStream_t stream);

/* The product grouped by expert:
 *     out[i] = scale2[e] * W_e x[r(i)],   offsets[e] <= i < offsets[e + 1],
 * r(i) = i, or rows[i] / top_k where `rows` is given (tokens' rows, read where
 * they are). Rows of `out` outside all experts are left as they were.
 *   x        device [x_rows, K] of `dtype` (FFN_MOE_BF16 or FFN_MOE_F16);
 *            x_rows >= R where `rows` is NULL (else FFN_NVFP4_ERR_BATCH)
 *   rows     device int32 [R], 0 <= rows[i] < x_rows * top_k, or NULL
 *   top_k    1 .. 32; 1 where `rows` is NULL (else FFN_NVFP4_ERR_BATCH)
 *   offsets  device int32 [E + 1], ascending, 0 <= offsets[e] <= R
 *   R        0 .. 2097152 (else FFN_NVFP4_ERR_BATCH); R = 0 is empty
 *   w        host struct of weights [N, K]
 *   out      device [R, N] of `out_dtype`: `dtype` or FFN_MOE_F32 (written)
 * N: 1 .. 1048576, any number. */
int ffn_moe_gemm(const void *x, int x_rows, int dtype, const int32_t *rows, int top_k, const int32_t *offsets,
                 int R, int E, int K, int N, const ffn_moe_weight *w, int out_dtype, void *out,
                 hipStream_t stream);

/* Bytes of device workspace ffn_moe_forward needs (the plan, h and the
 * experts' outputs); 0 if T = 0 or the shape is unsupported. Contents need no
 * initialisation. */
size_t ffn_moe_workspace_bytes(int T, int top_k, int E, int K, int N);

/* The whole sparse FFN (formula above). h is rounded to `dtype` once (in f16 a
 * magnitude past 65504 becomes infinite, and its token's outputs with it); the
 * experts' outputs stay in fp32 until their weighted sum, which runs with j
 * ascending, is rounded.
 *   x          device [T, K] of `dtype` (FFN_MOE_BF16 or FFN_MOE_F16)
 *   ids        device int32 [T, top_k]; weights: device fp32 [T, top_k]
 *   gate, up   host structs of weights [N, K]; down: of weights [K, N]
 *   workspace  device, >= ffn_moe_workspace_bytes(T, top_k, E, K, N) bytes;
 *              clobbered; calls that share it must not overlap
 *   out        device [T, K] of `dtype` (written; zeros for a token without
 *              an expert); may be x */
int ffn_moe_forward(const void *x, int T, int K, int N, int E, int top_k, int dtype, const int32_t *ids,
                    const float *weights, const ffn_moe_weight *gate, const ffn_moe_weight *up,
                    const ffn_moe_weight *down, int act, void *workspace, size_t workspace_bytes, void *out,
                    hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* FFN_MOE_H */
