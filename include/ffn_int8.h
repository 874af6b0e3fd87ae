/*
 * ffn_int8.h -- C ABI of the int8 (W8A8) gated FFN of libffn_nvfp4 and of the
 * operators around it: the root-mean-square norm with the residual's addition
 * and an int8 output, the row quantiser, and the int8 matrix product with a
 * scale for each token and each channel.
 *
 * Int8 rows. A row v of real values is held as codes q (int8) and one fp32
 * scale s, v[j] ~ s * q[j]:
 *     s = max_j |v[j]| / 127,    q[j] = rint(v[j] * (1 / s)),
 * each step one correctly rounded fp32 operation, rint to the nearest integer
 * with ties to even, so |q| <= 127 and q = +-127 where |v| is largest.
 *   - A row whose largest magnitude is below 127 * 2^-126 (a row of zeros
 *     among them) has s = 0 and codes 0: 1 / s would not be finite.
 *   - A row that holds an infinity or a NaN has s = NaN and codes 0: every
 *     product with it is NaN, and the other rows are not touched.
 * Activations are rows of tokens [M, K] (a scale for each token); weights are
 * rows of output channels [N, K] (a scale for each channel).
 *
 * The product: out[m, n] = sx[m] * sw[n] * sum_k qx[m, k] qw[n, k] + bias[n].
 * The sum runs in int32 and is exact (at most 65536 * 128 * 128 = 2^30), so
 * no order of summation, batch size or split of the work changes it: every
 * entry gives row m of a batch the same bits as a call on that row alone. The
 * sum is converted to fp32 once (to nearest), multiplied by sx[m], then by
 * sw[n], then the bias is added, and the result rounded once to the output's
 * type. Any int8 code is taken, -128 too, though the quantisers never
 * produce it.
 *
 * The gated FFN (dense_ffn.rs page, DenseFfnLayer::forward with the int8
 * weights of DenseFfnLayer::ensure_int8_weight):
 *     gate = W_g x, up = W_u x, h = act(gate) * up, out = W_d q(h),
 * gate, up and h in fp32 and h quantised as int8 rows, one scale for each
 * token (h rounded to bf16 first would move one code in a hundred of a
 * heavy-tailed row).
 *
 * Conventions are those of ffn_nvfp4.h: device pointers owned by the caller,
 * row-major dense matrices, asynchronous on `stream`, host-side validation
 * before anything is enqueued, deterministic results, M = 0 a validated empty
 * call, status codes FFN_NVFP4_*, activations ffn_nvfp4_act.
 *   - K, N: positive multiples of 16, at most 65536, unless an entry says
 *     otherwise (else FFN_NVFP4_ERR_SHAPE).
 *   - M: 0 .. 65536 (else FFN_NVFP4_ERR_BATCH).
 *   - matrices of codes or values, and workspaces, are 16-byte aligned; fp32
 *     vectors (scales, bias) 4-byte aligned (else FFN_NVFP4_ERR_ALIGN).
 *   - an unknown type is FFN_NVFP4_ERR_ACT.
 *   - outputs and workspaces overlap no other buffer of the call, unless an
 *     entry says otherwise.
 */
#ifndef FFN_INT8_H
#define FFN_INT8_H

#include <stddef.h>
#include <stdint.h>
#include <hip/hip_runtime_api.h>

#include "ffn_nvfp4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Types of real-valued inputs and outputs. */
typedef enum ffn_int8_dtype {
    FFN_INT8_BF16 = 0,
    FFN_INT8_F16 = 1,
    FFN_INT8_F32 = 2
} ffn_int8_dtype;

/* One int8 weight [rows, cols]: codes device, 16-byte aligned; scales device
 * fp32 [rows], 4-byte aligned. */
typedef struct ffn_int8_weight {
    const int8_t *codes;
    const float *scales;
} ffn_int8_weight;

/* Root-mean-square norm of x + residual, with int8 output:
 *   t[m, k] = x[m, k] + residual[m, k]                     (fp32)
 *   y[m, k] = t[m, k] / sqrt(mean_k t[m, k]^2 + eps) * (weight_offset + weight[k])
 *   sum_out = t, y_out = y, each rounded once to `dtype`;
 *   codes, scales = the int8 rows of y (of the unrounded y).
 * The norm is taken of t before it is rounded. Every row of finite t has its
 * norm: one whose squares do not fit fp32 is scaled by a power of two first. A
 * row with an infinity or a NaN in t has s = NaN and codes 0.
 *   x          device [M, K] of `dtype`
 *   residual   device [M, K] of `dtype`, or NULL (t = x)
 *   weight     device [K] of `weight_dtype`, 16-byte aligned
 *   eps        finite, >= 0; weight_offset finite (1 for weights stored as
 *              w - 1); else FFN_NVFP4_ERR_SCALE2. With eps = 0 a row of zeros
 *              has no norm: its y is NaN
 *   codes      device int8 [M, K] (written); scales: device fp32 [M] (written)
 *   sum_out    device [M, K] of `dtype` (written), or NULL; may be x or
 *              residual itself
 *   y_out      device [M, K] of `dtype` (written), or NULL; may be x or
 *              residual itself, not sum_out
 * Any other overlap of what is written with another buffer is
 * FFN_NVFP4_ERR_ALIAS. */
int ffn_int8_rmsnorm(const void *x, const void *residual, const void *weight, int M, int K, int dtype,
                     int weight_dtype, float eps, float weight_offset, int8_t *codes, float *scales,
                     void *sum_out, void *y_out, hipStream_t stream);

/* Int8 rows of x: activations that no norm precedes, or a weight at load.
 *   x       device [rows, cols] of `dtype`
 *   codes   device int8 [rows, cols] (written); scales: device fp32 [rows] (written) */
int ffn_int8_quantize(const void *x, int rows, int cols, int dtype, int8_t *codes, float *scales,
                      hipStream_t stream);

/* NVFP4 -> int8 weight, once at load: the int8 rows of e2m1 * e4m3, with the
 * row's scale multiplied by scale2 (which must be finite, else
 * FFN_NVFP4_ERR_SCALE2). cols a multiple of 32.
 *   w   host struct of an NVFP4 weight [rows, cols] (scales 2-byte aligned) */
int ffn_int8_prepare_weight(const ffn_nvfp4_weight *w, int rows, int cols, int8_t *codes, float *scales,
                            hipStream_t stream);

/* Bytes of device workspace ffn_int8_gemm needs; 0 where it needs none, M = 0
 * or the shape is unsupported. Contents need no initialisation; calls that
 * share a workspace must not overlap. */
size_t ffn_int8_gemm_workspace_bytes(int M, int K, int N);

/* The int8 product (formula above).
 *   xq, xs      device int8 [M, K] and fp32 [M]
 *   w           host struct of an int8 weight [N, K]
 *   bias        device fp32 [N], or NULL
 *   out         device [M, N] of `out_dtype` (written)
 *   workspace   device, >= ffn_int8_gemm_workspace_bytes(M, K, N) bytes
 *               (may be NULL where that is 0)
 * N: 1 .. 1048576, any number (a vocabulary, say). */
int ffn_int8_gemm(const int8_t *xq, const float *xs, int M, int K, int N, const ffn_int8_weight *w,
                  const float *bias, int out_dtype, void *out, void *workspace, size_t workspace_bytes,
                  hipStream_t stream);

/* Bytes of device workspace ffn_int8_dual_gemm and ffn_int8_forward need (h
 * in fp32, its codes and scales, and split reductions); 0 if M = 0 or the
 * shape is unsupported. Contents need no initialisation. */
size_t ffn_int8_workspace_bytes(int M, int K, int N);

/* The gated pair of products with an int8 output:
 * hq, hs = int8 rows of act(W_g x) * (W_u x).
 *   xq, xs     device int8 [M, K] and fp32 [M]
 *   gate, up   host structs of int8 weights [N, K]
 *   hq, hs     device int8 [M, N] and fp32 [M] (written)
 *   workspace  device, >= ffn_int8_workspace_bytes(M, K, N) bytes; clobbered;
 *              calls that share it must not overlap */
int ffn_int8_dual_gemm(const int8_t *xq, const float *xs, int M, int K, int N, const ffn_int8_weight *gate,
                       const ffn_int8_weight *up, int act, int8_t *hq, float *hs, void *workspace,
                       size_t workspace_bytes, hipStream_t stream);

/* The whole FFN: out[M, K] = W_d q(act(W_g x) * (W_u x)); the same bits as
 * ffn_int8_dual_gemm followed by ffn_int8_gemm.
 *   down   host struct of an int8 weight [K, N]
 *   out    device [M, K] of `out_dtype` (written)
 * The other arguments as ffn_int8_dual_gemm. */
int ffn_int8_forward(const int8_t *xq, const float *xs, int M, int K, int N, const ffn_int8_weight *gate,
                     const ffn_int8_weight *up, const ffn_int8_weight *down, int act, int out_dtype,
                     void *workspace, size_t workspace_bytes, void *out, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* FFN_INT8_H */
