// abi_int8.cpp -- the C entry points of the int8 operators: host-side
// validation and dispatch. Every check runs before anything is enqueued, and
// no HIP call is made when a check fails.
#include "ffn_int8.h"

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "int8.h"
#include "kernels.h"

namespace {

constexpr int kMaxDim = 65536;
constexpr int kMaxChannels = 1 << 20;  // of a single product

bool aligned(const void *p, uintptr_t a)
{
    return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

bool dim_ok(int d)
{
    return d > 0 && d <= kMaxDim && d % 16 == 0;
}

bool batch_ok(int M)
{
    return M >= 0 && M <= 65536;
}

bool dtype_ok(int t)
{
    return t == FFN_INT8_BF16 || t == FFN_INT8_F16 || t == FFN_INT8_F32;
}

bool act_ok(int act)
{
    return act == FFN_NVFP4_ACT_SILU || act == FFN_NVFP4_ACT_GELU_TANH;
}

int check_weight(const ffn_int8_weight *w)
{
    if (!w || !w->codes || !w->scales)
        return FFN_NVFP4_ERR_NULL;
    if (!aligned(w->codes, 16) || !aligned(w->scales, 4))
        return FFN_NVFP4_ERR_ALIGN;
    return FFN_NVFP4_OK;
}

int check_ffn(int M, int K, int N)
{
    if (!dim_ok(K) || !dim_ok(N))
        return FFN_NVFP4_ERR_SHAPE;
    return batch_ok(M) ? FFN_NVFP4_OK : FFN_NVFP4_ERR_BATCH;
}

int check_gemm(int M, int K, int N)
{
    if (!dim_ok(K) || N <= 0 || N > kMaxChannels)
        return FFN_NVFP4_ERR_SHAPE;
    return batch_ok(M) ? FFN_NVFP4_OK : FFN_NVFP4_ERR_BATCH;
}

int launch_status(hipError_t e)
{
    return e == hipSuccess ? FFN_NVFP4_OK : FFN_NVFP4_ERR_LAUNCH;
}

size_t round256(size_t b)
{
    return (b + 255) & ~static_cast<size_t>(255);
}

size_t dtype_bytes(int t)
{
    return t == FFN_INT8_F32 ? 4 : 2;
}

// A buffer of a call. (A null one overlaps nothing.)
struct Span {
    const void *p;
    size_t bytes;
};

bool overlap(const Span &a, const Span &b)
{
    const uintptr_t i = reinterpret_cast<uintptr_t>(a.p), j = reinterpret_cast<uintptr_t>(b.p);
    return i && j && i < j + b.bytes && j < i + a.bytes;
}

ffn::Int8Out out_kind(int dtype)
{
    return dtype == FFN_INT8_BF16 ? ffn::I8_BF16 : dtype == FFN_INT8_F16 ? ffn::I8_F16 : ffn::I8_F32;
}

// The workspace of the gated FFN: h fp32 [M, N], its codes [M, N] and scales
// [M], then what the split products need (one at a time).
struct Workspace {
    size_t h, codes, scales, split, total;
};

Workspace layout(int M, int K, int N, int cus)
{
    Workspace w;
    const size_t e = static_cast<size_t>(M) * static_cast<size_t>(N);
    w.h = 0;
    w.codes = round256(4 * e);
    w.scales = w.codes + round256(e);
    w.split = w.scales + round256(4 * static_cast<size_t>(M));
    w.total = w.split + std::max(ffn::int8_gemm_workspace(M, K, N, ffn::I8_H_SILU, cus),
                                 ffn::int8_gemm_workspace(M, N, K, ffn::I8_BF16, cus));
    return w;
}

// h = act(gate) * up in fp32.
hipError_t gated(const int8_t *xq, const float *xs, int M, int K, int N, const ffn_int8_weight *gate,
                 const ffn_int8_weight *up, int act, char *workspace, const Workspace &w, int cus,
                 hipStream_t stream)
{
    float *h = reinterpret_cast<float *>(workspace + w.h);
    const ffn::Int8GemmArgs a{xq, xs, nullptr, gate->codes, up->codes, gate->scales, up->scales, nullptr, h,
                              M,  K,  N,       cus};
    return ffn::launch_int8_gemm(a, act == FFN_NVFP4_ACT_SILU ? ffn::I8_H_SILU : ffn::I8_H_GELU,
                                 workspace + w.split, stream);
}

// Its int8 rows.
hipError_t quantize_h(int M, int N, int8_t *hq, float *hs, const char *workspace, const Workspace &w,
                      hipStream_t stream)
{
    ffn::Int8RowsArgs r{};
    r.x = workspace + w.h;
    r.rows = M;
    r.cols = N;
    r.codes = hq;
    r.scales = hs;
    return ffn::launch_int8_quantize(r, FFN_INT8_F32, stream);
}

}  // namespace

extern "C" {

int ffn_int8_rmsnorm(const void *x, const void *residual, const void *weight, int M, int K, int dtype,
                     int weight_dtype, float eps, float weight_offset, int8_t *codes, float *scales,
                     void *sum_out, void *y_out, hipStream_t stream)
{
    if (!weight)
        return FFN_NVFP4_ERR_NULL;
    if (!aligned(weight, 16))
        return FFN_NVFP4_ERR_ALIGN;
    if (!dim_ok(K))
        return FFN_NVFP4_ERR_SHAPE;
    if (!batch_ok(M))
        return FFN_NVFP4_ERR_BATCH;
    if (!dtype_ok(dtype) || !dtype_ok(weight_dtype))
        return FFN_NVFP4_ERR_ACT;
    if (!std::isfinite(eps) || eps < 0.0f || !std::isfinite(weight_offset))
        return FFN_NVFP4_ERR_SCALE2;
    if (M == 0)
        return FFN_NVFP4_OK;
    if (!x || !codes || !scales)
        return FFN_NVFP4_ERR_NULL;
    if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(codes, 16) || !aligned(scales, 4) ||
        !aligned(sum_out, 16) || !aligned(y_out, 16))
        return FFN_NVFP4_ERR_ALIGN;
    // A row is in registers before any of it is written, so x or residual may be
    // written in place; rows that overlap others would be read after that.
    const size_t elements = static_cast<size_t>(M) * static_cast<size_t>(K);
    const size_t real = elements * dtype_bytes(dtype);
    const Span in[] = {{x, real}, {residual, real}, {weight, static_cast<size_t>(K) * dtype_bytes(weight_dtype)}};
    const Span out[] = {{sum_out, real}, {y_out, real}, {codes, elements}, {scales, 4 * static_cast<size_t>(M)}};
    for (int o = 0; o < 4; ++o) {
        for (int i = 0; i < 3; ++i) {
            const bool in_place = o < 2 && i < 2 && out[o].p == in[i].p;
            if (!in_place && overlap(out[o], in[i]))
                return FFN_NVFP4_ERR_ALIAS;
        }
        for (int other = 0; other < o; ++other)
            if (overlap(out[o], out[other]))
                return FFN_NVFP4_ERR_ALIAS;
    }
    const ffn::Int8RowsArgs a{x, residual, weight, M, K, eps, weight_offset, codes, scales, sum_out, y_out};
    return launch_status(ffn::launch_int8_rmsnorm(a, dtype, weight_dtype, stream));
}

int ffn_int8_quantize(const void *x, int rows, int cols, int dtype, int8_t *codes, float *scales,
                      hipStream_t stream)
{
    if (!dim_ok(cols))
        return FFN_NVFP4_ERR_SHAPE;
    if (rows < 0 || rows > kMaxChannels)
        return FFN_NVFP4_ERR_BATCH;
    if (!dtype_ok(dtype))
        return FFN_NVFP4_ERR_ACT;
    if (rows == 0)
        return FFN_NVFP4_OK;
    if (!x || !codes || !scales)
        return FFN_NVFP4_ERR_NULL;
    if (!aligned(x, 16) || !aligned(codes, 16) || !aligned(scales, 4))
        return FFN_NVFP4_ERR_ALIGN;
    ffn::Int8RowsArgs a{};
    a.x = x;
    a.rows = rows;
    a.cols = cols;
    a.codes = codes;
    a.scales = scales;
    return launch_status(ffn::launch_int8_quantize(a, dtype, stream));
}

int ffn_int8_prepare_weight(const ffn_nvfp4_weight *w, int rows, int cols, int8_t *codes, float *scales,
                            hipStream_t stream)
{
    if (!w || !w->codes || !w->scales || !codes || !scales)
        return FFN_NVFP4_ERR_NULL;
    if (!aligned(w->codes, 16) || !aligned(w->scales, 2) || !aligned(codes, 16) || !aligned(scales, 4))
        return FFN_NVFP4_ERR_ALIGN;
    if (rows <= 0 || rows > kMaxDim || cols <= 0 || cols > kMaxDim || cols % 32 != 0)
        return FFN_NVFP4_ERR_SHAPE;
    if (!std::isfinite(w->scale2))
        return FFN_NVFP4_ERR_SCALE2;
    return launch_status(
        ffn::launch_int8_requant(w->codes, w->scales, w->scale2, rows, cols, codes, scales, stream));
}

size_t ffn_int8_gemm_workspace_bytes(int M, int K, int N)
{
    if (M == 0 || check_gemm(M, K, N) != FFN_NVFP4_OK)
        return 0;
    return ffn::int8_gemm_workspace(M, K, N, ffn::I8_BF16, ffn::device_cu_count());
}

int ffn_int8_gemm(const int8_t *xq, const float *xs, int M, int K, int N, const ffn_int8_weight *w,
                  const float *bias, int out_dtype, void *out, void *workspace, size_t workspace_bytes,
                  hipStream_t stream)
{
    int rc;
    if ((rc = check_weight(w)) || (rc = check_gemm(M, K, N)))
        return rc;
    if (!dtype_ok(out_dtype))
        return FFN_NVFP4_ERR_ACT;
    if (M == 0)
        return FFN_NVFP4_OK;
    const int cus = ffn::device_cu_count();
    const size_t need = ffn::int8_gemm_workspace(M, K, N, ffn::I8_BF16, cus);
    if (!xq || !xs || !out || (need > 0 && !workspace))
        return FFN_NVFP4_ERR_NULL;
    if (!aligned(xq, 16) || !aligned(xs, 4) || !aligned(bias, 4) || !aligned(out, 16) || !aligned(workspace, 16))
        return FFN_NVFP4_ERR_ALIGN;
    if (workspace_bytes < need)
        return FFN_NVFP4_ERR_WORKSPACE;
    const ffn::Int8GemmArgs a{xq, xs, nullptr, w->codes, nullptr, w->scales, nullptr, bias, out, M, K, N, cus};
    return launch_status(ffn::launch_int8_gemm(a, out_kind(out_dtype), workspace, stream));
}

size_t ffn_int8_workspace_bytes(int M, int K, int N)
{
    if (M == 0 || check_ffn(M, K, N) != FFN_NVFP4_OK)
        return 0;
    return layout(M, K, N, ffn::device_cu_count()).total;
}

int ffn_int8_dual_gemm(const int8_t *xq, const float *xs, int M, int K, int N, const ffn_int8_weight *gate,
                       const ffn_int8_weight *up, int act, int8_t *hq, float *hs, void *workspace,
                       size_t workspace_bytes, hipStream_t stream)
{
    int rc;
    if ((rc = check_weight(gate)) || (rc = check_weight(up)) || (rc = check_ffn(M, K, N)))
        return rc;
    if (!act_ok(act))
        return FFN_NVFP4_ERR_ACT;
    if (M == 0)
        return FFN_NVFP4_OK;
    if (!xq || !xs || !hq || !hs || !workspace)
        return FFN_NVFP4_ERR_NULL;
    if (!aligned(xq, 16) || !aligned(xs, 4) || !aligned(hq, 16) || !aligned(hs, 4) || !aligned(workspace, 16))
        return FFN_NVFP4_ERR_ALIGN;
    const int cus = ffn::device_cu_count();
    const Workspace w = layout(M, K, N, cus);
    if (workspace_bytes < w.total)
        return FFN_NVFP4_ERR_WORKSPACE;
    char *ws = static_cast<char *>(workspace);
    const hipError_t e = gated(xq, xs, M, K, N, gate, up, act, ws, w, cus, stream);
    return launch_status(e != hipSuccess ? e : quantize_h(M, N, hq, hs, ws, w, stream));
}

int ffn_int8_forward(const int8_t *xq, const float *xs, int M, int K, int N, const ffn_int8_weight *gate,
                     const ffn_int8_weight *up, const ffn_int8_weight *down, int act, int out_dtype,
                     void *workspace, size_t workspace_bytes, void *out, hipStream_t stream)
{
    int rc;
    if ((rc = check_weight(gate)) || (rc = check_weight(up)) || (rc = check_weight(down)) ||
        (rc = check_ffn(M, K, N)))
        return rc;
    if (!act_ok(act) || !dtype_ok(out_dtype))
        return FFN_NVFP4_ERR_ACT;
    if (M == 0)
        return FFN_NVFP4_OK;
    if (!xq || !xs || !out || !workspace)
        return FFN_NVFP4_ERR_NULL;
    if (!aligned(xq, 16) || !aligned(xs, 4) || !aligned(out, 16) || !aligned(workspace, 16))
        return FFN_NVFP4_ERR_ALIGN;
    const int cus = ffn::device_cu_count();
    const Workspace w = layout(M, K, N, cus);
    if (workspace_bytes < w.total)
        return FFN_NVFP4_ERR_WORKSPACE;
    char *ws = static_cast<char *>(workspace);
    int8_t *hq = reinterpret_cast<int8_t *>(ws + w.codes);
    float *hs = reinterpret_cast<float *>(ws + w.scales);
    // One token's h goes into the down product as it is, which quantises it by
    // the same rule (5120/17408: 4.7 us and a launch saved).
    const bool row = M == 1 && N <= ffn::kInt8RowMost;
    hipError_t e = gated(xq, xs, M, K, N, gate, up, act, ws, w, cus, stream);
    if (e == hipSuccess && !row)
        e = quantize_h(M, N, hq, hs, ws, w, stream);
    if (e != hipSuccess)
        return FFN_NVFP4_ERR_LAUNCH;
    const float *h = row ? reinterpret_cast<const float *>(ws + w.h) : nullptr;
    const ffn::Int8GemmArgs a{hq, hs, h, down->codes, nullptr, down->scales, nullptr, nullptr, out, M, N, K, cus};
    return launch_status(ffn::launch_int8_gemm(a, out_kind(out_dtype), ws + w.split, stream));
}

}  // extern "C"
