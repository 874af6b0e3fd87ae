// abi_moe.cpp -- the C entry points of the sparse FFN's operators: host-side
// validation and dispatch. Every check runs before anything is enqueued, and
// no HIP call is made when a check fails.
#include "ffn_moe.h"

#include <cmath>
#include <cstdint>

#include "moe.h"
#include "span.h"

namespace {

using ffn::Span;

constexpr int kMaxDim = 65536;
constexpr int kMaxChannels = 1 << 20;  // of a single product
constexpr int kMaxTokens = 65536;
constexpr int kMaxTopK = 32;
constexpr int kMaxExperts = 1024;
constexpr int kMaxRows = kMaxTokens * kMaxTopK;

bool aligned(const void *p, uintptr_t a)
{
    return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

bool dim_ok(int d)
{
    return d > 0 && d <= kMaxDim && d % 32 == 0;
}

bool experts_ok(int E)
{
    return E > 0 && E <= kMaxExperts;
}

bool tokens_ok(int T, int top_k)
{
    return T >= 0 && T <= kMaxTokens && top_k >= 1 && top_k <= kMaxTopK;
}

bool half_ok(int dtype)
{
    return dtype == FFN_MOE_BF16 || dtype == FFN_MOE_F16;
}

int check_weight(const ffn_moe_weight *w)
{
    if (!w || !w->codes || !w->scales || !w->scale2)
        return FFN_NVFP4_ERR_NULL;
    if (!aligned(w->codes, 16) || !aligned(w->scales, 2) || !aligned(w->scale2, 4))
        return FFN_NVFP4_ERR_ALIGN;
    return FFN_NVFP4_OK;
}

// The buffers of weights [rows, cols] of E experts.
struct WeightSpans {
    Span codes, scales, scale2;
};

WeightSpans spans(const ffn_moe_weight *w, int E, int rows, int cols)
{
    const size_t e = static_cast<size_t>(E) * rows * cols;
    return {{w->codes, e / 2}, {w->scales, e / 16}, {w->scale2, 4 * static_cast<size_t>(E)}};
}

size_t dtype_bytes(int t)
{
    return t == FFN_MOE_F32 ? 4 : 2;
}

int launch_status(hipError_t e)
{
    return e == hipSuccess ? FFN_NVFP4_OK : FFN_NVFP4_ERR_LAUNCH;
}

size_t round256(size_t b)
{
    return (b + 255) & ~static_cast<size_t>(255);
}

ffn::MoeWeightArg weight(const ffn_moe_weight *w)
{
    return ffn::MoeWeightArg{w->codes, w->scales, w->scale2};
}

// The workspace of the whole FFN: the plan, h [R, N] of two bytes an element and
// the experts' outputs y [R, K] in fp32, R = T * top_k.
struct Workspace {
    size_t rows, offsets, places, plan, h, y, total;
};

Workspace layout(int T, int top_k, int E, int K, int N)
{
    const size_t R = static_cast<size_t>(T) * top_k;
    Workspace w;
    w.rows = 0;
    w.offsets = w.rows + round256(4 * R);
    w.places = w.offsets + round256(4 * (static_cast<size_t>(E) + 1));
    w.plan = w.places + round256(4 * R);
    w.h = w.plan + round256(ffn::moe_plan_workspace(static_cast<int>(R), E));
    w.y = w.h + round256(2 * R * N);
    w.total = w.y + round256(4 * R * K);
    return w;
}

int check_ffn(int T, int top_k, int E, int K, int N)
{
    if (!dim_ok(K) || !dim_ok(N) || !experts_ok(E))
        return FFN_NVFP4_ERR_SHAPE;
    return tokens_ok(T, top_k) ? FFN_NVFP4_OK : FFN_NVFP4_ERR_BATCH;
}

}  // namespace

extern "C" {

int ffn_moe_route(const void *logits, int T, int E, int dtype, const float *bias, int top_k, int score,
                  int normalize, float scale, int32_t *ids, float *weights, hipStream_t stream)
{
    if (!experts_ok(E))
        return FFN_NVFP4_ERR_SHAPE;
    if (!tokens_ok(T, top_k) || top_k > E)
        return FFN_NVFP4_ERR_BATCH;
    if ((!half_ok(dtype) && dtype != FFN_MOE_F32) || (score != FFN_MOE_SOFTMAX && score != FFN_MOE_SIGMOID))
        return FFN_NVFP4_ERR_ACT;
    if (!std::isfinite(scale))
        return FFN_NVFP4_ERR_SCALE2;
    if (T == 0)
        return FFN_NVFP4_OK;
    if (!logits || !ids || !weights)
        return FFN_NVFP4_ERR_NULL;
    if (!aligned(logits, 16) || !aligned(bias, 4) || !aligned(ids, 4) || !aligned(weights, 4))
        return FFN_NVFP4_ERR_ALIGN;
    const size_t chosen = 4 * static_cast<size_t>(T) * top_k, experts = static_cast<size_t>(E);
    if (ffn::any_overlap<2, 2>({{ids, chosen}, {weights, chosen}},
                               {{logits, T * experts * dtype_bytes(dtype)}, {bias, 4 * experts}}))
        return FFN_NVFP4_ERR_ALIAS;
    const ffn::MoeRouteArgs a{logits, bias, T, E, top_k, score == FFN_MOE_SIGMOID, normalize != 0, scale, ids, weights};
    return launch_status(ffn::launch_moe_route(a, dtype, stream));
}

size_t ffn_moe_plan_workspace_bytes(int T, int top_k, int E)
{
    if (!experts_ok(E) || !tokens_ok(T, top_k) || T == 0)
        return 0;
    return ffn::moe_plan_workspace(T * top_k, E);
}

int ffn_moe_plan(const int32_t *ids, int T, int top_k, int E, int32_t *rows, int32_t *offsets, int32_t *places,
                 void *workspace, size_t workspace_bytes, hipStream_t stream)
{
    if (!experts_ok(E))
        return FFN_NVFP4_ERR_SHAPE;
    if (!tokens_ok(T, top_k))
        return FFN_NVFP4_ERR_BATCH;
    const int R = T * top_k;
    const size_t need = R > 0 ? ffn::moe_plan_workspace(R, E) : 0;
    if (!offsets || (R > 0 && (!ids || !rows || !places)) || (need > 0 && !workspace))
        return FFN_NVFP4_ERR_NULL;
    if (!aligned(ids, 4) || !aligned(rows, 4) || !aligned(offsets, 4) || !aligned(places, 4) ||
        !aligned(workspace, 16))
        return FFN_NVFP4_ERR_ALIGN;
    if (workspace_bytes < need)
        return FFN_NVFP4_ERR_WORKSPACE;
    const size_t slots = 4 * static_cast<size_t>(R);
    if (ffn::any_overlap<4, 1>(
            {{rows, slots}, {offsets, 4 * (static_cast<size_t>(E) + 1)}, {places, slots}, {workspace, need}},
            {{ids, slots}}))
        return FFN_NVFP4_ERR_ALIAS;
    return launch_status(ffn::launch_moe_plan(ids, R, E, rows, offsets, places, workspace, stream));
}

int ffn_moe_gemm(const void *x, int x_rows, int dtype, const int32_t *rows, int top_k, const int32_t *offsets,
                 int R, int E, int K, int N, const ffn_moe_weight *w, int out_dtype, void *out,
                 hipStream_t stream)
{
    if (const int rc = check_weight(w))
        return rc;
    if (!dim_ok(K) || N <= 0 || N > kMaxChannels || !experts_ok(E))
        return FFN_NVFP4_ERR_SHAPE;
    if (R < 0 || R > kMaxRows || x_rows < 0 || x_rows > kMaxRows || top_k < 1 || top_k > kMaxTopK)
        return FFN_NVFP4_ERR_BATCH;
    if (rows ? R > 0 && x_rows == 0 : x_rows < R || top_k != 1)
        return FFN_NVFP4_ERR_BATCH;
    if (!half_ok(dtype) || (out_dtype != dtype && out_dtype != FFN_MOE_F32))
        return FFN_NVFP4_ERR_ACT;
    if (R == 0)
        return FFN_NVFP4_OK;
    if (!x || !offsets || !out)
        return FFN_NVFP4_ERR_NULL;
    if (!aligned(x, 16) || !aligned(rows, 4) || !aligned(offsets, 4) || !aligned(out, 16))
        return FFN_NVFP4_ERR_ALIGN;
    const WeightSpans ws = spans(w, E, N, K);
    const size_t slots = static_cast<size_t>(R);
    if (ffn::any_overlap<1, 6>({{out, slots * N * dtype_bytes(out_dtype)}},
                               {{x, static_cast<size_t>(x_rows) * K * 2}, {rows, 4 * slots},
                                {offsets, 4 * (static_cast<size_t>(E) + 1)}, ws.codes, ws.scales, ws.scale2}))
        return FFN_NVFP4_ERR_ALIAS;
    const ffn::MoeGemmArgs a{x, rows, offsets, nullptr, weight(w), {}, out, x_rows, top_k, R, E, K, N};
    return launch_status(
        ffn::launch_moe_gemm(a, dtype, out_dtype == FFN_MOE_F32 ? ffn::MOE_F32 : ffn::MOE_SAME, stream));
}

size_t ffn_moe_workspace_bytes(int T, int top_k, int E, int K, int N)
{
    if (T == 0 || check_ffn(T, top_k, E, K, N) != FFN_NVFP4_OK)
        return 0;
    return layout(T, top_k, E, K, N).total;
}

int ffn_moe_forward(const void *x, int T, int K, int N, int E, int top_k, int dtype, const int32_t *ids,
                    const float *weights, const ffn_moe_weight *gate, const ffn_moe_weight *up,
                    const ffn_moe_weight *down, int act, void *workspace, size_t workspace_bytes, void *out,
                    hipStream_t stream)
{
    int rc;
    if ((rc = check_weight(gate)) || (rc = check_weight(up)) || (rc = check_weight(down)) ||
        (rc = check_ffn(T, top_k, E, K, N)))
        return rc;
    if (!half_ok(dtype) || (act != FFN_NVFP4_ACT_SILU && act != FFN_NVFP4_ACT_GELU_TANH))
        return FFN_NVFP4_ERR_ACT;
    if (T == 0)
        return FFN_NVFP4_OK;
    if (!x || !ids || !weights || !workspace || !out)
        return FFN_NVFP4_ERR_NULL;
    if (!aligned(x, 16) || !aligned(ids, 4) || !aligned(weights, 4) || !aligned(workspace, 16) || !aligned(out, 16))
        return FFN_NVFP4_ERR_ALIGN;
    const Workspace w = layout(T, top_k, E, K, N);
    if (workspace_bytes < w.total)
        return FFN_NVFP4_ERR_WORKSPACE;
    // x is read before any of out is written, so out may be x.
    const size_t hidden = static_cast<size_t>(T) * K * 2, chosen = 4 * static_cast<size_t>(T) * top_k;
    const WeightSpans g = spans(gate, E, N, K), u = spans(up, E, N, K), d = spans(down, E, K, N);
    if (ffn::any_overlap<2, 12>({{workspace, w.total}, {out, hidden}},
                                {{out == x ? nullptr : x, hidden}, {ids, chosen}, {weights, chosen}, g.codes, g.scales,
                                 g.scale2, u.codes, u.scales, u.scale2, d.codes, d.scales, d.scale2}))
        return FFN_NVFP4_ERR_ALIAS;
    char *ws = static_cast<char *>(workspace);
    int32_t *rows = reinterpret_cast<int32_t *>(ws + w.rows);
    int32_t *offsets = reinterpret_cast<int32_t *>(ws + w.offsets);
    int32_t *places = reinterpret_cast<int32_t *>(ws + w.places);
    const int R = T * top_k;
    const ffn::MoeOut gated = act == FFN_NVFP4_ACT_SILU ? ffn::MOE_H_SILU : ffn::MOE_H_GELU;
    const bool by_slots = ffn::moe_by_slots(R, E, K, N);
    hipError_t e = by_slots ? hipSuccess
                            : ffn::launch_moe_plan(ids, R, E, rows, offsets, places, ws + w.plan, stream);
    if (e != hipSuccess)
        return FFN_NVFP4_ERR_LAUNCH;
    // h and the experts' outputs are in expert order, or without a plan in that
    // of the slots.
    const int32_t *slots = by_slots ? ids : nullptr;
    const ffn::MoeGemmArgs first{x, rows, offsets, slots, weight(gate), weight(up), ws + w.h, T, top_k, R, E, K, N};
    const ffn::MoeGemmArgs last{ws + w.h, nullptr, offsets, slots, weight(down), {}, ws + w.y, R, 1, R, E, N, K};
    if ((e = ffn::launch_moe_gemm(first, dtype, gated, stream)) != hipSuccess ||
        (e = ffn::launch_moe_gemm(last, dtype, ffn::MOE_F32, stream)) != hipSuccess)
        return FFN_NVFP4_ERR_LAUNCH;
    return launch_status(ffn::launch_moe_combine(reinterpret_cast<const float *>(ws + w.y), places, slots, weights, T,
                                                 top_k, R, E, K, dtype, out, stream));
}

}  // extern "C"
