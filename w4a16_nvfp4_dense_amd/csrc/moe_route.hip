// moe_route.hip -- the router's choice: the top_k experts of each token and
// their weights.
//
// One wave for each token, lane l holding experts l, l + 64, ... The keys are
// turned into unsigned integers of the same order (0 for an expert that is not
// available, 1 for NaN), so a choice is an integer maximum over the wave and,
// among the lanes that hold it, the lowest expert. Without a bias the key is
// the logit: exact, and both scores rise with it. With one it is score + bias
// in 64 bits: in 32, scores a rounding apart would swap places with the order
// of the sum, and a choice of experts is not something that may differ between
// two right programs.
#include <hip/hip_runtime.h>

#include <cmath>

#include "moe.h"
#include "nvfp4_device.h"

namespace ffn {
namespace {

constexpr int kTokens = 4;  // tokens (waves) of a workgroup
constexpr int kMoeNoExpert = 1 << 20;

template <class V>
__device__ __forceinline__ V wave_sum_all(V v)
{
#pragma unroll
    for (int d = 32; d > 0; d /= 2)
        v += __shfl_xor(v, d);
    return v;
}

template <class V>
__device__ __forceinline__ V wave_max_all(V v)
{
#pragma unroll
    for (int d = 32; d > 0; d /= 2) {
        const V o = __shfl_xor(v, d);
        v = o > v ? o : v;
    }
    return v;
}

// An integer that orders like v: 0 for -infinity, 1 for NaN (below every
// number), -0 as +0.
__device__ __forceinline__ uint32_t key_of(float v)
{
    const uint32_t u = __float_as_uint(v + 0.0f);
    if (v != v)
        return 1u;
    if (v == -INFINITY)
        return 0u;
    return u >> 31 ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ unsigned long long key_of(double v)
{
    const unsigned long long u = __double_as_longlong(v + 0.0);
    if (v != v)
        return 1ull;
    if (v == -INFINITY)
        return 0ull;
    return u >> 63 ? ~u : u | 0x8000000000000000ull;
}

template <class L>
__device__ __forceinline__ float logit(const void *p, size_t i)
{
    return static_cast<float>(static_cast<const L *>(p)[i]);
}

// PER: experts of a lane. S: the type of scores and keys (double with a bias).
template <class L, class S, int PER>
__global__ __launch_bounds__(kTokens * 64) void moe_route_kernel(const MoeRouteArgs a)
{
    typedef decltype(key_of(S())) Key;
    const int lane = threadIdx.x & 63;
    const int t = blockIdx.x * kTokens + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (t >= a.T)
        return;
    S score[PER];
    Key key[PER];
    float l[PER];
    float most = -INFINITY;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = i * 64 + lane;
        l[i] = e < a.E ? logit<L>(a.logits, static_cast<size_t>(t) * a.E + e) : -INFINITY;
        most = fmaxf(most, l[i]);
    }
    if (a.sigmoid) {
#pragma unroll
        for (int i = 0; i < PER; ++i)
            score[i] = S(1) / (S(1) + exp(-static_cast<S>(l[i])));
    } else {
        most = wave_max_all(most);
        S sum = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            // (an expert that is not there adds nothing, whatever `most` is)
            score[i] = i * 64 + lane < a.E ? exp(static_cast<S>(l[i]) - static_cast<S>(most)) : S(0);
            sum += score[i];
        }
        sum = wave_sum_all(sum);
#pragma unroll
        for (int i = 0; i < PER; ++i)
            score[i] /= sum;
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = i * 64 + lane;
        key[i] = key_of(l[i]);
        if constexpr (sizeof(S) == 8)
            key[i] = e < a.E && l[i] != -INFINITY ? key_of(score[i] + static_cast<S>(a.bias[e])) : Key(0);
    }
    int id = -1;    // lane j: the token's j-th expert
    S weight = 0;   // and its score
    for (int j = 0; j < a.top_k; ++j) {
        Key best = key[0];
        int at = 0;
#pragma unroll
        for (int i = 1; i < PER; ++i)
            if (key[i] > best) {
                best = key[i];
                at = i;
            }
        const Key top = wave_max_all(best);
        if (top == 0)
            break;
        // The lowest expert with this key: a lane's own are ascending.
        int e = best == top ? at * 64 + lane : kMoeNoExpert;
#pragma unroll
        for (int d = 32; d > 0; d /= 2)
            e = min(e, __shfl_xor(e, d));
        S s = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (e == i * 64 + lane) {
                s = score[i];
                key[i] = 0;
            }
        s = __shfl(s, e & 63);
        if (lane == j) {
            id = e;
            weight = s;
        }
    }
    if (a.normalize) {
        const S sum = wave_sum_all(weight);
        weight = sum == 0 ? S(0) : weight / sum;
    }
    if (lane < a.top_k) {
        const size_t o = static_cast<size_t>(t) * a.top_k + lane;
        a.ids[o] = id;
        a.weights[o] = static_cast<float>(weight * static_cast<S>(a.scale));
    }
}

template <class L, class S>
hipError_t launch_per(const MoeRouteArgs &a, hipStream_t stream)
{
    const dim3 grid((a.T + kTokens - 1) / kTokens), block(kTokens * 64);
    if (a.E <= 64)
        hipLaunchKernelGGL((moe_route_kernel<L, S, 1>), grid, block, 0, stream, a);
    else if (a.E <= 128)
        hipLaunchKernelGGL((moe_route_kernel<L, S, 2>), grid, block, 0, stream, a);
    else if (a.E <= 256)
        hipLaunchKernelGGL((moe_route_kernel<L, S, 4>), grid, block, 0, stream, a);
    else
        hipLaunchKernelGGL((moe_route_kernel<L, S, 16>), grid, block, 0, stream, a);
    return hipGetLastError();
}

template <class L>
hipError_t launch_score(const MoeRouteArgs &a, hipStream_t stream)
{
    return a.bias ? launch_per<L, double>(a, stream) : launch_per<L, float>(a, stream);
}

}  // namespace

hipError_t launch_moe_route(const MoeRouteArgs &a, int dtype, hipStream_t stream)
{
    if (dtype == kMoeBf16)
        return launch_score<__bf16>(a, stream);
    if (dtype == kMoeF16)
        return launch_score<_Float16>(a, stream);
    return launch_score<float>(a, stream);
}

}  // namespace ffn
