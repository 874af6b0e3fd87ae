// moe_route.hip -- the router's choice: the top_k experts of each token and
// their weights.
//
// One wave for each token, lane l holding experts l, l + 64, ... The keys are
// turned into unsigned integers of the same order (0 for an expert that is not
// available, 1 for NaN), so a choice is an integer maximum over the wave and the
// lowest expert that has it. Without a bias the key is
// the logit: exact, and both scores rise with it. With one it is score + bias
// in 64 bits: in 32, scores a rounding apart would swap places with the order
// of the sum, and a choice of experts is not something that may differ between
// two right programs.
//
// Logits are read once, and a token's choices never leave its wave. Vector
// instructions bound it (top_k maxima one after another): 16384 tokens of 256
// experts, top 8, bf16 11.6 us, where the 9.4 MB are 2, fp32 15.5, with a bias (E
// exponentials of 64 bits for each token) 24 - 26; 333 tokens of 160 experts, fp32
// with a bias 5.3; one token a launch, 2.2, with a bias 3.3.
#include <hip/hip_runtime.h>

#include <cmath>
#include <type_traits>

#include "int8_device.h"
#include "moe.h"
#include "nvfp4_device.h"

namespace ffn {
namespace {

constexpr int kTokens = 4;  // tokens (waves) of a workgroup

template <class V>
__device__ __forceinline__ V wave_sum_all(V v)
{
#pragma unroll
    for (int d = 32; d > 0; d /= 2)
        v += __shfl_xor(v, d);
    return v;
}

__device__ __forceinline__ uint32_t from_lane(uint32_t v, int lane)
{
    return __builtin_amdgcn_readlane(v, lane);
}
__device__ __forceinline__ float from_lane(float v, int lane)
{
    return __uint_as_float(from_lane(__float_as_uint(v), lane));
}

// The largest key of the wave, by lane moves (shuffles through LDS instead: 25 us
// for 17 at 16384 tokens of 256 experts); of 64 bits the upper halves first.
__device__ __forceinline__ uint32_t wave_top(uint32_t v)
{
    return from_lane(wave_max(v), 63);
}
__device__ __forceinline__ unsigned long long wave_top(unsigned long long v)
{
    const uint32_t hi = static_cast<uint32_t>(v >> 32), top = wave_top(hi);
    const uint32_t lo = wave_top(hi == top ? static_cast<uint32_t>(v) : 0u);
    return static_cast<unsigned long long>(top) << 32 | lo;
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

// 1 / (1 + e^-l); where that e^-l may be infinite e^l, the same number.
__device__ __forceinline__ double logistic(float l)
{
    const bool low = l < -700.0f;
    const double z = exp(static_cast<double>(low ? l : -l));
    return low ? z : 1.0 / (1.0 + z);
}

__device__ __forceinline__ float wave_most(float v)
{
#pragma unroll
    for (int d = 32; d > 0; d /= 2)
        v = fmaxf(v, __shfl_xor(v, d));
    return v;
}

// `normalize`: a choice's weight over the sum of the wave's. (In 32 bits the sum has
// the order of its kernel, that of fp32 logits or of 16-bit ones.)
template <class L, class S>
__device__ __forceinline__ S share(S weight, bool normalize)
{
    if (!normalize)
        return weight;
    S sum;
    if constexpr (sizeof(S) == 8 || sizeof(L) == 4)
        sum = wave_sum_all(weight);
    else
        sum = from_lane(segment_sum<64>(weight), 63);
    return sum == 0 ? S(0) : weight / sum;
}

// The weight of lane j's choice (`there`: it has one), of logit l: scale * score,
// `normalize`: over the sum of the wave's choices. S: float where 32 bits do, which
// is not so far below 0 (of a softmax: below the largest logit): there a score is 0
// from -104 on, as a sigmoid from -89, while its product with scale, or its quotient
// by scores as small, is as good as any. So such choices have 64 bits; and where
// all of them are below -40, the scores of a quotient are times e^-(the largest of
// their logits), for 64 bits alone end at -745.

// A sigmoid. (Below -40 it is e^l to 2^-57 of it.) The type's lowest value is what
// masks put in: its score is 0.
template <class L, class S>
__device__ __forceinline__ float logistic_weight(float l, bool there, bool normalize, float scale)
{
    if (sizeof(S) == 4 && !__any(there && l < -80.0f))
        return share<L>(there ? 1.0f / (1.0f + expf(-l)) : 0.0f, normalize) * scale;
    constexpr float lowest = std::is_same<L, float>::value    ? -3.40282347e38f
                             : std::is_same<L, __bf16>::value ? -3.38953139e38f
                                                              : -65504.0f;
    double weight;
    if (normalize && !__any(there && !(l < -40.0f)))
        weight = exp(static_cast<double>(l) - static_cast<double>(wave_most(there ? l : -INFINITY)));
    else
        weight = logistic(l);
    weight = share<L>(there && l != lowest ? weight : 0.0, normalize);
    return static_cast<float>(weight * scale);
}

// A softmax; `most`: the largest logit of all, `sum`: that of e^(l - most). (Only a
// bias chooses experts that are all far below the largest.)
template <class L, class S>
__device__ __forceinline__ float softmax_weight(float l, bool there, float most, S sum, bool normalize, float scale)
{
    if (sizeof(S) == 4 && !__any(there && l - most < -80.0f))
        return share<L>(there ? expf(l - most) / static_cast<float>(sum) : 0.0f, normalize) * scale;
    double weight = static_cast<double>(l) - static_cast<double>(most);
    const bool apart = normalize && !__any(there && !(weight < -40.0));
    if (apart)
        weight = static_cast<double>(l) - static_cast<double>(wave_most(there ? l : -INFINITY));
    weight = exp(weight);
    if (!apart || sum != sum)
        weight /= sum;
    weight = share<L>(there ? weight : 0.0, normalize);
    return static_cast<float>(weight * scale);
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
    Key key[PER];
    float l[PER];
    float most = -INFINITY;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = i * 64 + lane;
        l[i] = e < a.E ? logit<L>(a.logits, static_cast<size_t>(t) * a.E + e) : -INFINITY;
        key[i] = key_of(l[i]);
        most = fmaxf(most, l[i]);
    }
    S sum = 0;  // of a softmax
    S score[PER];
    if (!a.sigmoid) {
        most = wave_most(most);
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            // (an expert that is not there adds nothing, whatever `most` is)
            score[i] = i * 64 + lane < a.E ? exp(static_cast<S>(l[i]) - static_cast<S>(most)) : S(0);
            sum += score[i];
        }
        sum = wave_sum_all(sum);
    }
    if constexpr (sizeof(S) == 8) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = i * 64 + lane;
            const S s = a.sigmoid ? logistic(l[i]) : score[i] / sum;
            key[i] = e < a.E && l[i] != -INFINITY ? key_of(s + static_cast<S>(a.bias[e])) : Key(0);
        }
    }
    int id = -1;  // lane j: the token's j-th expert
    for (int j = 0; j < a.top_k; ++j) {
        Key best = key[0];
#pragma unroll
        for (int i = 1; i < PER; ++i)
            best = max(best, key[i]);
        const Key top = wave_top(best);
        if (top == 0)
            break;
        // The lowest expert with this key: the first i that any lane has it for,
        // and of those lanes the first.
        unsigned long long lanes = 0;
        int at = 0;
#pragma unroll
        for (int i = PER - 1; i >= 0; --i) {
            const unsigned long long have = __ballot(key[i] == top);
            if (have) {
                lanes = have;
                at = i;
            }
        }
        const int first = __ffsll(lanes) - 1;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (i == at && lane == first)
                key[i] = 0;
        if (lane == j)
            id = at * 64 + first;
    }
    // The weights, of the chosen logits alone.
    const bool there = id >= 0;
    float chosen = -INFINITY;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const float v = __shfl(l[i], id & 63);
        chosen = there && id >> 6 == i ? v : chosen;
    }
    const float weight = a.sigmoid ? logistic_weight<L, S>(chosen, there, a.normalize, a.scale)
                                   : softmax_weight<L, S>(chosen, there, most, sum, a.normalize, a.scale);
    if (lane < a.top_k) {
        const size_t o = static_cast<size_t>(t) * a.top_k + lane;
        a.ids[o] = id;
        a.weights[o] = weight;
    }
}

// A logit of 16 bits and its expert in one integer, which orders as the choice
// does: the larger logit, of equal ones the lower expert. 0 for an expert that is
// not available.
template <class L>
__device__ __forceinline__ uint32_t packed_key(L l, int e)
{
    uint32_t u = __builtin_bit_cast(uint16_t, l);
    const float v = static_cast<float>(l);
    if (v == -INFINITY)
        return 0;
    if (u == 0x8000u)
        u = 0;  // (-0 is +0)
    const uint32_t key = v != v ? 1u : u >> 15 ? ~u & 0xFFFFu : u | 0x8000u;
    return key << 16 | (0xFFFFu - e);
}
template <class L>
__device__ __forceinline__ float packed_logit(uint32_t packed)
{
    const uint32_t key = packed >> 16;
    const uint16_t u = key >> 15 ? key & 0x7FFFu : ~key;
    return key == 1 ? __uint_as_float(0x7FC00000u) : static_cast<float>(__builtin_bit_cast(L, u));
}

// Logits of 16 bits and no bias. What is chosen carries its expert and its logit,
// so a choice is one maximum over the wave.
template <class L, int PER>
__global__ __launch_bounds__(kTokens * 64) void moe_route_packed_kernel(const MoeRouteArgs a)
{
    const int lane = threadIdx.x & 63;
    const int t = blockIdx.x * kTokens + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (t >= a.T)
        return;
    const L *logits = static_cast<const L *>(a.logits) + static_cast<size_t>(t) * a.E;
    float l[PER];
    uint32_t key[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = i * 64 + lane;
        const L v = e < a.E ? logits[e] : static_cast<L>(-INFINITY);
        l[i] = static_cast<float>(v);
        key[i] = packed_key(v, e);
    }
    uint32_t mine = 0, first = 0;  // lane j: the token's j-th choice; the best one
    for (int j = 0; j < a.top_k; ++j) {
        uint32_t best = key[0];
#pragma unroll
        for (int i = 1; i < PER; ++i)
            best = max(best, key[i]);
        const uint32_t top = wave_top(best);
        if (top == 0)
            break;
        if (j == 0)
            first = top;
        if (lane == j)
            mine = top;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            key[i] = key[i] == top ? 0u : key[i];
    }
    const float chosen = packed_logit<L>(mine);
    float weight;
    if (a.sigmoid) {
        weight = logistic_weight<L, float>(chosen, mine != 0, a.normalize, a.scale);
    } else {
        const float most = packed_logit<L>(first);
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            sum += i * 64 + lane < a.E ? expf(l[i] - most) : 0.0f;
        sum = from_lane(segment_sum<64>(sum), 63);
        weight = softmax_weight<L, float>(chosen, mine != 0, most, sum, a.normalize, a.scale);
    }
    if (lane < a.top_k) {
        const size_t o = static_cast<size_t>(t) * a.top_k + lane;
        a.ids[o] = mine ? static_cast<int>(0xFFFFu - (mine & 0xFFFFu)) : -1;
        a.weights[o] = weight;
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
hipError_t launch_packed(const MoeRouteArgs &a, hipStream_t stream)
{
    const dim3 grid((a.T + kTokens - 1) / kTokens), block(kTokens * 64);
    if (a.E <= 64)
        hipLaunchKernelGGL((moe_route_packed_kernel<L, 1>), grid, block, 0, stream, a);
    else if (a.E <= 128)
        hipLaunchKernelGGL((moe_route_packed_kernel<L, 2>), grid, block, 0, stream, a);
    else if (a.E <= 256)
        hipLaunchKernelGGL((moe_route_packed_kernel<L, 4>), grid, block, 0, stream, a);
    else
        hipLaunchKernelGGL((moe_route_packed_kernel<L, 16>), grid, block, 0, stream, a);
    return hipGetLastError();
}

template <class L>
hipError_t launch_half(const MoeRouteArgs &a, hipStream_t stream)
{
    return a.bias ? launch_per<L, double>(a, stream) : launch_packed<L>(a, stream);
}

}  // namespace

hipError_t launch_moe_route(const MoeRouteArgs &a, int dtype, hipStream_t stream)
{
    if (dtype == kMoeBf16)
        return launch_half<__bf16>(a, stream);
    if (dtype == kMoeF16)
        return launch_half<_Float16>(a, stream);
    return a.bias ? launch_per<float, double>(a, stream) : launch_per<float, float>(a, stream);
}

}  // namespace ffn
