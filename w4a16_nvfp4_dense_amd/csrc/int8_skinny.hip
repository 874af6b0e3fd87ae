// int8_skinny.hip -- the int8 product for few tokens (M <= 64): the weights
// are read once, straight into the matrix instruction's registers.
//
// Mathematics. out[m, n] = xs[m] s[n] sum_k x[m, k] w[n, k] with exact int32
// sums, so the reduction is split over the waves of a workgroup and added in
// any order: in LDS with integer atomics, whose order cannot change the sum.
//
// What bounds it: the weight stream from HBM (N K bytes); the products cost
// one v_mfma_i32_16x16x64_i8 for each KB of weights and 16 tokens.
//
// Layout. The weight is the instruction's first operand: lane l holds row
// l % 16 of a fragment of 16 channels and the 16 bytes at column
// 16 (l / 16) of a 64-column step; the tokens are the second operand, laid
// out alike, so accumulator v of lane l is channel 4 (l / 16) + v of token
// l % 16 and a lane ends with four consecutive channels of one token. Rows
// past the end repeat the last one (their results are not stored).
#include <hip/hip_runtime.h>

#include <algorithm>

#include "int8.h"
#include "int8_device.h"
#include "kernels.h"

namespace ffn {
namespace {

constexpr int kStep = 64;               // columns of one product
constexpr int kUnitSteps = 4;           // steps of a wave's unit
constexpr int kUnit = kStep * kUnitSteps;

__device__ __forceinline__ i32x4_t load16(const int8_t *p)
{
    return *reinterpret_cast<const i32x4_t *>(p);
}

// NF fragments of 16 weight rows (for two weights: the first half of them
// from w0, the second half the same channels of w1), TG fragments of 16
// tokens.
template <int NF, int TG, int OUT>
__global__ __launch_bounds__(1024) void int8_skinny_kernel(Int8GemmArgs a)
{
    constexpr bool TWO = int8_two_weights(OUT);
    constexpr int NC = TWO ? NF / 2 : NF;  // fragments of channels
    extern __shared__ int32_t red[];       // [NF][TG][4][64]
    const int waves = blockDim.x >> 6, wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int r = lane & 15, q = lane >> 4;
    const int n0 = blockIdx.x * (16 * NC);
    const int K = a.K;

    const int8_t *wp[NF];
#pragma unroll
    for (int f = 0; f < NF; ++f) {
        const int n = min(n0 + 16 * (f % NC) + r, a.N - 1);
        wp[f] = (TWO && f >= NC ? a.w1 : a.w0) + static_cast<size_t>(n) * K + q * 16;
    }
    const int8_t *xp[TG];
#pragma unroll
    for (int t = 0; t < TG; ++t)
        xp[t] = a.x + static_cast<size_t>(min(16 * t + r, a.M - 1)) * K + q * 16;

    for (int i = threadIdx.x; i < NF * TG * 256; i += blockDim.x)
        red[i] = 0;
    __syncthreads();

    i32x4_t acc[NF][TG];
#pragma unroll
    for (int f = 0; f < NF; ++f)
#pragma unroll
        for (int t = 0; t < TG; ++t)
            acc[f][t] = i32x4_t{0, 0, 0, 0};

    const int units = K / kUnit;
    for (int u = wave; u < units; u += waves) {
        i32x4_t w[kUnitSteps][NF], x[kUnitSteps][TG];
#pragma unroll
        for (int s = 0; s < kUnitSteps; ++s) {
#pragma unroll
            for (int f = 0; f < NF; ++f)
                w[s][f] = load16(wp[f] + u * kUnit + s * kStep);
#pragma unroll
            for (int t = 0; t < TG; ++t)
                x[s][t] = load16(xp[t] + u * kUnit + s * kStep);
        }
#pragma unroll
        for (int s = 0; s < kUnitSteps; ++s)
#pragma unroll
            for (int f = 0; f < NF; ++f)
#pragma unroll
                for (int t = 0; t < TG; ++t)
                    acc[f][t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[s][f], x[s][t], acc[f][t], 0, 0, 0);
    }
    // the last columns, fewer than a unit: one step for each wave, pieces of
    // 16 bytes past the end zero in both operands
    const int rest = K - units * kUnit;
    for (int s = wave; s * kStep < rest; s += waves) {
        const int k = units * kUnit + s * kStep;
        const bool in = k + q * 16 < K;
        i32x4_t w[NF], x[TG];
#pragma unroll
        for (int f = 0; f < NF; ++f)
            w[f] = in ? load16(wp[f] + k) : i32x4_t{0, 0, 0, 0};
#pragma unroll
        for (int t = 0; t < TG; ++t)
            x[t] = in ? load16(xp[t] + k) : i32x4_t{0, 0, 0, 0};
#pragma unroll
        for (int f = 0; f < NF; ++f)
#pragma unroll
            for (int t = 0; t < TG; ++t)
                acc[f][t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[f], x[t], acc[f][t], 0, 0, 0);
    }

#pragma unroll
    for (int f = 0; f < NF; ++f)
#pragma unroll
        for (int t = 0; t < TG; ++t)
#pragma unroll
            for (int v = 0; v < 4; ++v)
                atomicAdd(&red[((f * TG + t) * 4 + v) * 64 + lane], acc[f][t][v]);
    __syncthreads();

    for (int i = threadIdx.x; i < NC * TG * 64; i += blockDim.x) {
        const int f = i / (TG * 64), t = i / 64 % TG, l = i & 63;
        const int m = 16 * t + (l & 15), n = n0 + 16 * f + 4 * (l >> 4);
        if (m >= a.M || n >= a.N)
            continue;
        i32x4_t s0, s1{};
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            s0[v] = red[((f * TG + t) * 4 + v) * 64 + l];
            if constexpr (TWO)
                s1[v] = red[(((f + NC) * TG + t) * 4 + v) * 64 + l];
        }
        int8_finish4<OUT>(a, m, n, s0, s1);
    }
}

template <int NF, int TG, int OUT>
hipError_t launch_t(const Int8GemmArgs &a, hipStream_t stream)
{
    constexpr int channels = 16 * (int8_two_weights(OUT) ? NF / 2 : NF);
    const int groups = (a.N + channels - 1) / channels;
    // about 16 waves for each compute unit, none without a unit of its own
    const int want = std::max(1, 16 * device_cu_count() / groups);
    int waves = 4;
    while (waves < 16 && waves < want)
        waves *= 2;
    while (waves > 1 && waves * kUnit > std::max(a.K, kUnit))
        waves /= 2;
    hipLaunchKernelGGL((int8_skinny_kernel<NF, TG, OUT>), dim3(groups), dim3(waves * 64), NF * TG * 256 * 4, stream,
                       a);
    return hipGetLastError();
}

template <int OUT>
hipError_t launch_out(const Int8GemmArgs &a, hipStream_t stream)
{
    constexpr int NF = int8_two_weights(OUT) ? 2 : 1;
    if (a.M <= 16)
        return launch_t<NF, 1, OUT>(a, stream);
    if (a.M <= 32)
        return launch_t<2, 2, OUT>(a, stream);
    return launch_t<2, 4, OUT>(a, stream);
}

}  // namespace

hipError_t launch_int8_skinny(const Int8GemmArgs &a, Int8Out out, hipStream_t stream)
{
    switch (out) {
    case I8_BF16:
        return launch_out<I8_BF16>(a, stream);
    case I8_F16:
        return launch_out<I8_F16>(a, stream);
    case I8_F32:
        return launch_out<I8_F32>(a, stream);
    case I8_H_SILU:
        return launch_out<I8_H_SILU>(a, stream);
    default:
        return launch_out<I8_H_GELU>(a, stream);
    }
}

}  // namespace ffn
