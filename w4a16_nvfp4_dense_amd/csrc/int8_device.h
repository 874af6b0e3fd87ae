// int8_device.h -- device pieces shared by the int8 kernels: element types,
// the rule that turns a row's largest magnitude into a scale, and the
// epilogue that turns exact int32 sums into outputs.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "int8.h"
#include "nvfp4_device.h"

namespace ffn {

typedef int i32x4_t __attribute__((ext_vector_type(4)));

// Magnitude bits of an fp32: for finite values their unsigned order is the
// order of magnitudes, an infinity lies above them and a NaN above that, so
// an integer maximum keeps both (an fp32 maximum drops NaN).
__device__ __forceinline__ uint32_t magnitude_bits(float v)
{
    return __float_as_uint(v) & 0x7FFFFFFFu;
}

// A row's scale and the factor of its codes, from the largest magnitude's
// bits: s = amax / 127 and 1 / s, each correctly rounded; 0 and 0 where s
// would be subnormal (1 / s could overflow); NaN and 0 for a row with an
// infinity or a NaN.
__device__ __forceinline__ void int8_scale(uint32_t amax_bits, float &scale, float &inv)
{
    const float s = __uint_as_float(amax_bits) / 127.0f;
    const bool finite = amax_bits < 0x7F800000u;
    const bool live = finite && s >= 1.17549435e-38f;
    scale = live ? s : (finite ? 0.0f : __uint_as_float(0x7FC00000u));
    inv = live ? 1.0f / s : 0.0f;
}

// Four codes rint(v * inv), code i in byte i. Adding 1.5 * 2^23 to a value of
// magnitude at most 2^22 rounds it to the nearest integer, ties to even, and
// leaves the integer's two's complement in the low bits (no contraction: the
// product is rounded first). A row without a factor (inv = 0: zeros, or an
// infinity or NaN in it) has codes 0 whatever its values are.
__device__ __forceinline__ uint32_t int8_pack4(float a, float b, float c, float d, float inv)
{
#pragma clang fp contract(off)
    constexpr float magic = 12582912.0f;
    const uint32_t ia = __float_as_uint(a * inv + magic), ib = __float_as_uint(b * inv + magic);
    const uint32_t ic = __float_as_uint(c * inv + magic), id = __float_as_uint(d * inv + magic);
    const uint32_t lo = __builtin_amdgcn_perm(ib, ia, 0x0C0C0400u);  // bytes: ia.0, ib.0, 0, 0
    const uint32_t hi = __builtin_amdgcn_perm(id, ic, 0x04000C0Cu);  // bytes: 0, 0, ic.0, id.0
    return inv != 0.0f ? lo | hi : 0u;
}

// ------------------------------------------------------------------ epilogue
// The value of one output from its exact sum. Written without contraction, so
// every kernel gives the same bits.
__device__ __forceinline__ float int8_scaled(int sum, float xs, float ws)
{
#pragma clang fp contract(off)
    return static_cast<float>(sum) * xs * ws;
}

__device__ __forceinline__ float int8_biased(float v, float b)
{
#pragma clang fp contract(off)
    return v + b;
}

// act(g) * u in fp32, both gates as g / (1 + e^z): z = -g for SiLU and
// z = -2 sqrt(2/pi) (g + 0.044715 g^3) for GELU-tanh.
template <int OUT>
__device__ __forceinline__ float int8_gated(float g, float u)
{
#pragma clang fp contract(off)
    float z;
    if constexpr (OUT == I8_H_SILU)
        z = -g;
    else
        z = -1.5957691216057308f * (g + 0.044715f * g * g * g);
    return g * __builtin_amdgcn_rcpf(1.0f + __expf(z)) * u;
}

// Four results of channels n .. n + 3 of token m (those below N), in the
// output's type: one vector store where the row length keeps it aligned.
template <int OUT>
__device__ __forceinline__ void int8_store4(const Int8GemmArgs &a, int m, int n, const float (&v)[4])
{
    const size_t at = static_cast<size_t>(m) * a.N + n;
    const bool whole = (a.N & 3) == 0;  // n is a multiple of 4
    if constexpr (OUT == I8_BF16) {
        uint16_t *o = static_cast<uint16_t *>(a.out) + at;
        if (whole) {
            *reinterpret_cast<uint2 *>(o) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (n + i < a.N)
                    o[i] = to_bf16_bits(v[i]);
        }
    } else if constexpr (OUT == I8_F16) {
        _Float16 *o = static_cast<_Float16 *>(a.out) + at;
        if (whole) {
            typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
            *reinterpret_cast<f16x4 *>(o) = f16x4{static_cast<_Float16>(v[0]), static_cast<_Float16>(v[1]),
                                                  static_cast<_Float16>(v[2]), static_cast<_Float16>(v[3])};
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (n + i < a.N)
                    o[i] = static_cast<_Float16>(v[i]);
        }
    } else {
        float *o = static_cast<float *>(a.out) + at;
        if (whole) {
            *reinterpret_cast<f32x4_t *>(o) = f32x4_t{v[0], v[1], v[2], v[3]};
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (n + i < a.N)
                    o[i] = v[i];
        }
    }
}

// Sums of channels n .. n + 3 (n a multiple of 4, n < N) of token m -> output.
// s0 and s1: the sums of the first and second weight.
template <int OUT>
__device__ __forceinline__ void int8_finish4(const Int8GemmArgs &a, int m, int n, const i32x4_t &s0,
                                             const i32x4_t &s1)
{
    const float xs = a.xs[m];
    float v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int c = min(n + i, a.N - 1);
        const float y = int8_scaled(s0[i], xs, a.s0[c]);
        if constexpr (int8_two_weights(OUT))
            v[i] = int8_gated<OUT>(y, int8_scaled(s1[i], xs, a.s1[c]));
        else
            v[i] = a.bias ? int8_biased(y, a.bias[c]) : y;
    }
    int8_store4<OUT>(a, m, n, v);
}

}  // namespace ffn
