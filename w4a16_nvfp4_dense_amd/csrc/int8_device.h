// int8_device.h -- device pieces shared by the int8 kernels: element types,
// the rule that turns a row's largest magnitude into a scale, and the
// epilogue that turns exact int32 sums into outputs.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

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

// The maximum over a wave's lanes, valid in the last one (lane 63), by the
// lane moves of segment_sum (masked lanes give 0, below everything).
__device__ __forceinline__ uint32_t wave_max(uint32_t v)
{
    const auto other = [&](auto move) __attribute__((always_inline)) {
        v = max(v, __float_as_uint(move(__uint_as_float(v))));
    };
    other([](float x) { return dpp_move<0xB1>(x); });
    other([](float x) { return dpp_move<0x4E>(x); });
    other([](float x) { return dpp_move<0x141>(x); });
    other([](float x) { return dpp_move<0x140>(x); });
    other([](float x) { return dpp_move<0x142, 0xA>(x); });
    other([](float x) { return dpp_move<0x143, 0xC>(x); });
    return v;
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
// z = -2 sqrt(2/pi) (g + 0.044715 g^3) for GELU-tanh. (gate_act's formulas, again
// because that leaves it to the compiler where a product and a sum are fused:
// here every tile shape has to round alike.)
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

// C results of channels n .. n + C - 1 of token m (those below N), n a
// multiple of C, in the output's type: one store where the row length keeps it
// aligned.
template <int OUT, int C>
__device__ __forceinline__ void int8_store(const Int8GemmArgs &a, int m, int n, const float (&v)[C])
{
    const size_t at = static_cast<size_t>(m) * a.N + n;
    const bool whole = a.N % C == 0;
    if constexpr (OUT == I8_BF16) {
        uint16_t *o = static_cast<uint16_t *>(a.out) + at;
        if (C > 1 && whole) {
            typedef uint32_t pairs __attribute__((ext_vector_type(C > 1 ? C / 2 : 1)));
            pairs p;
#pragma unroll
            for (int i = 0; i < C / 2; ++i)
                p[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
            *reinterpret_cast<pairs *>(o) = p;
        } else {
#pragma unroll
            for (int i = 0; i < C; ++i)
                if (n + i < a.N)
                    o[i] = to_bf16_bits(v[i]);
        }
    } else {
        typedef typename std::conditional<OUT == I8_F16, _Float16, float>::type T;
        typedef T vec __attribute__((ext_vector_type(C)));
        T *o = static_cast<T *>(a.out) + at;
        if (whole) {
            vec p;
#pragma unroll
            for (int i = 0; i < C; ++i)
                p[i] = static_cast<T>(v[i]);
            *reinterpret_cast<vec *>(o) = p;
        } else {
#pragma unroll
            for (int i = 0; i < C; ++i)
                if (n + i < a.N)
                    o[i] = static_cast<T>(v[i]);
        }
    }
}

}  // namespace ffn
