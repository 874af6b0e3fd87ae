// moe_device.h -- device pieces shared by the grouped products: the 16-bit
// types' operations, NVFP4 weights as operands of the matrix cores, and an
// expert's rows.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "moe.h"
#include "nvfp4_device.h"

namespace ffn {

typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));

// What pieces past the last column are loaded from.
__device__ const u32x4_t kZeros = {0, 0, 0, 0};

// The element type's operations.
template <class T>
struct Half;
template <>
struct Half<__bf16> {
    typedef bf16x8_t vec8;
    // Eight codes times a block scale: exact, so the upper halves of the fp32
    // products are the bf16 values.
    static __device__ __forceinline__ vec8 weights(uint32_t codes, float scale)
    {
        const f32x2_t p0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 0);
        const f32x2_t p1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 1);
        const f32x2_t p2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 2);
        const f32x2_t p3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 3);
        const u32x4_t w = {upper(p0, scale), upper(p1, scale), upper(p2, scale), upper(p3, scale)};
        return __builtin_bit_cast(vec8, w);
    }
    static __device__ __forceinline__ f32x16_t mfma(const vec8 &a, const vec8 &b, const f32x16_t &c)
    {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
    }
    static __device__ __forceinline__ f32x4_t mfma(const vec8 &a, const vec8 &b, const f32x4_t &c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }

private:
    static __device__ __forceinline__ uint32_t upper(const f32x2_t &p, float scale)
    {
        return __builtin_amdgcn_perm(__float_as_uint(p[1] * scale), __float_as_uint(p[0] * scale), 0x07060302u);
    }
};
template <>
struct Half<_Float16> {
    typedef f16x8_t vec8;
    static __device__ __forceinline__ vec8 weights(uint32_t codes, float scale)
    {
        const _Float16 s = static_cast<_Float16>(scale);
        const f16x2_t s2 = {s, s};
        const f16x2_t p0 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 1.0f, 0) * s2;
        const f16x2_t p1 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 1.0f, 1) * s2;
        const f16x2_t p2 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 1.0f, 2) * s2;
        const f16x2_t p3 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 1.0f, 3) * s2;
        return vec8{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
    }
    static __device__ __forceinline__ f32x16_t mfma(const vec8 &a, const vec8 &b, const f32x16_t &c)
    {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
    }
    static __device__ __forceinline__ f32x4_t mfma(const vec8 &a, const vec8 &b, const f32x4_t &c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    }
};

// A load from global memory of an address that was chosen between two. (Without
// the address space the compiler takes it for any memory's, and waits for all
// loads in flight where one such is among them.)
template <class V>
__device__ __forceinline__ V load_global(uintptr_t at)
{
    return *(const __attribute__((address_space(1))) V *)at;
}

// Lanes 32 .. 63 of lo and lanes 0 .. 31 of hi change places.
__device__ __forceinline__ void swap_halves(uint32_t &lo, uint32_t &hi)
{
    const auto both = __builtin_amdgcn_permlane32_swap(lo, hi, false, false);
    lo = both[0];
    hi = both[1];
}

// A byte offset past any buffer.
constexpr uint32_t kPast = 0xE0000000u;

// A buffer whose base and size are the same in all lanes, which the compiler
// does not always see.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t uniform_buffer(const void *base, int bytes)
{
    const uint64_t at = reinterpret_cast<uintptr_t>(base);
    const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(at));
    const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(at >> 32));
    return raw_buffer(reinterpret_cast<const void *>(static_cast<uint64_t>(hi) << 32 | lo),
                      __builtin_amdgcn_readfirstlane(bytes));
}

// An expert's rows, whatever the offsets hold.
__device__ __forceinline__ void rows_of(const MoeGemmArgs &a, int e, int &begin, int &end)
{
    begin = min(max(a.offsets[e], 0), a.R);
    end = min(max(a.offsets[e + 1], begin), a.R);
}

// The value of a result: scale2 times the sum, or of two weights the gated
// product.
template <int OUT>
__device__ __forceinline__ float moe_value(float sum0, float sum1, float scale0, float scale1)
{
    if constexpr (moe_two_weights(OUT)) {
        constexpr int A = OUT == MOE_H_SILU ? ACT_SILU : ACT_GELU_TANH;
        return gate_act<A>(sum0 * scale0) * (sum1 * scale1);
    } else {
        return sum0 * scale0;
    }
}

template <class T, int OUT>
__device__ __forceinline__ void moe_store(void *out, size_t at, float v)
{
    if constexpr (OUT == MOE_F32)
        static_cast<float *>(out)[at] = v;
    else
        static_cast<T *>(out)[at] = static_cast<T>(v);
}

}  // namespace ffn
