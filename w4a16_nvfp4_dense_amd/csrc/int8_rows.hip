// int8_rows.hip -- rows of real values to int8 codes with one scale for each
// row: after a root-mean-square norm with the residual's addition (what feeds
// the FFN), as they are (activations without a norm, weights at load), or
// from an NVFP4 weight.
//
// Mathematics. t = x + r in fp32; y = t / sqrt(mean t^2 + eps) * (off + w), of
// a row scaled by a power of two where the squares leave fp32's range;
// s = max |y| / 127; q = rint(y * (1 / s)). The row's sum of squares and its
// maximum need the whole row before its first output, so a row is held in
// registers between them: one pass over memory, each element read once and
// each output written once.
//
// Layout. A thread holds C chunks of 8 consecutive elements (16 bytes of a
// 16-bit type), chunk c * threads + t, so a wave reads 1 KB contiguously. One
// workgroup for each row: rows are independent, and from about a thousand of
// them on that fills the card.
//
// What bounds it, measured on one MI355X: memory for many rows, and for few the
// launch and the two reductions' latency.
//   norm with residual, bf16, 8192 x 5120   52.4 us, 294 MB: 5.6 TB/s (47.4
//                                           where x was written just before)
//   the same, 1 x 5120                       3.6 us
//   norm with residual, fp32, 333 x 5376     7.9 us, 23 MB
//   bf16 rows, 17408 x 5120                 45.0 us, 267 MB: 6.0 TB/s
//   fp16 rows, 3 x 17408                     3.2 us
//   fp32 rows, 2048 x 17408, just written   27.1 us, 178 MB: 6.6 TB/s
//   NVFP4 rows, 17408 x 5120                44.6 us, 139 MB, two thirds of them
//                                           written: 3.1 TB/s
#include <hip/hip_runtime.h>

#include <algorithm>

#include "int8.h"
#include "int8_device.h"

namespace ffn {
namespace {

constexpr int kVec = 8;
constexpr int kRowThreads = 1024;  // the most threads of a row

enum Source { SRC_BF16 = 0, SRC_F16 = 1, SRC_F32 = 2, SRC_NVFP4 = 3 };

template <int T>
__device__ __forceinline__ void load8(const void *p, size_t at, float (&v)[kVec])
{
    if constexpr (T == SRC_F32) {
        const f32x4_t a = *reinterpret_cast<const f32x4_t *>(static_cast<const float *>(p) + at);
        const f32x4_t b = *reinterpret_cast<const f32x4_t *>(static_cast<const float *>(p) + at + 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = a[i];
            v[4 + i] = b[i];
        }
    } else {
        const u32x4_t a = *reinterpret_cast<const u32x4_t *>(static_cast<const uint16_t *>(p) + at);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (T == SRC_BF16) {
                v[2 * i] = __uint_as_float(a[i] << 16);
                v[2 * i + 1] = __uint_as_float(a[i] & 0xFFFF0000u);
            } else {
                typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
                const uint32_t pair = a[i];  // (a bit cast of a vector's element would take element 0)
                const f16x2 h = __builtin_bit_cast(f16x2, pair);
                v[2 * i] = static_cast<float>(h[0]);
                v[2 * i + 1] = static_cast<float>(h[1]);
            }
        }
    }
}

template <int T>
__device__ __forceinline__ void store8(void *p, size_t at, const float (&v)[kVec])
{
    if constexpr (T == SRC_F32) {
        float *o = static_cast<float *>(p) + at;
        *reinterpret_cast<f32x4_t *>(o) = f32x4_t{v[0], v[1], v[2], v[3]};
        *reinterpret_cast<f32x4_t *>(o + 4) = f32x4_t{v[4], v[5], v[6], v[7]};
    } else if constexpr (T == SRC_BF16) {
        *reinterpret_cast<u32x4_t *>(static_cast<uint16_t *>(p) + at) =
            u32x4_t{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                    pack_bf16x2(v[6], v[7])};
    } else {
        typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
        f16x8 h;
#pragma unroll
        for (int i = 0; i < kVec; ++i)
            h[i] = static_cast<_Float16>(v[i]);
        *reinterpret_cast<f16x8 *>(static_cast<_Float16 *>(p) + at) = h;
    }
}

// The norm's mean square in fp32. From kLeastSquare on, squares too small for
// fp32 (below 2^-126) are under 2^-30 of the mean. Where it is smaller, or not
// finite, the row is scaled first, by the power of two that brings its largest
// magnitude, or eps's root if that is larger, to [1, 4): the squares then sum to
// between 1 and 16 cols, and t factor / sqrt(mean (t factor)^2 + eps factor^2)
// is the same norm. (2^126 at most: a row of subnormals stays below 1, its
// squares above 2^-46.)
constexpr float kLeastSquare = 0x1p-96f;

__device__ __forceinline__ float norm_factor(float most)
{
    const int exponent = static_cast<int>(__float_as_uint(most) >> 23);  // of a finite value: 0 .. 254
    return __uint_as_float(static_cast<uint32_t>(254 - min(max(exponent, 1), 253)) << 23);
}

struct Rows {
    Int8RowsArgs a;
    const uint8_t *nv_codes, *nv_scales;
    float scale2;
};

// One workgroup for each row; C chunks of 8 elements per thread.
template <int T, int WT, int C, bool NORM>
__global__ __launch_bounds__(kRowThreads) void int8_rows_kernel(Rows p)
{
    __shared__ float sh_sum[kRowThreads / 64];
    __shared__ uint32_t sh_max[kRowThreads / 64];
    const int row = blockIdx.x, t = threadIdx.x, threads = blockDim.x;
    const int waves = threads >> 6, wave = t >> 6, lane = t & 63;
    const int chunks = p.a.cols / kVec;
    const size_t base = static_cast<size_t>(row) * p.a.cols;

    // the norm's weights are loaded with the row where registers allow it, so
    // that the outputs do not wait for them
    constexpr bool AHEAD = NORM && C <= 4;
    float v[C][kVec], nw[AHEAD ? C : 1][kVec];
    float sum = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int ch = c * threads + t;
#pragma unroll
        for (int i = 0; i < kVec; ++i)
            v[c][i] = 0.0f;
        if (ch < chunks) {
            const size_t at = base + static_cast<size_t>(ch) * kVec;
            if constexpr (T == SRC_NVFP4) {
                const uint32_t d = reinterpret_cast<const uint32_t *>(p.nv_codes)[at / kVec];
                const float s = e4m3_to_f32<0>(p.nv_scales[at / 16]);
                const f32x2_t p0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(d, 1.0f, 0);
                const f32x2_t p1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(d, 1.0f, 1);
                const f32x2_t p2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(d, 1.0f, 2);
                const f32x2_t p3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(d, 1.0f, 3);
                const float e[kVec] = {p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
#pragma unroll
                for (int i = 0; i < kVec; ++i)
                    v[c][i] = e[i] * s;  // exact
            } else {
                load8<T>(p.a.x, at, v[c]);
            }
            if constexpr (AHEAD)
                load8<WT>(p.a.weight, static_cast<size_t>(ch) * kVec, nw[c]);
            if constexpr (NORM) {
                if (p.a.residual) {
                    float r[kVec];
                    load8<T>(p.a.residual, at, r);
#pragma unroll
                    for (int i = 0; i < kVec; ++i)
                        v[c][i] += r[i];
                }
#pragma unroll
                for (int i = 0; i < kVec; ++i)
                    sum += v[c][i] * v[c][i];
            }
        }
    }
    if constexpr (NORM) {
        sum = segment_sum<64>(sum);
        if (lane == 63)
            sh_sum[wave] = sum;
        __syncthreads();
        sum = 0.0f;
        for (int w = 0; w < waves; ++w)
            sum += sh_sum[w];
        const float cols = static_cast<float>(p.a.cols);
        float square = sum / cols + p.a.eps, factor = 1.0f;
        if (!(square >= kLeastSquare && square < __builtin_inff())) {
            // (the same for every thread of the row)
            uint32_t most = 0;
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int i = 0; i < kVec; ++i)
                    most = max(most, magnitude_bits(v[c][i]));
            most = wave_max(most);
            if (lane == 63)
                sh_max[wave] = most;
            __syncthreads();
            for (int w = 0; w < waves; ++w)
                most = w == 0 ? sh_max[0] : max(most, sh_max[w]);
            if (most > 0 && most < 0x7F800000u) {
                factor = norm_factor(fmaxf(__uint_as_float(most), sqrtf(p.a.eps)));
                sum = 0.0f;
#pragma unroll
                for (int c = 0; c < C; ++c)
#pragma unroll
                    for (int i = 0; i < kVec; ++i)
                        sum += (v[c][i] * factor) * (v[c][i] * factor);
                sum = segment_sum<64>(sum);
                if (lane == 63)
                    sh_sum[wave] = sum;
                __syncthreads();
                sum = 0.0f;
                for (int w = 0; w < waves; ++w)
                    sum += sh_sum[w];
                square = sum / cols + p.a.eps * factor * factor;
            }
            __syncthreads();  // sh_max is used again below
        }
        const float rstd = 1.0f / sqrtf(square);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int ch = c * threads + t;
            if (ch < chunks) {
                const size_t at = base + static_cast<size_t>(ch) * kVec;
                if (p.a.sum_out)
                    store8<T>(p.a.sum_out, at, v[c]);
                float w[kVec];
                if constexpr (AHEAD)
#pragma unroll
                    for (int i = 0; i < kVec; ++i)
                        w[i] = nw[c][i];
                else
                    load8<WT>(p.a.weight, static_cast<size_t>(ch) * kVec, w);
#pragma unroll
                for (int i = 0; i < kVec; ++i)
                    v[c][i] = v[c][i] * factor * rstd * (p.a.weight_offset + w[i]);
                if (p.a.y_out)
                    store8<T>(p.a.y_out, at, v[c]);
            }
        }
    }
    uint32_t m = 0;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int i = 0; i < kVec; ++i)
            m = max(m, magnitude_bits(v[c][i]));
    m = wave_max(m);
    if (lane == 63)
        sh_max[wave] = m;
    __syncthreads();
    m = 0;
    for (int w = 0; w < waves; ++w)
        m = max(m, sh_max[w]);
    float scale, inv;
    int8_scale(m, scale, inv);
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int ch = c * threads + t;
        if (ch < chunks)
            reinterpret_cast<uint2 *>(p.a.codes)[(base + static_cast<size_t>(ch) * kVec) / kVec] =
                make_uint2(int8_pack4(v[c][0], v[c][1], v[c][2], v[c][3], inv),
                           int8_pack4(v[c][4], v[c][5], v[c][6], v[c][7], inv));
    }
    if (t == 0)
        p.a.scales[row] = T == SRC_NVFP4 ? scale * p.scale2 : scale;
}

template <int T, int WT, bool NORM>
hipError_t launch_rows(const Rows &p, hipStream_t stream)
{
    const int chunks = p.a.cols / kVec;
    // the fewest chunks per thread that 1024 threads cover the row with, at
    // least 2 (32 bytes in flight per tensor: 8192 rows of 5120 with a norm,
    // x just written, 47.4 us; 57.3 with one, which is 0.1 faster for a single
    // row)
    int c = 2;
    while (c * kRowThreads < chunks)
        c *= 2;
    const int threads = std::max(64, (((chunks + c - 1) / c) + 63) / 64 * 64);
    const dim3 grid(p.a.rows), block(threads);
    if (c == 2)
        hipLaunchKernelGGL((int8_rows_kernel<T, WT, 2, NORM>), grid, block, 0, stream, p);
    else if (c == 4)
        hipLaunchKernelGGL((int8_rows_kernel<T, WT, 4, NORM>), grid, block, 0, stream, p);
    else
        hipLaunchKernelGGL((int8_rows_kernel<T, WT, 8, NORM>), grid, block, 0, stream, p);
    return hipGetLastError();
}

template <int T>
hipError_t launch_norm(const Rows &p, int weight_dtype, hipStream_t stream)
{
    switch (weight_dtype) {
    case SRC_BF16:
        return launch_rows<T, SRC_BF16, true>(p, stream);
    case SRC_F16:
        return launch_rows<T, SRC_F16, true>(p, stream);
    default:
        return launch_rows<T, SRC_F32, true>(p, stream);
    }
}

}  // namespace

hipError_t launch_int8_rmsnorm(const Int8RowsArgs &a, int dtype, int weight_dtype, hipStream_t stream)
{
    const Rows p{a, nullptr, nullptr, 1.0f};
    switch (dtype) {
    case SRC_BF16:
        return launch_norm<SRC_BF16>(p, weight_dtype, stream);
    case SRC_F16:
        return launch_norm<SRC_F16>(p, weight_dtype, stream);
    default:
        return launch_norm<SRC_F32>(p, weight_dtype, stream);
    }
}

hipError_t launch_int8_quantize(const Int8RowsArgs &a, int dtype, hipStream_t stream)
{
    const Rows p{a, nullptr, nullptr, 1.0f};
    switch (dtype) {
    case SRC_BF16:
        return launch_rows<SRC_BF16, SRC_BF16, false>(p, stream);
    case SRC_F16:
        return launch_rows<SRC_F16, SRC_BF16, false>(p, stream);
    default:
        return launch_rows<SRC_F32, SRC_BF16, false>(p, stream);
    }
}

hipError_t launch_int8_requant(const uint8_t *codes, const uint8_t *scales, float scale2, int rows, int cols,
                               int8_t *q, float *qs, hipStream_t stream)
{
    Rows p{};
    p.a.rows = rows;
    p.a.cols = cols;
    p.a.codes = q;
    p.a.scales = qs;
    p.nv_codes = codes;
    p.nv_scales = scales;
    p.scale2 = scale2;
    return launch_rows<SRC_NVFP4, SRC_BF16, false>(p, stream);
}

}  // namespace ffn
