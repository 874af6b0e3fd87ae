// moe_combine.hip -- the weighted sum of a token's experts' outputs:
// out[t] = sum_j weights[t, j] y[place of (t, j)], in fp32 with j ascending.
//
// It moves top_k rows in and one out for each token and computes almost
// nothing. A thread has four columns (16 bytes of every row) and asks for
// kAtOnce rows before it adds the first. The rows are in fp32: in 16 bits their
// rounding would add to that of h and of the result (error against 64 bits 0.0029
// for 0.0024 in bf16, where the result's own rounding alone is 0.0017). 4096 tokens,
// top 8, 5120 columns: 700 MB in 141 - 144 us, 4.9 TB/s, about the copy rate (5.1).
#include <hip/hip_runtime.h>

#include "moe.h"
#include "nvfp4_device.h"

namespace ffn {
namespace {

constexpr int kThreads = 256;
constexpr int kAtOnce = 8;

template <class T>
__global__ __launch_bounds__(kThreads) void moe_combine_kernel(const float *y, const int32_t *places,
                                                               const int32_t *ids, const float *weights, int top_k,
                                                               int R, int E, int K, T *out)
{
    typedef T vec4 __attribute__((ext_vector_type(4)));
    const int t = blockIdx.x;
    const int c = (blockIdx.y * kThreads + threadIdx.x) * 4;
    if (c >= K)
        return;
    const int slot = t * top_k;
    const int32_t *place = (ids ? ids : places) + slot;
    const int most = ids ? E : R;
    const float *weight = weights + slot;
    f32x4_t sum = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int j0 = 0; j0 < top_k; j0 += kAtOnce) {
        f32x4_t v[kAtOnce];
        float w[kAtOnce];
        bool there[kAtOnce];
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
            const int at = j0 + j < top_k ? place[j0 + j] : -1;
            there[j] = at >= 0 && at < most;
            if (there[j]) {
                w[j] = weight[j0 + j];
                v[j] = *reinterpret_cast<const f32x4_t *>(y + static_cast<size_t>(ids ? slot + j0 + j : at) * K + c);
            }
        }
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j)
            if (there[j])
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    sum[i] += w[j] * v[j][i];
    }
    vec4 o;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        o[i] = static_cast<T>(sum[i]);
    *reinterpret_cast<vec4 *>(out + static_cast<size_t>(t) * K + c) = o;
}

}  // namespace

hipError_t launch_moe_combine(const float *y, const int32_t *places, const int32_t *ids, const float *weights, int T,
                              int top_k, int R, int E, int K, int dtype, void *out, hipStream_t stream)
{
    const dim3 grid(T, (K / 4 + kThreads - 1) / kThreads);
    if (dtype == kMoeBf16)
        hipLaunchKernelGGL((moe_combine_kernel<__bf16>), grid, dim3(kThreads), 0, stream,
                           y, places, ids, weights, top_k, R, E, K, static_cast<__bf16 *>(out));
    else
        hipLaunchKernelGGL((moe_combine_kernel<_Float16>), grid, dim3(kThreads), 0, stream,
                           y, places, ids, weights, top_k, R, E, K, static_cast<_Float16 *>(out));
    return hipGetLastError();
}

}  // namespace ffn
