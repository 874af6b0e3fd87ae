// int8_tile.hip -- the int8 product for many tokens: tiles of tokens and
// channels, both operands staged through LDS.
//
// Mathematics. As int8_skinny.hip; here the reduction of a tile stays in one
// workgroup's accumulators.
//
// What bounds it: the matrix instructions (2 M N K operations), and for
// middling M the weight stream.
//
// Layout. A stage holds 128 columns of BM token rows and BN weight rows, 128
// bytes a row, written by direct global -> LDS loads of 16 bytes a lane (eight
// rows for each wave instruction). Piece s of row i holds columns
// 16 (s ^ (i / 2 % 8)), chosen by the address each lane loads from, so the 16
// lanes that read one column piece of 16 consecutive rows touch all 64 banks
// once. STAGES stages form a ring: stage k + STAGES - 1 is loaded while stage
// k is multiplied, one barrier for each stage.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "int8.h"
#include "int8_device.h"
#include "kernels.h"

namespace ffn {
namespace {

constexpr int kBk = 128;  // columns (bytes of a row) of a stage

// Swizzle of row i's pieces.
__device__ __forceinline__ int piece_swizzle(int i)
{
    return (i >> 1) & 7;
}

// BM tokens x BN weight rows, WM x WN waves. For two weights each wave's weight
// rows are its channels of w0 followed by the same channels of w1.
template <int BM, int BN, int WM, int WN, int STAGES, int OUT>
__global__ __launch_bounds__(WM *WN * 64) void int8_tile_kernel(Int8GemmArgs a, int tiles_m, int tiles_n)
{
    constexpr bool TWO = int8_two_weights(OUT);
    constexpr int WAVES = WM * WN;
    constexpr int ROWS = BM + BN;
    constexpr int LOADS = ROWS / 8 / WAVES;          // direct loads of a wave and stage
    constexpr int FM = BM / WM / 16, FN = BN / WN / 16;  // fragments of a wave
    constexpr int WR = BN / WN;                      // weight rows of a wave
    constexpr int WC = TWO ? WR / 2 : WR;            // channels of a wave
    constexpr int BC = WC * WN;                      // channels of a tile
    static_assert(ROWS % (8 * WAVES) == 0 && BM % 8 == 0, "whole loads");
    extern __shared__ int8_t lds[];  // [STAGES][ROWS][kBk], tokens first

    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int r = lane & 15, q = lane >> 4;
    const int wm = wave / WN, wn = wave % WN;
    const int K = a.K;
    const int tm = blockIdx.x % tiles_m, tn = blockIdx.x / tiles_m;
    const int m0 = tm * BM, n0 = tn * BC;

    // Lane l of a load covers piece l % 8 of row l / 8 of eight rows.
    const int8_t *src[LOADS];
    int col[LOADS];
#pragma unroll
    for (int j = 0; j < LOADS; ++j) {
        const int row = (wave * LOADS + j) * 8 + (lane >> 3);
        col[j] = ((lane & 7) ^ piece_swizzle(row)) * 16;
        if (row < BM) {
            src[j] = a.x + static_cast<size_t>(min(m0 + row, a.M - 1)) * K + col[j];
        } else {
            const int i = row - BM, part = i / WR, in = i % WR;
            const int n = min(n0 + part * WC + (TWO ? in % WC : in), a.N - 1);
            src[j] = (TWO && in >= WC ? a.w1 : a.w0) + static_cast<size_t>(n) * K + col[j];
        }
    }
    const int whole = K / kBk, stages = (K + kBk - 1) / kBk;

    // Loads stage k into its ring slot: direct loads, or (a last stage of
    // fewer columns) through registers with zeros past the end.
    auto issue = [&](int k) {
        int8_t *to = lds + (k % STAGES) * (ROWS * kBk);
        if (k < whole) {
#pragma unroll
            for (int j = 0; j < LOADS; ++j)
                __builtin_amdgcn_global_load_lds(reinterpret_cast<const void *>(src[j] + k * kBk),
                                                 (FFN_LDS void *)(to + (wave * LOADS + j) * 8 * kBk), 16, 0, 0);
        } else {
#pragma unroll
            for (int j = 0; j < LOADS; ++j) {
                i32x4_t v = {0, 0, 0, 0};
                if (k * kBk + col[j] < K)
                    v = *reinterpret_cast<const i32x4_t *>(src[j] + k * kBk);
                *reinterpret_cast<i32x4_t *>(to + (wave * LOADS + j) * 8 * kBk + lane * 16) = v;
            }
        }
    };

    i32x4_t acc[FN][FM];
#pragma unroll
    for (int f = 0; f < FN; ++f)
#pragma unroll
        for (int t = 0; t < FM; ++t)
            acc[f][t] = i32x4_t{0, 0, 0, 0};

#pragma unroll
    for (int s = 0; s < STAGES - 1; ++s)
        if (s < stages)
            issue(s);

    // row i, piece p of a stage at i * kBk + (p ^ swizzle(i)) * 16; the
    // swizzle of a fragment's row is that of r (fragments start at multiples
    // of 16), and pieces 4 .. 7 are those of the second half with bit 2 set
    const int frag = r * kBk + ((q ^ piece_swizzle(r)) * 16);
    const int xoff = wm * (BM / WM) * kBk + frag;
    const int woff = (BM + wn * WR) * kBk + frag;

    for (int k = 0; k < stages; ++k) {
        // stage k has landed once at most the later stages' loads are in flight
        if (k + STAGES - 1 <= whole)
            wait_vmcnt<(STAGES - 2) * LOADS>();
        else
            wait_vmcnt<0>();
        lds_barrier();
        if (k + STAGES - 1 < stages)
            issue(k + STAGES - 1);
        const int8_t *st = lds + (k % STAGES) * (ROWS * kBk);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            i32x4_t w[FN], x[FM];
#pragma unroll
            for (int f = 0; f < FN; ++f)
                w[f] = *reinterpret_cast<const i32x4_t *>(st + (woff ^ (h * 64)) + f * 16 * kBk);
#pragma unroll
            for (int t = 0; t < FM; ++t)
                x[t] = *reinterpret_cast<const i32x4_t *>(st + (xoff ^ (h * 64)) + t * 16 * kBk);
#pragma unroll
            for (int f = 0; f < FN; ++f)
#pragma unroll
                for (int t = 0; t < FM; ++t)
                    acc[f][t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[f], x[t], acc[f][t], 0, 0, 0);
        }
    }

    constexpr int FC = WC / 16;  // fragments of channels
#pragma unroll
    for (int f = 0; f < FC; ++f) {
        const int n = n0 + wn * WC + 16 * f + 4 * q;
        if (n >= a.N)
            continue;
#pragma unroll
        for (int t = 0; t < FM; ++t) {
            const int m = m0 + wm * (BM / WM) + 16 * t + r;
            if (m < a.M)
                int8_finish4<OUT>(a, m, n, acc[f][t], acc[TWO ? f + FC : f][t]);
        }
    }
}

template <int BM, int BN, int WM, int WN, int STAGES, int OUT>
hipError_t launch_t(const Int8GemmArgs &a, hipStream_t stream)
{
    constexpr int channels = int8_two_weights(OUT) ? BN / 2 : BN;
    auto kern = int8_tile_kernel<BM, BN, WM, WN, STAGES, OUT>;
    constexpr int lds = STAGES * (BM + BN) * kBk;
    static std::atomic<uint64_t> lds_done{0};
    hipError_t e = allow_lds(reinterpret_cast<const void *>(kern), lds, lds_done);
    if (e != hipSuccess)
        return e;
    const int tm = (a.M + BM - 1) / BM, tn = (a.N + channels - 1) / channels;
    hipLaunchKernelGGL(kern, dim3(static_cast<unsigned>(tm) * tn), dim3(WM * WN * 64), lds, stream, a, tm, tn);
    return hipGetLastError();
}

template <int OUT>
hipError_t launch_out(const Int8GemmArgs &a, hipStream_t stream)
{
    return launch_t<128, 128, 2, 2, 2, OUT>(a, stream);
}

}  // namespace

hipError_t launch_int8_tile(const Int8GemmArgs &a, Int8Out out, hipStream_t stream)
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
