// moe_stream.h -- the product grouped by expert for few rows of each expert:
// what it costs is reading the weights, so they go from memory to registers
// once, and everything else is arranged around that.
//
// A tile is 16 rows of one expert (the matrix cores' smallest; rows that are not
// there cost nothing but idle lanes). Eight waves of a workgroup share its
// reduction: wave w takes the 128-column chunks w, w + 8, ... of every weight
// row, and keeps the tile's activations of those columns in registers. A pass
// is 32 weight rows (16 channels of two weights): each wave multiplies its
// chunks of them, the eight partial sums meet in LDS, and one thread finishes
// each result. The weights of the next pass are loaded before those of the
// present one are used, so memory never waits for the arithmetic.
//
// The passes of all tiles, in the order of experts, are dealt out as equal runs
// to as many workgroups as fit the device at once: how many tiles there are is
// known on the device only.
#pragma once

#include "kernels.h"
#include "moe.h"
#include "moe_device.h"

namespace ffn {

constexpr int kStreamRows = 16;
constexpr int kStreamWaves = 8;
constexpr int kStreamThreads = kStreamWaves * 64;
constexpr int kStreamChunk = 128;  // columns of a wave's chunk
constexpr int kStreamMostChunks = 6;
constexpr int kMoeMostExperts = 1024;

// Tiles of 16 rows of experts before this thread's (it has experts 2 tid and
// 2 tid + 1), and of all. Every thread of the workgroup calls it.
__device__ __forceinline__ int stream_tiles_before(int mine, int *wave_sum, int &total)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int sum = mine;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int other = __shfl_up(sum, d);
        sum += lane >= d ? other : 0;
    }
    if (lane == 63)
        wave_sum[wave] = sum;
    __syncthreads();
    total = 0;
    sum -= mine;
#pragma unroll
    for (int w = 0; w < kStreamWaves; ++w) {
        sum += w < wave ? wave_sum[w] : 0;
        total += wave_sum[w];
    }
    return sum;
}

// CH: chunks of a wave.
template <class T, int CH, int OUT>
__global__ __launch_bounds__(kStreamThreads, CH <= 2 ? 4 : 2) void moe_stream_kernel(const MoeGemmArgs a)
{
    constexpr bool TWO = moe_two_weights(OUT);
    constexpr int BN = TWO ? 16 : 32;  // channels of a pass
    typedef typename Half<T>::vec8 vec8;

    __shared__ int begins[kMoeMostExperts + 1];  // where the experts' rows begin
    __shared__ int ends[kMoeMostExperts];
    __shared__ int wave_sum[kStreamWaves];
    __shared__ int start[2];  // expert and tile of it that the run begins with
    __shared__ f32x4_t part[2][2][kStreamWaves][64];  // partial sums: pass parity, fragment, wave, lane

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int q = lane >> 4, r = lane & 15;
    const int K = a.K, N = a.N;
    const int passes = (N + BN - 1) / BN;  // of a tile

    // This workgroup's run of passes.
    int mine = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int e = 2 * threadIdx.x + i;
        if (e < a.E) {
            int b, n;
            rows_of(a, e, b, n);
            begins[e] = b;
            ends[e] = n;
            mine += (n - b + kStreamRows - 1) / kStreamRows;
        }
    }
    int total;
    const int before = stream_tiles_before(mine, wave_sum, total);
    const long all = static_cast<long>(total) * passes;
    const long from = all * blockIdx.x / gridDim.x, to = all * (blockIdx.x + 1) / gridDim.x;
    if (from == to)
        return;
    const int first = static_cast<int>(from / passes);  // the run's first tile
    if (first >= before && first < before + mine) {
        int e = 2 * threadIdx.x, t = first - before;
        const int tiles = (ends[e] - begins[e] + kStreamRows - 1) / kStreamRows;
        if (t >= tiles) {
            t -= tiles;
            ++e;
        }
        start[0] = e;
        start[1] = t;
    }
    __syncthreads();
    const auto scalar = [](int v) { return __builtin_amdgcn_readfirstlane(v); };
    int e = scalar(start[0]);
    int row0 = scalar(begins[e]) + scalar(start[1]) * kStreamRows, row_end = scalar(ends[e]);
    int pass = scalar(static_cast<int>(from - static_cast<long>(first) * passes));
    int left = scalar(static_cast<int>(to - from));

    // Chunk i of this lane: columns 128 (w + 8 i) + 32 q .. + 31. The last of a
    // wave's chunks may lie past the end: then its weights and activations are
    // zeros (and the addresses those of column 0).
    const int col0 = wave * kStreamChunk + 32 * q;
    const bool there = col0 + (CH - 1) * kStreamWaves * kStreamChunk < K;
    const auto col_of = [&](int i) { return i == CH - 1 && !there ? 0 : col0 + i * kStreamWaves * kStreamChunk; };

    // The weight rows of a pass in registers: 32 columns of one row for each
    // fragment and chunk.
    struct Rows {
        u32x4_t codes[2][CH];
        uint32_t scales[2][CH];
    };
    const size_t row_codes = static_cast<size_t>(K) / 2, row_scales = static_cast<size_t>(K) / 16;
    const auto load = [&](Rows &w, int expert, int p) {
#pragma unroll
        for (int f = 0; f < 2; ++f) {
            const uint8_t *codes = TWO && f == 1 ? a.w1.codes : a.w0.codes;
            const uint8_t *scales = TWO && f == 1 ? a.w1.scales : a.w0.scales;
            const int n = min(p * BN + (TWO ? 0 : 16 * f) + r, N - 1);
            const size_t row = static_cast<size_t>(expert) * N + n;
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                const int col = col_of(i);
                w.codes[f][i] = *reinterpret_cast<const u32x4_t *>(codes + row * row_codes + col / 2);
                w.scales[f][i] = *reinterpret_cast<const uint16_t *>(scales + row * row_scales + col / 16);
            }
        }
    };
    vec8 x[CH][4];
    float s0 = 0.0f, s1 = 0.0f;
    const auto load_tile = [&]() {
        int row = min(row0 + r, row_end - 1);
        if (a.rows)
            row = min(max(a.rows[row], 0) / a.top_k, a.x_rows - 1);
        const T *xr = static_cast<const T *>(a.x) + static_cast<size_t>(row) * K;
#pragma unroll
        for (int i = 0; i < CH; ++i)
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                x[i][t] = *reinterpret_cast<const vec8 *>(xr + col_of(i) + 8 * t);
                if (i == CH - 1 && !there)
                    x[i][t] = vec8{};
            }
        s0 = a.w0.scale2[e];
        s1 = TWO ? a.w1.scale2[e] : s0;
    };
    // The pass after this one: of this tile, of the expert's next or of the
    // next expert that has rows.
    int next_e, next_row0, next_end, next_pass;
    const auto find_next = [&]() {
        next_e = e;
        next_row0 = row0;
        next_end = row_end;
        next_pass = pass + 1;
        if (next_pass < passes)
            return;
        next_pass = 0;
        next_row0 += kStreamRows;
        while (next_row0 >= next_end && next_e + 1 < a.E) {
            ++next_e;
            next_row0 = scalar(begins[next_e]);
            next_end = scalar(ends[next_e]);
        }
    };
    int parity = 0;
    const auto multiply = [&](const Rows &w) {
        f32x4_t acc[2] = {};
#pragma unroll
        for (int i = 0; i < CH; ++i)
#pragma unroll
            for (int f = 0; f < 2; ++f) {
                const bool zero = i == CH - 1 && !there;
                const float sc0 = zero ? 0.0f : e4m3_to_f32<0>(w.scales[f][i]);
                const float sc1 = zero ? 0.0f : e4m3_to_f32<1>(w.scales[f][i]);
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    acc[f] = Half<T>::mfma(x[i][t], Half<T>::weights(w.codes[f][i][t], t < 2 ? sc0 : sc1), acc[f]);
            }
#pragma unroll
        for (int f = 0; f < 2; ++f)
            part[parity][f][wave][lane] = acc[f];
    };
    // One thread for each result: value c of lane l is row 4 (l / 16) + c of
    // channel l % 16. Threads 256 .. 511 have the second fragment's.
    const auto finish = [&]() {
        lds_barrier();
        const int j = threadIdx.x & 255, f = threadIdx.x >> 8;
        const int l = j & 63, c = j >> 6;
        const int row = row0 + 4 * (l >> 4) + c, n = pass * BN + (TWO ? 0 : 16 * f) + (l & 15);
        float sum0 = 0.0f, sum1 = 0.0f;
        if (!(TWO && f == 1)) {
#pragma unroll
            for (int w = 0; w < kStreamWaves; ++w) {
                sum0 += reinterpret_cast<const float *>(&part[parity][f][w][l])[c];
                if (TWO)
                    sum1 += reinterpret_cast<const float *>(&part[parity][1][w][l])[c];
            }
            if (row < row_end && n < N)
                moe_store<T, OUT>(a.out, static_cast<size_t>(row) * N + n, moe_value<OUT>(sum0, sum1, s0, s1));
        }
        parity ^= 1;
    };

    Rows even, odd;
    load(even, e, pass);
    load_tile();
    const auto step = [&](Rows &now, Rows &next) {
        find_next();
        if (left > 1)
            load(next, next_e, next_pass);
        multiply(now);
        finish();
        const bool tile = next_pass == 0;
        e = next_e;
        row0 = next_row0;
        row_end = next_end;
        pass = next_pass;
        --left;
        if (tile && left > 0)
            load_tile();
    };
    while (true) {
        step(even, odd);
        if (left == 0)
            return;
        step(odd, even);
        if (left == 0)
            return;
    }
}

template <class T, int CH, int OUT>
hipError_t launch_stream_chunks(const MoeGemmArgs &a, hipStream_t stream)
{
    constexpr int BN = moe_two_weights(OUT) ? 16 : 32;
    const long most = (a.R / kStreamRows + (a.R < a.E ? a.R : a.E)) * static_cast<long>((a.N + BN - 1) / BN);
    const long room = device_cu_count() * (CH <= 2 ? 2 : 1);
    hipLaunchKernelGGL((moe_stream_kernel<T, CH, OUT>), dim3(most < room ? most : room), dim3(kStreamThreads), 0,
                       stream, a);
    return hipGetLastError();
}

// hipErrorNotSupported where the tiles of moe_gemm.hip are faster or K is too
// long for a wave's registers.
template <class T, int OUT>
hipError_t launch_moe_stream(const MoeGemmArgs &a, hipStream_t stream)
{
    if (a.R > 16 * a.E)
        return hipErrorNotSupported;
    switch ((a.K + kStreamWaves * kStreamChunk - 1) / (kStreamWaves * kStreamChunk)) {
    case 1:
        return launch_stream_chunks<T, 1, OUT>(a, stream);
    case 2:
        return launch_stream_chunks<T, 2, OUT>(a, stream);
    case 3:
        return launch_stream_chunks<T, 3, OUT>(a, stream);
    case 4:
        return launch_stream_chunks<T, 4, OUT>(a, stream);
    case 5:
        return launch_stream_chunks<T, 5, OUT>(a, stream);
    case 6:
        return launch_stream_chunks<T, 6, OUT>(a, stream);
    default:
        return hipErrorNotSupported;
    }
}

}  // namespace ffn
