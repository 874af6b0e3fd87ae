// moe_stream.h -- the product grouped by expert for few rows of each expert:
// what it costs is reading the weights, so they go from memory to registers
// once, and everything else is arranged around that.
//
// A tile is 16 rows of one expert (the matrix cores' smallest; rows that are not
// there cost nothing but idle lanes). Eight waves of a workgroup share its
// reduction: each takes some 128-column chunks of every weight row, and keeps
// the tile's activations of those columns in registers. A pass
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
constexpr int kStreamSlots = kStreamThreads;  // a thread for each
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

// SLOTS: there is no plan; a.ids has the experts of the R slots (at most
// kStreamSlots), row s of the product is of x[s / top_k] and is written to
// out[s]. Every workgroup counts the experts' slots for itself, and finds the
// slots of a tile by looking through the ids, kept in LDS.
// WK: waves that share a reduction (the workgroup's 8 / WK groups of them have
// 32 weight rows of a pass each). CH: chunks of a wave.
template <class T, bool SLOTS, int WK, int CH, int OUT>
__global__ __launch_bounds__(kStreamThreads, CH <= 2 ? 4 : 2) void moe_stream_kernel(const MoeGemmArgs a)
{
    constexpr bool TWO = moe_two_weights(OUT);
    constexpr int GROUPS = kStreamWaves / WK;
    constexpr int GN = TWO ? 16 : 32;   // channels of a group
    constexpr int BN = GN * GROUPS;     // and of a pass
    constexpr int FRAGS = 2 * GROUPS;   // fragments of 16 weight rows of a pass
    constexpr int BLOCK = CH * WK * kStreamChunk;  // most bytes of a fragment's scales: the most columns
    constexpr int SLOTS_EACH = BLOCK / 1024;       // 64 pieces of 16 bytes each
    constexpr int PIECES = (FRAGS * SLOTS_EACH + kStreamWaves - 1) / kStreamWaves;  // of a thread
    static_assert(BLOCK % 1024 == 0, "whole waves");
    typedef typename Half<T>::vec8 vec8;

    __shared__ int bound[kMoeMostExperts + 1];  // where the experts' rows begin; SLOTS: how many they are
    __shared__ int slot_ids[SLOTS ? kStreamSlots : 1];
    __shared__ int tile_slots[SLOTS ? kStreamWaves : 1][kStreamRows];  // the tile's, for each wave
    __shared__ int wave_sum[kStreamWaves];
    __shared__ int start[2];  // expert and tile of it that the run begins with
    __shared__ __attribute__((aligned(16))) uint8_t scales_lds[2][FRAGS * BLOCK];  // pass parity
    __shared__ f32x4_t part[2][2][kStreamWaves][64];  // partial sums: pass parity, fragment, wave, lane

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int q = lane >> 4, r = lane & 15;
    const int wk = wave % WK, group = wave / WK;
    const int K = a.K, N = a.N;
    const int passes = (N + BN - 1) / BN;  // of a tile

    const auto scalar = [](int v) { return __builtin_amdgcn_readfirstlane(v); };

    // This workgroup's run of passes.
    int mine = 0;
    if constexpr (SLOTS) {
        for (int e = threadIdx.x; e < a.E; e += kStreamThreads)
            bound[e] = 0;
        const int id = static_cast<int>(threadIdx.x) < a.R ? a.ids[threadIdx.x] : -1;
        slot_ids[threadIdx.x] = id;
        __syncthreads();
        if (id >= 0 && id < a.E)
            atomicAdd(&bound[id], 1);
    } else {
        for (int e = threadIdx.x; e <= a.E; e += kStreamThreads)
            bound[e] = min(max(a.offsets[e], 0), a.R);
    }
    __syncthreads();
    const auto begin_of = [&](int e) { return SLOTS ? 0 : bound[e]; };
    const auto end_of = [&](int e) { return SLOTS ? bound[e] : max(bound[e + 1], bound[e]); };
    const auto tiles_of = [&](int e) { return (end_of(e) - begin_of(e) + kStreamRows - 1) / kStreamRows; };
#pragma unroll
    for (int i = 0; i < 2; ++i)
        if (2 * static_cast<int>(threadIdx.x) + i < a.E)
            mine += tiles_of(2 * threadIdx.x + i);
    int total;
    const int before = stream_tiles_before(mine, wave_sum, total);
    // Offsets that do not ascend could ask for any number of tiles; such a product
    // is left undone.
    if (total > a.R / kStreamRows + min(a.R, a.E))
        return;
    const unsigned all = static_cast<unsigned>(total) * passes;  // (2048 tiles of 65536 passes at most)
    const unsigned share = all / gridDim.x, over = all % gridDim.x, b = blockIdx.x;
    const unsigned from = b * share + min(b, over);
    const int count = scalar(share + (b < over ? 1 : 0));
    if (count == 0)
        return;
    const int first = static_cast<int>(from / passes);  // the run's first tile
    if (first >= before && first < before + mine) {
        int e = 2 * threadIdx.x, t = first - before;
        if (t >= tiles_of(e)) {
            t -= tiles_of(e);
            ++e;
        }
        start[0] = e;
        start[1] = t;
    }
    __syncthreads();
    int e = scalar(start[0]);
    int row_end = scalar(end_of(e)), row0 = scalar(begin_of(e) + start[1] * kStreamRows);
    int pass = scalar(static_cast<int>(from) - first * passes);  // (divisions run on the vector unit)
    int left = count;

    // Chunks go in pairs, so that a lane has 64 consecutive columns of a row and a
    // wave whole lines of memory: chunks 2 j and 2 j + 1 are its columns 256 (w +
    // WK j) + 64 q .. + 31 and .. + 63; the last chunk of an odd number is columns
    // 128 (WK (CH - 1) + w) + 32 q .. + 31.
    constexpr int PAIRS = CH / 2;
    const auto col_of = [&](int i) {
        return i < 2 * PAIRS ? (wk + i / 2 * WK) * 256 + 64 * q + i % 2 * 32 : (wk + i * WK) * 128 + 32 * q;
    };

    // The weight rows of a pass in registers: 32 columns of one row for each
    // fragment and chunk. They are loaded by buffer, whose bounds check gives
    // zeros for rows past the last channel (and for the pass behind the run's
    // last, of no rows: the same number of loads on every path, so that the
    // compiler's waits for the pass at hand are not waits for the next one);
    // columns past the end have an offset past any buffer.
    struct Rows {
        u32x4_t codes[2][CH];
    };
    const int row_codes = K / 2, row_scales = K / 16;
    uint32_t code_at[CH];
    int scale_at[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        code_at[i] = col_of(i) < K ? r * row_codes + col_of(i) / 2 : kPast;
        scale_at[i] = group * 2 * BLOCK + (col_of(i) < K ? r * row_scales + col_of(i) / 16 : 0);
    }
    // The block scales of a fragment are K consecutive bytes, 16 of them for each
    // thread; they come to LDS by way of registers. (Each lane loading those of
    // its own chunks touches many lines for a few bytes each: 2048 -> 5120, 32
    // experts met, 43.1 us for 42.4; one token's layer 5120/2048 47.7 for 45.4.)
    u32x4_t piece[PIECES];
    const auto slot_of = [&](int j) { return j * kStreamWaves + wave; };  // of 64 pieces
    const auto piece_at = [&](int j) { return slot_of(j) % SLOTS_EACH * 1024 + lane * 16; };
    // The bounds check is made for each four bytes. Where a block's are two more
    // than a multiple of four (an odd number of rows, K not a multiple of 64), it
    // is taken with the two bytes before it (the first of all, with the two behind).
    const auto rows_from = [&](int n) { return min(max(N - n, 0), 16); };
    const auto extra_of = [&](int n) { return rows_from(n) * row_scales & 2; };
    const auto skew_of = [&](int expert, int n) { return expert == 0 && n == 0 ? 0 : extra_of(n); };
    const auto load = [&](Rows &w, int expert, int p, bool real) {
        const auto block = [&](const uint8_t *m, int n, int row_bytes, int extra) {  // 16 rows from channel n on
            const size_t row = static_cast<size_t>(scalar(expert)) * N + n;
            return uniform_buffer(m + row * row_bytes, real ? rows_from(n) * row_bytes + extra : 0);
        };
        const int n0 = scalar(p) * BN;
#pragma unroll
        for (int j = 0; j < PIECES; ++j) {
            const int fr = slot_of(j) / SLOTS_EACH, f = fr % 2, n = n0 + fr / 2 * GN + (TWO ? 0 : 16 * f);
            const auto scales = block((TWO && f == 1 ? a.w1.scales : a.w0.scales) - skew_of(expert, n), n, row_scales,
                                      extra_of(n));
            const int at = piece_at(j);
            piece[j] = __builtin_amdgcn_raw_buffer_load_b128(scales, fr < FRAGS && at < K ? at : kPast, 0, 0);
        }
#pragma unroll
        for (int f = 0; f < 2; ++f) {
            const auto codes = block(TWO && f == 1 ? a.w1.codes : a.w0.codes,
                                     n0 + group * GN + (TWO ? 0 : 16 * f), row_codes, 0);
#pragma unroll
            for (int i = 0; i < CH; ++i)
                w.codes[f][i] = __builtin_amdgcn_raw_buffer_load_b128(codes, code_at[i], 0, 0);
        }
        __builtin_amdgcn_sched_barrier(0);  // (nothing that waits for earlier loads goes before these)
    };
    const auto keep_scales = [&](int to) {
#pragma unroll
        for (int j = 0; j < PIECES; ++j)
            if (slot_of(j) < FRAGS * SLOTS_EACH)
                *reinterpret_cast<u32x4_t *>(scales_lds[to] + slot_of(j) * 1024 + lane * 16) = piece[j];
    };
    vec8 x[CH][4];
    float s0 = 0.0f, s1 = 0.0f;
    const auto load_tile = [&]() {
        int row = min(row0 + r, row_end - 1);
        if constexpr (SLOTS) {
            int rank = -row0;  // of the expert's slots, from the tile's first
            for (int s0 = 0; s0 < a.R; s0 += 64) {
                const bool ours = slot_ids[s0 + lane] == e;
                const unsigned long long lanes = __ballot(ours);
                const int at = rank + __popcll(lanes & ((1ull << lane) - 1));
                if (ours && at >= 0 && at < kStreamRows)
                    tile_slots[wave][at] = s0 + lane;
                rank += __popcll(lanes);
            }
            __builtin_amdgcn_wave_barrier();
            row = tile_slots[wave][row - row0] / a.top_k;
        } else if (a.rows) {
            row = min(max(a.rows[row], 0) / a.top_k, a.x_rows - 1);
        }
        const T *xr = static_cast<const T *>(a.x) + static_cast<size_t>(row) * K;
#pragma unroll
        for (int i = 0; i < CH; ++i)
#pragma unroll
            for (int t = 0; t < 4; ++t)
                x[i][t] = load_global<vec8>(col_of(i) < K ? reinterpret_cast<uintptr_t>(xr + col_of(i) + 8 * t)
                                                          : reinterpret_cast<uintptr_t>(&kZeros));
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
            next_row0 = scalar(begin_of(next_e));
            next_end = scalar(end_of(next_e));
        }
    };
    int parity = 0;
    const auto multiply = [&](const Rows &w) {
        f32x4_t acc[2] = {};
#pragma unroll
        for (int f = 0; f < 2; ++f) {  // (in the order of their loads)
            const int skew = scalar(skew_of(e, pass * BN + group * GN + (TWO ? 0 : 16 * f)));
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                uint32_t both = *reinterpret_cast<const uint16_t *>(scales_lds[parity] + f * BLOCK + skew + scale_at[i]);
                if (i >= CH - 2 && col_of(i) >= K)  // (codes are zeros: a scale of NaN would not be)
                    both = 0;
                const float sc0 = e4m3_to_f32<0>(both), sc1 = e4m3_to_f32<1>(both);
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    acc[f] = Half<T>::mfma(x[i][t], Half<T>::weights(w.codes[f][i][t], t < 2 ? sc0 : sc1), acc[f]);
            }
        }
#pragma unroll
        for (int f = 0; f < 2; ++f)
            part[parity][f][wave][lane] = acc[f];
    };
    // One thread for each result: value c of lane l is row 4 (l / 16) + c of
    // channel l % 16 of a fragment.
    const auto finish = [&]() {
        lds_barrier();
#pragma unroll
        for (int k = 0; k < GROUPS * (TWO ? 1 : 2); k += 2) {
            const int j = threadIdx.x & 255, i = k + (threadIdx.x >> 8);  // i: which 256 results
            if (TWO && GROUPS == 1 && i == 1)
                break;
            const int f = TWO ? 0 : i & 1, g = TWO ? i : i >> 1;
            const int l = j & 63, c = j >> 6;
            const int row = row0 + 4 * (l >> 4) + c, n = pass * BN + g * GN + 16 * f + (l & 15);
            const int to = SLOTS ? tile_slots[wave][row - row0] : row;
            float sum0 = 0.0f, sum1 = 0.0f;
#pragma unroll
            for (int w = 0; w < WK; ++w) {
                sum0 += reinterpret_cast<const float *>(&part[parity][f][g * WK + w][l])[c];
                if (TWO)
                    sum1 += reinterpret_cast<const float *>(&part[parity][1][g * WK + w][l])[c];
            }
            if (row < row_end && n < N)
                moe_store<T, OUT>(a.out, static_cast<size_t>(to) * N + n, moe_value<OUT>(sum0, sum1, s0, s1));
        }
        parity ^= 1;
    };

    Rows even, odd;
    load(even, e, pass, true);
    load_tile();
    keep_scales(0);
    lds_barrier();
    const auto step = [&](Rows &now, Rows &next) {
        find_next();
        load(next, next_e, next_pass, left > 1);
        multiply(now);
        keep_scales(parity ^ 1);
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

// The most passes that a product can have.
template <int OUT>
long stream_passes(const MoeGemmArgs &a, int WK)
{
    const int BN = (moe_two_weights(OUT) ? 16 : 32) * kStreamWaves / WK;
    return (a.R / kStreamRows + (a.R < a.E ? a.R : a.E)) * static_cast<long>((a.N + BN - 1) / BN);
}

template <class T, bool SLOTS, int WK, int CH, int OUT>
hipError_t launch_stream_chunks(const MoeGemmArgs &a, hipStream_t stream)
{
    const long most = stream_passes<OUT>(a, WK), room = device_cu_count() * (CH <= 2 ? 2 : 1);
    hipLaunchKernelGGL((moe_stream_kernel<T, SLOTS, WK, CH, OUT>), dim3(most < room ? most : room), dim3(kStreamThreads), 0,
                       stream, a);
    return hipGetLastError();
}

// Whether a reduction fits the waves' registers (and the weights have two bytes
// of scales before or behind any block of rows).
inline bool stream_fits(int E, int K, int N)
{
    return K <= kStreamMostChunks * kStreamWaves * kStreamChunk && (E > 1 || N >= 16 || K % 64 == 0 || N % 2 == 0);
}

template <class T, bool SLOTS, int OUT>
hipError_t launch_moe_stream(const MoeGemmArgs &a, hipStream_t stream)
{
    switch ((a.K + kStreamWaves * kStreamChunk - 1) / (kStreamWaves * kStreamChunk)) {
    case 1:
        if (a.K > 512 && stream_passes<OUT>(a, 4) >= 4 * device_cu_count())
            return launch_stream_chunks<T, SLOTS, 4, 2, OUT>(a, stream);
        return launch_stream_chunks<T, SLOTS, 8, 1, OUT>(a, stream);
    case 2:
        return launch_stream_chunks<T, SLOTS, 8, 2, OUT>(a, stream);
    case 3:
        return launch_stream_chunks<T, SLOTS, 8, 3, OUT>(a, stream);
    case 4:
        return launch_stream_chunks<T, SLOTS, 8, 4, OUT>(a, stream);
    case 5:
        return launch_stream_chunks<T, SLOTS, 8, 5, OUT>(a, stream);
    default:
        return launch_stream_chunks<T, SLOTS, 8, 6, OUT>(a, stream);
    }
}

}  // namespace ffn
