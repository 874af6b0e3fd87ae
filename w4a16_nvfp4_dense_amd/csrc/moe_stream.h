// moe_stream.h -- the product grouped by expert for few rows of each expert:
// what it costs is reading the weights, so they go from memory to registers
// once, and everything else is arranged around that.
//
// A tile is 16 rows of one expert (the matrix cores' smallest; rows that are not
// there cost nothing but idle lanes). Eight waves of a workgroup share its
// reduction: each takes some 128-column chunks of every weight row, and keeps
// the tile's activations of those columns in registers. A pass is 32 weight rows
// (16 channels of two weights): each wave multiplies its chunks of them, the eight
// partial sums meet in LDS, and one thread finishes each result. The weights of the
// next pass are loaded before those of the present one are used, so memory never
// waits for the arithmetic. Reductions too long for the registers go in blocks.
//
// The passes of all tiles, in the order of experts, are dealt out as equal runs
// to as many workgroups as fit the device at once: how many tiles there are is
// known on the device only.
//
// What bounds it is the stream of weights: reads alone reach 6.0 - 7.0 TB/s. 64
// rows of 64 experts (41 of them met), 2048 -> 5120: 239 MB in 42 us, 5.7 TB/s. 32
// tokens, 8 of 128 experts each, 2048/1024: gate and up 254 MB in 49.6 us, 5.1
// TB/s, down 127 MB in 29.3. One token, 8 of 64 experts, 5120/2048: gate and up 94 MB
// in 27.2 us, down 47 MB in 14.0, 3.4 TB/s, for there the start of a launch (its
// first data comes after 4 - 5 us) and the last pass, which nothing hides, are
// most of what is above the floor. Weights are fetched once (94.8 and 47.6 MB
// counted). Measured without gain: loads two passes ahead (25.9 us for 27.6 of that
// gate and up, but 14.9 for 13.4 of down), non-temporal loads (30.7 for 27.6), a
// wave's priority raised for its products.
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
// 32 weight rows of a pass each). CH: chunks of a wave. LONG: a reduction of any
// length, in blocks of CH WK chunks one after another; the activations of a block
// are read again for each pass.
template <class T, bool SLOTS, int WK, int CH, int OUT, bool LONG>
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
    static_assert(!LONG || CH == 2, "one pair, all of whose columns may be past the end");
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
    const int blocks = LONG ? (K + BLOCK - 1) / BLOCK : 1;  // of a pass

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
    int block = 0;
    int left = count * blocks;  // steps

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
        code_at[i] = LONG || col_of(i) < K ? r * row_codes + col_of(i) / 2 : kPast;
        scale_at[i] = group * 2 * BLOCK + (LONG ? r * (BLOCK / 16) + col_of(i) / 16
                                           : col_of(i) < K ? r * row_scales + col_of(i) / 16 : 0);
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
    const auto extra_of = [&](int n) { return LONG ? 0 : rows_from(n) * row_scales & 2; };
    const auto skew_of = [&](int expert, int n) { return expert == 0 && n == 0 ? 0 : extra_of(n); };
    const auto load = [&](Rows &w, int expert, int p, int blk, bool real) {
        const auto rows_at = [&](const uint8_t *m, int n, int row_bytes, int extra) {  // 16 rows from channel n on
            const size_t row = static_cast<size_t>(scalar(expert)) * N + n;
            return uniform_buffer(m + row * row_bytes, real ? rows_from(n) * row_bytes + extra : 0);
        };
        const int n0 = scalar(p) * BN;
#pragma unroll
        for (int j = 0; j < PIECES; ++j) {
            const int fr = slot_of(j) / SLOTS_EACH, f = fr % 2, n = n0 + fr / 2 * GN + (TWO ? 0 : 16 * f);
            const auto scales = rows_at((TWO && f == 1 ? a.w1.scales : a.w0.scales) - skew_of(expert, n), n, row_scales,
                                        extra_of(n));
            const int at = piece_at(j);
            uint32_t offset = fr < FRAGS && at < K ? at : kPast;
            if constexpr (LONG) {  // of a row's scales those of the block
                const int col = blk * (BLOCK / 16) + at % (BLOCK / 16);
                offset = fr < FRAGS && col < row_scales ? at / (BLOCK / 16) * row_scales + col : kPast;
            }
            piece[j] = __builtin_amdgcn_raw_buffer_load_b128(scales, offset, 0, 0);
        }
#pragma unroll
        for (int f = 0; f < 2; ++f) {
            const auto codes = rows_at(TWO && f == 1 ? a.w1.codes : a.w0.codes,
                                       n0 + group * GN + (TWO ? 0 : 16 * f), row_codes, 0);
#pragma unroll
            for (int i = 0; i < CH; ++i)
                w.codes[f][i] = __builtin_amdgcn_raw_buffer_load_b128(
                    codes, !LONG || blk * BLOCK + col_of(i) < K ? code_at[i] : kPast, blk * (BLOCK / 2), 0);
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
    uintptr_t x_row;
    const auto load_x = [&]() {
#pragma unroll
        for (int i = 0; i < CH; ++i)
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const int col = (LONG ? block * BLOCK : 0) + col_of(i);
                x[i][t] = load_global<vec8>(col < K ? x_row + (col + 8 * t) * sizeof(T)
                                                    : reinterpret_cast<uintptr_t>(&kZeros));
            }
    };
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
        x_row = reinterpret_cast<uintptr_t>(static_cast<const T *>(a.x) + static_cast<size_t>(row) * K);
        if constexpr (!LONG)
            load_x();
        s0 = a.w0.scale2[e];
        s1 = TWO ? a.w1.scale2[e] : s0;
    };
    // The step after this one: the pass's next block, or the next pass: of this
    // tile, of the expert's next or of the next expert that has rows.
    int next_e, next_row0, next_end, next_pass, next_block;
    const auto find_next = [&]() {
        next_e = e;
        next_row0 = row0;
        next_end = row_end;
        next_pass = pass;
        next_block = block + 1;
        if (next_block < blocks)
            return;
        next_block = 0;
        ++next_pass;
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
    f32x4_t acc[2];
    const auto multiply = [&](const Rows &w) {
        if (!LONG || block == 0)
            acc[0] = acc[1] = f32x4_t{};
#pragma unroll
        for (int f = 0; f < 2; ++f) {  // (in the order of their loads)
            const int skew = scalar(skew_of(e, pass * BN + group * GN + (TWO ? 0 : 16 * f)));
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                uint32_t both = *reinterpret_cast<const uint16_t *>(scales_lds[parity] + f * BLOCK + skew + scale_at[i]);
                if (i >= CH - 2 && (LONG ? block * BLOCK : 0) + col_of(i) >= K)  // (codes are zeros: a scale of NaN would not be)
                    both = 0;
                const float sc0 = e4m3_to_f32<0>(both), sc1 = e4m3_to_f32<1>(both);
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    acc[f] = Half<T>::mfma(x[i][t], Half<T>::weights(w.codes[f][i][t], t < 2 ? sc0 : sc1), acc[f]);
            }
        }
        if (next_block == 0)
#pragma unroll
            for (int f = 0; f < 2; ++f)
                part[parity][f][wave][lane] = acc[f];
    };
    // One thread for each result: value c of lane l is row 4 (l / 16) + c of
    // channel l % 16 of a fragment.
    const auto finish = [&]() {
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
    };

    Rows even, odd;
    load(even, e, pass, 0, true);
    load_tile();
    keep_scales(0);
    lds_barrier();
    const auto step = [&](Rows &now, Rows &next) {
        find_next();
        if constexpr (LONG)
            load_x();
        load(next, next_e, next_pass, next_block, left > 1);
        multiply(now);
        keep_scales(parity ^ 1);
        lds_barrier();
        if (next_block == 0)
            finish();
        parity ^= 1;
        const bool tile = next_pass == 0 && next_block == 0;
        e = next_e;
        row0 = next_row0;
        row_end = next_end;
        pass = next_pass;
        block = next_block;
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

template <class T, bool SLOTS, int WK, int CH, int OUT, bool LONG = false>
hipError_t launch_stream_chunks(const MoeGemmArgs &a, hipStream_t stream)
{
    const long most = stream_passes<OUT>(a, WK), room = device_cu_count() * (CH <= 2 ? 2 : 1);
    hipLaunchKernelGGL((moe_stream_kernel<T, SLOTS, WK, CH, OUT, LONG>), dim3(most < room ? most : room),
                       dim3(kStreamThreads), 0, stream, a);
    return hipGetLastError();
}

// Whether this kernel is the one for a product (of TWO weights); if not, tiles are.
// Up to 16 rows of an expert on average (figures at the tiles' launcher), provided
// that the weights have two bytes of scales before or behind any block of rows. The
// mean is all that the host knows: where one expert has all rows its weights are
// read, from L2, once for 16 of them (64 experts, 5120 -> 2048, all rows with one: 256
// rows 31 us for 34 on tiles of 64 x 128, 512 50 for 36, 1024 82 for 38).
// With the reduction in blocks, whose activations are read again for each pass, up
// to 4, or 16 where the tiles are fewer than the compute units; us, this kernel
// and tiles of 32 rows, experts x rows:
//   8192 -> 4096, two weights, 8 x 2 / 4 / 6 / 8:   78 / 80 / 91 / 103   82 / 82 / 82 / 82
//   8192 -> 4096, 32 x 4 / 6 / 8:                   167 / 180 / 205      162 / 165 / 167
//   14336 -> 4096, 2 x 1, 8 x 1 / 4 / 8 / 16: 19, 57 / 65 / 83 / 117     116, 117 / 118 / 119 / 121
template <bool TWO>
bool stream_fits(int R, int E, int K, int N)
{
    if (R > kStreamRows * E)
        return false;
    if (K <= kStreamMostChunks * kStreamWaves * kStreamChunk)
        return E > 1 || N >= 16 || K % 64 == 0 || N % 2 == 0;
    constexpr int BN = TWO ? 128 : 256;
    const long tiles = (R / 32 + (R < E ? R : E)) * static_cast<long>((N + BN - 1) / BN);
    return K % 64 == 0 && (R <= 4 * E || tiles < device_cu_count());
}

template <class T, bool SLOTS, int OUT>
hipError_t launch_moe_stream(const MoeGemmArgs &a, hipStream_t stream)
{
    // Up to 1024 columns, two groups of four waves with two chunks each (whole lines
    // of memory for a wave), where every compute unit has several passes: 34 - 38
    // us for 38 - 42 at K = 1024. At 2048 four chunks of four waves: 16.9 us for 13.9.
    // Six chunks of a wave are a few registers more than there are, so few rows go
    // by blocks there: 6144 -> 4096, 2 rows of 2 experts 10.5 us for 15.2, 4 rows of each
    // of 8 30.4 for 33.6, but 16 of each 51.7 for 40.2. With five, 5120 -> 4096: 11.7 for
    // 12.6 (2 of 2), 29.2 for 27.3 (1 of 8), 32.7 for 27.6 (4 of 8).
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
    case 6:
        if (a.R > 4 * a.E || a.K % 64)
            return launch_stream_chunks<T, SLOTS, 8, 6, OUT>(a, stream);
        [[fallthrough]];
    default:
        return launch_stream_chunks<T, SLOTS, 8, 2, OUT, true>(a, stream);
    }
}

}  // namespace ffn
