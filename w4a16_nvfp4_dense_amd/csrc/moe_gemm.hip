// moe_gemm.hip -- the product grouped by expert over NVFP4 weights, on tiles of
// tokens and channels, for any number of rows of each expert.
//
// Mathematics. Rows offsets[e] .. offsets[e + 1] - 1 of the product are
// scale2[e] W_e x, with W_e = e2m1 * e4m3. A weight has at most six significant
// bits and exponents from -10 to 12, so it is exact in bf16 and in f16, and
// the only rounding in a sum is that of the matrix core's fp32 accumulation.
//
// Tiles. A tile is 32 MT rows of one expert by 256 weight rows (128 channels of
// two weights), or by 128 of one weight where the others would be too few. How many
// tiles an expert has is known on the device only, so the grid is the most there
// can be, and each workgroup finds its tile from the offsets (a scan over experts);
// workgroups past the last tile end at once. Tiles are numbered expert by expert,
// the rows fastest, and dealt to the eight XCDs in runs, so that an XCD's L2 holds
// what its tiles share.
//
// A workgroup has four waves; each dequantises 32 NF weight rows of the tile, 64
// (32 of either weight) or 32, and multiplies them with all its rows. Activations come
// through a ring of LDS units of 64 columns, by direct loads of 16 bytes a lane,
// the pieces swizzled so that reads meet no bank twice (none counted). Codes and
// scales are used by one wave only, so they come to registers, by stages of 128
// columns: lane half h = lane / 32 has columns 64 h .. + 63, two 16-byte pieces, and
// unit v of a stage is columns 64 h + 32 v .. + 31 of either half; in step t (of
// four) of a unit a lane multiplies eight of them. One barrier a unit.
//
// What bounds it. Many rows of an expert: the matrix cores, at the clock that
// the card's power leaves. 4019 tokens, 8 of 64 experts each, 5120/2048: gate and up
// 1.35 TFLOP in 1300 - 1391 us, 970 - 1037 TFLOP/s; down 674 GFLOP in 706 - 750, 899 -
// 955; 16384 rows of 64 experts, 5120 -> 2048: 343.6 GFLOP in 375 - 405 us, 848 - 916.
// A large bf16 library product reaches 1450. The matrix cores are busy 51 -
// 57% of the time. The vector instructions before the products are a small part of
// it: in f16, which has half as many, those 16384 rows take 382 us for 402. With
// operands of zeros, so at the full clock, the same kernel
// does 1697 TFLOP/s, without its reads of LDS it is 17% faster, with all weights in
// L2 10%. Tiles of 512 channels and eight waves (half the reads of activations
// from L2): 2213 us for 2172 of the whole layer; channels fastest instead of rows:
// 2229. Few rows: the weights' way in, a tile's worth of latency; two groups of
// waves that share the columns of a tile: 49.9 us for 48.4 at 777 rows of 17
// experts. Weights through LDS as well, in pieces of 32 bytes a row: 172 us for 134
// at 32 rows each of 64 experts, 5120 -> 2048.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "kernels.h"
#include "moe.h"
#include "moe_device.h"
#include "moe_stream.h"

namespace ffn {
namespace {

constexpr int kThreads = 256;
constexpr int kStageCols = 128;

// The tile of a workgroup.
struct Tile {
    int e;           // expert, or -1: none
    int begin, end;  // its rows of the product
    int nt;          // which channels
};

// Finds tile number `at` (of this workgroup, see above) among tiles of BM rows
// and `nts` groups of channels. Every thread calls it; it has barriers.
template <int BM>
__device__ __forceinline__ Tile find_tile(const MoeGemmArgs &a, int nts, int *note)
{
    // note: [0..3] sums of the waves, [4..7] the tile
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int per = (a.E + kThreads - 1) / kThreads;
    const int e0 = threadIdx.x * per, e1 = min(e0 + per, a.E);
    int mine = 0;
    for (int e = e0; e < e1; ++e) {
        int begin, end;
        rows_of(a, e, begin, end);
        mine += (end - begin + BM - 1) / BM;
    }
    int sum = mine;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int other = __shfl_up(sum, d);
        sum += lane >= d ? other : 0;
    }
    if (lane == 63)
        note[wave] = sum;
    if (threadIdx.x == 0)
        note[4] = -1;
    __syncthreads();
    int total = 0;
    sum -= mine;
#pragma unroll
    for (int w = 0; w < kThreads / 64; ++w) {
        sum += w < wave ? note[w] : 0;
        total += note[w];
    }
    // runs of tiles for the XCDs; workgroup b runs on XCD b % 8
    const int tiles = total * nts, run = (tiles + 7) / 8;
    const int within = blockIdx.x / 8, number = static_cast<int>(blockIdx.x % 8) * run + within;
    if (within < run && number < tiles) {
        const int group = number / nts;  // within the expert's share
        if (group >= sum && group < sum + mine) {
            for (int e = e0; e < e1; ++e) {
                int begin, end;
                rows_of(a, e, begin, end);
                const int count = (end - begin + BM - 1) / BM;
                if (group < sum + count) {
                    const int local = number - sum * nts;
                    note[5] = begin + local % count * BM;
                    note[6] = end;
                    note[7] = local / count;
                    note[4] = e;
                    break;
                }
                sum += count;
            }
        }
    }
    __syncthreads();
    const auto scalar = [](int v) { return __builtin_amdgcn_readfirstlane(v); };
    Tile t;
    t.e = scalar(note[4]);
    t.begin = scalar(note[5]);
    t.end = min(scalar(note[6]), t.begin + BM);
    t.nt = scalar(note[7]);
    return t;
}

// How deep a tile's loads run ahead: units of activations (LDS) and stages of
// weights (registers).
template <int MT>
constexpr int units_ahead()
{
    return MT == 4 ? 4 : 8;
}
template <int MT>
constexpr int stages_ahead()
{
    return MT == 4 ? 2 : 4;
}
// Channels of a tile: four waves have NF fragments of 32 weight rows each.
template <int NF, int OUT>
constexpr int tile_channels()
{
    return moe_two_weights(OUT) ? 128 : 128 * NF;
}
// On the way out: bytes of a row of results in LDS, and how many fragments of rows
// go at once.
template <int NF, int OUT>
constexpr int out_row_bytes()
{
    return tile_channels<NF, OUT>() * (OUT == MOE_F32 ? 4 : 2) + 16;
}
template <int MT, int OUT>
constexpr int out_pass()
{
    return OUT == MOE_F32 && MT == 4 ? 2 : MT;
}
// Bytes of LDS, the last 32 of them what find_tile notes.
template <int MT, int NF, int OUT>
constexpr int tile_lds()
{
    constexpr int ring = units_ahead<MT>() * MT * 4096, out = 32 * out_pass<MT, OUT>() * out_row_bytes<NF, OUT>();
    return (ring > out ? ring : out) + 32;
}

// WIDE: x does not fit a buffer of 32-bit offsets.
template <class T, int MT, int NF, int OUT, bool WIDE>
__global__ __launch_bounds__(kThreads, 2) void moe_tile_kernel(const MoeGemmArgs a)
{
    constexpr bool TWO = moe_two_weights(OUT);
    constexpr int BM = 32 * MT;
    constexpr int BN = tile_channels<NF, OUT>(), WR = BN / 4;  // channels of the tile and of a wave
    static_assert(!TWO || NF == 2, "a fragment of either weight");
    constexpr int S = units_ahead<MT>(), D = stages_ahead<MT>(), UNIT = MT * 4096;
    typedef typename Half<T>::vec8 vec8;

    extern __shared__ u32x4_t lds_raw[];
    FFN_LDS uint8_t *lds = (FFN_LDS uint8_t *)lds_raw;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int h = lane >> 5, r = lane & 31;
    const int K = a.K, N = a.N;
    const Tile tile =
        find_tile<BM>(a, (N + BN - 1) / BN, reinterpret_cast<int *>(reinterpret_cast<char *>(lds_raw) + tile_lds<MT, NF, OUT>() - 32));
    if (tile.e < 0)
        return;

    // Whatever is past an end (rows of the tile, channels, columns, stages) is
    // loaded with an offset past its buffer, which gives zeros.
    const int whole = K / kStageCols, stages = (K + kStageCols - 1) / kStageCols;
    const int rest = K - whole * kStageCols;  // columns of a last stage that is not whole
    // This lane's 16-byte pieces of the activations: piece P = 64 i + lane of
    // the wave's, of row P / 8 of the tile, piece c = (P % 8) ^ (row / 2 % 8) of a
    // unit: columns 64 (c / 4) + 8 (c % 4) of a stage, 32 further on in its second unit.
    uint32_t x_at[MT];
    int x_col[MT];
    const T *x_from[WIDE ? MT : 1];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const int m = (wave * MT + i) * 8 + (lane >> 3);
        const int c = (lane & 7) ^ ((m >> 1) & 7);
        const bool there = tile.begin + m < tile.end;
        const int row = !there ? 0 : a.rows ? min(max(a.rows[tile.begin + m], 0) / a.top_k, a.x_rows - 1) : m;
        x_col[i] = 64 * (c >> 2) + 8 * (c & 3);
        x_at[i] = there ? static_cast<uint32_t>(row) * (2 * K) + 2 * x_col[i] : kPast;
        if constexpr (WIDE)
            x_from[i] = there ? static_cast<const T *>(a.x) + static_cast<size_t>(row) * K + x_col[i] : nullptr;
    }
    const T *x_base = static_cast<const T *>(a.x) + (a.rows ? size_t{0} : static_cast<size_t>(tile.begin) * K);
    const auto x_buffer =
        uniform_buffer(x_base, a.rows ? static_cast<int>(static_cast<uint32_t>(a.x_rows) * (2 * K)) : 2 * BM * K);
    const auto direct = [&](const __amdgpu_buffer_rsrc_t &from, int to, uint32_t at, int offset) {
        __builtin_amdgcn_raw_ptr_buffer_load_lds(from, reinterpret_cast<FFN_LDS void *>(lds + to), 16, at, offset, 0, 0);
    };
    const auto load_x = [&](int s, int v, int slot) {
        const int to = slot * UNIT + wave * MT * 1024;
        const int most = (s < whole ? kStageCols : s < stages ? rest : 0) - v * 32;
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const bool there = x_col[i] < most;
            if constexpr (WIDE) {
                const uintptr_t from = there && x_from[i] ? reinterpret_cast<uintptr_t>(x_from[i] + s * kStageCols + v * 32)
                                                          : reinterpret_cast<uintptr_t>(&kZeros);
                __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)from,
                                                 reinterpret_cast<FFN_LDS void *>(lds + to + i * 1024), 16, 0, 0);
            } else {
                direct(x_buffer, to + i * 1024, there ? x_at[i] : kPast, s * 256 + v * 64);
            }
        }
    };
    // The weights: lane (h, r) holds columns 64 h + 32 v .. + 31 of a stage's unit
    // v, of row r of a fragment. Its four scale bytes of a stage come with those
    // of three more: lane (h, r) loads bytes 16 h .. + 15 of a row's 32, and the
    // halves of the wave swap what is the other's.
    const int row_codes = K / 2, row_scales = K / 16;
    const int n0 = tile.nt * BN + wave * WR;  // the wave's first channel
    const auto rows_of_weight = [&](const uint8_t *m, int first, int row_bytes) {
        return uniform_buffer(m + (static_cast<size_t>(tile.e) * N + first) * row_bytes,
                              min(max(N - first, 0), 32) * row_bytes);
    };
    __amdgpu_buffer_rsrc_t codes[NF], scales[NF];
#pragma unroll
    for (int f = 0; f < NF; ++f) {
        const int first = n0 + (TWO ? 0 : 32 * f);
        codes[f] = rows_of_weight(TWO && f == 1 ? a.w1.codes : a.w0.codes, first, row_codes);
        scales[f] = rows_of_weight(TWO && f == 1 ? a.w1.scales : a.w0.scales, first, row_scales);
    }
    const uint32_t code_at = r * row_codes + 32 * h, scale_at = r * row_scales + 16 * h;
    u32x4_t code[D][NF][2];  // stage, fragment, unit
    const auto load_w = [&](int s, int slot) {
        const int most = (s < whole ? kStageCols : s < stages ? rest : 0) - 64 * h;
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            const uint32_t at = 32 * v < most ? code_at + 16 * v : kPast;
#pragma unroll
            for (int f = 0; f < NF; ++f)
                code[slot][f][v] = __builtin_amdgcn_raw_buffer_load_b128(codes[f], at, s * 64, 0);
        }
    };
    u32x4_t scale[NF], scale_next[NF];  // of four stages
    const auto load_scales = [&](int s) {
#pragma unroll
        for (int f = 0; f < NF; ++f)
            scale_next[f] = __builtin_amdgcn_raw_buffer_load_b128(scales[f], scale_at, s * 8, 0);
    };
    const auto take_scales = [&]() {
#pragma unroll
        for (int f = 0; f < NF; ++f)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                uint32_t lo = scale_next[f][2 * i], hi = scale_next[f][2 * i + 1];
                swap_halves(lo, hi);
                scale[f][i] = lo;
                scale[f][2 + i] = hi;
            }
    };
    // Those of a last stage that is not whole: the bounds check, made for each four
    // bytes, would drop the last two of an odd number of rows.
    uint32_t last_scale[NF] = {};
    if (rest) {
#pragma unroll
        for (int f = 0; f < NF; ++f) {
            const uint32_t at = r * row_scales + whole * 8 + 4 * h;
            const uint32_t lo = __builtin_amdgcn_raw_buffer_load_b16(scales[f], 64 * h < rest ? at : kPast, 0, 0);
            const uint32_t hi = __builtin_amdgcn_raw_buffer_load_b16(scales[f], 64 * h + 32 < rest ? at + 2 : kPast, 0, 0);
            last_scale[f] = lo | hi << 16;
        }
    }

    f32x16_t acc[NF][MT];
#pragma unroll
    for (int f = 0; f < NF; ++f)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
            acc[f][mt] = f32x16_t{};
    // A unit's products, of the first R fragments of rows.
    const auto multiply = [&](auto fragments, int v, int slot, const u32x4_t (&q)[NF][2], const uint32_t (&sc)[NF]) {
        constexpr int R = decltype(fragments)::value;
        const FFN_LDS uint8_t *x = lds + slot * UNIT;
        float s[NF][2];
#pragma unroll
        for (int f = 0; f < NF; ++f) {
            s[f][0] = v ? e4m3_to_f32<2>(sc[f]) : e4m3_to_f32<0>(sc[f]);
            s[f][1] = v ? e4m3_to_f32<3>(sc[f]) : e4m3_to_f32<1>(sc[f]);
        }
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            vec8 w[NF];
#pragma unroll
            for (int f = 0; f < NF; ++f)
                w[f] = Half<T>::weights(q[f][v][t], s[f][t >> 1]);
#pragma unroll
            for (int mt = 0; mt < R; ++mt) {
                const int m = 32 * mt + r;
                const vec8 xv = *reinterpret_cast<const FFN_LDS vec8 *>(x + m * 128 + (((4 * h + t) ^ ((m >> 1) & 7)) * 16));
#pragma unroll
                for (int f = 0; f < NF; ++f)
                    acc[f][mt] = Half<T>::mfma(xv, w[f], acc[f][mt]);
            }
        }
    };

    const auto run = [&](auto fragments) {
        load_scales(0);
#pragma unroll
        for (int u = 0; u < S - 1; ++u) {
            if (u % 2 == 1 && u / 2 < D - 1)
                load_w(u / 2, u / 2);
            load_x(u / 2, u % 2, u);
            __builtin_amdgcn_sched_barrier(0);  // (in this order: the waits below count on it)
        }
        static_assert(S == 2 * D && 4 % D == 0, "every round has the rings' places alike");
        for (int s0 = 0; s0 < stages; s0 += 4) {
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int s = s0 + u / 2, v = u % 2;
                if (v == 0 && s >= stages)
                    break;
                // This unit's activations have landed here once at most the loads
                // of the S - 2 units after them are in flight (and the weights of
                // every other one), and in every wave behind the barrier, where
                // all are done with the unit before. (In whichever order a step's
                // loads are issued, no fewer than these are younger.)
                wait_vmcnt<(S - 2) * MT + (S - 2) / 2 * 2 * NF>();
                lds_barrier();
                if (u == 0) {
                    take_scales();
                    load_scales(s + 4);
                }
                if (v == 0)
                    load_w(s + D - 1, (u / 2 + D - 1) % D);
                const int next = u + S - 1;
                load_x(s0 + next / 2, next % 2, next % S);
                uint32_t sc[NF];
#pragma unroll
                for (int f = 0; f < NF; ++f)
                    sc[f] = s < whole ? scale[f][u / 2] : last_scale[f];
                multiply(fragments, v, u % S, code[(u / 2) % D], sc);
            }
        }
    };
    // A tile of fewer rows takes as many products as it needs.
    const int rows = tile.end - tile.begin;
    if (MT >= 2 && rows <= 32)
        run(std::integral_constant<int, 1>{});
    else if (MT >= 4 && rows <= 64)
        run(std::integral_constant<int, (MT >= 4 ? 2 : 1)>{});
    else
        run(std::integral_constant<int, MT>{});

    // Results go through LDS, so that the channels of a row leave as whole lines
    // (two bytes a lane straight from the accumulators: 15 - 28 us a tile for
    // 2 - 4). Value 4 g + c of acc[f][mt] is row 32 mt + 8 g + 4 h + c, weight row r
    // of fragment f. The padding of a row keeps both halves of a wave apart.
    typedef typename std::conditional<OUT == MOE_F32, float, T>::type Out;
    constexpr int PASS = out_pass<MT, OUT>(), ROW = out_row_bytes<NF, OUT>();
    constexpr int EACH = 16 / sizeof(Out), PIECES = BN / EACH;  // pieces of 16 bytes of a row
    const float s0 = a.w0.scale2[tile.e], s1 = TWO ? a.w1.scale2[tile.e] : s0;
    Out *out = static_cast<Out *>(a.out);
    wait_vmcnt<0>();  // (also of loads behind the last unit)
#pragma unroll
    for (int mt0 = 0; mt0 < MT; mt0 += PASS) {
        lds_barrier();
#pragma unroll
        for (int mt = mt0; mt < mt0 + PASS; ++mt)
#pragma unroll
            for (int v = 0; v < 16; ++v) {
                const int i = 32 * (mt - mt0) + 8 * (v >> 2) + 4 * h + (v & 3);
                FFN_LDS Out *to = reinterpret_cast<FFN_LDS Out *>(lds + i * ROW) + wave * WR + r;
                const float y0 = acc[0][mt][v], y1 = acc[NF - 1][mt][v];
                *to = static_cast<Out>(moe_value<OUT>(y0, y1, s0, s1));
                if constexpr (!TWO && NF == 2)
                    to[32] = static_cast<Out>(moe_value<OUT>(y1, 0.0f, s0, s1));
            }
        lds_barrier();
        const int first = tile.begin + 32 * mt0, most = min(32 * PASS, tile.end - first);
        if (N % EACH == 0) {
            const int n = static_cast<int>(threadIdx.x) % PIECES * EACH, to = tile.nt * BN + n;
            for (int i = threadIdx.x / PIECES; i < most; i += kThreads / PIECES)
                if (to < N)
                    *reinterpret_cast<u32x4_t *>(out + static_cast<size_t>(first + i) * N + to) =
                        *reinterpret_cast<const FFN_LDS u32x4_t *>(lds + i * ROW + n * sizeof(Out));
        } else {
            const int n = static_cast<int>(threadIdx.x) % BN, to = tile.nt * BN + n;
            for (int i = threadIdx.x / BN; i < most; i += kThreads / BN)
                if (to < N)
                    out[static_cast<size_t>(first + i) * N + to] =
                        reinterpret_cast<const FFN_LDS Out *>(lds + i * ROW)[n];
        }
    }
}

// The most tiles that R rows make: every expert with rows may have one that is not
// full.
inline long most_tiles(const MoeGemmArgs &a, int BM, int BN)
{
    return (a.R / BM + static_cast<long>(a.R < a.E ? a.R : a.E)) * ((a.N + BN - 1) / BN);
}

template <class T, int MT, int NF, int OUT, bool WIDE = false>
hipError_t launch_tiles(const MoeGemmArgs &a, hipStream_t stream)
{
    constexpr int BM = 32 * MT, BN = tile_channels<NF, OUT>(), lds = tile_lds<MT, NF, OUT>();
    auto kern = moe_tile_kernel<T, MT, NF, OUT, WIDE>;
    static std::atomic<uint64_t> lds_done{0};
    const hipError_t e = allow_lds(reinterpret_cast<const void *>(kern), lds, lds_done);
    if (e != hipSuccess)
        return e;
    const long grid = (most_tiles(a, BM, BN) + 7) / 8 * 8;
    hipLaunchKernelGGL(kern, dim3(grid), dim3(kThreads), lds, stream, a);
    return hipGetLastError();
}

template <class T, int OUT>
hipError_t launch_out(const MoeGemmArgs &a, hipStream_t stream)
{
    // Which kernel, by the mean rows of an expert; us at experts x mean rows, bf16,
    // rows gathered. Three counts each: all experts alike / as random logits choose /
    // as such logits with a popularity of their own deviation for each expert choose.
    //                             few rows        32 x 256        64 x 256        128 x 256
    //   64 x 8,  5120 -> 2048    93/ 98/ 79     107/105/ 84     107/106/ 93     113/114/103
    //   64 x 16, 5120 -> 2048    92/121/114     104/104/126     108/107/103     116/115/125
    //   64 x 16, 2048 -> 5120    87/104/ 97      99/100/ 95     102/103/ 97     110/111/100
    //  128 x 16, 2048 -> 1024    36/ 49/ 47      40/ 41/ 47      41/ 41/ 39      44/ 45/ 49
    //   64 x 20, 5120 -> 2048   146/148/134     103/103/126     106/106/107     117/116/130
    //   64 x 24, 5120 -> 2048   151/150/155     105/105/130     107/108/105     117/117/132
    //   64 x 32, 5120 -> 2048   150/196/189     109/145/162     109/113/146     118/120/147
    //   64 x 32, 2048 -> 5120   135/175/169     107/139/130     110/113/119     115/121/131
    //  128 x 32, 2048 -> 1024    57/ 71/ 72      42/ 51/ 57      42/ 45/ 55      44/ 47/ 57
    //   64 x 64, 5120 -> 2048                   169/202/217     125/168/188     137/154/197
    //   64 x 96, 5120 -> 2048                   234/261/281     200/203/225     180/176/211
    //   64 x 128, 2048 -> 5120                  297/329/334     224/260/263     192/245/241
    // A router's counts scatter, so from a mean of about 24 on many experts need a
    // second tile of 32 rows. At 16 they need a second one of the stream's 16, and tiles
    // would be up to a sixth faster there on scattered counts, but slower on even
    // ones and at 8. Where the large tiles are fewer than the compute units, smaller
    // ones (from a mean of 25 on; 8 x 20, 4096 -> 2048 would be 25 on 64 x 128 and 23 by
    // the stream for the 34 of 32 x 256): 8 x 200, 2048 -> 1024: 34.7 us with 128 x 256,
    // 24.9 with 64 x 256, 20.6 with 64 x 128, 21.0 with 32 x 128; 64 x 128, 2048 ->
    // 5120, which has enough: 207 with 128 x 256, 227 with 128 x 128.
    if (stream_fits<moe_two_weights(OUT)>(a.R, a.E, a.K, a.N))
        return launch_moe_stream<T, false, OUT>(a, stream);
    // (rows of x past 32-bit offsets: a 64-row variant only)
    if (a.rows && static_cast<uint64_t>(a.x_rows) * a.K * 2 >= kPast)
        return launch_tiles<T, 2, 2, OUT, true>(a, stream);
    const int mean = a.R / a.E, cus = device_cu_count();
    constexpr int BN = tile_channels<2, OUT>();
    if (mean > 64 && most_tiles(a, 128, BN) >= cus)
        return launch_tiles<T, 4, 2, OUT>(a, stream);
    if constexpr (!moe_two_weights(OUT))
        if (mean > 24 && most_tiles(a, 64, BN) < cus)
            return launch_tiles<T, 2, 1, OUT>(a, stream);
    if (mean > 24)
        return launch_tiles<T, 2, 2, OUT>(a, stream);
    return launch_tiles<T, 1, 2, OUT>(a, stream);
}

template <class T, int OUT>
hipError_t launch_either(const MoeGemmArgs &a, hipStream_t stream)
{
    if constexpr (OUT != MOE_SAME)
        if (a.ids)
            return launch_moe_stream<T, true, OUT>(a, stream);
    return launch_out<T, OUT>(a, stream);
}

template <class T>
hipError_t launch_type(const MoeGemmArgs &a, MoeOut out, hipStream_t stream)
{
    switch (out) {
    case MOE_SAME:
        return launch_either<T, MOE_SAME>(a, stream);
    case MOE_F32:
        return launch_either<T, MOE_F32>(a, stream);
    case MOE_H_SILU:
        return launch_either<T, MOE_H_SILU>(a, stream);
    default:
        return launch_either<T, MOE_H_GELU>(a, stream);
    }
}

}  // namespace

bool moe_by_slots(int R, int E, int K, int N)
{
    return R <= kStreamSlots && stream_fits<true>(R, E, K, N) && stream_fits<false>(R, E, N, K);
}

hipError_t launch_moe_gemm(const MoeGemmArgs &a, int dtype, MoeOut out, hipStream_t stream)
{
    return dtype == kMoeBf16 ? launch_type<__bf16>(a, out, stream) : launch_type<_Float16>(a, out, stream);
}

}  // namespace ffn
