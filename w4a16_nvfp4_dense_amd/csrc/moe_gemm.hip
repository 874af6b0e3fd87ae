// moe_gemm.hip -- the product grouped by expert over NVFP4 weights, on tiles of
// tokens and channels, for any number of rows of each expert.
//
// Mathematics. Rows offsets[e] .. offsets[e + 1] - 1 of the product are
// scale2[e] W_e x, with W_e = e2m1 * e4m3. A weight has at most six significant
// bits and exponents from -10 to 12, so it is exact in bf16 and in f16, and
// the only rounding in a sum is that of the matrix core's fp32 accumulation.
//
// Tiles. A tile is 32 MT rows of one expert by 256 weight rows (128 channels of
// two weights). How many tiles an expert has is known on the device only, so
// the grid is the most there can be, and each workgroup finds its tile from the
// offsets (a scan over experts); workgroups past the last tile end at once.
// Tiles are numbered expert by expert, the rows fastest, and dealt to the eight
// XCDs in runs, so that an XCD's L2 holds what its tiles share.
//
// A workgroup has four waves; each dequantises 64 weight rows of the tile (32
// of either weight) and multiplies them with all its rows.
// Columns go by stages of 128 (weights) in two units of 64 (activations). In
// stage s, unit v and step t (of four), lane half h = lane / 32 holds columns
// 128 s + 64 h + 32 v + 8 t .. + 7 of either operand: a lane's weights of a
// stage are then 64 consecutive columns with four scale bytes.
//
// Activations and codes come through LDS by direct loads of 16 bytes a lane,
// two units and two stages deep, the 16-byte pieces swizzled so that reads meet
// no bank twice; scales come in registers, a stage ahead.
#include <hip/hip_runtime.h>

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

template <int MT>
constexpr int unit_bytes()
{
    return MT * 4096;  // activations of a unit
}
constexpr int kStageBytes = 256 * 64;  // codes of a stage
template <int MT>
constexpr int tile_lds()
{
    return 2 * unit_bytes<MT>() + 2 * kStageBytes + 32;
}

template <class T, int MT, int OUT>
__global__ __launch_bounds__(kThreads, 2) void moe_tile_kernel(const MoeGemmArgs a)
{
    constexpr bool TWO = moe_two_weights(OUT);
    constexpr int BM = 32 * MT;
    constexpr int WR = TWO ? 32 : 64;     // channels of a wave
    constexpr int BN = 4 * WR;
    typedef typename Half<T>::vec8 vec8;
    constexpr int LOADS_W = 4;            // direct loads of a stage's codes, for each wave

    extern __shared__ u32x4_t lds_raw[];
    FFN_LDS uint8_t *lds = (FFN_LDS uint8_t *)lds_raw;
    constexpr int XRING = 2 * unit_bytes<MT>();
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int h = lane >> 5, r = lane & 31;
    const int K = a.K, N = a.N;
    const Tile tile = find_tile<BM>(a, (N + BN - 1) / BN,
                                    reinterpret_cast<int *>(reinterpret_cast<char *>(lds_raw) + XRING + 2 * kStageBytes));
    if (tile.e < 0)
        return;

    // This lane's 16-byte pieces of the activations: piece P = 64 i + lane of
    // the wave's, of row P / 8 of the tile, piece (P % 8) ^ (row / 2 % 8) of a
    // unit, which are columns 64 (piece / 4) + 8 (piece % 4) of it.
    const T *xp[MT];
    int xcol[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const int m = (wave * MT + i) * 8 + (lane >> 3);
        const int c = (lane & 7) ^ ((m >> 1) & 7);
        int row = min(tile.begin + m, tile.end - 1);
        if (a.rows)
            row = min(max(a.rows[row], 0) / a.top_k, a.x_rows - 1);
        xcol[i] = 64 * (c >> 2) + 8 * (c & 3);
        xp[i] = static_cast<const T *>(a.x) + static_cast<size_t>(row) * K + xcol[i];
    }
    // Its pieces of the codes: piece j of four, of row 16 j + lane / 4 of the
    // wave's 64, columns 32 ((lane % 4) ^ (row / 4 % 4)) .. of a stage.
    const size_t row_codes = static_cast<size_t>(K) / 2, row_scales = static_cast<size_t>(K) / 16;
    const size_t expert = static_cast<size_t>(tile.e) * N;
    const auto channel = [&](int i) {  // of weight row i of the wave
        return min(tile.nt * BN + wave * WR + (TWO ? i & 31 : i), N - 1);
    };
    const uint8_t *wp[4];
    int wcol[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int i = 16 * j + (lane >> 2);
        const int c = (lane & 3) ^ ((i >> 2) & 3);
        const uint8_t *codes = TWO && j >= 2 ? a.w1.codes : a.w0.codes;
        wcol[j] = 32 * c;
        wp[j] = codes + (expert + channel(i)) * row_codes + 16 * c;
    }
    const uint8_t *sp[2];
#pragma unroll
    for (int f = 0; f < 2; ++f) {
        const uint8_t *scales = TWO && f == 1 ? a.w1.scales : a.w0.scales;
        sp[f] = scales + (expert + channel(32 * f + r)) * row_scales + 4 * h;
    }

    // Of a last stage of fewer columns, pieces past the end are loaded from zeros.
    const auto load_x = [&](int s, int v) {
        FFN_LDS uint8_t *to = lds + v * unit_bytes<MT>() + wave * MT * 1024;
        const int k0 = s * kStageCols + v * 32;
        const bool whole = (s + 1) * kStageCols <= K;
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const void *from = xp[i] + k0;
            if (!whole && k0 + xcol[i] >= K)
                from = &kZeros;
            __builtin_amdgcn_global_load_lds(from, reinterpret_cast<FFN_LDS void *>(to + i * 1024), 16, 0, 0);
        }
    };
    uint32_t scale_next[2];
    const auto load_w = [&](int s) {
        FFN_LDS uint8_t *to = lds + XRING + (s & 1) * kStageBytes + wave * 4096;
        const int k0 = s * kStageCols;
        const bool whole = k0 + kStageCols <= K;
        if (whole) {
#pragma unroll
            for (int f = 0; f < 2; ++f)
                scale_next[f] = reinterpret_cast<const pair16_t *>(sp[f] + s * 8)->both;
        } else {
#pragma unroll
            for (int f = 0; f < 2; ++f) {
                const uint16_t *p = reinterpret_cast<const uint16_t *>(sp[f] + s * 8);
                const uint32_t lo = k0 + 64 * h < K ? p[0] : 0, hi = k0 + 64 * h + 32 < K ? p[1] : 0;
                scale_next[f] = lo | hi << 16;
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const void *from = wp[j] + k0 / 2;
            if (!whole && k0 + wcol[j] >= K)
                from = &kZeros;
            __builtin_amdgcn_global_load_lds(from, reinterpret_cast<FFN_LDS void *>(to + j * 1024), 16, 0, 0);
        }
    };

    f32x16_t acc[2][MT];
#pragma unroll
    for (int f = 0; f < 2; ++f)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
            acc[f][mt] = f32x16_t{};
    uint32_t scale[2];
    const auto multiply = [&](int s, int v) {
        const FFN_LDS uint8_t *codes = lds + XRING + (s & 1) * kStageBytes + wave * 4096;
        const FFN_LDS uint8_t *x = lds + v * unit_bytes<MT>();
        u32x4_t q[2];
        float sc[2][2];
#pragma unroll
        for (int f = 0; f < 2; ++f) {
            const int i = 32 * f + r;
            q[f] = *reinterpret_cast<const FFN_LDS u32x4_t *>(codes + i * 64 + (((2 * h + v) ^ ((i >> 2) & 3)) * 16));
            const uint32_t two = scale[f] >> (16 * v);
            sc[f][0] = e4m3_to_f32<0>(two);
            sc[f][1] = e4m3_to_f32<1>(two);
        }
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            vec8 w[2];
#pragma unroll
            for (int f = 0; f < 2; ++f)
                w[f] = Half<T>::weights(q[f][t], sc[f][t >> 1]);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                const int m = 32 * mt + r;
                const vec8 xv = *reinterpret_cast<const FFN_LDS vec8 *>(x + m * 128 + (((4 * h + t) ^ ((m >> 1) & 7)) * 16));
                acc[0][mt] = Half<T>::mfma(xv, w[0], acc[0][mt]);
                acc[1][mt] = Half<T>::mfma(xv, w[1], acc[1][mt]);
            }
        }
    };

    const int stages = (K + kStageCols - 1) / kStageCols;
    load_w(0);
    load_x(0, 0);
    for (int s = 0; s < stages; ++s) {
        wait_vmcnt<0>();
        lds_barrier();
        scale[0] = scale_next[0];
        scale[1] = scale_next[1];
        load_x(s, 1);
        if (s + 1 < stages)
            load_w(s + 1);
        multiply(s, 0);
        if (s + 1 < stages)
            wait_vmcnt<LOADS_W>();
        else
            wait_vmcnt<0>();
        lds_barrier();
        if (s + 1 < stages)
            load_x(s + 1, 0);
        multiply(s, 1);
    }

    // Value 4 g + c of acc[f][mt]: row 32 mt + 8 g + 4 h + c, weight row r of
    // fragment f.
    const float s0 = a.w0.scale2[tile.e], s1 = TWO ? a.w1.scale2[tile.e] : s0;
    const int n0 = tile.nt * BN + wave * WR + r;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int v = 0; v < 16; ++v) {
            const int i = tile.begin + 32 * mt + 8 * (v >> 2) + 4 * h + (v & 3);
            if (i >= tile.end)
                continue;
            const float y0 = acc[0][mt][v], y1 = acc[1][mt][v];
            const size_t o = static_cast<size_t>(i) * N + n0;
            if (n0 < N)
                moe_store<T, OUT>(a.out, o, moe_value<OUT>(y0, y1, s0, s1));
            if (!TWO && n0 + 32 < N)
                moe_store<T, OUT>(a.out, o + 32, moe_value<OUT>(y1, 0.0f, s0, s1));
        }
}

template <class T, int MT, int OUT>
hipError_t launch_tiles(const MoeGemmArgs &a, hipStream_t stream)
{
    constexpr int BM = 32 * MT, BN = moe_two_weights(OUT) ? 128 : 256;
    auto kern = moe_tile_kernel<T, MT, OUT>;
    static std::atomic<uint64_t> lds_done{0};
    const hipError_t e = allow_lds(reinterpret_cast<const void *>(kern), tile_lds<MT>(), lds_done);
    if (e != hipSuccess)
        return e;
    // The most tiles of rows that R rows make: every expert with rows may have
    // one that is not full.
    const long most = a.R / BM + (a.R < a.E ? a.R : a.E);
    const long grid = (most * ((a.N + BN - 1) / BN) + 7) / 8 * 8;
    hipLaunchKernelGGL(kern, dim3(grid), dim3(kThreads), tile_lds<MT>(), stream, a);
    return hipGetLastError();
}

template <class T, int OUT>
hipError_t launch_out(const MoeGemmArgs &a, hipStream_t stream)
{
    if (a.R <= kStreamRows * a.E && stream_fits(a.E, a.K, a.N))
        return launch_moe_stream<T, false, OUT>(a, stream);
    const int mean = a.R / a.E;  // rows of an expert
    if (mean > 64)
        return launch_tiles<T, 4, OUT>(a, stream);
    if (mean > 24)
        return launch_tiles<T, 2, OUT>(a, stream);
    return launch_tiles<T, 1, OUT>(a, stream);
}

template <class T, int OUT>
hipError_t launch_either(const MoeGemmArgs &a, hipStream_t stream)
{
    if constexpr (OUT != MOE_F32)
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
    return R <= kStreamSlots && R <= kStreamRows * E && stream_fits(E, K, N) && stream_fits(E, N, K);
}

hipError_t launch_moe_gemm(const MoeGemmArgs &a, int dtype, MoeOut out, hipStream_t stream)
{
    return dtype == kMoeBf16 ? launch_type<__bf16>(a, out, stream) : launch_type<_Float16>(a, out, stream);
}

}  // namespace ffn
