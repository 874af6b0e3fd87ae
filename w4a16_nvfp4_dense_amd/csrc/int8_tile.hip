// int8_tile.hip -- the int8 product on tiles of tokens and channels, both
// operands staged through LDS, by one persistent workgroup for each compute
// unit.
//
// Mathematics. out[m, n] = xs[m] s[n] sum_k x[m, k] w[n, k] with exact int32
// sums, so a reduction may be cut anywhere and added in any order.
//
// What bounds it: the weight stream for few tokens, the matrix instructions
// (2 M N K operations) for many, at the clock that the card's power leaves
// them: 1.4 - 1.7 GHz in long runs, where products without any loads reach
// 2450 - 2640 TOPS. In short runs at 2.1 GHz the matrix cores are busy 57% of the
// time, and LDS reads and writes take as many cycles as the products. Measured
// on one MI355X, weights not in a cache at M <= 128 (K/N; "dual" with h):
//   M = 1     dual 5120/17408  32.2 - 32.6 us, 178 MB: 5.5 TB/s
//             17408/5120, h quantised here too  19.5 - 21.8 us, 89 MB: 4.1 -
//             4.6 TB/s; 5120/17408 18.0 us
//   M = 32    dual 5376/21504  46.4 - 47.2 us, 231 MB: 5.0 TB/s
//             21504/5376       27.0 us, 116 MB: 4.3 TB/s
//   M = 128   dual 5120/17408  53.0 - 53.9 us, 860 TOPS; 17408/5120 33.2 us
//   M = 300   4112/4099 fp32   21.2 us, 478 TOPS
//   M = 2048  dual 5120/17408  369 - 388 us, 1880 - 1980 TOPS; 17408/5120
//             184 - 193 us, 1890 - 1980 TOPS
//   M = 4096  5120/17408       346 us, 2110 TOPS (4 waves of 128 x 128 instead
//             of 8 of 64 x 128, which read LDS less: 8% slower)
//
// Layout. A stage holds 128 columns of BM token rows and BN weight rows, 128
// bytes a row, written by direct global -> LDS loads of 16 bytes a lane (eight
// rows, whole 128-byte lines, for each wave instruction). Piece s of row i
// holds columns 16 (s ^ (i / 2 % 8)), chosen by the address each lane loads
// from, so the 16 lanes that read one column piece of 16 consecutive rows
// touch all 64 banks once. STAGES stages form a ring that runs on over the
// workgroup's tiles; one barrier for each stage.
//
// Work split (int8_split.h). Every workgroup takes whole tiles and then an equal
// share of the units of the tiles that are left, walked downwards: the tile that
// its share ends in the middle of comes first, the one that its share begins in
// the middle of last. The tile's last workgroup, which reaches it last in its
// walk, adds the sums that the others have written to the workspace to its own
// and stores the tile. It looks for them a bounded time; whatever is late then,
// some workgroup finishes the tile (part_words.h), so launches beside each other
// cannot hold each other up, and int32 sums give the same bits whoever adds
// them. (Every workgroup writing its sums, and the last one counted adding them:
// 1-2% slower at M <= 64; 44.2 us for 40.9 at M = 256, K = 5120, N = 17408.)
//
// A single token's real row (`row`, what is between the two products of a
// decoded token) is quantised by every workgroup for itself before its first
// stage, into LDS: the same codes as a launch of their own would give, without
// that launch.
#include <hip/hip_runtime.h>

#include <climits>

#include "int8.h"
#include "int8_device.h"
#include "int8_split.h"
#include "kernels.h"
#include "part_words_device.h"

// Every piece of the kernel is inlined: a closure left in memory would put the
// loop's state there.
#define FFN_INLINE __attribute__((always_inline))

namespace ffn {
namespace {

constexpr int kPieces = kBk / 16;        // 16-byte pieces of a row and stage
constexpr int kLoadRows = 64 / kPieces;  // rows of a direct load

// Swizzle of row i's pieces: the 16 lanes that read one piece of 16 consecutive
// rows touch all 64 banks once.
__device__ __forceinline__ int piece_swizzle(int i)
{
    return (i >> 1) & 7;
}

// The matrix instruction on fragments of F tokens x F channels (F = 16: 64
// columns at a time, F = 32: 32 columns). Lane l holds row l % F of either
// operand and the 16 bytes at piece l / F of a step; group g of its results
// is channel l % F of tokens 8 g + 4 (l / F) .. + 3.
template <int F>
struct Mfma;
template <>
struct Mfma<16> {
    typedef i32x4_t acc_t;
    static __device__ __forceinline__ void go(acc_t &c, const i32x4_t &x, const i32x4_t &w)
    {
        c = __builtin_amdgcn_mfma_i32_16x16x64_i8(x, w, c, 0, 0, 0);
    }
};
template <>
struct Mfma<32> {
    typedef int acc_t __attribute__((ext_vector_type(16)));
    static __device__ __forceinline__ void go(acc_t &c, const i32x4_t &x, const i32x4_t &w)
    {
        c = __builtin_amdgcn_mfma_i32_32x32x32_i8(x, w, c, 0, 0, 0);
    }
};
// A direct load of 16 bytes a lane to LDS, lane l to byte `at` + 16 l. Written in
// assembly because the compiler makes the next LDS read wait for every direct
// load that it knows of; here the waits are those of the ring. It has no
// output register, and the other waits stay right: the compiler's counts of
// loads in flight are at most too low, so its waits are at most too long. The
// wait states are those between a vector instruction's write of a scalar
// register, or a write of m0, and this.
template <bool NT>
__device__ __forceinline__ void load_to_lds(const u32x4_t &rsrc, uint32_t at, int offset, int scalar_offset)
{
    const auto scalar = [](uint32_t v) { return static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(v)); };
    const u32x4_t buffer = {scalar(rsrc[0]), scalar(rsrc[1]), scalar(rsrc[2]), scalar(rsrc[3])};
    if constexpr (NT)
        asm volatile("s_nop 4\n\tbuffer_load_dwordx4 %0, %1, %2 offen nt lds"
                     :
                     : "v"(offset), "s"(buffer), "s"(scalar(scalar_offset)), "{m0}"(scalar(at))
                     : "memory");
    else
        asm volatile("s_nop 4\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds"
                     :
                     : "v"(offset), "s"(buffer), "s"(scalar(scalar_offset)), "{m0}"(scalar(at))
                     : "memory");
}

template <class A>
__device__ __forceinline__ i32x4_t group_of(const A &c, int g)
{
    return i32x4_t{c[4 * g], c[4 * g + 1], c[4 * g + 2], c[4 * g + 3]};
}

// BM tokens x BN weight rows, WM x WN waves, fragments of F x F. A wave has
// FC fragments of channels; row c of fragment f is channel FC c + f of the
// wave's, so that a lane ends with FC consecutive channels of a token and a
// wave stores whole lines. For two weights each wave's rows are its channels of
// w0 followed by the same channels of w1. NT: the weights are read
// non-temporally. ROW: one token, given as its real row (a.row); the stages
// hold weights only, and its codes lie behind the ring.
template <int BM, int BN, int WM, int WN, int F, int STAGES, bool NT, int OUT, bool ROW>
__global__ __launch_bounds__(WM *WN * 64, 2) void int8_tile_kernel(Int8GemmArgs a, Split sp)
{
    constexpr bool TWO = int8_two_weights(OUT);
    constexpr int WAVES = WM * WN;
    constexpr int XR = ROW ? 0 : BM;                     // token rows of a stage
    constexpr int ROWS = XR + BN;
    constexpr int LOADS_ALL = ROWS / kLoadRows;          // direct loads of a stage
    constexpr int LOADS = (LOADS_ALL + WAVES - 1) / WAVES;  // the most of one wave
    constexpr int FULL = LOADS_ALL - (LOADS - 1) * WAVES;   // waves with LOADS; the others have one fewer
    constexpr int FM = BM / WM / F, FN = BN / WN / F;    // fragments of a wave
    constexpr int NG = F * F / 256;                      // groups of four results of a lane and fragment
    constexpr int STEPS = kBk * F / 1024;                // steps of a stage
    constexpr int WR = BN / WN;                          // weight rows of a wave
    constexpr int WC = TWO ? WR / 2 : WR;                // channels of a wave
    constexpr int BC = WC * WN;                          // channels of a tile
    constexpr int FC = WC / F;                           // fragments of channels of a wave
    constexpr int STAGE = ROWS * kBk;
    static_assert(XR % kLoadRows == 0 && WR % kLoadRows == 0 && WC % F == 0, "whole loads and fragments");
    extern __shared__ int8_t lds[];  // [STAGES][ROWS][kBk], tokens first

    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    __builtin_assume(wave >= 0 && wave < WAVES);
    const int r = lane % F, q = lane / F;
    const int wm = wave / WN, wn = wave % WN;
    const int K = a.K;
    const int G = gridDim.x, b = blockIdx.x;
    const int whole_k = K / kBk;  // stages of whole 128 columns

    // Load j of a wave covers rows (j * WAVES + wave) * kLoadRows .. of a stage, all
    // of the tokens, of w0 or of w1; lane l has one piece of row l / kPieces of
    // those. `off` is that piece's place in its matrix, from the first row of
    // the tile being loaded; rows past the end repeat the last one. (The
    // buffers' bounds check would stop a read past a matrix all the same.)
    const int lrow = lane / kPieces;
    const auto column = [&](int j) FFN_INLINE {
        return ((lane % kPieces) ^ piece_swizzle((j * WAVES + wave) * kLoadRows + lrow)) * 16;
    };
    // Tiles are numbered in bands of kBand tiles of tokens, the tokens fastest:
    // 32 neighbours (an XCD's share of a round) are at most 8 x 4 tiles.
    const auto tile_at = [&](int tile, int &m, int &n) FFN_INLINE {
        const int band = sp.by_band.divide(tile), in = tile - band * sp.by_band.d;
        const bool last = (band + 1) * kBand > sp.tiles_m;
        n = last ? sp.by_last_rows.divide(in) : sp.by_rows.divide(in);
        m = band * kBand + in - n * (last ? sp.by_last_rows.d : sp.by_rows.d);
    };
    const auto rows_from = [&](const int8_t *m, int row, int rows) FFN_INLINE {
        // base, stride 0, size (of a tile's rows at most), raw-buffer format (as raw_buffer)
        const uint64_t base = reinterpret_cast<uintptr_t>(m) + static_cast<uint64_t>(row) * K;
        return u32x4_t{static_cast<uint32_t>(base), static_cast<uint32_t>(base >> 32) & 0xFFFF,
                       static_cast<uint32_t>(min(rows - row, 256) * K), 0x00020000};
    };
    u32x4_t from_x, from_w0, from_w1;
    int off[LOADS];
    const auto aim = [&](int tile) FFN_INLINE {
        int m0, n0;
        tile_at(tile, m0, n0);
        m0 *= BM;
        n0 *= BC;
        from_x = rows_from(a.x, m0, a.M);
        from_w0 = rows_from(a.w0, n0, a.N);
        from_w1 = TWO ? rows_from(a.w1, n0, a.N) : from_w0;
#pragma unroll
        for (int j = 0; j < LOADS; ++j) {
            const int row = (j * WAVES + wave) * kLoadRows + lrow;
            const int i = row - XR, f = i % WR / F % FC;
            const int from = i < 0 ? min(row, a.M - 1 - m0) : min(i / WR * WC + i % F * FC + f, a.N - 1 - n0);
            off[j] = from * K + column(j);
        }
    };
    const auto source = [&](int j) FFN_INLINE {
        const int i = (j * WAVES + wave) * kLoadRows - XR;
        // (copies first: a choice between the variables would keep them in memory)
        const u32x4_t x = from_x, w0 = from_w0, w1 = from_w1;
        return i < 0 ? x : TWO && i % WR >= WC ? w1 : w0;
    };
    // Loads stage k into the ring at `to`. Of a last stage of fewer columns the
    // pieces past the end get an offset past the buffer, which reads as zeros.
    const auto issue = [&](int k, int to) FFN_INLINE {
        const uint32_t at = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((FFN_LDS int8_t *)lds)) + to;
        const auto load = [&](int j, int offset) FFN_INLINE {
            if (j == LOADS - 1 && wave >= FULL)
                return;
            const uint32_t rows = at + (j * WAVES + wave) * kLoadRows * kBk;
            if (NT && (j * WAVES + wave) * kLoadRows >= XR)
                load_to_lds<NT>(source(j), rows, offset, k * kBk);
            else
                load_to_lds<false>(source(j), rows, offset, k * kBk);
        };
        if (k < whole_k) {
#pragma unroll
            for (int j = 0; j < LOADS; ++j)
                load(j, off[j]);
        } else {
#pragma unroll
            for (int j = 0; j < LOADS; ++j)
                load(j, k * kBk + column(j) < K ? off[j] : INT_MIN);
        }
    };

    typename Mfma<F>::acc_t acc[FN][FM];
    const auto clear = [&]() FFN_INLINE {
#pragma unroll
        for (int f = 0; f < FN; ++f)
#pragma unroll
            for (int t = 0; t < FM; ++t)
                acc[f][t] = typename Mfma<F>::acc_t{};
    };

    // row i, piece p of a stage at i * kBk + (p ^ swizzle(i)) * 16; the
    // swizzle of a fragment's row is that of r (fragments start at multiples
    // of 16), and a step's number is in the bits of p above q's
    const int frag = r * kBk + ((q ^ piece_swizzle(r)) * 16);
    const int xoff = wm * (BM / WM) * kBk + frag;
    const int woff = (XR + wn * WR) * kBk + frag;
    typedef i32x4_t Weights[FN];
    typedef i32x4_t Tokens[FM];
    const auto read = [&](int st, int k, int s, Weights &w, Tokens &x) FFN_INLINE {
        const int flip = s * (1024 / F);
#pragma unroll
        for (int f = 0; f < FN; ++f)
            w[f] = *reinterpret_cast<const i32x4_t *>(lds + st + (woff ^ flip) + f * F * kBk);
#pragma unroll
        for (int t = 0; t < FM; ++t)
            x[t] = *reinterpret_cast<const i32x4_t *>(
                ROW ? lds + STAGES * STAGE + k * kBk + (q + s * (64 / F)) * 16
                    : lds + st + (xoff ^ flip) + t * F * kBk);
    };
    const auto products = [&](const Weights &w, const Tokens &x, int f0, int f1) FFN_INLINE {
#pragma unroll
        for (int f = f0; f < f1; ++f)
#pragma unroll
            for (int t = 0; t < FM; ++t)
                Mfma<F>::go(acc[f][t], x[t], w[f]);
    };

    const auto slot_at = [&](int f, int t, int g) FFN_INLINE {
        return (((wave * FN + f) * FM + t) * NG + g) * 1024 + lane * 16;
    };
    const auto slot_of = [&](int number) FFN_INLINE {
        return raw_buffer(sp.part + static_cast<size_t>(number) * (BM * BN), BM * BN * 4);
    };
    // Tokens in a tile from this lane's first one on; the sums of others are not
    // kept.
    const auto tokens_of = [&](int tile) FFN_INLINE {
        int m, n;
        tile_at(tile, m, n);
        return a.M - (m * BM + wm * (BM / WM) + 4 * q);
    };
    // This workgroup's sums of a tile that it shares, to its slot.
    const auto publish = [&](int tile, int number) FFN_INLINE {
        const auto mine = slot_of(number);
        const int tokens = tokens_of(tile);
#pragma unroll
        for (int t = 0; t < FM; ++t)
#pragma unroll
            for (int g = 0; g < NG; ++g)
                if (F * t + 8 * g < tokens)
#pragma unroll
                    for (int f = 0; f < FN; ++f)
                        store_device_coherent(mine, slot_at(f, t, g),
                                              __builtin_bit_cast(f32x4_t, group_of(acc[f][t], g)));
        wait_vmcnt<0>();
        lds_barrier();  // every wave's stores have completed
    };
    // What the first wave finds, to every thread. (16 bytes behind the ring and
    // a row's codes; two uses have a barrier between them.)
    const int note_at = STAGES * STAGE + (ROW ? sp.stages * kBk : 0);
    const auto agree = [&](auto find) FFN_INLINE {
        int *note = reinterpret_cast<int *>(lds + note_at);
        if (wave == 0) {
            const bool found = find();
            if (lane == 0)
                *note = found;
        }
        lds_barrier();
        return __builtin_amdgcn_readfirstlane(*note) != 0;
    };
    // Whether this workgroup, with its part of a tile that `in` share, finishes the
    // tile: then the others' sums are in their slots.
    const auto take = [&](int tile, const Sharers &in) FFN_INLINE {
        const int parts = in.last - in.first + 1;
        const auto word = [&](int i) FFN_INLINE {
            return PartWord{sp.words + slot_number(sp, in, in.first + i)};
        };
        bool mine = b == in.last && agree([&]() FFN_INLINE { return all_come(word, parts - 1, sp.tag); });
        if (!mine) {
            publish(tile, slot_number(sp, in, b));
            mine = agree([&]() FFN_INLINE {
                if (lane != 0)
                    return false;
                return b == in.last ? last_gives_up(word, word(parts - 1), sp.tag, parts)
                                    : word(b - in.first).swap(marked(sp.tag)) == given_up(sp.tag) &&
                                          late_part(word(parts - 1), sp.tag, parts);
            });
        }
        if (mine && threadIdx.x < parts)
            word(threadIdx.x).clear();
        return mine;
    };
    // The scales of a tile, for this lane's FC channels and GROUPS groups of
    // four tokens. Small tiles read them when a tile begins, so that they are
    // there when it ends; large ones, which have no registers to spare, a
    // piece at a time when it ends.
    constexpr int GROUPS = FM * NG;
    constexpr bool DEEP = FN * FM * F * F / 64 >= 128;
    float row_scale = 0.0f;  // of ROW
    float scale_x[GROUPS][4], scale_0[FC], scale_1[FC], add[FC];
    const auto place = [&](int tile, int &m, int &n) FFN_INLINE {
        tile_at(tile, m, n);
        m = m * BM + wm * (BM / WM) + 4 * q;
        n = n * BC + wn * WC + FC * r;
    };
    const auto channel_scales = [&](int n) FFN_INLINE {
#pragma unroll
        for (int i = 0; i < FC; ++i) {
            const int c = min(n + i, a.N - 1);
            scale_0[i] = a.s0[c];
            scale_1[i] = TWO ? a.s1[c] : 0.0f;
            add[i] = !TWO && a.bias ? a.bias[c] : 0.0f;
        }
    };
    const auto token_scales = [&](int m, int j0, int count) FFN_INLINE {  // of groups j0 .., into place 0 on
#pragma unroll
        for (int j = 0; j < count; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                scale_x[j][e] = ROW ? row_scale : a.xs[min(m + F * ((j0 + j) / NG) + 8 * ((j0 + j) % NG) + e, a.M - 1)];
    };
    const auto begin = [&](int tile) FFN_INLINE {
        clear();
        if constexpr (!DEEP) {
            int m, n;
            place(tile, m, n);
            channel_scales(n);
            token_scales(m, 0, GROUPS);
        }
    };
    // Finishes a tile: outputs of this workgroup's sums plus those of the
    // `others` workgroups that share it with this one. Their loads come a few
    // groups of a few slots at a time, 32 registers in flight.
    const auto store = [&](int tile, const Sharers &in, int others) FFN_INLINE {
        int m0, n;
        place(tile, m0, n);
        const int tokens = a.M - m0;
        constexpr int ROOM = 8;  // groups in flight
        constexpr int ONCE = FN >= ROOM ? 1 : (GROUPS < ROOM / FN ? GROUPS : ROOM / FN);
        constexpr int SLOTS = ROOM / (FN * ONCE) > 0 ? ROOM / (FN * ONCE) : 1;
        static_assert(GROUPS % ONCE == 0, "whole pieces");
        float xs[ONCE][4];
        if constexpr (DEEP) {
            channel_scales(n);
            token_scales(m0, 0, ONCE);
        }
#pragma unroll
        for (int j0 = 0; j0 < GROUPS; j0 += ONCE) {
#pragma unroll
            for (int j = 0; j < ONCE; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    xs[j][e] = scale_x[DEEP ? j : j0 + j][e];
            if constexpr (DEEP)
                if (j0 + ONCE < GROUPS)
                    token_scales(m0, j0 + ONCE, ONCE);
            i32x4_t sum[ONCE][FN];
#pragma unroll
            for (int j = 0; j < ONCE; ++j)
#pragma unroll
                for (int f = 0; f < FN; ++f)
                    sum[j][f] = group_of(acc[f][(j0 + j) / NG], (j0 + j) % NG);
            for (int w0 = 0; w0 < others; w0 += SLOTS) {
                i32x4_t v[SLOTS][ONCE][FN];
#pragma unroll
                for (int i = 0; i < SLOTS; ++i) {
                    const auto theirs = slot_of(slot_number(sp, in, other_sharer(in, b, min(w0 + i, others - 1))));
#pragma unroll
                    for (int j = 0; j < ONCE; ++j)
#pragma unroll
                        for (int f = 0; f < FN; ++f) {
                            const int t = (j0 + j) / NG, g = (j0 + j) % NG;
                            v[i][j][f] = w0 + i < others && F * t + 8 * g < tokens
                                             ? __builtin_bit_cast(i32x4_t,
                                                                  load_device_coherent(theirs, slot_at(f, t, g)))
                                             : i32x4_t{0, 0, 0, 0};
                        }
                }
#pragma unroll
                for (int i = 0; i < SLOTS; ++i)
#pragma unroll
                    for (int j = 0; j < ONCE; ++j)
#pragma unroll
                        for (int f = 0; f < FN; ++f)
                            sum[j][f] += v[i][j][f];
            }
#pragma unroll
            for (int j = 0; j < ONCE; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int at = F * ((j0 + j) / NG) + 8 * ((j0 + j) % NG) + e;  // token, from m0
                    if (at >= tokens || n >= a.N)
                        continue;
                    float v[FC];
#pragma unroll
                    for (int f = 0; f < FC; ++f) {
                        const float y = int8_scaled(sum[j][f][e], xs[j][e], scale_0[f]);
                        if constexpr (TWO)
                            v[f] = int8_gated<OUT>(y, int8_scaled(sum[j][f + FC][e], xs[j][e], scale_1[f]));
                        else
                            v[f] = a.bias ? int8_biased(y, add[f]) : y;
                    }
                    int8_store<OUT, FC>(a, m0 + at, n, v);
                }
            __builtin_amdgcn_sched_barrier(0);  // (one piece's values at a time in registers)
        }
    };

    // One read among the products of a step, again and again.
    const auto interleave = [&]() FFN_INLINE {
#pragma unroll
        for (int i = 0; i < FN + FM; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x008, FN * FM / (FN + FM), 0);  // products
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);                    // LDS read
        }
        __builtin_amdgcn_sched_group_barrier(0x008, FN * FM, 0);
        __builtin_amdgcn_sched_barrier(0);
    };

    const int total = sp.whole * sp.stages + share(sp, b + 1) - share(sp, b);
    if (total == 0)
        return;
    Cursor ld, at;
    ld.start(sp, b, G);
    at = ld;
    int to = 0;        // where in the ring the next unit is loaded
    int st = 0;        // and where the unit to multiply is
    int rest = total;  // units to load
    int ld_units = ld.k_end - ld.k;
    const auto load_next = [&]() FFN_INLINE {
        issue(ld.k, to);
        to = to + STAGE == STAGES * STAGE ? 0 : to + STAGE;
        if (--rest > 0 && ++ld.k == ld.k_end) {
            ld.advance(sp, b, G, ld_units);
            ld_units = ld.k_end - ld.k;
            aim(ld.tile);
        }
    };
    constexpr int THREADS = WAVES * 64;
    constexpr int CHUNKS = ROW ? kInt8RowMost / (4 * THREADS) : 1;  // of four elements of the row, for each thread
    f32x4_t row[CHUNKS];
    if constexpr (ROW) {
        const auto reals = raw_buffer(a.row, K * 4);  // (past its end: zeros)
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c)
            row[c] = __builtin_bit_cast(
                f32x4_t, __builtin_amdgcn_raw_buffer_load_b128(reals, (c * THREADS + threadIdx.x) * 16, 0, 0));
        wait_vmcnt<0>();  // (before the ring's first loads, which the next wait would include)
    }
    aim(ld.tile);
#pragma unroll 1
    for (int s = 0; s < STAGES - 1 && rest > 0; ++s)
        load_next();
    if constexpr (ROW) {
        uint32_t most = 0;
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                most = max(most, magnitude_bits(row[c][i]));
        most = wave_max(most);
        const int codes = STAGES * STAGE, span = sp.stages * kBk;
        uint32_t *wave_most = reinterpret_cast<uint32_t *>(lds + note_at);
        if (lane == 63)
            wave_most[wave] = most;
        lds_barrier();
#pragma unroll
        for (int i = 0; i < WAVES; ++i)
            most = max(most, wave_most[i]);
        float inverse;
        int8_scale(most, row_scale, inverse);
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c)  // (zeros up to the last stage's end)
            if (const int at = (c * THREADS + threadIdx.x) * 4; at < span)
                *reinterpret_cast<uint32_t *>(lds + codes + at) =
                    int8_pack4(row[c][0], row[c][1], row[c][2], row[c][3], inverse);
        // (the first stage's barrier is also between these writes and their reads)
    }
    int spare = total - (STAGES - 1);  // units past those the ring holds now
    // To the next unit, every wave being done with the one before: it has
    // landed once at most the STAGES - 2 later ones' loads are in flight (loads
    // return in order). Its predecessor's slot takes the next load.
    const auto enter = [&]() FFN_INLINE {
        if (spare < 0)
            wait_vmcnt<0>();
        else if (FULL == WAVES || wave < FULL)
            wait_vmcnt<(STAGES - 2) * LOADS>();
        else
            wait_vmcnt<(STAGES - 2) * (LOADS - 1)>();
        lds_barrier();
        if (spare > 0)
            load_next();
        --spare;
    };
    const auto leave = [&]() FFN_INLINE { st = st + STAGE == STAGES * STAGE ? 0 : st + STAGE; };
    // After a tile's last unit; false after the workgroup's last.
    const auto finish = [&]() FFN_INLINE {
        Sharers in{b, b};
        if (at.k > 0 || at.k_end < sp.stages) {
            in = sharers_of(sp, at.tile - sp.whole * G);
            // (divisions run on the vector unit; back to scalar registers)
            in.first = __builtin_amdgcn_readfirstlane(in.first);
            in.last = __builtin_amdgcn_readfirstlane(in.last);
        }
        if (in.first == in.last || take(at.tile, in))
            store(at.tile, in, in.last - in.first);
        // nothing that the compiler knows to be in flight goes into the next
        // tile's loop: its waits there would take the ring's loads along
        wait_vmcnt<0>();
        return at.advance(sp, b, G, at.k_end - at.k);
    };
    if constexpr (!DEEP) {
        // few fragments: all of a unit's are read, then all multiplied, so the
        // read latency is met once a unit
        do {
            begin(at.tile);
            for (int n = at.k_end - at.k; n > 0; --n) {
                enter();
                Weights w[STEPS];
                Tokens x[STEPS];
#pragma unroll
                for (int s = 0; s < STEPS; ++s)
                    read(st, at.k_end - n, s, w[s], x[s]);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int s = 0; s < STEPS; ++s)
                    products(w[s], x[s], 0, FN);
                leave();
            }
        } while (finish());
    } else {
        static_assert(!ROW, "a single row has small tiles");
        // many: the next step's fragments are read while one step's are
        // multiplied, over the units' bounds too
        Weights w[2];
        Tokens x[2];
        enter();
        read(st, 0, 0, w[0], x[0]);
        for (;;) {
            begin(at.tile);
            for (int n = at.k_end - at.k; n > 1; --n) {
#pragma unroll
                for (int s = 0; s < STEPS; ++s) {
                    // (products on either side of the barrier keep the matrix
                    // cores busy over it)
                    const int before = s + 1 == STEPS ? FN / 2 : 0;
                    if (s + 1 == STEPS) {
                        products(w[s % 2], x[s % 2], 0, before);
                        __builtin_amdgcn_sched_barrier(0);
                        enter();
                        leave();
                    }
                    read(st, 0, (s + 1) % STEPS, w[(s + 1) % 2], x[(s + 1) % 2]);
                    products(w[s % 2], x[s % 2], before, FN);
                    interleave();
                }
            }
#pragma unroll
            for (int s = 0; s < STEPS; ++s) {
                if (s + 1 < STEPS)
                    read(st, 0, s + 1, w[(s + 1) % 2], x[(s + 1) % 2]);
                products(w[s % 2], x[s % 2], 0, FN);
            }
            if (!finish())
                return;
            enter();
            leave();
            read(st, 0, 0, w[0], x[0]);
        }
    }
}

template <int BM, int BN, int WM, int WN, int F, int STAGES, bool NT, int OUT, bool ROW = false>
hipError_t launch_t(const Int8GemmArgs &a, void *workspace, size_t *need, hipStream_t stream)
{
    Plan p = int8_plan(a.M, a.K, a.N, BM, BN, int8_two_weights(OUT) ? BN / 2 : BN, a.cus);
    if (need) {
        *need = p.part_bytes + p.word_bytes;
        return hipSuccess;
    }
    auto kern = int8_tile_kernel<BM, BN, WM, WN, F, STAGES, NT, OUT, ROW>;
    // the ring, a row's codes, and 16 bytes for what the waves tell each other (a
    // row's maximum of each wave, then whether a tile is finished here)
    constexpr int ring = STAGES * ((ROW ? 0 : BM) + BN) * kBk, most = ring + (ROW ? kInt8RowMost : 0) + 16;
    static_assert(most <= 160 * 1024, "LDS of a compute unit");
    static_assert(!ROW || WM * WN <= 4, "a maximum of each wave");
    const int lds = ring + (ROW ? p.split.stages * kBk : 0) + 16;
    static std::atomic<uint64_t> lds_done{0};
    hipError_t e = allow_lds(reinterpret_cast<const void *>(kern), most, lds_done);
    if (e != hipSuccess)
        return e;
    if (p.split.shared > 0) {
        p.split.tag = tag_of_launch(launch_tag());
        p.split.part = static_cast<int32_t *>(workspace);
        p.split.words = reinterpret_cast<unsigned long long *>(static_cast<char *>(workspace) + p.part_bytes);
    }
    hipLaunchKernelGGL(kern, dim3(p.groups), dim3(WM * WN * 64), lds, stream, a, p.split);
    return hipGetLastError();
}

// Weights of this size are read non-temporally where every byte is read once:
// with those of the layer before them they do not stay in the 256 MB
// last-level cache anyway. (178 MB at M = 1: 32.0 us for 35.4 with other
// weights in between, but 30.6 for 29.0 if the same ones are read again and
// again; 89 MB: no difference.)
constexpr size_t kStreamBytes = size_t{128} << 20;

// The tile of a product, by the tokens and by how many tiles it makes (times
// on one MI355X, K/N as given, G the dual of K = 5120 and N = 17408):
//   M <= 16, 32     the smallest that hold the tokens, 128 weight rows; 64 rows
//                   where 128 at a time leave half the compute units without a
//                   tile (17408/5120: M = 1 19.4 us for 20.8, M = 32 19.8 for
//                   22.0; 21504/5376, M = 32: 26.1 for 27.0)
//   M <= 64         64 x 128 (G, M = 64: 46.3 us; 64 x 64: 48.6), 64 x 64
//                   where 128 channels at a time leave half the compute units
//                   without a tile (17408/5120: 23.1 us for 24.6)
//   M <= 128, and more tokens that fill tiles of 256 badly: 128 x 128 (G,
//                   M = 128: 53.9 us; 128 x 64: 65.9), 128 x 64 by the same
//                   rule (17408/5120: 29.8 us for 33.1; M = 300, 4112/4099:
//                   21.1 for 21.4)
//   more            256 x 256 from 0.6 tiles a compute unit on (5120/17408,
//                   M = 4096, traced: 387 us; 256 x 128: 431; 128 x 128: 484),
//                   256 x 128 from half a tile a compute unit on (G, M = 256:
//                   72.5 us; 128 x 128: 88.4)
template <int OUT>
hipError_t launch_out(const Int8GemmArgs &a, void *workspace, size_t *need, hipStream_t stream)
{
    constexpr bool TWO = int8_two_weights(OUT);
    const long cus = a.cus;
    const auto tiles = [&](long bm, long bn) {
        const long channels = TWO ? bn / 2 : bn;
        return (a.M + bm - 1) / bm * ((a.N + channels - 1) / channels);
    };
    if (a.M <= 64) {
        const bool nt = static_cast<size_t>(a.N) * a.K * (TWO ? 2 : 1) >= kStreamBytes;
        if constexpr (!TWO)
            if (a.row)
                return nt                         ? launch_t<16, 128, 1, 4, 16, 8, true, OUT, true>(a, workspace, need, stream)
                       : 2 * tiles(16, 128) < cus ? launch_t<16, 64, 1, 4, 16, 10, false, OUT, true>(a, workspace, need, stream)
                                                  : launch_t<16, 128, 1, 4, 16, 8, false, OUT, true>(a, workspace, need, stream);
        if (a.M <= 32 && !nt)
            if constexpr (!TWO)
                if (2 * tiles(32, 128) < cus)
                    return a.M <= 16 ? launch_t<16, 64, 1, 4, 16, 10, false, OUT>(a, workspace, need, stream)
                                     : launch_t<32, 64, 1, 4, 16, 12, false, OUT>(a, workspace, need, stream);
        if (a.M <= 16)
            return nt ? launch_t<16, 128, 1, 4, 16, 8, true, OUT>(a, workspace, need, stream)
                      : launch_t<16, 128, 1, 4, 16, 8, false, OUT>(a, workspace, need, stream);
        if (a.M <= 32)
            return nt ? launch_t<32, 128, 1, 4, 16, 7, true, OUT>(a, workspace, need, stream)
                      : launch_t<32, 128, 1, 4, 16, 7, false, OUT>(a, workspace, need, stream);
        if constexpr (!TWO)
            if (2 * tiles(64, 128) < cus)
                return launch_t<64, 64, 4, 2, 16, 8, false, OUT>(a, workspace, need, stream);
        return nt ? launch_t<64, 128, 2, 4, 16, 6, true, OUT>(a, workspace, need, stream)
                  : launch_t<64, 128, 2, 4, 16, 6, false, OUT>(a, workspace, need, stream);
    }
    const long padded = (a.M + 255) / 256 * 256, padded_128 = (a.M + 127) / 128 * 128;
    if (a.M > 128 && 8 * padded <= 9 * padded_128) {
        if (10 * tiles(256, 256) >= 6 * cus)
            return launch_t<256, 256, 4, 2, 32, 2, false, OUT>(a, workspace, need, stream);
        if (2 * tiles(256, 128) >= cus)
            return launch_t<256, 128, 4, 2, 32, 3, false, OUT>(a, workspace, need, stream);
    }
    if constexpr (!TWO)
        if (2 * tiles(128, 128) < cus)
            return launch_t<128, 64, 4, 2, 16, 6, false, OUT>(a, workspace, need, stream);
    return launch_t<128, 128, 2, 4, 16, 4, false, OUT>(a, workspace, need, stream);
}

hipError_t launch(const Int8GemmArgs &a, Int8Out out, void *workspace, size_t *need, hipStream_t stream)
{
    switch (out) {
    case I8_BF16:
        return launch_out<I8_BF16>(a, workspace, need, stream);
    case I8_F16:
        return launch_out<I8_F16>(a, workspace, need, stream);
    case I8_F32:
        return launch_out<I8_F32>(a, workspace, need, stream);
    case I8_H_SILU:
        return launch_out<I8_H_SILU>(a, workspace, need, stream);
    default:
        return launch_out<I8_H_GELU>(a, workspace, need, stream);
    }
}

}  // namespace

hipError_t launch_int8_gemm(const Int8GemmArgs &a, Int8Out out, void *workspace, hipStream_t stream)
{
    return launch(a, out, workspace, nullptr, stream);
}

size_t int8_gemm_workspace(int M, int K, int N, Int8Out out, int cus)
{
    Int8GemmArgs a{};
    a.cus = cus;
    a.M = M;
    a.K = K;
    a.N = N;
    size_t need = 0;
    return launch(a, out, nullptr, &need, nullptr) == hipSuccess ? need : 0;
}

}  // namespace ffn
