// int8_split.h -- how the int8 product's tiles are split over workgroups, and
// how workgroups that share a tile agree on the one that finishes it. Plain
// integer code for host and device.
//
// The tiles' stages, in tile order, are units. Every workgroup takes `whole`
// tiles and then an equal share of the units of the tiles that are left, so a
// tile may be shared by neighbouring workgroups, each with one part of its
// stages. A workgroup walks its share downwards.
//
// A shared tile is finished by its last workgroup, or whichever is late
// (part_words.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <algorithm>

#include "part_words.h"

namespace ffn {

constexpr int kBk = 128;  // columns (bytes of a row) of a stage

// Division by a number that the host knows: n / d = n m >> (31 + s) for
// n < 2^31, with s = ceil(log2 d) and m = ceil(2^(31 + s) / d). A few scalar
// instructions instead of two dozen: a kernel this short is held up by
// fetching its prologue's instructions.
struct Divisor {
    uint32_t d, m, s;
    __host__ __device__ __forceinline__ uint32_t divide(uint32_t n) const
    {
        return static_cast<uint32_t>((static_cast<uint64_t>(n) * m) >> (31 + s));
    }
};

inline Divisor divisor(uint32_t d)
{
    Divisor v{d, 0, 0};
    while ((uint64_t{1} << v.s) < d)
        ++v.s;
    v.m = static_cast<uint32_t>(((uint64_t{1} << (31 + v.s)) + d - 1) / d);
    return v;
}

constexpr int kXcds = 8;
constexpr int kBand = 8;  // tiles of tokens that are walked together

struct Split {
    int tiles_m, tiles_n;
    int whole;                  // whole tiles of every workgroup
    int shared;                 // tiles split over the workgroups, after those
    int sharers;                // workgroups that have a share of them, at most one for each unit
    int least, more;            // units of a share
    int stages;                 // stages of a tile
    int place_step;             // of a round's places between an XCD's and the next one's, or 0
    Divisor by_stages, by_band, by_rows, by_last_rows;  // tiles of a band; its tiles of tokens, and the last one's
    unsigned long long tag;     // of this launch, its low kCountBits zero
    int32_t *part;              // two slots of a tile's sums for each sharer
    unsigned long long *words;  // a word for each slot

    // Workgroup b's place in a round of whole tiles: those of one XCD (b % 8)
    // take neighbouring tiles, which share operands in its L2.
    __host__ __device__ __forceinline__ int chunk(int b, int G) const
    {
        return place_step ? b % kXcds * place_step + b / kXcds : b;
    }
};

// The units of workgroup b: its whole tiles, then units [share(b), share(b + 1))
// of the shared tiles: `least` each, one more for the first `more` sharers.
__host__ __device__ __forceinline__ int share(const Split &s, int b)
{
    b = b < s.sharers ? b : s.sharers;
    return b * s.least + (b < s.more ? b : s.more);
}

// The workgroup that has unit u of the shared tiles.
__host__ __device__ __forceinline__ int owner(const Split &s, int u)
{
    const int cut = s.more * (s.least + 1);
    const uint32_t n = u < cut ? u : u - cut, d = u < cut ? s.least + 1 : s.least;
    return static_cast<int>(n / d) + (u < cut ? 0 : s.more);
}

// The workgroups first .. last that have a part of shared tile t.
struct Sharers {
    int first, last;
};

__host__ __device__ __forceinline__ Sharers sharers_of(const Split &s, int t)
{
    return Sharers{owner(s, t * s.stages), owner(s, (t + 1) * s.stages - 1)};
}

// The slot of workgroup w's sums of a tile that it shares with others, and the
// number of its word. A share has at most one part that stops short of its
// tile's last stage and one that has that stage without the tile's first: the
// tile's last workgroup takes its second slot, every other one its first.
__host__ __device__ __forceinline__ int slot_number(const Split &s, const Sharers &t, int w)
{
    return w == t.last ? s.sharers + w : w;
}

// The i-th of a tile's other workgroups, seen from workgroup b.
__host__ __device__ __forceinline__ int other_sharer(const Sharers &t, int b, int i)
{
    return t.first + i + (t.first + i >= b ? 1 : 0);
}

// A position in a workgroup's units: the whole tiles, then the shared ones
// from the highest down, the stages of each upwards.
struct Cursor {
    int tile, k, k_end;  // stage k of a tile; the workgroup has it up to k_end
    int round, u0, u;    // units [u0, u) of the share are still to come, the tile's among them

    __host__ __device__ __forceinline__ void segment(const Split &s, int b, int G)
    {
        if (round < s.whole) {
            tile = round * G + s.chunk(b, G);
            k = 0;
            k_end = s.stages;
        } else {
            const int t = s.by_stages.divide(u - 1);
            tile = s.whole * G + t;
            k = u0 > t * s.stages ? u0 - t * s.stages : 0;
            k_end = u - t * s.stages;
        }
    }
    __host__ __device__ __forceinline__ void start(const Split &s, int b, int G)
    {
        round = 0;
        u0 = share(s, b);
        u = share(s, b + 1);
        segment(s, b, G);
    }
    // Past the `units` units of this tile; false if that was the last one.
    __host__ __device__ __forceinline__ bool advance(const Split &s, int b, int G, int units)
    {
        if (round < s.whole)
            ++round;
        else
            u -= units;
        if (round >= s.whole && u <= u0)
            return false;
        segment(s, b, G);
        return true;
    }
};

// ---------------------------------------------------------------- the launch
struct Plan {
    int groups;  // workgroups
    Split split;
    size_t part_bytes, word_bytes;
};

// The split of M x N outputs over tiles of BM tokens x BC channels (BN weight
// rows), K columns, on `cus` compute units.
inline Plan int8_plan(int M, int K, int N, int BM, int BN, int BC, int cus)
{
    const auto round256 = [](size_t n) { return (n + 255) & ~static_cast<size_t>(255); };
    Plan p{};
    Split &s = p.split;
    s.tiles_m = (M + BM - 1) / BM;
    s.tiles_n = (N + BC - 1) / BC;
    s.stages = (K + kBk - 1) / kBk;
    const long tiles = static_cast<long>(s.tiles_m) * s.tiles_n;
    p.groups = static_cast<int>(std::min<long>(cus, std::max<long>(tiles, tiles * s.stages / 4)));
    // With tiles left over after a single round, that round is shared out too,
    // so that a share is at least a tile long and a tile has at most two
    // parts. (After more rounds the left-over tiles alone are shared: 1-3%
    // faster at 4 rounds and a quarter, where a round's sums exchanged are
    // 64 MB.)
    s.whole = static_cast<int>(tiles / p.groups);
    if (s.whole == 1 && tiles % p.groups != 0)
        s.whole = 0;
    s.shared = static_cast<int>(tiles - static_cast<long>(s.whole) * p.groups);
    // At least four units to a share; and after whole rounds shares of half a
    // tile or more, so that a tile has two parts, or three where the shares'
    // ends drift off the tiles' middles (an odd number of stages, or more
    // left-over tiles than half the workgroups). (5120/17408, M = 4096: 387 us;
    // four parts 393, whole tiles 389.)
    const long units = static_cast<long>(s.shared) * s.stages;
    s.sharers = static_cast<int>(std::min<long>(s.whole > 0 ? std::min(p.groups, 2 * s.shared) : p.groups,
                                                std::max<long>(1, units / 4)));
    s.place_step = p.groups % kXcds == 0 ? p.groups / kXcds : 0;
    s.by_stages = divisor(s.stages);
    s.by_band = divisor(kBand * s.tiles_n);
    s.by_rows = divisor(kBand);
    s.by_last_rows = divisor(s.tiles_m % kBand ? s.tiles_m % kBand : kBand);
    if (s.shared > 0) {
        s.least = s.shared * s.stages / s.sharers;
        s.more = s.shared * s.stages % s.sharers;
        p.part_bytes = round256(2 * static_cast<size_t>(s.sharers) * BM * BN * 4);
        p.word_bytes = round256(2 * static_cast<size_t>(s.sharers) * 8);
    }
    return p;
}

}  // namespace ffn
