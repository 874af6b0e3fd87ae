// moe_plan.hip -- expert order of the chosen (token, expert) pairs: a stable
// counting sort of the slots by expert.
//
// The place of slot s with expert e is (slots of lower experts) + (earlier
// slots of e). Every wave owns a run of consecutive slots, taken 64 at a time.
// It counts its run's slots of each expert into a row of LDS of its own; a scan
// over experts and, for each expert, over the waves turns the counts into the
// place of the first such slot of the run; then the wave walks its run again,
// and a slot's place is that number plus how many lanes below it have the same
// expert, found from one ballot for each bit of the id. Integer counts and
// positions only, so the order does not hang on timing.
//
// Up to kOnce slots one workgroup does it all. More are cut into chunks of
// kChunk: a first launch counts the chunks, and in the second each chunk's
// workgroup adds up the counts of all of them, those of earlier chunks apart,
// instead of a launch between the two. That is chunks^2 E 4 bytes from L2: 4 MB for
// 131072 slots of 256 experts, 4 GB for 2097152 of 1024.
//
// It is bound by launches and latency: 256 slots of 128 experts 3.4 us, 131072 of
// 256 2.6 + 7.5 us (1.6 MB of ids, rows and places: 0.3 us of memory); at the largest
// sizes by the adding up: both launches 17 us for 524288 of 256, 27 of 1024; 78 for
// 2097152 of 256, 181 of 1024.
#include <hip/hip_runtime.h>

#include "kernels.h"
#include "moe.h"

namespace ffn {
namespace {

constexpr int kWaves = 16;
constexpr int kThreads = kWaves * 64;
constexpr int kMostExperts = 1024;
constexpr int kChunk = 2048;  // slots of a workgroup, where there are several
constexpr int kOnce = 8192;

static_assert(kMostExperts <= kThreads, "a thread for each expert");

// Which lanes of the wave hold this lane's value, of `bits` bits.
__device__ __forceinline__ unsigned long long lanes_alike(int v, int bits)
{
    unsigned long long alike = ~0ull;
    for (int b = 0; b < bits; ++b) {
        const bool set = (v >> b) & 1;
        const unsigned long long lanes = __ballot(set);
        alike &= set ? lanes : ~lanes;
    }
    return alike;
}

// The sum of v over the threads below this one, and over all of them.
__device__ __forceinline__ int scan_threads(int v, int *wave_sum, int &total)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int s = v;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int other = __shfl_up(s, d);
        s += lane >= d ? other : 0;
    }
    if (lane == 63)
        wave_sum[wave] = s;
    __syncthreads();
    int below = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        below += w < wave ? wave_sum[w] : 0;
        total += wave_sum[w];
    }
    return below + s - v;
}

// Counts of the slots [begin, end) of a wave.
__device__ __forceinline__ void count_run(const int32_t *ids, int begin, int end, int E, int *count)
{
    for (int s = begin + static_cast<int>(threadIdx.x & 63); s < end; s += 64) {
        const int e = ids[s];
        if (e >= 0 && e < E)
            atomicAdd(count + e, 1);
    }
}

// A chunk's slots of each expert, to counts[chunk][E].
__global__ __launch_bounds__(kThreads) void moe_count_kernel(const int32_t *ids, int R, int E, int *counts)
{
    __shared__ int count[kMostExperts];
    if (threadIdx.x < E)
        count[threadIdx.x] = 0;
    __syncthreads();
    const int wave = threadIdx.x >> 6, run = kChunk / kWaves;
    const int begin = blockIdx.x * kChunk + wave * run;
    count_run(ids, begin, min(begin + run, R), E, count);
    __syncthreads();
    if (threadIdx.x < E)
        counts[static_cast<size_t>(blockIdx.x) * E + threadIdx.x] = count[threadIdx.x];
}

// Places of a chunk's slots; `counts` null: one workgroup holds all slots.
__global__ __launch_bounds__(kThreads) void moe_place_kernel(const int32_t *ids, int R, int E, int chunk,
                                                             const int *counts, int32_t *rows, int32_t *offsets,
                                                             int32_t *places)
{
    extern __shared__ int at[];  // [kWaves][E], counts, then places
    __shared__ int wave_sum[kWaves];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int i = threadIdx.x; i < kWaves * E; i += kThreads)
        at[i] = 0;
    __syncthreads();
    const int run = (chunk + kThreads - 1) / kThreads * 64;  // of a wave: whole steps of 64
    const int first = blockIdx.x * chunk, last = min(first + chunk, R);
    const int begin = min(first + wave * run, last), end = min(begin + run, last);
    count_run(ids, begin, end, E, at + wave * E);
    __syncthreads();
    const int e = threadIdx.x;
    int mine = 0, earlier = 0;  // slots of expert e: all, and those of earlier chunks
    if (e < E) {
        if (counts)
#pragma unroll 16
            for (int b = 0; b < static_cast<int>(gridDim.x); ++b) {
                const int c = counts[static_cast<size_t>(b) * E + e];
                mine += c;
                earlier += b < static_cast<int>(blockIdx.x) ? c : 0;
            }
        else
            for (int w = 0; w < kWaves; ++w)
                mine += at[w * E + e];
    }
    int total;
    const int begins = scan_threads(mine, wave_sum, total);
    if (e < E) {
        int place = begins + earlier;
        for (int w = 0; w < kWaves; ++w) {
            const int c = at[w * E + e];
            at[w * E + e] = place;
            place += c;
        }
        if (blockIdx.x == 0)
            offsets[e] = begins;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0)
        offsets[E] = total;
    for (int i = max(first, total) + static_cast<int>(threadIdx.x); i < last; i += kThreads)
        rows[i] = -1;  // behind the last expert's
    __syncthreads();
    const int bits = 32 - __clz(E);  // of 0 .. E, E standing for none
    for (int s0 = begin; s0 < end; s0 += 64) {
        const int s = s0 + lane;
        int id = s < end ? ids[s] : -1;
        if (id < 0 || id >= E)
            id = E;
        const unsigned long long alike = lanes_alike(id, bits);
        const int rank = __popcll(alike & ((1ull << lane) - 1));
        int place = -1;
        if (id < E)
            place = at[wave * E + id] + rank;
        __builtin_amdgcn_wave_barrier();  // (every lane has read before one adds)
        if (id < E && rank == 0)
            at[wave * E + id] += __popcll(alike);
        __builtin_amdgcn_wave_barrier();
        if (s < end) {
            places[s] = place;
            if (place >= 0)
                rows[place] = s;
        }
    }
}

int chunks_of(int R)
{
    return R > kOnce ? (R + kChunk - 1) / kChunk : 1;
}

}  // namespace

size_t moe_plan_workspace(int R, int E)
{
    return chunks_of(R) > 1 ? static_cast<size_t>(chunks_of(R)) * E * sizeof(int) : 0;
}

hipError_t launch_moe_plan(const int32_t *ids, int R, int E, int32_t *rows, int32_t *offsets, int32_t *places,
                           void *workspace, hipStream_t stream)
{
    const int chunks = chunks_of(R);
    int *counts = chunks > 1 ? static_cast<int *>(workspace) : nullptr;
    if (counts)
        hipLaunchKernelGGL(moe_count_kernel, dim3(chunks), dim3(kThreads), 0, stream, ids, R, E, counts);
    static std::atomic<uint64_t> lds_done{0};
    const hipError_t e = allow_lds(reinterpret_cast<const void *>(moe_place_kernel),
                                   kWaves * kMostExperts * sizeof(int), lds_done);
    if (e != hipSuccess)
        return e;
    hipLaunchKernelGGL(moe_place_kernel, dim3(chunks), dim3(kThreads), kWaves * E * sizeof(int), stream, ids, R, E,
                       chunks > 1 ? kChunk : R, counts, rows, offsets, places);
    return hipGetLastError();
}

}  // namespace ffn
