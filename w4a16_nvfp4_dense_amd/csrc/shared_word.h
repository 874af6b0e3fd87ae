// shared_word.h -- how workgroups that hold parts of one result agree on the one
// that finishes it, without any of them depending on another's being started.
// Plain integer code for host and device.
//
// A shared result has one word in the workspace: the launch's tag with the
// count of the parts whose sums are in the workspace. Whoever has a part writes
// its sums, then counts itself there; the one that finds all others counted
// finishes the result. Whichever that is, and in whatever order and however late
// the workgroups of a launch run beside those of other launches, the result is
// finished exactly once, after all its parts are there.
//
// The low bits count parts, the rest is the launch's tag. A word of any other
// tag (what the workspace held before, or zero) stands for no parts: the first
// part replaces it. Whoever finishes sets the word to zero, by then being the
// only one left that uses it, so that a replay of the same launch starts afresh.
#pragma once

#include <hip/hip_runtime.h>

namespace ffn {

constexpr int kCountBits = 16;

// A launch's tag from its number (launch_tag()): not zero, its low bits zero.
__host__ __device__ __forceinline__ unsigned long long tag_of_launch(unsigned long long number)
{
    const unsigned long long tag = number >> kCountBits << kCountBits;
    return tag ? tag : 1ull << kCountBits;
}

__host__ __device__ __forceinline__ bool is_tagged(unsigned long long word, unsigned long long tag)
{
    return word >> kCountBits == tag >> kCountBits;
}

// Counts one part in the word; returns how many it holds now. `seen` is what
// the word may hold (a guess costs one more try). Word: exchange(seen, next)
// sets the word to `next` if it holds `seen`, else writes what it holds to
// `seen` and returns false; add_one() returns what the word held. Ends: a word
// that is tagged stays so until this part is counted, so exchange fails at most
// twice, for a wrong guess and for another first part.
template <class Word>
__host__ __device__ __forceinline__ int count_part(const Word &word, unsigned long long tag, unsigned long long seen)
{
    while (!is_tagged(seen, tag))
        if (word.exchange(seen, tag + 1))
            return 1;
    return static_cast<int>(word.add_one() - tag) + 1;
}

}  // namespace ffn
