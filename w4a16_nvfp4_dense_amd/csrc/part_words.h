// part_words.h -- the agreement of shared_word.h for results whose last part had
// rather wait a little than write its sums. Plain code for host and device.
//
// Every part has a word. A lower part writes its sums, then marks its word; the
// last part looks at those words for a bounded time and, finding them all
// marked, finishes the result with its own sums in registers: nothing else is
// exchanged. Should the time run out, as when launches on other streams hold
// the compute units that the lower parts need, it writes its sums too and
// leaves each of those words as given up, which tells it exactly which parts
// were there; a part that finds its word given up knows that nobody looks any
// more. The last part counts itself and those that were there in its own word,
// each of the others counts itself there, and the one that completes the count
// finishes the result. So it is finished exactly once, whoever is started when.
//
// The words need no initialisation: what is neither this launch's mark nor its
// giving up stands for nothing. Whoever finishes sets them to zero, by then
// being the only one left that uses them.
#pragma once

#include "shared_word.h"

namespace ffn {

// The two states of a lower part's word; their low bits are no count.
__host__ __device__ __forceinline__ unsigned long long marked(unsigned long long tag)
{
    return tag;
}
__host__ __device__ __forceinline__ unsigned long long given_up(unsigned long long tag)
{
    return tag | ((1ull << kCountBits) - 1);
}

// Counts n parts in the word, whatever it holds; returns how many it holds now.
// Word: as count_part's, and add(n), which returns what the word held.
template <class Word>
__host__ __device__ __forceinline__ int count_parts(const Word &word, unsigned long long tag, int n)
{
    unsigned long long seen = 0;
    while (!is_tagged(seen, tag))
        if (word.exchange(seen, tag + n))
            return n;
    return static_cast<int>(word.add(n) - tag) + n;
}

// A lower part, its sums written, swaps its word for marked(tag). What the word
// held says whether the last part still looks; if it has given up, the lower
// part finishes the result of `parts` parts if it completes the count.
template <class Word>
__host__ __device__ __forceinline__ bool late_part(const Word &last, unsigned long long tag, int parts)
{
    return count_parts(last, tag, 1) == parts;
}

// The last part, whose time ran out, its sums written; whether it finishes the
// result all the same. lower(i): the word of lower part i, with swap(v), which
// returns what the word held.
template <class LowerWord, class Word>
__host__ __device__ __forceinline__ bool last_gives_up(LowerWord lower, const Word &last, unsigned long long tag,
                                                       int parts)
{
    int there = 1;
    for (int i = 0; i < parts - 1; ++i)
        there += lower(i).swap(given_up(tag)) == marked(tag);
    return count_parts(last, tag, there) == parts;
}

// Looks of the last part at a lower part's word; each is a round trip to memory,
// all of them about 0.1 ms.
constexpr int kLooks = 64;

}  // namespace ffn
