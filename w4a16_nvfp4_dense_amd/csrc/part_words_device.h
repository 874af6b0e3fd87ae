// part_words_device.h -- the words of part_words.h on the device.
#pragma once

#include <hip/hip_runtime.h>

#include "part_words.h"
#include "shared_word_device.h"

namespace ffn {

struct PartWord : SharedWord {
    __device__ __forceinline__ unsigned long long add(int n) const
    {
        return __hip_atomic_fetch_add(at, static_cast<unsigned long long>(n), __ATOMIC_RELAXED,
                                      __HIP_MEMORY_SCOPE_AGENT);
    }
    __device__ __forceinline__ unsigned long long swap(unsigned long long v) const
    {
        return __hip_atomic_exchange(at, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
};

// Whether the words of the first n parts, lower(i), come to be marked within the
// last part's time. A wave looks at 64 of them together; every lane of it calls
// this, and has the same answer.
template <class LowerWord>
__device__ __forceinline__ bool all_come(LowerWord lower, int n, unsigned long long tag)
{
    const int lane = threadIdx.x & 63;
    for (int i = 0; i < kLooks; ++i) {
        bool there = true;
        for (int k = lane; k < n; k += 64)
            there = there && lower(k).load() == marked(tag);
        if (__all(there))
            return true;
        __builtin_amdgcn_s_sleep(1);
    }
    return false;
}

}  // namespace ffn
