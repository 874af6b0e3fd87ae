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

// Whether a lower part's word comes to be marked within the last part's time (the
// same answer in every active lane of a wave).
__device__ __forceinline__ bool comes(const PartWord &word, unsigned long long tag)
{
    for (int i = 0; i < kLooks; ++i) {
        if (__builtin_amdgcn_readfirstlane(word.load() == marked(tag)))
            return true;
        __builtin_amdgcn_s_sleep(1);
    }
    return false;
}

}  // namespace ffn
