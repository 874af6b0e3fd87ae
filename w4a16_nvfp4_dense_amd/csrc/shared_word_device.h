// shared_word_device.h -- the words of shared_word.h on the device.
#pragma once

#include <hip/hip_runtime.h>

#include "shared_word.h"

namespace ffn {

// A word of the workspace in which workgroups on any XCD count: relaxed
// agent-scope atomics. The parts' sums move with device-coherent stores and
// loads (nvfp4_device.h); a part is counted once its stores have completed.
struct SharedWord {
    unsigned long long *at;
    __device__ __forceinline__ bool exchange(unsigned long long &seen, unsigned long long next) const
    {
        return __hip_atomic_compare_exchange_strong(at, &seen, next, __ATOMIC_RELAXED, __ATOMIC_RELAXED,
                                                    __HIP_MEMORY_SCOPE_AGENT);
    }
    __device__ __forceinline__ unsigned long long add_one() const
    {
        return __hip_atomic_fetch_add(at, 1ull, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __device__ __forceinline__ unsigned long long load() const
    {
        return __hip_atomic_load(at, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __device__ __forceinline__ void clear() const
    {
        __hip_atomic_store(at, 0ull, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
};

}  // namespace ffn
