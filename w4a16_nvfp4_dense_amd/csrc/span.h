// span.h -- the buffers of a call, for the checks of what may overlap (host).
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace ffn {

// A buffer of a call. (A null or an empty one overlaps nothing.)
struct Span {
    const void *p;
    size_t bytes;
};

inline bool overlap(const Span &a, const Span &b)
{
    const uintptr_t i = reinterpret_cast<uintptr_t>(a.p), j = reinterpret_cast<uintptr_t>(b.p);
    return i && j && a.bytes && b.bytes && i < j + b.bytes && j < i + a.bytes;
}

// Whether one of the `written` overlaps another of them or an input.
template <int W, int R>
bool any_overlap(const Span (&written)[W], const Span (&in)[R])
{
    for (int w = 0; w < W; ++w) {
        for (int r = 0; r < R; ++r)
            if (overlap(written[w], in[r]))
                return true;
        for (int other = 0; other < w; ++other)
            if (overlap(written[w], written[other]))
                return true;
    }
    return false;
}

}  // namespace ffn
