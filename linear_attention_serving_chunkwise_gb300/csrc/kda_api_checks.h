// Checks that the C entry points share: alignment, and buffers that may not overlap.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/kda.h"

namespace kda {
namespace checks {

struct Span {
    uintptr_t lo, hi;   // [lo, hi); empty for a null pointer
};
inline Span span(const void* p, size_t bytes)
{
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    return p ? Span{lo, lo + bytes} : Span{0, 0};
}
inline bool meet(Span a, Span b) { return a.lo < b.hi && b.lo < a.hi; }
inline bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

// the outputs (the first `n_out` spans) overlap neither one another nor an input
template <int N>
inline bool apart(const Span (&s)[N], int n_out)
{
    for (int i = 0; i < n_out; ++i)
        for (int j = i + 1; j < N; ++j)
            if (meet(s[i], s[j])) return false;
    return true;
}

inline bool known_dtype(int32_t t) { return t == KDA_F32 || t == KDA_BF16; }
inline kda_status of(cudaError_t e) { return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA; }

}  // namespace checks
}  // namespace kda
