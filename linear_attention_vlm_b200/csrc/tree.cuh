// Device helpers shared by the kernels over drafted trees and bounded caches.
#pragma once

#include <stdint.h>

#include "gdn_internal.h"

namespace gdn {

constexpr int kMaxNodes = 64;

// Rows [bos, bos + n) of sequence b in a packed tensor of `total` rows, never
// more than `most` of them and never past the end.
__device__ __forceinline__ int seq_rows(const int32_t *cu, int64_t uniform_len, int64_t total, int b, int most,
                                        int64_t &bos) {
    int64_t eos;
    SeqBounds{cu, uniform_len}.get(b, bos, eos);
    bos = max((int64_t)0, bos);
    eos = min(eos, min(total, bos + most));
    return eos > bos ? (int)(eos - bos) : 0;
}

// Cached slots of sequence b, within [0, capacity].
__device__ __forceinline__ int cached_slots(const int32_t *lens, int64_t capacity, int b) {
    if (capacity == 0) return 0;
    const int n = lens[b];
    return n < 0 ? 0 : (n > capacity ? (int)capacity : n);
}

// Parent of node i (of a tree whose first row is bos): -1, or an index below
// i; anything else is read as -1.  Without a table the tree is a chain.
__device__ __forceinline__ int tree_parent(const int32_t *parents, int64_t bos, int i) {
    if (!parents) return i - 1;
    const int p = parents[bos + i];
    return p >= 0 && p < i ? p : -1;
}

}  // namespace gdn
