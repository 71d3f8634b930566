// Device helpers shared by the kernels over drafted trees and bounded caches.
#pragma once

#include <stdint.h>

#include "gdn_internal.h"
#include "sm100.cuh"

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

__device__ __forceinline__ bool mbar_test_wait(uint32_t bar, uint32_t parity) {   // never suspends the thread
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

static __device__ __noinline__ bool wait_long(uint32_t bar, uint32_t parity, uint64_t limit_ns, const volatile int *abort) {
    if (limit_ns == 0) return mbar_test_wait(bar, parity);
#pragma unroll 1
    for (int i = 0; i < 8; ++i) {
        if (sm100::mbar_try_wait(bar, parity)) return true;
        if (*abort) return false;
    }
    return sm100::mbar_wait(bar, parity, limit_ns, abort);
}

// sm100::mbar_wait, with three differences: a limit of 0 gives up at once where
// the phase is not complete (try_wait alone may suspend for longer than a copy
// takes); the clock is read only once a wait has become long; and all but the
// first try is a call, which keeps the loops of the issuing warps short enough
// for the instruction cache (inlined, they ran at half the speed).
__device__ __forceinline__ bool wait_phase(uint32_t bar, uint32_t parity, uint64_t limit_ns, const volatile int *abort) {
    if (limit_ns != 0 && sm100::mbar_try_wait(bar, parity)) return true;
    return wait_long(bar, parity, limit_ns, abort);
}

// A wait gave up: the CTA's other waits end, and the first code stays.
static __device__ __noinline__ void record_failure(volatile int *abort, int *err, int code) {
    *abort = 1;
    atomicCAS(err, 0, code);
}

// True in one lane of a converged warp.  The issuing warps run their loops with
// all lanes and elect one per batch of instructions: addresses and descriptors
// then stay in uniform registers, where a branch on the lane number would move
// every operand of every product there (about 100 cycles a product).
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// Work of W units cut evenly over N CTAs: CTA c takes [start(c), start(c + 1)),
// where start(c) = floor(c W / N), with one wide division.
struct Cut {
    int64_t whole;
    int rest, n;
    __device__ __forceinline__ Cut(int64_t W, int N) : n(N) {
        if (W <= INT32_MAX) {
            whole = (uint32_t)W / (uint32_t)N;
            rest = (int)((uint32_t)W % (uint32_t)N);
        } else {
            whole = W / N;
            rest = (int)(W % N);
        }
    }
    __device__ __forceinline__ int64_t start(int c) const { return whole * c + rest * c / n; }   // n, c < 2^15
};

// Parent of node i (of a tree whose first row is bos): -1, or an index below
// i; anything else is read as -1.  Without a table the tree is a chain.
__device__ __forceinline__ int tree_parent(const int32_t *parents, int64_t bos, int i) {
    if (!parents) return i - 1;
    const int p = parents[bos + i];
    return p >= 0 && p < i ? p : -1;
}

}  // namespace gdn
