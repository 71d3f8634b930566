// New tokens enter a cache of constant size in place of its lightest slots.
//
// Per (sequence, key/value head) the candidates are the cached slots and the
// new tokens, in this order, each with a 32-bit key that orders them: the
// bits of the weight made monotone, all ones for a recent position, zero for
// NaN.  E = candidates - capacity of them give way: those below the E-th
// smallest key tau and, of the ones equal to it, the latest.  tau is found
// digit by digit (8 bits, a histogram in shared memory each).  Evicted slots and
// empty ones, ascending, take the new tokens that stay, ascending: slots that
// stay do not move, so the rows copied are the new tokens' alone, and no copy
// reads what another writes.
//
// Two kernels: the selection, one CTA per (sequence, head), which also writes
// weights and positions; then the copy of keys and values, one warp per row.
#include <cuda_runtime.h>
#include <math.h>

#include "tree.cuh"

namespace gdn {
namespace {

constexpr int kSelThreads = 1024, kSelWarps = kSelThreads / 32;
constexpr unsigned kAll = 0xffffffffu;

// order-preserving bits of a weight; NaN below everything, -0 as 0
__device__ __forceinline__ uint32_t weight_key(float w) {
    if (isnan(w)) return 0u;
    const uint32_t u = __float_as_uint(w + 0.f);
    return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}

// Exclusive prefix over the CTA's warps of a per-warp count; every thread of
// a warp gets its warp's prefix, `total` the sum.
__device__ __forceinline__ int warp_prefix(int count, int *sh, int &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    __syncthreads();
    if (lane == 0) sh[warp] = count;
    __syncthreads();
    int v = sh[lane];
    int incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(kAll, incl, o);
        if (lane >= o) incl += t;
    }
    total = __shfl_sync(kAll, incl, 31);
    return __shfl_sync(kAll, incl - v, warp);
}

__global__ void __launch_bounds__(kSelThreads) cache_select_kernel(const CacheInsertLaunch L, int64_t uniform_len) {
    __shared__ unsigned hist[256];
    __shared__ int scan_sh[kSelWarps];
    __shared__ unsigned prefix_sh;
    __shared__ int rest_sh;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int b = blockIdx.x / L.Hkv, h = blockIdx.x % L.Hkv;
    int64_t t0;
    const int m = seq_rows(L.cu_seqlens, uniform_len, L.total_tokens, b, INT32_MAX, t0);
    const int cap = (int)L.capacity;
    const int len = cached_slots(L.lens_in, L.capacity, b);
    const int64_t seen = L.seen_in[b];
    const int C = len + m, keep = min(cap, C), evict = C - keep;
    const int64_t base = ((int64_t)b * L.Hkv + h) * cap;
    auto new_weight = [&](int j) { return L.w_new ? L.w_new[(t0 + j) * L.Hkv + h] : 0.f; };
    auto key_of = [&](int i) -> uint32_t {
        if (i < len) return seen + m - L.pos_in[base + i] <= L.recent ? 0xffffffffu : weight_key(L.w_in[base + i]);
        return C - i <= L.recent ? 0xffffffffu : weight_key(new_weight(i - len));
    };

    // tau, and how many of the candidates equal to it give way
    uint32_t tau = 0;
    int ties = 0;
    if (evict > 0) {
        int rest = evict;
        for (int shift = 24; shift >= 0; shift -= 8) {
            __syncthreads();
            if (tid < 256) hist[tid] = 0;
            __syncthreads();
            for (int i = tid; i < C; i += kSelThreads) {
                const uint32_t key = key_of(i);
                if (shift == 24 || (key >> (shift + 8)) == (tau >> (shift + 8))) atomicAdd(&hist[(key >> shift) & 255], 1u);
            }
            __syncthreads();
            if (tid == 0) {
                int r = rest, d = 0;
                while (d < 255 && (int)hist[d] < r) r -= hist[d++];
                prefix_sh = d;
                rest_sh = r;
            }
            __syncthreads();
            tau |= prefix_sh << shift;
            rest = rest_sh;
        }
        ties = rest;
    }

    // a warp owns consecutive candidates, so ranks are running counts
    const int span = ((C + kSelThreads - 1) / kSelThreads) * 32, c0 = warp * span, c1 = min(C, c0 + span);
    int n_eq = 0, all_eq = 0;
    if (evict > 0)
        for (int i = c0 + lane; i - lane < c1; i += 32) n_eq += __popc(__ballot_sync(kAll, i < c1 && key_of(i) == tau));
    const int eq0 = warp_prefix(n_eq, scan_sh, all_eq);
    const unsigned below = (1u << lane) - 1;
    // calls f(candidate, gives way) for the warp's candidates, all lanes together
    auto walk = [&](auto f) {
        int eq = eq0;
        for (int i = c0 + lane; i - lane < c1; i += 32) {
            const bool in = i < c1;
            const uint32_t key = in && evict > 0 ? key_of(i) : 0xffffffffu;
            const unsigned same = __ballot_sync(kAll, in && evict > 0 && key == tau);
            const bool gone = in && evict > 0 && (key < tau || (key == tau && eq + __popc(same & below) >= all_eq - ties));
            eq += __popc(same);
            f(i, in, gone);
        }
    };
    int n_gone = 0, n_new = 0, all_gone, all_new;
    walk([&](int i, bool in, bool gone) {
        n_gone += __popc(__ballot_sync(kAll, in && gone && i < len));
        n_new += __popc(__ballot_sync(kAll, in && !gone && i >= len));
    });
    int gone0 = warp_prefix(n_gone, scan_sh, all_gone), new0 = warp_prefix(n_new, scan_sh, all_new);

    // places for the new tokens, ascending: evicted slots, then empty ones
    int32_t *places = static_cast<int32_t *>(L.workspace) + (int64_t)h * L.total_tokens + t0;
    for (int s = len + tid; s < keep; s += kSelThreads) places[all_gone + s - len] = s;
    walk([&](int i, bool in, bool gone) {
        const unsigned out = __ballot_sync(kAll, in && gone && i < len), enter = __ballot_sync(kAll, in && !gone && i >= len);
        if (in && i < len) {
            if (gone) {
                places[gone0 + __popc(out & below)] = i;
            } else if (L.w_out != L.w_in || L.pos_out != L.pos_in) {
                L.w_out[base + i] = L.w_in[base + i];
                L.pos_out[base + i] = L.pos_in[base + i];
            }
        } else if (in) {
            L.slots[(t0 + i - len) * L.Hkv + h] = gone ? -1 : new0 + __popc(enter & below);   // a rank for now
        }
        gone0 += __popc(out);
        new0 += __popc(enter);
    });
    __syncthreads();
    for (int j = tid; j < m; j += kSelThreads) {
        int32_t *slot = L.slots + (t0 + j) * L.Hkv + h;
        const int r = *slot;
        if (r < 0) continue;
        const int s = places[r];
        *slot = s;
        L.w_out[base + s] = new_weight(j);
        L.pos_out[base + s] = (int32_t)(seen + j);
    }
}

constexpr int kCopyWarps = 8;

__global__ void __launch_bounds__(kCopyWarps * 32) cache_copy_kernel(const CacheInsertLaunch L, int64_t uniform_len) {
    const int b = blockIdx.y, lane = threadIdx.x & 31;
    int64_t t0;
    const int m = seq_rows(L.cu_seqlens, uniform_len, L.total_tokens, b, INT32_MAX, t0);
    const int64_t rows = (int64_t)m * L.Hkv;
    const int64_t vecs = L.row_bytes / 16;
    for (int64_t r = (int64_t)blockIdx.x * kCopyWarps + (threadIdx.x >> 5); r < rows; r += (int64_t)gridDim.x * kCopyWarps) {
        const int64_t at = t0 * L.Hkv + r;
        const int s = L.slots[at], h = (int)(r % L.Hkv);
        if (s < 0) continue;
        const int64_t to = ((int64_t)b * L.capacity + s) * L.Hkv + h;
        for (int64_t x = lane; x < 2 * vecs; x += 32) {
            const bool value = x >= vecs;
            const int64_t c = value ? x - vecs : x;
            const uint4 *src = static_cast<const uint4 *>(value ? L.v : L.k) + at * vecs + c;
            static_cast<uint4 *>(value ? L.v_cache : L.k_cache)[to * vecs + c] = *src;
        }
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        const int len = cached_slots(L.lens_in, L.capacity, b);
        const int32_t seen = L.seen_in[b];
        L.lens_out[b] = (int32_t)min(L.capacity, (int64_t)len + m);
        L.seen_out[b] = seen + m;
    }
}

}  // namespace

size_t cache_insert_workspace(int64_t total_tokens, int Hkv) {
    return ((size_t)total_tokens * Hkv * 4 + 255) & ~(size_t)255;   // places of the new tokens
}

cudaError_t launch_cache_insert(const CacheInsertLaunch &L, cudaStream_t stream) {
    const int64_t uniform_len = L.cu_seqlens ? 0 : L.total_tokens / L.num_seqs;
    cache_select_kernel<<<L.num_seqs * L.Hkv, kSelThreads, 0, stream>>>(L, uniform_len);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    int64_t x = (L.total_tokens * L.Hkv / L.num_seqs + kCopyWarps - 1) / kCopyWarps;
    x = x < 1 ? 1 : x > 4096 ? 4096 : x;
    cache_copy_kernel<<<dim3((unsigned)x, L.num_seqs), kCopyWarps * 32, 0, stream>>>(L, uniform_len);
    return cudaGetLastError();
}

}  // namespace gdn
