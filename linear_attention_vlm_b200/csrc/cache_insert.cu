// New tokens enter a cache of constant size in place of its lightest slots.
//
// Per (sequence, key/value head) the candidates are the cached slots and the
// new tokens, in this order, each with a 32-bit key that orders them: the
// bits of the weight made monotone, all ones for a recent position, zero for
// NaN.  E = candidates - capacity of them give way: those below the E-th
// smallest key tau and, of the ones equal to it, the latest.  tau is found
// digit by digit (11, 11 and 10 bits), a histogram in shared memory each.
// Evicted slots and empty ones, ascending, take the new tokens that stay, ascending:
// slots that stay do not move, so the rows copied are the new tokens' alone,
// and no copy reads what another writes.
//
// Two kernels: the selection, which also writes weights and positions, then
// the copy of keys and values, one warp per row.  Weights and positions are 8
// bytes a slot and are read once: the keys stay in registers, kKeep a thread.
// What bounds the selection is the chain of histograms (latency, a
// few microseconds), so a (sequence, head) with more candidates than one CTA
// keeps is spread over a cluster of CTAs that read one another's histograms.
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <math.h>

#include "sm100.cuh"
#include "tree.cuh"

namespace gdn {
namespace {

namespace cg = cooperative_groups;

constexpr int kSelThreads = 1024, kSelWarps = kSelThreads / 32;
constexpr int kKeep = 10;          // keys a thread holds: 10240 candidates a CTA; the rest are read again
constexpr int kBins = 2048;
constexpr int kMaxCluster = 8;     // the portable limit
constexpr unsigned kAll = 0xffffffffu;
constexpr uint32_t kProtected = 0xffffffffu, kZero = 0x80000000u;   // keys of recent positions and of weight 0

// order-preserving bits of a weight; NaN below everything, -0 as 0
__device__ __forceinline__ uint32_t weight_key(float w) {
    if (isnan(w)) return 0u;
    const uint32_t u = __float_as_uint(w + 0.f);
    return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}

// One more in hist[digit] for every lane of `on`.  Equal keys share a bin, so
// the lanes that have the first lane's digit add once.
__device__ __forceinline__ void count_digit(unsigned *hist, unsigned on, uint32_t digit) {
    if (!on) return;
    const int lane = threadIdx.x & 31, first = __ffs(on) - 1;
    const uint32_t lead = __shfl_sync(kAll, digit, first);
    const bool in = on >> lane & 1;
    const unsigned same = __ballot_sync(kAll, in && digit == lead);
    if (lane == first) atomicAdd(&hist[lead], __popc(same));
    else if (in && digit != lead) atomicAdd(&hist[digit], 1u);
}

struct Counts {
    int below_slot, below_new, equal_slot, equal_new;   // keys below tau and equal to it, among slots and new tokens
};

__global__ void __launch_bounds__(kSelThreads) cache_select_kernel(const CacheInsertLaunch L, int64_t uniform_len) {
    __shared__ unsigned hist[3][kBins];
    __shared__ int scan_sh[4][kSelWarps];
    __shared__ Counts tot_sh;
    __shared__ int found_sh[2];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    cg::cluster_group cluster = cg::this_cluster();
    const int ctas = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    auto sync_all = [&] {
        if (ctas > 1) cluster.sync();
        else __syncthreads();
    };
    const int bh = blockIdx.x / ctas, b = bh / L.Hkv, h = bh % L.Hkv;
    sm100::grid_dep_launch();
    int64_t t0;
    const int m = seq_rows(L.cu_seqlens, uniform_len, L.total_tokens, b, INT32_MAX, t0);
    const int cap = (int)L.capacity;
    const int len = cached_slots(L.lens_in, L.capacity, b);
    const int64_t seen = L.seen_in[b];
    const int C = len + m, keep = min(cap, C), evict = C - keep;
    const int64_t base = ((int64_t)b * L.Hkv + h) * cap;
    auto new_weight = [&](int j) { return L.w_new ? L.w_new[(t0 + j) * L.Hkv + h] : 0.f; };
    const int32_t *pos_in = L.pos_in + base;
    const float *w_in = L.w_in + base;
    // positions above `old` are among the last `recent`
    const int old = (int)max((int64_t)INT32_MIN, min((int64_t)INT32_MAX, seen + m - L.recent - 1));
    auto key_of = [&](int i) -> uint32_t {
        if (i < len) {
            const int pos = pos_in[i];
            const float w = w_in[i];
            return pos > old ? kProtected : weight_key(w);
        }
        return C - i <= L.recent ? kProtected : weight_key(new_weight(i - len));
    };
    // a warp owns `rounds` x 32 consecutive candidates from c0 on, so ranks are running counts
    const int rounds = (int)(((int64_t)C + ctas * kSelThreads - 1) / (ctas * kSelThreads));
    const int64_t c0_ = ((int64_t)rank * kSelWarps + warp) * rounds * 32;
    const int c0 = (int)min((int64_t)C, c0_);
    uint32_t kept[kKeep];
    if (evict > 0) {
#pragma unroll
        for (int k = 0; k < kKeep; ++k) {
            const int i = c0 + 32 * k + lane;
            kept[k] = k < rounds && i < C ? key_of(i) : 0u;
        }
    }
    // calls f(first candidate, mask of those that exist, key) for the warp's rounds, all lanes together
    auto walk = [&](auto f) {
        const int left = C - c0;
#pragma unroll
        for (int k = 0; k < kKeep; ++k) {
            if (k >= rounds || 32 * k >= left) break;
            f(c0 + 32 * k, left - 32 * k >= 32 ? kAll : (1u << (left - 32 * k)) - 1, kept[k]);
        }
        for (int k = kKeep; k < rounds && 32 * k < left; ++k) {
            const int i = c0 + 32 * k + lane;
            f(c0 + 32 * k, left - 32 * k >= 32 ? kAll : (1u << (left - 32 * k)) - 1, evict > 0 && i < C ? key_of(i) : 0u);
        }
    };
    // which of 32 candidates from i on are slots
    auto slots_of = [&](int i) { return i + 32 <= len ? kAll : i >= len ? 0u : (1u << (len - i)) - 1; };

    // tau, and how many of the candidates equal to it give way
    uint32_t tau = 0;
    int ties = 0;
    if (evict > 0) {
        for (int i = tid; i < 3 * kBins; i += kSelThreads) (&hist[0][0])[i] = 0;
        __syncthreads();
        int rest = evict;
#pragma unroll 1
        for (int pass = 0; pass < 3; ++pass) {
            const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 1 ? 11 : 10;   // of the later passes
            if (pass == 0) {
                // the two keys that many candidates share are counted apart
                int recents = 0, zeros = 0;
                walk([&](int, unsigned in, uint32_t key) {
                    const unsigned r = __ballot_sync(kAll, key == kProtected) & in, z = __ballot_sync(kAll, key == kZero) & in;
                    recents += __popc(r);
                    zeros += __popc(z);
                    count_digit(hist[0], in & ~(r | z), key >> 21);
                });
                if (lane == 0 && recents) atomicAdd(&hist[0][kProtected >> 21], recents);
                if (lane == 0 && zeros) atomicAdd(&hist[0][kZero >> 21], zeros);
            } else {
                walk([&](int, unsigned in, uint32_t key) {
                    const unsigned on = __ballot_sync(kAll, (key ^ tau) >> (shift + bits) == 0) & in;
                    count_digit(hist[pass], on, (key >> shift) & ((1u << bits) - 1));
                });
            }
            sync_all();
            // bins 2 tid, 2 tid + 1 of all CTAs, and what lies before them
            unsigned n0 = 0, n1 = 0;
            for (int c = 0; c < ctas; ++c) {
                const unsigned *other = ctas > 1 ? cluster.map_shared_rank(&hist[pass][0], c) : hist[pass];
                const uint2 v = *reinterpret_cast<const uint2 *>(other + 2 * tid);
                n0 += v.x;
                n1 += v.y;
            }
            int incl = (int)(n0 + n1);
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int t = __shfl_up_sync(kAll, incl, o);
                if (lane >= o) incl += t;
            }
            if (lane == 31) scan_sh[0][warp] = incl;
            __syncthreads();
            int add = lane < warp ? scan_sh[0][lane] : 0;
            add = __reduce_add_sync(kAll, add);
            const int before = add + incl - (int)(n0 + n1);
            if (before < rest && rest <= before + (int)(n0 + n1)) {
                const bool second = rest > before + (int)n0;
                found_sh[0] = 2 * tid + second;
                found_sh[1] = rest - before - (second ? (int)n0 : 0);
            }
            __syncthreads();
            tau |= (uint32_t)found_sh[0] << shift;
            rest = found_sh[1];
        }
        ties = rest;
    }

    // counts before this warp, over the cluster
    Counts mine = {0, 0, 0, 0};
    if (evict > 0)
        walk([&](int i, unsigned in, uint32_t key) {
            const unsigned below = __ballot_sync(kAll, key < tau) & in, same = __ballot_sync(kAll, key == tau) & in;
            if (!(below | same)) return;
            const unsigned slots = slots_of(i);
            mine.below_slot += __popc(below & slots);
            mine.below_new += __popc(below & ~slots);
            mine.equal_slot += __popc(same & slots);
            mine.equal_new += __popc(same & ~slots);
        });
    __syncthreads();
    if (lane == 0) {
        scan_sh[0][warp] = mine.below_slot;
        scan_sh[1][warp] = mine.below_new;
        scan_sh[2][warp] = mine.equal_slot;
        scan_sh[3][warp] = mine.equal_new;
    }
    __syncthreads();
    int pre[4], all[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int v = scan_sh[e][lane];
        pre[e] = __reduce_add_sync(kAll, lane < warp ? v : 0);
        all[e] = __reduce_add_sync(kAll, v);
    }
    if (ctas > 1) {
        if (tid == 0) tot_sh = Counts{all[0], all[1], all[2], all[3]};
        cluster.sync();
#pragma unroll
        for (int e = 0; e < 4; ++e) all[e] = 0;
        for (int c = 0; c < ctas; ++c) {
            const Counts o = *cluster.map_shared_rank(&tot_sh, c);
            const int v[4] = {o.below_slot, o.below_new, o.equal_slot, o.equal_new};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (c < rank) pre[e] += v[e];
                all[e] += v[e];
            }
        }
    }
    // the last `ties` of the equal ones give way: those from the `stay`-th on
    const int stay = all[2] + all[3] - ties;
    int equal = pre[2] + pre[3];                                     // equal ones before
    int gone = pre[0] + max(0, pre[2] - stay);                       // evicted slots before
    const int all_gone = all[0] + max(0, all[2] - stay);
    int entered = max(0, c0 - len) - pre[1] - max(0, equal - max(stay, pre[2]));   // new tokens that stay before

    // places for the new tokens, ascending: evicted slots, then empty ones
    int32_t *places = static_cast<int32_t *>(L.workspace) + (int64_t)h * L.total_tokens + t0;
    for (int s = len + rank * kSelThreads + tid; s < keep; s += ctas * kSelThreads) places[all_gone + s - len] = s;
    const unsigned lower = (1u << lane) - 1;
    const bool copy = L.w_out != L.w_in || L.pos_out != L.pos_in;
    walk([&](int i0, unsigned in, uint32_t key) {
        unsigned leave = 0;
        if (evict > 0) {
            const unsigned same = __ballot_sync(kAll, key == tau) & in;
            leave = __ballot_sync(kAll, key < tau) & in;
            if (same) {
                leave |= __ballot_sync(kAll, key == tau && equal + __popc(same & lower) >= stay) & in;
                equal += __popc(same);
            }
        }
        const unsigned slots = slots_of(i0) & in, out = leave & slots, enter = in & ~slots & ~leave;
        const int i = i0 + lane;
        if (slots >> lane & 1) {
            if (out >> lane & 1) {
                places[gone + __popc(out & lower)] = i;
            } else if (copy) {
                L.w_out[base + i] = w_in[i];
                L.pos_out[base + i] = pos_in[i];
            }
        } else if (in >> lane & 1) {
            L.slots[(t0 + i - len) * L.Hkv + h] = leave >> lane & 1 ? -1 : entered + __popc(enter & lower);   // a rank for now
        }
        gone += __popc(out);
        entered += __popc(enter);
    });
    sync_all();
    for (int64_t j = rank * kSelThreads + tid; j < m; j += ctas * kSelThreads) {
        int32_t *slot = L.slots + (t0 + j) * L.Hkv + h;
        const int r = *slot;
        if (r < 0) continue;
        const int s = places[r];
        *slot = s;
        L.w_out[base + s] = new_weight((int)j);
        L.pos_out[base + s] = (int32_t)(seen + j);
    }
}

constexpr int kCopyWarps = 8;

__global__ void __launch_bounds__(kCopyWarps * 32) cache_copy_kernel(const CacheInsertLaunch L, int64_t uniform_len) {
    const int b = blockIdx.y, lane = threadIdx.x & 31;
    sm100::grid_dep_wait();
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
    // a cluster per (sequence, head) where its candidates, at the sequences'
    // mean, are more than one CTA keeps, or where SMs would stay idle
    const int64_t candidates = L.capacity + (L.total_tokens + L.num_seqs - 1) / L.num_seqs;
    const int64_t lists = (int64_t)L.num_seqs * L.Hkv;
    int ctas = 1;
    while (ctas < kMaxCluster && (candidates > (int64_t)ctas * kKeep * kSelThreads ||
                                  (2 * ctas * lists <= 148 && candidates > 2048 * ctas)))
        ctas *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(L.num_seqs * L.Hkv * ctas));
    cfg.blockDim = dim3(kSelThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ctas;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, cache_select_kernel, L, uniform_len);
    if (e != cudaSuccess) return e;
    int64_t x = (L.total_tokens * L.Hkv / L.num_seqs + kCopyWarps - 1) / kCopyWarps;
    x = x < 1 ? 1 : x > 4096 ? 4096 : x;
    cfg.gridDim = dim3((unsigned)x, L.num_seqs);
    cfg.blockDim = dim3(kCopyWarps * 32);
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    return cudaLaunchKernelEx(&cfg, cache_copy_kernel, L, uniform_len);
}

}  // namespace gdn
