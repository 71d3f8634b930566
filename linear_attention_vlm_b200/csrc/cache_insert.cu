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
// The selection also writes weights and positions; keys and values are copied
// by it or by a second kernel, one warp per row.  Weights and positions are 8
// bytes a slot and are read once: the keys stay in registers, kKeep a thread.
// What bounds the selection is the chain of histograms, scans and walks over
// the keys, each a barrier apart: 19 us for 8192 slots, of which the bytes take
// 3, for one list and for 128 alike.  A (sequence, head) with more candidates
// than one CTA keeps is spread over a cluster of CTAs that read one another's
// histograms: 34 against 79 us for 40960 candidates.  With fewer the barriers
// of a cluster cost more than the shared work gives (23 against 19.5 us, 8193
// candidates over 4 CTAs).
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
constexpr int kRowsAhead = 4;      // rows of a warp in flight
constexpr int64_t kWholeBytes = 64 << 10;
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

__device__ __forceinline__ void write_counts(const CacheInsertLaunch &L, int b, int len, int m) {
    const int32_t seen = L.seen_in[b];
    L.lens_out[b] = (int32_t)min(L.capacity, (int64_t)len + m);
    L.seen_out[b] = seen + m;
}

struct Counts {
    int below_slot, below_new, equal_slot, equal_new;   // keys below tau and equal to it, among slots and new tokens
};

__global__ void __launch_bounds__(kSelThreads) cache_select_kernel(const CacheInsertLaunch L, int64_t uniform_len, int ctas,
                                                                    bool whole) {
    __shared__ unsigned hist[3][kBins];
    __shared__ int scan_sh[4][kSelWarps];
    __shared__ Counts tot_sh;
    __shared__ int found_sh[2];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank() % ctas, first = (int)cluster.block_rank() - rank;
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
    // a warp owns `rounds` x 32 consecutive candidates from c0 on, so ranks are
    // running counts; a lane without one has the highest key, which no histogram
    // minds, and is told apart where it matters
    const int rounds = (int)(((int64_t)C + ctas * kSelThreads - 1) / (ctas * kSelThreads));
    const int c0 = (int)min((int64_t)C, ((int64_t)rank * kSelWarps + warp) * rounds * 32);
    uint32_t kept[kKeep];
    auto load_key = [&](int k) -> uint32_t {
        const int i = c0 + 32 * k + lane;
        return i < C ? key_of(i) : kProtected;
    };
    if (evict > 0) {
        // slots alone: all loads first
        if (c0 + 32 * min(rounds, kKeep) <= len) {
            float w[kKeep];
            int pos[kKeep];
#pragma unroll
            for (int k = 0; k < kKeep; ++k) {
                w[k] = 0.f;
                pos[k] = 0;
                if (k < rounds) {
                    w[k] = w_in[c0 + 32 * k + lane];
                    pos[k] = pos_in[c0 + 32 * k + lane];
                }
            }
#pragma unroll
            for (int k = 0; k < kKeep; ++k) kept[k] = pos[k] > old ? kProtected : weight_key(w[k]);
        } else {
#pragma unroll
            for (int k = 0; k < kKeep; ++k) kept[k] = k < rounds ? load_key(k) : kProtected;
        }
    }
    // calls f(first candidate, key) for the warp's rounds, all lanes together
    auto walk = [&](auto f) {
#pragma unroll
        for (int k = 0; k < kKeep; ++k)
            if (k < rounds) f(c0 + 32 * k, kept[k]);
#pragma unroll 1
        for (int k = kKeep; k < rounds; ++k) f(c0 + 32 * k, evict > 0 ? load_key(k) : 0u);
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
                walk([&](int, uint32_t key) {
                    const bool r = key == kProtected, z = key == kZero;
                    recents += r;
                    zeros += z;
                    count_digit(hist[0], __ballot_sync(kAll, !r && !z), key >> 21);
                });
                recents = __reduce_add_sync(kAll, recents);
                zeros = __reduce_add_sync(kAll, zeros);
                if (lane == 0) {
                    atomicAdd(&hist[0][kProtected >> 21], recents);
                    atomicAdd(&hist[0][kZero >> 21], zeros);
                }
            } else {
                walk([&](int, uint32_t key) {
                    count_digit(hist[pass], __ballot_sync(kAll, (key ^ tau) >> (shift + bits) == 0), (key >> shift) & ((1u << bits) - 1));
                });
            }
            sync_all();
            // bins 2 tid, 2 tid + 1 of all CTAs, and what lies before them
            unsigned n0 = 0, n1 = 0;
            for (int c = 0; c < ctas; ++c) {
                const unsigned *other = ctas > 1 ? cluster.map_shared_rank(&hist[pass][0], first + c) : hist[pass];
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
        walk([&](int i0, uint32_t key) {
            // a lane's own counts
            const int i = i0 + lane;
            if (key <= tau && i < C) {
                const bool same = key == tau, slot = i < len;
                mine.below_slot += !same && slot;
                mine.below_new += !same && !slot;
                mine.equal_slot += same && slot;
                mine.equal_new += same && !slot;
            }
        });
    mine.below_slot = __reduce_add_sync(kAll, mine.below_slot);
    mine.below_new = __reduce_add_sync(kAll, mine.below_new);
    mine.equal_slot = __reduce_add_sync(kAll, mine.equal_slot);
    mine.equal_new = __reduce_add_sync(kAll, mine.equal_new);
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
            const Counts o = *cluster.map_shared_rank(&tot_sh, first + c);
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
    walk([&](int i0, uint32_t key) {
        const int i = i0 + lane;
        const bool here = i < C;
        unsigned leave = 0;
        if (evict > 0 && __any_sync(kAll, here && key <= tau)) {
            const unsigned same = __ballot_sync(kAll, here && key == tau);
            leave = __ballot_sync(kAll, here && (key < tau || (key == tau && equal + __popc(same & lower) >= stay)));
            equal += __popc(same);
        }
        if (i0 + 32 <= len && !leave && !copy) return;
        const unsigned in = __ballot_sync(kAll, here), slots = slots_of(i0) & in, out = leave & slots, enter = in & ~slots & ~leave;
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
    // A new token that stays: its slot, weight and position.  (Where cu_seqlens
    // decreases, sequences share tokens and may find one another's ranks.)
    auto settle = [&](int64_t j) -> int {
        int32_t *slot = L.slots + (t0 + j) * L.Hkv + h;
        const int r = *slot;
        const int s = (unsigned)r < (unsigned)m ? places[r] : -1;
        if ((unsigned)s >= (unsigned)cap) {
            if (r >= 0) *slot = -1;
            return -1;
        }
        *slot = s;
        L.w_out[base + s] = new_weight((int)j);
        L.pos_out[base + s] = (int32_t)(seen + j);
        return s;
    };
    if (!whole) {
        // four a thread at a time, so that their loads overlap
        const int64_t all_threads = ctas * kSelThreads;
        for (int64_t j = rank * kSelThreads + tid; j < m; j += 4 * all_threads) {
            int r[4], s[4];
            float w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int64_t at = j + e * all_threads;
                r[e] = at < m ? L.slots[(t0 + at) * L.Hkv + h] : -1;
                w[e] = at < m ? new_weight((int)at) : 0.f;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) s[e] = (unsigned)r[e] < (unsigned)m ? places[r[e]] : -1;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int64_t at = j + e * all_threads;
                if ((unsigned)s[e] >= (unsigned)cap) {
                    if (r[e] >= 0) L.slots[(t0 + at) * L.Hkv + h] = -1;
                    continue;
                }
                L.slots[(t0 + at) * L.Hkv + h] = s[e];
                L.w_out[base + s[e]] = w[e];
                L.pos_out[base + s[e]] = (int32_t)(seen + at);
            }
        }
        return;
    }
    // and its key and value, kRowsAhead rows of a warp at a time, so that their loads overlap
    const int64_t vecs = L.row_bytes / 16;
    for (int64_t j0 = (rank * kSelWarps + warp) * kRowsAhead; j0 < m; j0 += ctas * kSelWarps * kRowsAhead) {
        const int mine = lane < kRowsAhead && j0 + lane < m ? settle(j0 + lane) : -1;
        int slot[kRowsAhead];
#pragma unroll
        for (int e = 0; e < kRowsAhead; ++e) slot[e] = __shfl_sync(kAll, mine, e);
        for (int64_t x = lane; x < 2 * vecs; x += 32) {
            const bool value = x >= vecs;
            const int64_t c = value ? x - vecs : x;
            const uint4 *src = static_cast<const uint4 *>(value ? L.v : L.k) + ((t0 + j0) * L.Hkv + h) * vecs + c;
            uint4 *dst = static_cast<uint4 *>(value ? L.v_cache : L.k_cache) + ((int64_t)b * cap * L.Hkv + h) * vecs + c;
            uint4 data[kRowsAhead];
#pragma unroll
            for (int e = 0; e < kRowsAhead; ++e)
                if (slot[e] >= 0) data[e] = src[(int64_t)e * L.Hkv * vecs];
#pragma unroll
            for (int e = 0; e < kRowsAhead; ++e)
                if (slot[e] >= 0) dst[(int64_t)slot[e] * L.Hkv * vecs] = data[e];
        }
    }
    // every head has read the counts
    if (L.Hkv * ctas > 1) cluster.sync();
    if (h == 0 && rank == 0 && tid == 0) write_counts(L, b, len, m);
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
    if (blockIdx.x == 0 && threadIdx.x == 0) write_counts(L, b, cached_slots(L.lens_in, L.capacity, b), m);
}

}  // namespace

size_t cache_insert_workspace(int64_t total_tokens, int Hkv) {
    return ((size_t)total_tokens * Hkv * 4 + 255) & ~(size_t)255;   // places of the new tokens
}

cudaError_t launch_cache_insert(const CacheInsertLaunch &L, cudaStream_t stream) {
    static int sms[64] = {0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!sms[dev]) {
        e = cudaDeviceGetAttribute(&sms[dev], cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return e;
    }
    const int64_t uniform_len = L.cu_seqlens ? 0 : L.total_tokens / L.num_seqs;
    // a cluster per (sequence, head) where its candidates, at the sequences'
    // mean, are more than one CTA keeps
    const int64_t candidates = L.capacity + (L.total_tokens + L.num_seqs - 1) / L.num_seqs;
    int ctas = 1;
    while (ctas < kMaxCluster && candidates > (int64_t)ctas * kKeep * kSelThreads)
        ctas *= 2;
    // The kernel that selects copies too, in one cluster of all heads of a
    // sequence (whose counts are written once all have read them), where a CTA
    // has few rows or the lists alone fill the SMs.  With both sides' kernels at
    // 8192 slots of 2 heads of 128 in bf16: 19.0 against 19.8 us for 64
    // sequences of 4 tokens, 45 against 55 of 1024; one sequence of 1 token 19.0
    // against 19.5, of 256 23.3 against 20.0.  A launch less is 2 us of the host.
    // The lengths of the lists are not known here, only their mean: a list far above it is
    // left to one CTA a head (one of 16384 tokens among 63 of one token takes
    // 195 us, alone 30).
    const int64_t list_bytes = 2 * (L.total_tokens / L.num_seqs) * L.row_bytes;
    const bool whole = ctas == 1 && L.Hkv <= kMaxCluster &&
                       (list_bytes <= kWholeBytes || 2 * (int64_t)L.num_seqs * L.Hkv >= sms[dev]);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(L.num_seqs * L.Hkv * ctas));
    cfg.blockDim = dim3(kSelThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = whole ? L.Hkv * ctas : ctas;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, cache_select_kernel, L, uniform_len, ctas, whole);
    if (e != cudaSuccess || whole) return e;
    int64_t x = (L.total_tokens * L.Hkv / L.num_seqs + kCopyWarps - 1) / kCopyWarps;
    x = x < 1 ? 1 : x > 4096 ? 4096 : x;
    cfg.gridDim = dim3((unsigned)x, L.num_seqs);
    cfg.blockDim = dim3(kCopyWarps * 32);
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    return cudaLaunchKernelEx(&cfg, cache_copy_kernel, L, uniform_len);
}

}  // namespace gdn
