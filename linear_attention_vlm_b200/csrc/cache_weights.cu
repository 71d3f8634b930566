// Attention weight that the newest tokens of a sequence lay on every slot of
// its cache and on one another, added up per key.
//
// w[s] += sum over queries i and the heads of the group of
// exp(scale q_i . k_s - lse_i).  A thread owns one key and walks the queries
// in a fixed order, so no sum depends on scheduling.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>

#include "tree.cuh"

namespace gdn {
namespace {

constexpr int kD = 128, kKeys = 128;
constexpr float kLog2e = 1.4426950408889634f;

__global__ void __launch_bounds__(kKeys) cache_weights_kernel(const CacheWeightsLaunch L, int64_t uq, int64_t ut,
                                                              int cache_tiles) {
    __shared__ __nv_bfloat16 qs[kD];
    const int tid = threadIdx.x, kvh = blockIdx.y, b = blockIdx.z;
    const int group = L.Hq / L.Hkv;
    int64_t q0, t0;
    int nq = seq_rows(L.cu_queries, uq, L.total_queries, b, INT32_MAX, q0);
    const int m = seq_rows(L.cu_tokens, ut, L.total_tokens, b, INT32_MAX, t0);
    if (nq > m) {
        q0 += nq - m;
        nq = m;
    }
    const int len = cached_slots(L.cache_lens, L.capacity, b);
    const bool cached = (int)blockIdx.x < cache_tiles;
    const int s = (cached ? blockIdx.x : blockIdx.x - cache_tiles) * kKeys + tid;
    const int lim = cached ? len : m;
    if ((int)(s - tid) >= lim) return;
    const bool mine = s < lim;
    const int64_t slot = ((int64_t)b * L.Hkv + kvh) * L.capacity + s;
    const __nv_bfloat16 *key = cached ? static_cast<const __nv_bfloat16 *>(L.k_cache) + (((int64_t)b * L.capacity + s) * L.Hkv + kvh) * kD
                                      : static_cast<const __nv_bfloat16 *>(L.k) + ((t0 + s) * L.Hkv + kvh) * kD;
    const int64_t seen = L.window && L.cache_pos ? L.seen[b] : len;
    const int64_t kpos = !mine ? 0 : !cached ? seen + s : L.window && L.cache_pos ? L.cache_pos[slot] : s;
    float sum = 0.f;
    for (int i = 0; i < nq; ++i) {
        const int64_t reach = seen + m - nq + i - kpos;
        const bool sees = mine && (cached || reach >= 0) && (!L.window || reach < L.window);
        for (int g = 0; g < group; ++g) {
            const int64_t row = (q0 + i) * L.Hq + kvh * group + g;
            __syncthreads();
            qs[tid] = static_cast<const __nv_bfloat16 *>(L.q)[row * kD + tid];
            __syncthreads();
            const float lse = L.lse[row];
            if (!sees || lse == -INFINITY) continue;
            float x = 0.f;
            for (int c = 0; c < kD; ++c) x = fmaf(__bfloat162float(qs[c]), __bfloat162float(key[c]), x);
            sum += exp2f((x * L.scale - lse) * kLog2e);
        }
    }
    if (!mine) return;
    if (cached) L.w_out[slot] = L.w_in[slot] + sum;
    else L.w_new[(t0 + s) * L.Hkv + kvh] = sum;
}

}  // namespace

size_t cache_weights_workspace() { return 256; }

cudaError_t launch_cache_weights(const CacheWeightsLaunch &L, cudaStream_t stream) {
    const int64_t uq = L.cu_queries ? 0 : L.total_queries / L.num_seqs, ut = L.cu_tokens ? 0 : L.total_tokens / L.num_seqs;
    const int64_t ct = (L.capacity + kKeys - 1) / kKeys, nt = ((L.cu_tokens ? L.total_tokens : ut) + kKeys - 1) / kKeys;
    if (ct + nt == 0) return cudaSuccess;
    cache_weights_kernel<<<dim3((unsigned)(ct + nt), L.Hkv, L.num_seqs), kKeys, 0, stream>>>(L, uq, ut, (int)ct);
    return cudaGetLastError();
}

}  // namespace gdn
