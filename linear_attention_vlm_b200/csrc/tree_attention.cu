// Attention of a tree of drafted tokens over a cache of keys and values.
//
// Per (node, query head): scores over the sequence's cached slots and over the
// node and its ancestors, softmax with a running maximum and sum, weighted
// values.  One CTA per (node, head); a thread scores one key of a 128-key
// block, then sums one value channel over the block.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>

#include "tree.cuh"

namespace gdn {
namespace {

constexpr int kD = 128, kKeys = 128;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float dot_row(const __nv_bfloat16 *row, const float *q) {
    float a = 0.f;
    for (int c = 0; c < kD; c += 8) {
        const uint4 u = *reinterpret_cast<const uint4 *>(row + c);
        const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(&u);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            a = fmaf(__low2float(h[e]), q[c + 2 * e], a);
            a = fmaf(__high2float(h[e]), q[c + 2 * e + 1], a);
        }
    }
    return a;
}

__device__ __forceinline__ float block_max(float v, float *red) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    return fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
}

__global__ void __launch_bounds__(kKeys) tree_attention_kernel(const TreeAttnLaunch L, int64_t uniform_len) {
    __shared__ float qs[kD], ps[kKeys], red[4];
    __shared__ unsigned long long anc_sh;
    __shared__ int depth_sh;
    const int tid = threadIdx.x, b = blockIdx.z, h = blockIdx.y, node = blockIdx.x;
    const int kvh = h / (L.Hq / L.Hkv);
    int64_t bos;
    const int n = seq_rows(L.cu_seqlens, uniform_len, L.total_nodes, b, L.max_nodes, bos);
    if (node >= n) return;
    const int len = cached_slots(L.cache_lens, L.capacity, b);
    const int64_t row = (bos + node) * L.Hq + h;
    const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(L.q) + row * kD;
    const __nv_bfloat16 *kc = static_cast<const __nv_bfloat16 *>(L.k_cache), *vc = static_cast<const __nv_bfloat16 *>(L.v_cache);
    const __nv_bfloat16 *kn = static_cast<const __nv_bfloat16 *>(L.k), *vn = static_cast<const __nv_bfloat16 *>(L.v);
    qs[tid] = __bfloat162float(q[tid]) * L.scale * kLog2e;
    if (tid == 0) {
        unsigned long long anc = 0;
        int depth = -1;
        for (int p = node; p >= 0; p = tree_parent(L.parents, bos, p)) {
            if (!L.window || depth + 1 < L.window) anc |= 1ull << p;
            ++depth;
        }
        anc_sh = anc;
        depth_sh = depth;
    }
    __syncthreads();
    const int32_t *pos = L.cache_pos ? L.cache_pos + ((int64_t)b * L.Hkv + kvh) * L.capacity : nullptr;
    const int64_t here = (int64_t)(pos && L.window ? L.seen[b] : len) + depth_sh;
    float m = -INFINITY, l = 0.f, acc = 0.f;
    for (int k0 = 0; k0 < len + n; k0 += kKeys) {
        const int s = k0 + tid;
        float x = -INFINITY;
        if (s < len) {
            if (!L.window || here - (pos ? pos[s] : s) < L.window)
                x = dot_row(kc + (((int64_t)b * L.capacity + s) * L.Hkv + kvh) * kD, qs);
        } else if (s < len + n && (anc_sh >> (s - len) & 1)) {
            x = dot_row(kn + ((bos + s - len) * L.Hkv + kvh) * kD, qs);
        }
        const float mb = fmaxf(m, block_max(x, red));
        const float alpha = mb == -INFINITY ? 1.f : exp2f(m - mb);
        ps[tid] = mb == -INFINITY ? 0.f : exp2f(x - mb);
        m = mb;
        __syncthreads();
        acc *= alpha;
        l *= alpha;
        for (int j = 0; j < kKeys && k0 + j < len + n; ++j) {
            const float p = ps[j];
            if (p == 0.f) continue;
            const int s2 = k0 + j;
            const __nv_bfloat16 *vr = s2 < len ? vc + (((int64_t)b * L.capacity + s2) * L.Hkv + kvh) * kD
                                               : vn + ((bos + s2 - len) * L.Hkv + kvh) * kD;
            l += p;
            acc = fmaf(p, __bfloat162float(vr[tid]), acc);
        }
        __syncthreads();
    }
    static_cast<__nv_bfloat16 *>(L.o)[row * kD + tid] = __float2bfloat16_rn(l > 0.f ? acc / l : 0.f);
    if (L.lse && tid == 0) L.lse[row] = l > 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
}

}  // namespace

size_t tree_attention_workspace() { return 256; }

cudaError_t launch_tree_attention(const TreeAttnLaunch &L, cudaStream_t stream) {
    const int64_t uniform_len = L.cu_seqlens ? 0 : L.total_nodes / L.num_seqs;
    const dim3 grid(L.max_nodes, L.Hq, L.num_seqs);
    tree_attention_kernel<<<grid, kKeys, 0, stream>>>(L, uniform_len);
    return cudaGetLastError();
}

}  // namespace gdn
