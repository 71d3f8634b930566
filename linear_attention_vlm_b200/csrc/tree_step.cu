// Gated DeltaNet over a tree of drafted tokens, from one state per sequence
// and head, without forming the states of the nodes.
//
// With anc(i) the node and its ancestors, G_i = sum of g over anc(i) and S the
// state before the tree, unrolling the recurrence along a path gives
//   S_i = exp(G_i) S + sum_{j in anc(i)} exp(G_i - G_j) u_j k_j^T
//   u_i = beta_i (v_i - exp(G_i) S k_i - sum_{j in anc(i), j != i} exp(G_i - G_j) (k_j . k_i) u_j)
//   o_i = exp(G_i) S q_i + sum_{j in anc(i)} exp(G_i - G_j) (k_j . q_i) u_j
// The exponents are sums of g over part of a path, so no factor exceeds 1.
// The products with S do not depend on the tree; u_i is solved node by node,
// every value channel (row of S) on its own.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "gdn.h"
#include "tree.cuh"

namespace gdn {
namespace {

// One CTA per (sequence, head), a thread per value channel.
template <typename T, int D>
__global__ void __launch_bounds__(D) tree_step_kernel(const TreeStepLaunch L, int64_t uniform_len) {
    extern __shared__ float sm[];
    float *ks = sm;                        // [64][D]
    float *qs = ks + kMaxNodes * D;        // [64][D]
    float *us = qs + kMaxNodes * D;        // [64][D], a thread's own column
    float *kk = us + kMaxNodes * D;        // [64][64] exp(G_i - G_j) k_j . k_i, 0 where j is no ancestor
    float *qk = kk + kMaxNodes * kMaxNodes;
    __shared__ float Gs[kMaxNodes];
    __shared__ unsigned long long anc[kMaxNodes];
    const int tid = threadIdx.x, b = blockIdx.x / L.H, h = blockIdx.x % L.H;
    int64_t bos;
    const int n = seq_rows(L.cu_seqlens, uniform_len, L.total_nodes, b, L.max_nodes, bos);
    const T *q = static_cast<const T *>(L.q), *k = static_cast<const T *>(L.k), *v = static_cast<const T *>(L.v);
    for (int i = 0; i < n; ++i) {
        const int64_t at = ((bos + i) * L.H + h) * D + tid;
        ks[i * D + tid] = to_f32(k[at]);
        qs[i * D + tid] = to_f32(q[at]);
    }
    if (tid < n) {
        unsigned long long a = 0;
        float G = 0.f;
        for (int p = tid; p >= 0; p = tree_parent(L.parents, bos, p)) {
            a |= 1ull << p;
            G += L.g[(bos + p) * L.H + h];
        }
        anc[tid] = a;
        Gs[tid] = G;
    }
    __syncthreads();
    for (int e = tid; e < n * n; e += D) {
        const int i = e / n, j = e % n;
        float a = 0.f, c = 0.f;
        if (anc[i] >> j & 1) {
            for (int x = 0; x < D; ++x) {
                a = fmaf(ks[j * D + x], ks[i * D + x], a);
                c = fmaf(ks[j * D + x], qs[i * D + x], c);
            }
            const float f = expf(Gs[i] - Gs[j]);
            a *= f;
            c *= f;
        }
        kk[i * kMaxNodes + j] = a;
        qk[i * kMaxNodes + j] = c;
    }
    __syncthreads();
    const float *srow = L.state ? L.state + ((int64_t)blockIdx.x * D + tid) * D : nullptr;
    for (int i = 0; i < n; ++i) {
        float sk = 0.f, sq = 0.f;
        if (srow)
            for (int x = 0; x < D; ++x) {
                const float s = srow[x];
                sk = fmaf(s, ks[i * D + x], sk);
                sq = fmaf(s, qs[i * D + x], sq);
            }
        const float gamma = expf(Gs[i]);
        const int64_t at = (bos + i) * L.H + h;
        float u = to_f32(v[at * D + tid]) - gamma * sk, o = gamma * sq;
        for (int j = 0; j < i; ++j) {
            u = fmaf(-kk[i * kMaxNodes + j], us[j * D + tid], u);
            o = fmaf(qk[i * kMaxNodes + j], us[j * D + tid], o);
        }
        u *= L.beta[at];
        us[i * D + tid] = u;
        o = fmaf(qk[i * kMaxNodes + i], u, o);
        static_cast<T *>(L.out)[at * D + tid] = from_f32<T>(o);
    }
}

template <typename T, int D>
cudaError_t launch(const TreeStepLaunch &L, cudaStream_t stream) {
    const int64_t uniform_len = L.cu_seqlens ? 0 : L.total_nodes / L.num_seqs;
    const int smem = (3 * kMaxNodes * D + 2 * kMaxNodes * kMaxNodes) * 4;
    cudaError_t e = cudaFuncSetAttribute(tree_step_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    tree_step_kernel<T, D><<<L.num_seqs * L.H, D, smem, stream>>>(L, uniform_len);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_tree_step(const TreeStepLaunch &L, cudaStream_t stream) {
    if (L.dtype == GDN_F32) return L.d == 128 ? launch<float, 128>(L, stream) : launch<float, 64>(L, stream);
    return L.d == 128 ? launch<__nv_bfloat16, 128>(L, stream) : launch<__nv_bfloat16, 64>(L, stream);
}

}  // namespace gdn
