// Gated DeltaNet over a tree of drafted tokens, from one state per sequence
// and head, without forming the states of the nodes.
//
// With anc(i) the node and its ancestors, G_i = sum of g over anc(i) and S the
// state before the tree, unrolling the recurrence along a path gives
//   S_i = e^G_i S + sum_{j in anc(i)} e^(G_i - G_j) u_j k_j^T
//   (I + A) U = R,   R_i = beta_i (v_i - e^G_i S k_i),   A_ij = beta_i e^(G_i - G_j) k_i . k_j  (j a proper ancestor)
//   o_i = e^G_i S q_i + sum_j M_ij R_j,   M = P (I + A)^-1,   P_ij = e^(G_i - G_j) q_i . k_j  (j in anc(i))
// The exponents are sums of g over part of a path, so no factor exceeds 1.
// Only S k and S q touch the state, and M needs no state at all: it is found by
// back substitution, a thread per row, while the tensor cores form S k and S q.
//
// What bounds it: the state, 4 d^2 bytes per head, read once; then the products
// (2 + 2 splits) n d^2.  One CTA per (sequence, head).  A warp owns 16 rows of S
// (value channels), which go from memory straight into the A fragments of
// mma.sync: lane quads read 64 consecutive bytes of a row, and the keys and
// queries are read in the same order of channels, so no shuffle or shared
// memory is needed for S.  The result fragments (value channel x node) are the
// A fragments of the second product, with M: nothing of size n x d leaves the
// registers between them.  (tcgen05, with S as bf16 pairs in tensor memory and the rows of
// keys and queries read once instead of by every warp, is not built: it would serve
// the larger trees.)
// With d = 128 in bf16, 64 sequences of 16 heads (67 MB of state) take 19.1 us
// at 4 nodes and 21.6 at 16 (3.7 TB/s with the rows); at 64 nodes 78, where
// the chain of the substitution (64 steps in two warps) and the products that
// wait for it take the time.  One sequence of 7 nodes takes 4.3, a launch's latency.
//
// Precision: with bf16 inputs S, R and M enter as hi + lo bf16 pairs (2^-17
// relative, far below the rounding of the output); with fp32 inputs every
// operand is split into two tf32 numbers and three products are taken (2^-21);
// the errors are then those of a plain fp32 evaluation token by token (1.3e-7 to 1.9e-7
// in the norm, whatever the gates; 1.6e-7 to 2.5e-7).  All sums are fp32, but the sums of g
// along a path, which are pairs of fp32: a decay is the exponential of the difference
// of two of them.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "gdn.h"
#include "tree.cuh"

namespace gdn {
namespace {

__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_tf32(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float4 load_stream(const float *p) {   // read once: keep it out of L1
    float4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(p));
    return v;
}

// 16 bytes to shared memory without passing a register; zeros where `there` is false.
__device__ __forceinline__ void copy16(void *dst, const void *src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(sm100::smem_u32(dst)), "l"(src), "r"(there ? 16 : 0) : "memory");
}

__device__ __forceinline__ uint32_t pack2(float x, float y) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// hi + lo = (x, y) up to 2^-17, two bf16 each
__device__ __forceinline__ void split_bf16(float x, float y, uint32_t &hi, uint32_t &lo) {
    hi = pack2(x, y);
    lo = pack2(x - __uint_as_float(hi << 16), y - __uint_as_float(hi & 0xffff0000u));
}

// hi + lo = x up to 2^-21: 11 significant bits each, hi rounded to nearest, so
// that lo has either sign and what the unit cuts off it does not add up.  A NaN
// stays one in lo.  (cvt.rna.tf32 rounds alike and took a quarter more time.)
__device__ __forceinline__ void split_tf32(float x, uint32_t &hi, uint32_t &lo) {
    hi = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;
    lo = __float_as_uint(x - __uint_as_float(hi));
}

// (h, l) += (x, y), each a sum of two floats that do not overlap: 2^-46 relative
// for terms of one sign.
__device__ __forceinline__ void add_two(float &h, float &l, float x, float y) {
    const float s = __fadd_rn(h, x), d = __fsub_rn(s, h);
    const float e = __fadd_rn(__fadd_rn(__fsub_rn(h, __fsub_rn(s, d)), __fsub_rn(x, d)), __fadd_rn(l, y));
    h = __fadd_rn(s, e);
    l = __fsub_rn(e, __fsub_rn(h, s));
}

// The product fragments of 16 channels.  An A fragment holds two rows (lane
// group g = lane / 4: rows g and g + 8), a B fragment one (row g); of a row, lane
// t = lane % 4 has channels 4 t .. 4 t + 3.  Both sides use the same order, so
// the sum over channels is the same.
template <typename T> struct Frag;

template <> struct Frag<__nv_bfloat16> {
    struct A { uint32_t hi[4], lo[4]; };
    struct B { uint32_t b[2]; };
    static constexpr int kPad = 16;     // elements behind a row of keys: conflict-free 8-byte reads
    __device__ static float exp(float x) { return __expf(x); }
    __device__ static void split(const float4 &u, const float4 &w, A &a) {
        split_bf16(u.x, u.y, a.hi[0], a.lo[0]);
        split_bf16(w.x, w.y, a.hi[1], a.lo[1]);
        split_bf16(u.z, u.w, a.hi[2], a.lo[2]);
        split_bf16(w.z, w.w, a.hi[3], a.lo[3]);
    }
    __device__ static void load_b(const __nv_bfloat16 *row, B &b) {
        const uint2 v = *reinterpret_cast<const uint2 *>(row);
        b.b[0] = v.x;
        b.b[1] = v.y;
    }
    __device__ static void mma(float (&c)[4], const A &a, const B &b) {
        mma_bf16(c, a.hi, b.b[0], b.b[1]);
        mma_bf16(c, a.lo, b.b[0], b.b[1]);
    }
    // keys and queries as A rows: exact in bf16
    __device__ static void mma_rows(float (&c)[4], const __nv_bfloat16 *r0, const __nv_bfloat16 *r1, const B &b) {
        const uint2 u = *reinterpret_cast<const uint2 *>(r0), w = *reinterpret_cast<const uint2 *>(r1);
        const uint32_t a[4] = {u.x, w.x, u.y, w.y};
        mma_bf16(c, a, b.b[0], b.b[1]);
    }
    // R (two accumulator fragments, 16 nodes) times M (row of node i: m at nodes 2t, 2t + 1 of each fragment)
    __device__ static void mma_nodes(float (&c)[4], const float (&x)[4], const float (&y)[4], const float2 &m0, const float2 &m1) {
        uint32_t hi[4], lo[4], mh[2], ml[2];
        split_bf16(x[0], x[1], hi[0], lo[0]);
        split_bf16(x[2], x[3], hi[1], lo[1]);
        split_bf16(y[0], y[1], hi[2], lo[2]);
        split_bf16(y[2], y[3], hi[3], lo[3]);
        split_bf16(m0.x, m0.y, mh[0], ml[0]);
        split_bf16(m1.x, m1.y, mh[1], ml[1]);
        mma_bf16(c, lo, mh[0], mh[1]);
        mma_bf16(c, hi, ml[0], ml[1]);
        mma_bf16(c, hi, mh[0], mh[1]);
    }
};

template <> struct Frag<float> {
    struct A { uint32_t hi[2][4], lo[2][4]; };
    struct B { uint32_t hi[4], lo[4]; };
    static constexpr int kPad = 16;     // conflict-free 16-byte reads
    __device__ static float exp(float x) { return expf(x); }
    __device__ static void split(const float4 &u, const float4 &w, A &a) {
        split_tf32(u.x, a.hi[0][0], a.lo[0][0]);
        split_tf32(w.x, a.hi[0][1], a.lo[0][1]);
        split_tf32(u.y, a.hi[0][2], a.lo[0][2]);
        split_tf32(w.y, a.hi[0][3], a.lo[0][3]);
        split_tf32(u.z, a.hi[1][0], a.lo[1][0]);
        split_tf32(w.z, a.hi[1][1], a.lo[1][1]);
        split_tf32(u.w, a.hi[1][2], a.lo[1][2]);
        split_tf32(w.w, a.hi[1][3], a.lo[1][3]);
    }
    __device__ static void load_b(const float *row, B &b) {
        const float4 v = *reinterpret_cast<const float4 *>(row);
        split_tf32(v.x, b.hi[0], b.lo[0]);
        split_tf32(v.y, b.hi[1], b.lo[1]);
        split_tf32(v.z, b.hi[2], b.lo[2]);
        split_tf32(v.w, b.hi[3], b.lo[3]);
    }
    // The unit cuts its sums, always towards zero, so a long sum in it drifts
    // (1e-6 over 128 channels).  It gets 16 channels at a time, the small products
    // first, and what it has is added here, rounded.
    __device__ static void mma(float (&c)[4], const A &a, const B &b) {
        float x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            mma_tf32(x, a.lo[s], b.hi[2 * s], b.hi[2 * s + 1]);
            mma_tf32(x, a.hi[s], b.lo[2 * s], b.lo[2 * s + 1]);
        }
#pragma unroll
        for (int s = 0; s < 2; ++s) mma_tf32(x, a.hi[s], b.hi[2 * s], b.hi[2 * s + 1]);
#pragma unroll
        for (int e = 0; e < 4; ++e) c[e] += x[e];
    }
    __device__ static void mma_rows(float (&c)[4], const float *r0, const float *r1, const B &b) {
        A a;
        split(*reinterpret_cast<const float4 *>(r0), *reinterpret_cast<const float4 *>(r1), a);
        mma(c, a, b);
    }
    __device__ static void mma_nodes(float (&c)[4], const float (&x)[4], const float (&y)[4], const float2 &m0, const float2 &m1) {
        const float *src[2] = {x, y};
        const float2 ms[2] = {m0, m1};
        uint32_t hi[2][4], lo[2][4], mh[2][2], ml[2][2];   // nodes 2t, 2t + 1 as the k indices t, t + 4
        float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            split_tf32(src[s][0], hi[s][0], lo[s][0]);
            split_tf32(src[s][2], hi[s][1], lo[s][1]);
            split_tf32(src[s][1], hi[s][2], lo[s][2]);
            split_tf32(src[s][3], hi[s][3], lo[s][3]);
            split_tf32(ms[s].x, mh[s][0], ml[s][0]);
            split_tf32(ms[s].y, mh[s][1], ml[s][1]);
            mma_tf32(d, lo[s], mh[s][0], mh[s][1]);
            mma_tf32(d, hi[s], ml[s][0], ml[s][1]);
        }
#pragma unroll
        for (int s = 0; s < 2; ++s) mma_tf32(d, hi[s], mh[s][0], mh[s][1]);
#pragma unroll
        for (int e = 0; e < 4; ++e) c[e] += d[e];
    }
};

// Shared memory of a CTA for up to NP nodes.
template <typename T, int D, int NP> struct Shape {
    static constexpr int kMain = D / 16;                       // warps with rows of S
    static constexpr int kSolve = NP >= 64 ? 2 : 1;            // warps with rows of M
    static constexpr int kThreads = 32 * (kMain + kSolve);
    static constexpr int kRow = D + Frag<T>::kPad;             // elements of a key or query row
    static constexpr int kVRow = D + (sizeof(T) == 2 ? 8 : 4); // of a value row, later the output
    static constexpr int kA = NP, kP = NP + 8;                 // floats of a row of A and of P (then M)
    static constexpr size_t kv = 2 * NP * kRow * sizeof(T), ka = kv + NP * kVRow * sizeof(T), kp = ka + NP * kA * 4,
                            kn = kp + NP * kP * 4, kBytes = kn + NP * (8 + 4 + 4 + 4 + 4);
};

// CTAs of an SM.  Two hide one another's phases, which outweighs the spills that
// their registers cost (64 sequences of 16 heads, d = 128, bf16: 47.1 -> 36.4 us
// at 32 nodes, 94.0 -> 80.6 at 64; fp32 87 -> 73 at 32, now 78), except where every
// fragment is held twice: fp32 at 64 nodes, 179 us with one and 233 with two (159 now).
template <typename T, int D, int NP> constexpr int kPerSm = sizeof(T) == 4 && D == 128 && NP == 64 ? 1 : 2;

template <typename T, int D, int NP>
__global__ void __launch_bounds__(Shape<T, D, NP>::kThreads, kPerSm<T, D, NP>)
    tree_step_kernel(const TreeStepLaunch L, int64_t uniform_len) {
    using S = Shape<T, D, NP>;
    using F = Frag<T>;
    extern __shared__ __align__(16) uint8_t sm[];
    T *kq = reinterpret_cast<T *>(sm);                        // [2 NP][kRow]: keys, then queries
    T *vo = reinterpret_cast<T *>(sm + S::kv);                // [NP][kVRow]
    float *as = reinterpret_cast<float *>(sm + S::ka);        // [NP][kA]
    float *ps = reinterpret_cast<float *>(sm + S::kp);        // [NP][kP]
    unsigned long long *anc = reinterpret_cast<unsigned long long *>(sm + S::kn);   // [NP]
    float *Gs = reinterpret_cast<float *>(anc + NP), *Gl = Gs + NP, *bs = Gl + NP;  // [NP]: G = Gs + Gl
    int *up = reinterpret_cast<int *>(bs + NP);                                      // [NP]
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int b = blockIdx.x / L.H, h = blockIdx.x % L.H;
    int64_t bos;
    const int n = seq_rows(L.cu_seqlens, uniform_len, L.total_nodes, b, min(L.max_nodes, NP), bos);
    if (n == 0) return;
    const bool main_warp = warp < S::kMain;

    // this warp's 16 rows of S, in flight while the tree is prepared
    constexpr int KS = D / 16;
    float4 s0[KS], s1[KS];
    if (main_warp) {
        const float *row = L.state + ((int64_t)blockIdx.x * D + 16 * warp + g) * D + 4 * t;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            s0[s] = L.state ? load_stream(row + 16 * s) : make_float4(0.f, 0.f, 0.f, 0.f);
            s1[s] = L.state ? load_stream(row + 8 * D + 16 * s) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
    }
    // keys, queries and values, all copies in flight at once; rows behind the last node are zero
    {
        constexpr int V = 16 / sizeof(T), per = D / V;
        const int64_t step = (int64_t)L.H * D;
        const int64_t first = bos * step + (int64_t)h * D;
#pragma unroll
        for (int m = 0; m < 3; ++m) {
            const T *src = static_cast<const T *>(m == 0 ? L.k : m == 1 ? L.q : L.v) + first;
            T *dst = m == 0 ? kq : m == 1 ? kq + NP * S::kRow : vo;
            const int row = m < 2 ? S::kRow : S::kVRow;
            for (int e = tid; e < NP * per; e += S::kThreads) {
                const int i = e / per, c = e % per * V;
                copy16(dst + i * row + c, src + min(i, n - 1) * step + c, i < n);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    if (!main_warp) {
        // ancestors and path sums by doubling: every round a node takes over
        // what its current ancestor pointer has gathered.  G is a sum of two floats: one
        // alone would leave the decays below a gate of -75 off by 2^-18 (4e-6 in the
        // norm of the outputs), below one of -1e6 by 3 % and more.
        const int i = tid - 32 * S::kMain;
        float G = 0.f, G_low = 0.f;
        unsigned long long a = 0;
        int p = -1;
        if (i < NP) {
            if (i < n) {
                p = tree_parent(L.parents, bos, i);
                G = L.g[(bos + i) * L.H + h];
                bs[i] = L.beta[(bos + i) * L.H + h];
                a = 1ull << i;
            } else {
                bs[i] = 0.f;
            }
        }
#pragma unroll 1
        for (int round = 1; round < NP; round *= 2) {
            if (i < NP) {
                Gs[i] = G;
                Gl[i] = G_low;
                anc[i] = a;
                up[i] = p;
            }
            asm volatile("bar.sync 1, %0;" ::"r"(32 * S::kSolve) : "memory");
            if (p >= 0) {
                add_two(G, G_low, Gs[p], Gl[p]);
                a |= anc[p];
                p = up[p];
            }
            asm volatile("bar.sync 1, %0;" ::"r"(32 * S::kSolve) : "memory");
        }
        if (i < NP) {
            Gs[i] = G;
            Gl[i] = G_low;
            anc[i] = a;
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();

    // A and P: products of keys and queries with keys, decayed, 0 where j is no ancestor
    const int tiles = (n + 7) / 8;   // 8 nodes each
    {
        // tiles of 16 rows (keys, then queries) by 8 keys, dealt to all warps; as
        // ancestors come before, row block r has 2 (r + 1) of them and nothing
        // reads what lies to their right
        constexpr int MT = NP / 16;
        const int nb = MT == 1 ? 1 : (n + 15) / 16, of_keys = nb * (nb + 1);
#pragma unroll 1
        for (int w = warp; w < 2 * of_keys; w += S::kThreads / 32) {
            const bool reads = w >= of_keys;                        // a tile of queries
            const int u = reads ? w - of_keys : w, r = MT == 1 ? 0 : (u >= 2) + (u >= 6) + (u >= 12);
            const int i0 = 16 * r, j0 = 8 * (u - r * (r + 1)), mt = r + (reads ? MT : 0);
            float c[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
            {
                const T *r0 = kq + (mt * 16 + g) * S::kRow + 4 * t, *r1 = r0 + 8 * S::kRow;
                const T *rb = kq + (j0 + g) * S::kRow + 4 * t;
#pragma unroll
                for (int s = 0; s < KS; ++s) {
                    typename F::B fb;
                    F::load_b(rb + 16 * s, fb);
                    F::mma_rows(c[s & 1], r0 + 16 * s, r1 + 16 * s, fb);
                }
            }
            const float2 Gj = *reinterpret_cast<const float2 *>(Gs + j0 + 2 * t), Gj_low = *reinterpret_cast<const float2 *>(Gl + j0 + 2 * t);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int i = i0 + g + 8 * e, j = j0 + 2 * t;
                const unsigned two = (unsigned)(anc[i] >> j) & 3u;
                const float G = Gs[i], G_low = Gl[i];
                float x = two & 1 ? (c[0][2 * e] + c[1][2 * e]) * F::exp((G - Gj.x) + (G_low - Gj_low.x)) : 0.f;
                float y = two & 2 ? (c[0][2 * e + 1] + c[1][2 * e + 1]) * F::exp((G - Gj.y) + (G_low - Gj_low.y)) : 0.f;
                if (!reads) {
                    const float be = bs[i];
                    x = j == i ? 0.f : x * be;
                    y = j + 1 == i ? 0.f : y * be;
                }
                *reinterpret_cast<float2 *>(reads ? ps + i * S::kP + j : as + i * S::kA + j) = make_float2(x, y);
            }
        }
    }
    __syncthreads();

    if (!main_warp) {
        // M = P (I + A)^-1, row i: m_l = p_l - sum over l' > l of m_l' A_l'l
        const int i = tid - 32 * S::kMain;
        if (i < NP) {
            float m[NP];
            // steps without a branch between them, so that the loads of the next run
            // ahead: 15.8 -> 12.9 us for 24 fp32 trees of 33 nodes (13.0 now); at 32 nodes the
            // registers this takes cost 2 %
            constexpr int kRun = NP == 64 ? 16 : 1;
            float *row = ps + i * S::kP;
#pragma unroll
            for (int j = 0; j < NP; j += 4) {
                const float4 v = i < n && (NP == 16 || j <= (i | 15)) ? *reinterpret_cast<const float4 *>(row + j) : make_float4(0.f, 0.f, 0.f, 0.f);
                m[j] = v.x;
                m[j + 1] = v.y;
                m[j + 2] = v.z;
                m[j + 3] = v.w;
            }
#pragma unroll
            for (int l0 = NP - kRun; l0 >= 0; l0 -= kRun) {
                if (l0 < n) {
#pragma unroll
                    for (int l = l0 + kRun - 1; l >= max(l0, 1); --l) {
#pragma unroll
                        for (int j = 0; j < l; j += 4) {
                            const float4 a = *reinterpret_cast<const float4 *>(as + l * S::kA + j);
                            m[j] = fmaf(-m[l], a.x, m[j]);
                            if (j + 1 < l) m[j + 1] = fmaf(-m[l], a.y, m[j + 1]);
                            if (j + 2 < l) m[j + 2] = fmaf(-m[l], a.z, m[j + 2]);
                            if (j + 3 < l) m[j + 3] = fmaf(-m[l], a.w, m[j + 3]);
                        }
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < NP; j += 4) *reinterpret_cast<float4 *>(row + j) = make_float4(m[j], m[j + 1], m[j + 2], m[j + 3]);
        }
        __syncthreads();
        return;
    }

    // S k and S q: value channels g, g + 8 of the warp's 16 by nodes 2t, 2t + 1 of each 8
    float xk[NP / 8][4], xq[NP / 8][4];
#pragma unroll
    for (int j = 0; j < NP / 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) xk[j][e] = xq[j][e] = 0.f;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
        typename F::A a;
        F::split(s0[s], s1[s], a);
#pragma unroll
        for (int j = 0; j < NP / 8; ++j) {
            if (j < tiles) {
                typename F::B fk, fq;
                F::load_b(kq + (8 * j + g) * S::kRow + 16 * s + 4 * t, fk);
                F::load_b(kq + (NP + 8 * j + g) * S::kRow + 16 * s + 4 * t, fq);
                F::mma(xk[j], a, fk);
                F::mma(xq[j], a, fq);
            }
        }
    }
    // R in place of S k, the first term of the output in place of S q
#pragma unroll
    for (int j = 0; j < NP / 8; ++j) {
        if (j < tiles) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = 8 * j + 2 * t + (e & 1), c = 16 * warp + g + 8 * (e >> 1);
                const float gamma = F::exp(Gs[i]);
                xk[j][e] = bs[i] * (to_f32(vo[i * S::kVRow + c]) - gamma * xk[j][e]);
                xq[j][e] *= gamma;
            }
        }
    }
    __syncthreads();   // M is there
#pragma unroll
    for (int i = 0; i < NP / 8; ++i) {
        if (i < tiles) {
#pragma unroll
            for (int k = 0; k <= i / 2; ++k) {   // 16 nodes: none after node tile i is an ancestor
                const float *m = ps + (8 * i + g) * S::kP + 16 * k + 2 * t;
                F::mma_nodes(xq[i], xk[2 * k], xk[2 * k + 1], *reinterpret_cast<const float2 *>(m), *reinterpret_cast<const float2 *>(m + 8));
            }
#pragma unroll
            for (int e = 0; e < 4; ++e)          // over the value that this thread alone has read
                vo[(8 * i + 2 * t + (e & 1)) * S::kVRow + 16 * warp + g + 8 * (e >> 1)] = from_f32<T>(xq[i][e]);
        }
    }
    __syncwarp();
    // the warp's 16 channels of every node
    constexpr int V = 16 / sizeof(T), per = 16 / V;
    for (int e = lane; e < n * per; e += 32) {
        const int i = e / per, c = 16 * warp + e % per * V;
        *reinterpret_cast<uint4 *>(static_cast<T *>(L.out) + ((bos + i) * L.H + h) * D + c) =
            *reinterpret_cast<const uint4 *>(vo + i * S::kVRow + c);
    }
}

template <typename T, int D, int NP> cudaError_t launch(const TreeStepLaunch &L, cudaStream_t stream) {
    using S = Shape<T, D, NP>;
    static bool done[64] = {false};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!done[dev]) {
        e = cudaFuncSetAttribute(tree_step_kernel<T, D, NP>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S::kBytes);
        if (e != cudaSuccess) return e;
        done[dev] = true;
    }
    const int64_t uniform_len = L.cu_seqlens ? 0 : L.total_nodes / L.num_seqs;
    tree_step_kernel<T, D, NP><<<L.num_seqs * L.H, S::kThreads, S::kBytes, stream>>>(L, uniform_len);
    return cudaGetLastError();
}

// The node count fixes the registers that hold S k, S q and a row of M, so it
// is a compile-time bound: 16, 32 or 64.  At 16 nodes (64 sequences of 16
// heads, d = 128, bf16) the bounds of 16 and 32 take 21.5 and 29.9 us; at 32
// nodes those of 32 and 64 take 36.4 and 71.6.
template <typename T, int D> cudaError_t launch_nodes(const TreeStepLaunch &L, cudaStream_t stream) {
    if (L.max_nodes <= 16) return launch<T, D, 16>(L, stream);
    if (L.max_nodes <= 32) return launch<T, D, 32>(L, stream);
    return launch<T, D, 64>(L, stream);
}

}  // namespace

cudaError_t launch_tree_step(const TreeStepLaunch &L, cudaStream_t stream) {
    if (L.dtype == GDN_F32) return L.d == 128 ? launch_nodes<float, 128>(L, stream) : launch_nodes<float, 64>(L, stream);
    return L.d == 128 ? launch_nodes<__nv_bfloat16, 128>(L, stream) : launch_nodes<__nv_bfloat16, 64>(L, stream);
}

}  // namespace gdn
