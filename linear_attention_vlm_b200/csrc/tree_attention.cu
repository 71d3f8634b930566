// Attention of a tree of drafted tokens over a cache of keys and values.
//
// A row is a (node, query head); the rows of one sequence that share a
// key/value head (n nodes x Hq / Hkv heads) see the same keys, so they form the
// M side of the tensor-core products, 128 rows a tile, node by node.  Per
// block of 128 keys: S = Q K^T (fp32 in tensor memory), P = 2^(c S - m) with a
// running maximum m and row sum, O += P V with P as the bf16 A operand in
// tensor memory.  The last block of an item holds the tree's own keys, masked
// by the ancestor bits of each node; a cache's last block ends inside the tile.
//
// What bounds it: K and V are read once, 512 bytes a slot and key/value head,
// against 512 Hq / Hkv n flops: memory up to about n Hq / Hkv = 260 rows, the
// tensor pipe above.  So the work is cut by keys, not by rows: all (sequence,
// key/value head, row tiles) items are laid end to end as key blocks and every
// CTA takes an equal run of them, whatever the lengths; an item that crosses
// CTAs leaves partial sums that a second kernel joins.
//
// Two streams keep the tensor pipe and the copies busy while a softmax runs,
// each with its own scores, accumulator, maximum and 8 softmax warps:
//   by keys (trees of at most one tile): the streams take alternate key
//     blocks of the same rows and are merged at the end;
//   by rows (larger trees): the streams take two row tiles of the same key
//     block, so a block is loaded once for 256 rows.
//   warps 0-7 / 8-15  softmax of stream 0 / 1 (warps w and w + 4 split the
//                     columns of the rows of TMEM lane quarter w % 4)
//   warp 16           TMA producer: Q per item, K and V through rings
//   warp 17           MMA issuer (one lane)
// Tensor memory: S_0, S_1, O_0, O_1, 128 columns each; the bf16 P of a block
// lies over the columns of its S, read by then.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>

#include "sm100.cuh"
#include "tma_maps.h"
#include "tree.cuh"

namespace gdn {
namespace {

using namespace sm100;

constexpr int kD = 128, kBM = 128, kBN = 128;
constexpr uint32_t kHalf = 16384;       // [128 rows][64 bf16] swizzled half tile
constexpr uint32_t kBlk = 2 * kHalf;    // [128 rows][128 bf16]
constexpr int kBox = 16;                // rows of a copy of the tree's own keys
constexpr float kLn2 = 0.6931471805599453f, kLog2e = 1.4426950408889634f;
constexpr float kRescaleThreshold = 8.f;   // log2 units, as in the window attention
constexpr int kMaxCtas = 160;

constexpr int kSoftmaxWarps = 16, kProducerWarp = 16, kMmaWarp = 17;
constexpr int kThreads = 32 * 18;

// shared memory: [Q tiles][K ring][V ring][barriers][exchange]
template <bool ROWS> struct Cfg {
    static constexpr int kStages = ROWS ? 2 : 3;
    static constexpr int kTiles = ROWS ? 2 : 1;       // Q tiles
    static constexpr uint32_t kQ = 0, kK = kTiles * kBlk, kV = kK + kStages * kBlk, kBar = kV + kStages * kBlk;
    static constexpr size_t kSmem = 232448;           // the per-CTA maximum; the rest is alignment slack
};
enum : int { B_QFULL = 0, B_QEMPTY, B_FIN, B_SFULL, B_PREADY = B_SFULL + 2, B_PVDONE = B_PREADY + 2, B_KFULL = B_PVDONE + 2,
             B_KEMPTY = B_KFULL + 3, B_VFULL = B_KEMPTY + 3, B_VEMPTY = B_VFULL + 3, B_NUM = B_VEMPTY + 3 };
// after the barriers (offsets from kBar); the exchange has 8 bytes a stream and
// row: a value of each half in fp32, or two of each in bf16
constexpr uint32_t kOffTmem = 8 * B_NUM, kOffAbort = kOffTmem + 4, kOffErr = kOffTmem + 8, kOffPlan = 192;
constexpr uint32_t kOffPar = 256;                     // [2 streams][64] parents, int8
constexpr uint32_t kOffXch = kOffPar + 128;           // [2 streams][128 rows] 8 bytes
static_assert(kOffErr + 4 <= kOffPlan, "barrier area");
static_assert(Cfg<false>::kBar + kOffXch + 2048 <= Cfg<false>::kSmem, "shared memory");
static_assert(Cfg<true>::kBar + kOffXch + 2048 + 1024 <= Cfg<true>::kSmem, "shared memory");

constexpr uint32_t TM_S = 0, TM_O = 256, kTmemCols = 512;   // + 128 * stream

struct Params {
    __nv_bfloat16 *o;
    float *lse;
    const int32_t *parents, *cu, *lens, *pos, *seen;
    int64_t uniform_len, total, capacity;
    int num_seqs, max_nodes, Hq, Hkv, group, tile_nodes, window;
    float c;                            // scale * log2(e)
    float *part;                        // [2 * CTAs][rows][128] partial sums
    float2 *ml;                         // [2 * CTAs][rows] their maxima (log2) and row sums
    int64_t *prefix;                    // [num_seqs + 1] key blocks before each sequence
    int *err;                           // [CTAs] what each CTA's waits left
    uint64_t timeout_ns, drain_ns;
};

// One sequence's share of the work.
struct Seq {
    int64_t bos;
    int n, len, kstart, blocks, tiles, items;
    __device__ __forceinline__ int64_t work(int Hkv) const { return (int64_t)Hkv * items * blocks; }
};

template <bool ROWS> __device__ __forceinline__ Seq load_seq(const Params &p, int b) {
    Seq s;
    s.n = seq_rows(p.cu, p.uniform_len, p.total, b, p.max_nodes, s.bos);
    s.len = cached_slots(p.lens, p.capacity, b);
    // in order, the slots before len + 1 - window are out of every node's window
    s.kstart = p.window && !p.pos ? max(0, s.len + 1 - p.window) : 0;
    if (s.kstart > s.len) s.kstart = s.len;
    s.blocks = (s.len - s.kstart + kBN - 1) / kBN + 1;
    s.tiles = (s.n + p.tile_nodes - 1) / p.tile_nodes;
    s.items = ROWS ? (s.tiles + 1) / 2 : s.tiles;
    return s;
}

// A CTA's run of key blocks, cut into segments of one item each.
template <bool ROWS> struct Walk {
    const Params &p;
    int64_t w, end, base;   // base: blocks before sequence b
    int b;
    Seq s;
    int h, it, blk0, blk1;  // the segment: key blocks [blk0, blk1) of item (h, it)
    __device__ Walk(const Params &p_, int64_t w_, int64_t end_, int b_, int64_t base_) : p(p_), w(w_), end(end_), base(base_), b(b_) {
        if (w < end) s = load_seq<ROWS>(p, b);
    }
    __device__ __forceinline__ bool next() {
        if (w >= end) return false;
        int64_t share;
        while (w >= base + (share = s.work(p.Hkv))) {
            base += share;
            s = load_seq<ROWS>(p, ++b);
        }
        const int64_t off = w - base, item = off / s.blocks;
        h = (int)(item / s.items);
        it = (int)(item % s.items);
        blk0 = (int)(off - item * s.blocks);
        blk1 = (int)min((int64_t)s.blocks, blk0 + (end - w));
        w += blk1 - blk0;
        return true;
    }
    __device__ __forceinline__ bool draft(int j) const { return j == s.blocks - 1; }
    __device__ __forceinline__ int key0(int j) const { return s.kstart + j * kBN; }
    __device__ __forceinline__ int valid(int j) const { return draft(j) ? s.n : min(kBN, s.len - key0(j)); }
};

// CTA c of N takes blocks [c W / N, (c + 1) W / N); with N <= W no run is empty.
__device__ __forceinline__ int64_t run_start(int64_t W, int c, int N) { return W * c / N; }

template <bool ROWS>
__global__ void __launch_bounds__(kThreads, 1)
    tree_attention_kernel(const __grid_constant__ CUtensorMap mQ, const __grid_constant__ CUtensorMap mKc,
                          const __grid_constant__ CUtensorMap mVc, const __grid_constant__ CUtensorMap mKn,
                          const __grid_constant__ CUtensorMap mVn, const Params p) {
    using C = Cfg<ROWS>;
    constexpr int NST = C::kStages;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t pad = (1024u - (smem_u32(smem_raw) & 1023u)) & 1023u;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, cta = blockIdx.x;
    constexpr unsigned kAll = 0xffffffffu;
    grid_dep_launch();
    if (pad + C::kBar + kOffXch + 2048 > C::kSmem) {   // cannot happen with an aligned dynamic base
        if (tid == 0) p.err[cta] = 80;
        return;
    }
    uint8_t *sm = smem_raw + pad, *ctl = sm + C::kBar;
    auto bar = [&](int i) { return smem_u32(ctl + 8 * i); };
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(ctl + kOffTmem);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(ctl + kOffAbort);
    int *err_sh = reinterpret_cast<int *>(ctl + kOffErr);
    auto fail = [&](int code) {
        *abort_flag = 1;
        atomicCAS(err_sh, 0, code);
    };

    // ---------------------------------------------------------------- plan
    // total blocks, then the sequence that this CTA's run starts in
    int64_t *plan = reinterpret_cast<int64_t *>(ctl + kOffPlan);                // W, base of the first sequence, its index
    int64_t *wsum = reinterpret_cast<int64_t *>(sm);                            // [18] scratch before any copy lands
    int64_t W = 0;
    for (int b = tid; b < p.num_seqs; b += kThreads) W += load_seq<ROWS>(p, b).work(p.Hkv);
#pragma unroll
    for (int o = 16; o; o >>= 1) W += __shfl_xor_sync(kAll, W, o);
    if (lane == 0) wsum[warp] = W;
    __syncthreads();
    W = 0;
    for (int i = 0; i < kThreads / 32; ++i) W += wsum[i];
    const int runs = (int)min((int64_t)gridDim.x, W);
    const int64_t w0 = cta < runs ? run_start(W, cta, runs) : W, w1 = cta < runs ? run_start(W, cta + 1, runs) : W;
    int64_t carry = 0;
    for (int b0 = 0; b0 < p.num_seqs && (carry <= w0 || cta == 0); b0 += kThreads) {
        const int b = b0 + tid;
        const int64_t mine = b < p.num_seqs ? load_seq<ROWS>(p, b).work(p.Hkv) : 0;
        int64_t incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t t = __shfl_up_sync(kAll, incl, o);
            if (lane >= o) incl += t;
        }
        __syncthreads();
        if (lane == 31) wsum[warp] = incl;
        __syncthreads();
        int64_t before = carry;
        for (int i = 0; i < warp; ++i) before += wsum[i];
        for (int i = 0; i < kThreads / 32; ++i) carry += wsum[i];
        const int64_t start = before + incl - mine;
        if (mine > 0 && start <= w0 && w0 < start + mine) {
            plan[0] = start;
            plan[1] = b;
        }
        if (cta == 0 && b < p.num_seqs) p.prefix[b] = start;
    }
    if (cta == 0 && tid == 0) p.prefix[p.num_seqs] = W;
    if (w0 == w1) {   // nothing for this CTA
        if (tid == 0) p.err[cta] = 0;
        return;
    }

    if (warp == 0) {
        tmem_alloc(smem_u32(tmem_slot), kTmemCols);
        tmem_relinquish();
    }
    if (tid == 32 * kProducerWarp) {
        mbar_init(bar(B_QFULL), 1);
        mbar_init(bar(B_QEMPTY), 1);
        mbar_init(bar(B_FIN), 1);
        for (int x = 0; x < 2; ++x) {
            mbar_init(bar(B_SFULL + x), 1);
            mbar_init(bar(B_PREADY + x), 32 * kSoftmaxWarps / 2);
            mbar_init(bar(B_PVDONE + x), 1);
        }
        for (int s = 0; s < NST; ++s) {
            mbar_init(bar(B_KFULL + s), 1);
            mbar_init(bar(B_KEMPTY + s), 1);
            mbar_init(bar(B_VFULL + s), 1);
            mbar_init(bar(B_VEMPTY + s), 1);
        }
        *abort_flag = 0;
        *err_sh = 0;
        fence_mbar_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = *tmem_slot;
    const uint64_t lim = p.timeout_ns, drain = p.drain_ns;
    Walk<ROWS> seg(p, w0, w1, (int)plan[1], plan[0]);

    if (warp == kProducerWarp) {
        // ------------------------------------------------------------ TMA producer
        if (lane == 0) {
            int used = 0, segs = 0;   // key blocks and segments so far
            int issued_k[NST] = {}, issued_v[NST] = {}, issued_q = 0;
            const uint32_t qbytes = 2u * 128u * (uint32_t)(p.group * p.tile_nodes);
            bool ok = true;
            for (; ok && seg.next(); ++segs) {
                const int tiles = ROWS ? min(2, seg.s.tiles - 2 * seg.it) : 1;
                if (segs && !mbar_wait(bar(B_QEMPTY), (segs - 1) & 1, lim, abort_flag)) { fail(81); break; }
                mbar_arrive_expect_tx(bar(B_QFULL), tiles * qbytes);
                for (int x = 0; x < tiles; ++x) {
                    const int row = (int)(seg.s.bos + (ROWS ? 2 * seg.it + x : 0) * p.tile_nodes);
                    tma_load_3d(smem_u32(sm + C::kQ + x * kBlk), &mQ, 0, seg.h * p.group, row, bar(B_QFULL));
                    tma_load_3d(smem_u32(sm + C::kQ + x * kBlk + kHalf), &mQ, 64, seg.h * p.group, row, bar(B_QFULL));
                }
                ++issued_q;
                for (int j = seg.blk0; j < seg.blk1; ++j, ++used) {
                    const int s = used % NST;
                    const uint32_t ph = ((used - NST) / NST) & 1;
                    const bool draft = seg.draft(j);
                    const int boxes = (seg.s.n + kBox - 1) / kBox;
                    const uint32_t bytes = draft ? boxes * kBox * 256u : kBlk;
                    auto copy = [&](uint32_t at, const CUtensorMap *cache, const CUtensorMap *nodes, uint32_t full) {
                        mbar_arrive_expect_tx(full, bytes);
                        if (draft) {
                            for (int i = 0; i < boxes; ++i) {
                                const int row = (int)seg.s.bos + i * kBox;
                                tma_load_3d(smem_u32(sm + at + i * kBox * 128), nodes, 0, seg.h, row, full);
                                tma_load_3d(smem_u32(sm + at + kHalf + i * kBox * 128), nodes, 64, seg.h, row, full);
                            }
                        } else {
                            const int row = (int)(seg.b * p.capacity + seg.key0(j));
                            tma_load_3d(smem_u32(sm + at), cache, 0, seg.h, row, full);
                            tma_load_3d(smem_u32(sm + at + kHalf), cache, 64, seg.h, row, full);
                        }
                    };
                    if (used >= NST && !mbar_wait(bar(B_KEMPTY + s), ph, lim, abort_flag)) { fail(82); ok = false; break; }
                    copy(C::kK + s * kBlk, &mKc, &mKn, bar(B_KFULL + s));
                    ++issued_k[s];
                    if (used >= NST && !mbar_wait(bar(B_VEMPTY + s), ph, lim, abort_flag)) { fail(83); ok = false; break; }
                    copy(C::kV + s * kBlk, &mVc, &mVn, bar(B_VFULL + s));
                    ++issued_v[s];
                }
            }
            const int zero = 0;   // no copy may still be landing in shared memory at exit
            if (issued_q) mbar_wait(bar(B_QFULL), (issued_q - 1) & 1, drain, &zero);
            for (int s = 0; s < NST; ++s) {
                if (issued_k[s]) mbar_wait(bar(B_KFULL + s), (issued_k[s] - 1) & 1, drain, &zero);
                if (issued_v[s]) mbar_wait(bar(B_VFULL + s), (issued_v[s] - 1) & 1, drain, &zero);
            }
        }
    } else if (warp == kMmaWarp) {
        // ------------------------------------------------------------ MMA issuer
        if (lane == 0) {
            const uint32_t id_s = idesc_bf16(kBM, kBN, false, false);   // Q (K-major) x K (K-major)
            const uint32_t id_o = idesc_bf16(kBM, kD, false, true);     // P (TMEM) x V (MN-major)
            const uint64_t dKm = desc_sw128(smem_u32(sm), 16, 1024);
            const uint64_t dMN = desc_sw128(smem_u32(sm), kHalf, 1024);
            int used = 0, segs = 0;
            int pvs[2] = {0, 0}, ps[2] = {0, 0};   // P V products issued, P blocks waited for, per stream
            // S_x = Q K^T of block `at` (its K already waited for), once P_x V of the block before has read S_x
            auto qk = [&](int x, int at) -> bool {
                if (pvs[x] && !mbar_wait(bar(B_PVDONE + x), (pvs[x] - 1) & 1, lim, abort_flag)) { fail(84); return false; }
                tc_fence_after();
                const uint32_t kofs = C::kK + (at % NST) * kBlk, qofs = C::kQ + (ROWS ? x * kBlk : 0);
#pragma unroll
                for (int ks = 0; ks < kD / 16; ++ks) {
                    const uint32_t off = (ks >> 2) * kHalf + (ks & 3) * 32;
                    mma_bf16_ss(tm + TM_S + x * kBN, dKm + ((qofs + off) >> 4), dKm + ((kofs + off) >> 4), id_s, ks > 0);
                }
                mma_commit(bar(B_SFULL + x));
                return true;
            };
            // O_x (+)= P_x V, over the keys that count (P is zero beyond them)
            auto pv = [&](int x, int at, int steps, bool first) -> bool {
                if (!mbar_wait(bar(B_PREADY + x), ps[x]++ & 1, lim, abort_flag)) { fail(85); return false; }
                if (!mbar_wait(bar(B_VFULL + at % NST), (at / NST) & 1, lim, abort_flag)) { fail(86); return false; }
                tc_fence_after();
                const uint32_t vofs = C::kV + (at % NST) * kBlk;
                for (int ks = 0; ks < steps; ++ks)
                    mma_bf16_ts(tm + TM_O + x * kD, tm + TM_S + x * kBN + (ks >> 2) * 64 + (ks & 3) * 8,
                                dMN + ((vofs + ks * 2048) >> 4), id_o, (!first || ks > 0) ? 1u : 0u);
                mma_commit(bar(B_PVDONE + x));
                ++pvs[x];
                return true;
            };
            auto k_ready = [&](int at) -> bool {
                if (mbar_wait(bar(B_KFULL + at % NST), (at / NST) & 1, lim, abort_flag)) return true;
                fail(87);
                return false;
            };
            bool ok = true;
            for (; ok && seg.next(); ++segs) {
                const int nblk = seg.blk1 - seg.blk0;
                if (!mbar_wait(bar(B_QFULL), segs & 1, lim, abort_flag)) { fail(88); break; }
                if (ROWS) {
                    const int tiles = min(2, seg.s.tiles - 2 * seg.it);
                    // the scores of block jj for stream x; after the last stream the K stage is free
                    auto scores = [&](int x, int jj) -> bool {
                        if ((x == 0 && !k_ready(used + jj)) || !qk(x, used + jj)) return false;
                        if (x == tiles - 1) {
                            mma_commit(bar(B_KEMPTY + (used + jj) % NST));
                            if (jj == nblk - 1) mma_commit(bar(B_QEMPTY));
                        }
                        return true;
                    };
                    for (int x = 0; ok && x < tiles; ++x) ok = scores(x, 0);
                    for (int jj = 0; ok && jj < nblk; ++jj) {
                        const int steps = (seg.valid(seg.blk0 + jj) + 15) / 16;
                        for (int x = 0; ok && x < tiles; ++x) {
                            ok = pv(x, used + jj, steps, jj == 0);
                            if (ok && x == tiles - 1) mma_commit(bar(B_VEMPTY + (used + jj) % NST));
                            if (ok && jj + 1 < nblk) ok = scores(x, jj + 1);
                        }
                    }
                } else {
                    auto scores = [&](int jj) -> bool {
                        if (!k_ready(used + jj) || !qk(jj & 1, used + jj)) return false;
                        mma_commit(bar(B_KEMPTY + (used + jj) % NST));
                        if (jj == nblk - 1) mma_commit(bar(B_QEMPTY));
                        return true;
                    };
                    ok = scores(0);
                    if (ok && nblk > 1) ok = scores(1);
                    for (int jj = 0; ok && jj < nblk; ++jj) {
                        ok = pv(jj & 1, used + jj, (seg.valid(seg.blk0 + jj) + 15) / 16, jj < 2);
                        if (ok) mma_commit(bar(B_VEMPTY + (used + jj) % NST));
                        if (ok && jj + 2 < nblk) ok = scores(jj + 2);
                    }
                }
                used += nblk;
            }
            mma_commit(bar(B_FIN));   // every issued MMA completes before TMEM is released
            const int zero = 0;
            mbar_wait(bar(B_FIN), 0, drain, &zero);
        }
    } else {
        // ------------------------------------------------------------ softmax (warps 0-15)
        // A wait that gives up does not leave the loops (others could be
        // waiting at an exchange): with the abort flag set the remaining waits
        // return at once and nothing is stored.
        const int x = warp >> 3, quarter = warp & 3, half = (warp >> 2) & 1, gtid = tid & 255;
        const int r = 32 * quarter + lane;
        const uint32_t lane_off = static_cast<uint32_t>(32 * quarter) << 16;
        const uint32_t sa = tm + lane_off + TM_S + x * kBN + 64 * half;
        const uint32_t oa = tm + lane_off + TM_O + x * kD + 64 * half;
        const float c = p.c;
        float *xch = reinterpret_cast<float *>(ctl + kOffXch);            // [stream][128 rows][2]
        float *mine = xch + (x * 128 + r) * 2 + half, *other = xch + (x * 128 + r) * 2 + (half ^ 1);
        int8_t *par = reinterpret_cast<int8_t *>(ctl + kOffPar) + x * 64;
        const int bar_pair = 1 + 4 * x + quarter, bar_group = 9 + x, bar_both = 11;
        // the sum of the halves' values of this row
        auto pair_sum = [&](float v) -> float {
            named_bar_sync(bar_pair, 64);
            *mine = v;
            named_bar_sync(bar_pair, 64);
            return v + *other;
        };
        // the larger of the halves' values as bf16: m only has to be the same in
        // both halves and within a factor of the maximum (two parities keep
        // consecutive exchanges apart)
        __nv_bfloat16 *mx_sh = reinterpret_cast<__nv_bfloat16 *>(xch) + (x * 128 + r) * 4;   // [2 parities][2 halves]
        int parity = 0;
        auto pair_max = [&](float v) -> float {
            const __nv_bfloat16 w = __float2bfloat16_rn(v);
            __nv_bfloat16 *at = mx_sh + 2 * parity;
            parity ^= 1;
            at[half] = w;
            named_bar_sync(bar_pair, 64);
            return fmaxf(__bfloat162float(w), __bfloat162float(at[half ^ 1]));
        };
        int used = 0, cnt = 0;                   // key blocks so far; blocks of this stream so far
        bool ok = true;
        auto wait = [&](int b, uint32_t parity, int code) {
            if (!__all_sync(kAll, mbar_wait(bar(b), parity, lim, abort_flag))) {
                fail(code);
                ok = false;
            }
        };
        while (seg.next()) {
            const int nblk = seg.blk1 - seg.blk0;
            const int tile = ROWS ? 2 * seg.it + x : 0;
            if (ROWS && tile >= seg.s.tiles) {   // an odd tile count leaves stream 1 without rows
                used += nblk;
                continue;
            }
            const int node = tile * p.tile_nodes + r / p.group;
            const bool vrow = r < p.group * p.tile_nodes && node < seg.s.n;
            const bool work = __any_sync(kAll, vrow);
            // ancestors and depth of the row's node
            uint64_t anc = 0;
            int depth = 0;
            const bool need_tree = seg.draft(seg.blk1 - 1) || p.window;
            if (need_tree && p.parents) {
                named_bar_sync(bar_group, 256);
                if (gtid < seg.s.n) par[gtid] = (int8_t)tree_parent(p.parents, seg.s.bos, gtid);
                named_bar_sync(bar_group, 256);
            }
            if (need_tree && vrow) {
                if (p.parents) {
                    int d = -1;
                    for (int a = node; a >= 0; a = par[a]) {
                        ++d;
                        if (!p.window || d < p.window) anc |= 1ull << a;
                    }
                    depth = d;
                } else {
                    depth = node;
                    anc = (2ull << node) - 1;
                    if (p.window && node >= p.window) anc &= ~0ull << (node - p.window + 1);
                }
            }
            // only keys at positions above `far` are inside the window
            const int32_t *pos = p.window && p.pos ? p.pos + ((int64_t)seg.b * p.Hkv + seg.h) * p.capacity : nullptr;
            const int far = p.window ? (pos ? p.seen[seg.b] : seg.s.len) + depth - p.window : INT32_MIN;
            // positions of this half's keys, two a lane, fetched a block ahead
            int p0 = INT32_MAX, p1 = INT32_MAX;
            auto fetch_pos = [&](int jj) {
                p0 = p1 = INT32_MAX;
                if (!pos || !work || jj >= nblk || seg.draft(seg.blk0 + jj)) return;
                const int k0 = seg.key0(seg.blk0 + jj) + 64 * half;
                if (k0 + lane < seg.s.len) p0 = pos[k0 + lane];
                if (k0 + 32 + lane < seg.s.len) p1 = pos[k0 + 32 + lane];
            };
            fetch_pos(ROWS ? 0 : x);
            const int top = p.window ? __reduce_max_sync(kAll, vrow ? far : INT32_MIN) : 0;   // the warp's last masked position
            float m = -INFINITY, l = 0.f;   // m: the same in both halves of a row; l: this half's share
            for (int jj = ROWS ? 0 : x; jj < nblk; jj += ROWS ? 1 : 2) {
                const int j = seg.blk0 + jj, valid = seg.valid(j);
                const bool draft = seg.draft(j);
                uint64_t vis;                // which of this half's 64 keys the row sees
                if (draft) {
                    vis = half ? 0 : anc;
                } else {
                    const int left = valid - 64 * half, k0 = seg.key0(j) + 64 * half;
                    vis = left >= 64 ? ~0ull : left <= 0 ? 0 : (1ull << left) - 1;
                    if (p.window && work) {
                        if (pos) {
                            if (__reduce_min_sync(kAll, min(p0, p1)) <= top) {
                                uint32_t lo = 0, hi = 0;
                                for (int i = 0; i < 32; ++i) {
                                    if (__shfl_sync(kAll, p0, i) > far) lo |= 1u << i;
                                    if (__shfl_sync(kAll, p1, i) > far) hi |= 1u << i;
                                }
                                vis &= (uint64_t)hi << 32 | lo;
                            }
                        } else if (k0 <= top) {
                            const int skip = far + 1 - k0;   // keys of this half before the window
                            if (skip > 0) vis &= skip >= 64 ? 0 : ~0ull << skip;
                        }
                    }
                }
                if (pos) fetch_pos(jj + (ROWS ? 1 : 2));
                wait(B_SFULL + x, cnt & 1, 89);
                ++cnt;
                tc_fence_after();
                if (work) {
                    const bool masked = !__all_sync(kAll, vis == ~0ull);
                    float mx = -INFINITY;
#pragma unroll 1
                    for (int c4 = 0; c4 < 2; ++c4) {
                        float v[32];
                        tmem_ld32(sa + 32 * c4, v);
                        float a[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                        if (masked) {
                            const uint32_t bits = (uint32_t)(vis >> (32 * c4));
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (bits >> i & 1) a[i & 3] = fmaxf(a[i & 3], v[i]);
                        } else {
#pragma unroll
                            for (int i = 0; i < 32; ++i) a[i & 3] = fmaxf(a[i & 3], v[i]);
                        }
                        mx = fmaxf(mx, fmaxf(fmaxf(a[0], a[1]), fmaxf(a[2], a[3])));
                    }
                    const float mb = pair_max(mx) * c;
                    float alpha = 1.f;
                    bool rescale = false;
                    if (mb > m + kRescaleThreshold) {   // also taken when m is still -inf
                        if (m != -INFINITY) {
                            alpha = ex2_approx(m - mb);
                            rescale = true;
                        }
                        m = mb;
                    }
                    const float msub = m == -INFINITY ? 0.f : m;
                    float sum = 0.f;
#pragma unroll 1
                    for (int c4 = 0; c4 < 2; ++c4) {
                        float v[32];
                        tmem_ld32(sa + 32 * c4, v);
                        uint32_t pk[16];
                        float sm4[4] = {0.f, 0.f, 0.f, 0.f};
                        const uint32_t bits = (uint32_t)(vis >> (32 * c4));
#pragma unroll
                        for (int i = 0; i < 32; i += 2) {
                            float p0 = ex2_approx(fmaf(v[i], c, -msub)), p1 = ex2_approx(fmaf(v[i + 1], c, -msub));
                            if (masked) {
                                if (!(bits >> i & 1)) p0 = 0.f;
                                if (!(bits >> (i + 1) & 1)) p1 = 0.f;
                            }
                            sm4[(i >> 1) & 3] += p0 + p1;
                            pk[i >> 1] = pack_bf16(p0, p1);
                        }
                        tmem_st16u(sa + 16 * c4, pk);   // over columns read by now
                        sum += (sm4[0] + sm4[1]) + (sm4[2] + sm4[3]);
                    }
                    l = l * alpha + sum;
                    if (__any_sync(kAll, rescale)) {    // O_x is stable: P_x V of the block before has completed
#pragma unroll 1
                        for (int c4 = 0; c4 < 2; ++c4) {
                            float v[32];
                            tmem_ld32(oa + 32 * c4, v);
#pragma unroll
                            for (int i = 0; i < 32; ++i) v[i] *= alpha;
                            tmem_st32(oa + 32 * c4, v);
                        }
                    }
                }
                // V rows behind the last key, up to the 16 of a product step, may hold
                // anything; P is zero there and the rows are cleared
                const int behind = (16 - valid % 16) % 16;
                if (behind && (!ROWS || x == 0)) {
                    const int at = used + jj, s = at % NST;
                    wait(B_VFULL + s, (at / NST) & 1, 90);
                    if (gtid < behind * 16) {
                        const int row = valid + gtid / 16, ch = gtid % 16;
                        st_shared_v4(smem_u32(sm + C::kV + s * kBlk + (ch >> 3) * kHalf + row * 128 + (ch & 7) * 16), 0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                }
                tc_fence_before();
                mbar_arrive(bar(B_PREADY + x));
            }
            used += nblk;
            const bool whole = seg.blk0 == 0 && seg.blk1 == seg.s.blocks;
            // an item that began in an earlier CTA goes to slot 2c, one that goes on into the next to 2c + 1
            const int slot = 2 * cta + (seg.blk0 > 0 ? 0 : 1);
            const int64_t row_at = (seg.s.bos + node) * p.Hq + (int64_t)seg.h * p.group + r % p.group;
            const int64_t part_at = (int64_t)slot * (C::kTiles * kBM) + (ROWS ? x * kBM : 0) + r;
            auto store = [&](int col, const float (&v)[32], float inv) {   // 32 columns from `col`
                if (whole) {
                    uint4 *dst = reinterpret_cast<uint4 *>(p.o + row_at * kD + col);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        dst[e] = make_uint4(pack_bf16(v[8 * e] * inv, v[8 * e + 1] * inv),
                                            pack_bf16(v[8 * e + 2] * inv, v[8 * e + 3] * inv),
                                            pack_bf16(v[8 * e + 4] * inv, v[8 * e + 5] * inv),
                                            pack_bf16(v[8 * e + 6] * inv, v[8 * e + 7] * inv));
                } else {
                    float4 *dst = reinterpret_cast<float4 *>(p.part + part_at * kD + col);
#pragma unroll
                    for (int e = 0; e < 8; ++e) dst[e] = make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
                }
            };
            auto store_ml = [&](float mm, float ll) {
                if (whole) {
                    if (p.lse) p.lse[row_at] = ll > 0.f ? (mm + log2f(ll)) * kLn2 : -INFINITY;
                } else {
                    p.ml[part_at] = make_float2(mm, ll);
                }
            };
            if (ROWS) {
                wait(B_PVDONE + x, (cnt - 1) & 1, 91);
                tc_fence_after();
                if (work) {
                    const float lsum = pair_sum(l);
                    const float inv = lsum > 0.f ? 1.f / lsum : 0.f;
#pragma unroll 1
                    for (int c4 = 0; c4 < 2; ++c4) {
                        float v[32];
                        tmem_ld32(oa + 32 * c4, v);
                        if (vrow && ok) store(64 * half + 32 * c4, v, inv);
                    }
                    if (vrow && ok && half == 0) store_ml(m, lsum);
                }
            } else {
                // merge the streams: each takes 32 of the half's 64 columns
                const bool two = nblk > 1;
                if (x == 0 || two) wait(B_PVDONE + x, (cnt - 1) & 1, 92);
                const float lrow = work ? pair_sum(l) : 0.f;   // a stream without blocks: m = -inf, l = 0
                tc_fence_before();
                named_bar_sync(bar_both, 32 * kSoftmaxWarps);     // both streams' products have completed
                tc_fence_after();
                if (half == 0) *mine = m;
                else *mine = lrow;
                named_bar_sync(bar_both, 32 * kSoftmaxWarps);
                if (work) {
                    const float m0 = xch[2 * r], l0 = xch[2 * r + 1], m1 = xch[256 + 2 * r], l1 = xch[257 + 2 * r];
                    const float mm = fmaxf(m0, m1);
                    const float f0 = m0 == -INFINITY ? 0.f : ex2_approx(m0 - mm), f1 = m1 == -INFINITY ? 0.f : ex2_approx(m1 - mm);
                    const float ll = f0 * l0 + f1 * l1, inv = ll > 0.f ? 1.f / ll : 0.f;
                    const uint32_t at = tm + lane_off + TM_O + 64 * half + 32 * x;
                    float v[32];
                    tmem_ld32(at, v);
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] *= f0;
                    if (two) {
                        float u[32];
                        tmem_ld32(at + kD, u);
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = fmaf(u[i], f1, v[i]);
                    }
                    if (vrow && ok) {
                        store(64 * half + 32 * x, v, inv);
                        if (half == 0 && x == 0) store_ml(mm, ll);
                    }
                }
                tc_fence_before();
                named_bar_sync(bar_both, 32 * kSoftmaxWarps);   // both accumulators read, the exchange free
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (tid == 0) p.err[cta] = *err_sh;
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tm, kTmemCols);
    }
}

// Joins the partial sums of the items that more than one CTA worked on: a
// group of `width` warps per row.  CTA 0 also gathers the status.
constexpr int kJoinWarps = 8;

template <bool ROWS>
__global__ void __launch_bounds__(kJoinWarps * 32) tree_join_kernel(const Params p, int ctas, int *status, int width) {
    __shared__ float4 acc_sh[kJoinWarps][32];
    __shared__ float l_sh[kJoinWarps];
    __shared__ int bad;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr unsigned kAll = 0xffffffffu;
    constexpr int kRows = Cfg<ROWS>::kTiles * kBM;
    const int part = warp % width, b = blockIdx.y;
    const int64_t at_row = (int64_t)blockIdx.x * (kJoinWarps / width) + warp / width;   // (node, head) of the sequence
    const int64_t node = at_row / p.Hq;
    const int hq = (int)(at_row % p.Hq), h = hq / p.group;
    const Seq s = load_seq<ROWS>(p, b);
    const int64_t row = s.bos * p.Hq + at_row;
    const bool here = node < s.n;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float M = -INFINITY, l = 0.f;
    bool split = false;
    grid_dep_wait();
    if (blockIdx.x == 0 && b == 0) {
        if (tid == 0) bad = 0;
        __syncthreads();
        for (int i = tid; i < ctas; i += blockDim.x)
            if (p.err[i]) bad = p.err[i];
        __syncthreads();
        if (tid == 0) *status = bad;
    }
    if (here) {
        const int tile = (int)node / p.tile_nodes, it = ROWS ? tile / 2 : tile;
        const int r = (ROWS ? (tile & 1) * kBM : 0) + ((int)node % p.tile_nodes) * p.group + hq % p.group;
        const int64_t W = p.prefix[p.num_seqs], runs = min((int64_t)ctas, W);
        const int64_t start = p.prefix[b] + ((int64_t)h * s.items + it) * s.blocks, last = start + s.blocks - 1;
        const int c0 = (int)(((start + 1) * runs - 1) / W), c1 = (int)(((last + 1) * runs - 1) / W);
        split = c1 > c0;
        if (split) {
            auto at = [&](int c) { return (int64_t)(c == c0 ? 2 * c + 1 : 2 * c) * kRows + r; };
            for (int c = c0 + lane; c <= c1; c += 32) M = fmaxf(M, p.ml[at(c)].x);
#pragma unroll
            for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kAll, M, o));
#pragma unroll 8
            for (int c = c0 + part; c <= c1; c += width) {
                const int64_t i = at(c);
                const float2 ml = p.ml[i];
                const float4 v = reinterpret_cast<const float4 *>(p.part)[i * 32 + lane];
                const float f = ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - M);
                l = fmaf(f, ml.y, l);
                acc.x = fmaf(f, v.x, acc.x);
                acc.y = fmaf(f, v.y, acc.y);
                acc.z = fmaf(f, v.z, acc.z);
                acc.w = fmaf(f, v.w, acc.w);
            }
        }
    }
    if (width > 1) {   // the same for the whole block
        acc_sh[warp][lane] = acc;
        if (lane == 0) l_sh[warp] = l;
        __syncthreads();
        if (part == 0) {
            for (int i = 1; i < width; ++i) {
                const float4 v = acc_sh[warp + i][lane];
                acc.x += v.x;
                acc.y += v.y;
                acc.z += v.z;
                acc.w += v.w;
                l += l_sh[warp + i];
            }
        }
    }
    if (split && part == 0) {
        const float inv = l > 0.f ? 1.f / l : 0.f;
        *reinterpret_cast<uint2 *>(p.o + row * kD + 4 * lane) = make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
        if (p.lse && lane == 0) p.lse[row] = l > 0.f ? (M + log2f(l)) * kLn2 : -INFINITY;
    }
}

// workspace: [status, 256 B][err: CTAs ints][prefix][ml][part]
struct Ws {
    size_t err, prefix, ml, part, total;
};
Ws ws_layout(int num_seqs, bool rows) {
    const size_t R = (rows ? 2 : 1) * (size_t)kBM * 2 * kMaxCtas;
    Ws w;
    w.err = 256;
    w.prefix = w.err + kMaxCtas * 4;
    w.ml = (w.prefix + (size_t)(num_seqs + 1) * 8 + 255) & ~(size_t)255;
    w.part = w.ml + R * 8;
    w.total = w.part + R * kD * 4;
    return w;
}

template <bool ROWS> cudaError_t launch(const TreeAttnLaunch &L, cudaStream_t stream) {
    static bool done[64] = {false};
    static int sms[64] = {0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64 || !done[dev]) {
        int count = 0;
        e = cudaFuncSetAttribute(tree_attention_kernel<ROWS>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Cfg<ROWS>::kSmem);
        if (e == cudaSuccess) e = cudaDeviceGetAttribute(&count, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return e;
        if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
        sms[dev] = count;
        done[dev] = true;
    }
    const int ctas = sms[dev] < kMaxCtas ? sms[dev] : kMaxCtas;
    const int group = L.Hq / L.Hkv, nodes = kBM / group;
    const Ws w = ws_layout(L.num_seqs, ROWS);
    uint8_t *ws = static_cast<uint8_t *>(L.workspace);
    Params p;
    p.o = static_cast<__nv_bfloat16 *>(L.o);
    p.lse = L.lse;
    p.parents = L.parents; p.cu = L.cu_seqlens; p.lens = L.cache_lens; p.pos = L.cache_pos; p.seen = L.seen;
    p.uniform_len = L.cu_seqlens ? 0 : L.total_nodes / L.num_seqs;
    p.total = L.total_nodes; p.capacity = L.capacity;
    p.num_seqs = L.num_seqs; p.max_nodes = L.max_nodes;
    p.Hq = L.Hq; p.Hkv = L.Hkv; p.group = group; p.tile_nodes = nodes; p.window = L.window;
    p.c = L.scale * kLog2e;
    p.err = reinterpret_cast<int *>(ws + w.err);
    p.prefix = reinterpret_cast<int64_t *>(ws + w.prefix);
    p.ml = reinterpret_cast<float2 *>(ws + w.ml);
    p.part = reinterpret_cast<float *>(ws + w.part);
    p.timeout_ns = L.timeout_ns; p.drain_ns = L.drain_ns;
    CUtensorMap mq, mkc, mvc, mkn, mvn;
    const int64_t rows = (int64_t)L.num_seqs * L.capacity;
    bool ok = make_rows_map(&mq, L.q, L.total_nodes, L.Hq, group, nodes) && make_rows_map(&mkn, L.k, L.total_nodes, L.Hkv, 1, kBox) &&
              make_rows_map(&mvn, L.v, L.total_nodes, L.Hkv, 1, kBox);
    if (ok && rows > 0) {
        ok = make_rows_map(&mkc, L.k_cache, rows, L.Hkv, 1, kBN) && make_rows_map(&mvc, L.v_cache, rows, L.Hkv, 1, kBN);
    } else {
        mkc = mkn;   // no cached block is ever read
        mvc = mvn;
    }
    if (!ok) return cudaErrorInvalidValue;
    tree_attention_kernel<ROWS><<<ctas, kThreads, Cfg<ROWS>::kSmem, stream>>>(mq, mkc, mvc, mkn, mvn, p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    // few items are cut many times: then a whole block joins a row
    const int64_t items = (int64_t)L.num_seqs * L.Hkv * (ROWS ? ((L.max_nodes + nodes - 1) / nodes + 1) / 2 : 1);
    const int width = items * 8 <= ctas ? kJoinWarps : 1;
    const int64_t per = kJoinWarps / width, blocks = ((int64_t)L.max_nodes * L.Hq + per - 1) / per;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks, (unsigned)L.num_seqs);
    cfg.blockDim = dim3(kJoinWarps * 32);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, tree_join_kernel<ROWS>, p, ctas, static_cast<int *>(L.workspace), width);
}

bool by_rows(int max_nodes, int Hq, int Hkv) { return max_nodes > kBM / (Hq / Hkv); }

}  // namespace

size_t tree_attention_workspace(int num_seqs, int max_nodes, int Hq, int Hkv) {
    return ws_layout(num_seqs, by_rows(max_nodes, Hq, Hkv)).total;
}

cudaError_t launch_tree_attention(const TreeAttnLaunch &L, cudaStream_t stream) {
    return by_rows(L.max_nodes, L.Hq, L.Hkv) ? launch<true>(L, stream) : launch<false>(L, stream);
}

}  // namespace gdn
