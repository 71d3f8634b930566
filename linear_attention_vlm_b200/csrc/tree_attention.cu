// Attention of a tree of drafted tokens over a cache of keys and values.
//
// A row is a (node, query head); the rows of one sequence that share a
// key/value head (n nodes x Hq / Hkv heads) see the same keys, so they form the
// M side of the tensor-core products, 128 rows a tile, node by node.  Per
// block of 128 keys: S = Q K^T (fp32 in tensor memory), P = 2^(c S - m) with a
// running maximum m and row sum, O += P V with P as the bf16 A operand in
// tensor memory (its rounding adds as much error as the output's: 2.2e-3 in the norm
// against 1.6e-3; the row sums take the unrounded P).  The last block of an item
// holds the tree's own keys, masked by the ancestor bits of each node; a cache's
// last block ends inside the tile.
//
// What bounds it: K and V, 512 bytes a slot and key/value head, against 512 Hq /
// Hkv n flops: memory up to about n Hq / Hkv = 260 rows, the tensor pipe above.
// An item has at most 256 rows, so up to there K and V are read once, and again
// for every further 256: 32 trees of 32 to 64 nodes (256 to 512 rows a head) at
// 8192 slots read 428 MB from memory where 279 would do; at 66 us of copy rate
// that is not what bounds their 166.  So the work is cut by keys, not by rows: all (sequence,
// key/value head, row tiles) items are laid end to end as key blocks and every
// CTA takes an equal run of them, whatever the lengths; an item that crosses
// CTAs leaves partial sums that a second kernel joins.
//
// A block is worked on in halves of 64 keys.  Two streams keep the tensor pipe
// and the copies busy while a softmax runs, each with its own accumulator,
// maximum and row sum and two score buffers of 64 columns:
//   by keys (trees of at most one tile): stream x takes half x of every block
//     for the same rows, and the streams are merged at the end;
//   by rows (larger trees): the streams take two row tiles of the same half
//     block, so a block is loaded once for 256 rows.  For a tree of one tile the
//     second stream would idle: 70 against 57 us for a token of 64 sequences
//     at 0 to 8192 slots, 53 against 48 for 32 trees of 16 nodes.
// With two buffers the scores of the next half are formed while the softmax of
// this one runs, so the softmax warps hardly wait; a thread holds a whole row of
// 64 scores in registers, so a row needs no exchange and its scores are read once.
//   warps 0-3 / 4-7   softmax of stream 0 / 1 (a thread per row)
//   warp 8            TMA producer: Q per item, K and V through rings
//   warps 9, 10       MMA issuers of stream 0 / 1: with one warp for both, its
//                     waits and issues (about 3000 cycles per half block) were
//                     longer than the products and the softmax (1200 each)
// Bandwidth and rates reached, bf16, 16 query and 2 key/value heads: a token of 64
// sequences at 0 to 8192 slots 59 us (4.4 TB/s, of which 13 us are the first
// copies, the merge and the join); 24 nodes at 262144 slots 84 to 91 us by the box
// (2.9 to 3.2 TB/s, 0.6 PFLOP/s); 32 trees of 64 nodes at 8192 slots 166 us.  With many rows the hand-over
// between softmax and products of a stream bounds it: a half block takes 2050
// cycles, 1350 of them the exponentials and the conversions of 128 rows x 64 keys
// a stream (the special-function units alone need 1100 for two streams).
// Tensor memory: per stream 2 x 64 columns of scores and 128 of output; the bf16
// P of a half block lies over the columns of its S, read by then.
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

constexpr int kSoftmaxWarps = 8, kProducerWarp = 8, kMmaWarp = 9;
constexpr int kThreads = 32 * 11;
constexpr int kSub = 64;                // keys of a half block
// Planning weight of an item beside its key blocks: starting one (its Q, the
// first scores) and ending it (merge and stores) take the time of one or two
// blocks.  Weights 0, 1 and 2: 50.1, 48.8, 46.7 us for 32 trees of 16 nodes at
// 8192 slots of 2 x 8 heads, 112, 107, 105 of 64 nodes, 58.7, 56.9, 58.1 for a
// token of 64 sequences, 60.1, 60.5, 58.8 for one of 512 at 100 slots.
constexpr int kItemCost = 2;

// shared memory: [Q tiles][K ring][V ring][barriers][exchange]
template <bool ROWS> struct Cfg {
    static constexpr int kStages = ROWS ? 2 : 3;
    static constexpr int kTiles = ROWS ? 2 : 1;       // Q tiles
    static constexpr uint32_t kQ = 0, kK = kTiles * kBlk, kV = kK + kStages * kBlk, kBar = kV + kStages * kBlk;
    static constexpr size_t kSmem = 232448;           // the per-CTA maximum; the rest is alignment slack
};
// A parity wait tells a phase only from the one before it, so what a softmax
// may run two half blocks ahead of has a barrier per score buffer (+ 2 stream + buffer).
enum : int { B_QFULL = 0, B_QEMPTY = 2, B_FIN = 4, B_SFULL = 5, B_PREADY = 9, B_PVDONE = 13, B_KFULL = 17, B_KEMPTY = 20,
             B_VFULL = 23, B_VEMPTY = 26, B_NUM = 29 };
// after the barriers (offsets from kBar)
constexpr uint32_t kOffTmem = 8 * B_NUM, kOffAbort = kOffTmem + 4, kOffErr = kOffTmem + 8, kOffPlan = 256;
constexpr uint32_t kOffPar = 320;                     // [2 streams][64] parents, int8
constexpr uint32_t kOffXch = kOffPar + 128;           // [2 streams][128 rows] maximum and row sum
constexpr uint32_t kCtlBytes = kOffXch + 2048;
static_assert(kOffErr + 4 <= kOffPlan, "barrier area");
static_assert(Cfg<false>::kBar + kCtlBytes <= Cfg<false>::kSmem, "shared memory");
static_assert(Cfg<true>::kBar + kCtlBytes + 1024 <= Cfg<true>::kSmem, "shared memory");

constexpr uint32_t TM_S = 0, TM_O = 256, kTmemCols = 512;   // + 128 * stream

// 32 lanes x 64 consecutive fp32 columns; waits for completion.
__device__ __forceinline__ void tmem_ld64(uint32_t taddr, float (&v)[64]) {
    uint32_t r[64];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x64.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,"
        "%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,"
        "%61,%62,%63}, [%64];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=r"(r[32]),
          "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]),
          "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]), "=r"(r[48]),
          "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]), "=r"(r[56]),
          "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
        : "r"(taddr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 64; ++i) v[i] = __uint_as_float(r[i]);
}

// Two fp32 operations an instruction.
__device__ __forceinline__ uint64_t pack_f32x2(float x, float y) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(x), "f"(y));
    return d;
}
__device__ __forceinline__ void unpack_f32x2(uint64_t d, float &x, float &y) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(d));
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

struct Params {
    __nv_bfloat16 *o;
    float *lse;
    const int32_t *parents, *cu, *lens, *pos, *seen;
    int64_t uniform_len, total, capacity;
    int num_seqs, max_nodes, Hq, Hkv, group, window;
    int tile_nodes;                     // nodes of a row tile
    int box_nodes, q_bufs;              // nodes of a copy of Q; buffers for it
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
    __device__ __forceinline__ int cost() const { return blocks + kItemCost; }   // of an item
    __device__ __forceinline__ int64_t work(int Hkv) const { return (int64_t)Hkv * items * cost(); }
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

// A CTA's run of work units, cut into segments of one item each.  The first
// kItemCost units of an item stand for its overhead, the others for its key blocks.
template <bool ROWS> struct Walk {
    const Params &p;
    int64_t w, end, base;   // base: units before sequence b
    int b;
    Seq s, after;           // of sequences b and b + 1, fetched ahead
    int h, it, blk0, blk1;  // the segment: key blocks [blk0, blk1) of item (h, it)
    __device__ Walk(const Params &p_, int64_t w_, int64_t end_, int b_, int64_t base_, const Seq &s_)
        : p(p_), w(w_), end(end_), base(base_), b(b_), s(s_) {
        after = load_seq<ROWS>(p, min(b + 1, p.num_seqs - 1));
    }
    __device__ __forceinline__ bool next() {
        while (w < end) {
            int64_t share;
            while (w >= base + (share = s.work(p.Hkv))) {
                base += share;
                ++b;
                s = after;
                after = load_seq<ROWS>(p, min(b + 1, p.num_seqs - 1));
            }
            const int cost = s.cost();
            const uint32_t off = (uint32_t)(w - base), item = off / cost;
            h = (int)(item / s.items);
            it = (int)(item % s.items);
            const int at = (int)(off - item * cost);
            const int upto = (int)min((int64_t)cost, at + (end - w));
            w += upto - at;
            blk0 = max(0, at - kItemCost);
            blk1 = upto - kItemCost;
            if (blk0 < blk1) return true;
        }
        return false;
    }
    __device__ __forceinline__ bool draft(int j) const { return j == s.blocks - 1; }
    __device__ __forceinline__ int key0(int j) const { return s.kstart + j * kBN; }
    __device__ __forceinline__ int valid(int j) const { return draft(j) ? s.n : min(kBN, s.len - key0(j)); }
    __device__ __forceinline__ int tiles() const { return ROWS ? min(2, s.tiles - 2 * it) : 1; }   // of the item
};

// The half blocks of a segment, in order: by rows both streams take half h of
// block j; by keys stream x takes half x of block j, if that has keys.
template <bool ROWS> struct Halves {
    int j, h;
    __device__ __forceinline__ int half(int x) const { return ROWS ? h : x; }
    __device__ __forceinline__ bool has(const Walk<ROWS> &seg, int x) const {
        return ROWS ? x < seg.tiles() : kSub * x < seg.valid(j);
    }
    __device__ __forceinline__ bool last(const Walk<ROWS> &seg) const { return !ROWS || h == 1 || seg.valid(j) <= kSub; }   // of its block
    __device__ __forceinline__ void step(const Walk<ROWS> &seg) {
        if (last(seg)) ++j, h = 0;
        else h = 1;
    }
    __device__ __forceinline__ bool done(const Walk<ROWS> &seg) const { return j >= seg.blk1; }
};

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
    if (pad + C::kBar + kCtlBytes > C::kSmem) {   // cannot happen with an aligned dynamic base
        if (tid == 0) p.err[cta] = 80;
        return;
    }
    uint8_t *sm = smem_raw + pad, *ctl = sm + C::kBar;
    auto bar = [&](int i) { return smem_u32(ctl + 8 * i); };
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(ctl + kOffTmem);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(ctl + kOffAbort);
    int *err_sh = reinterpret_cast<int *>(ctl + kOffErr);
    auto fail = [&](int code) { record_failure(abort_flag, err_sh, code); };

    if (warp == 0) {
        tmem_alloc(smem_u32(tmem_slot), kTmemCols);
        tmem_relinquish();
    }
    if (tid == 32 * kProducerWarp) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(B_QFULL + i), 1);
            mbar_init(bar(B_QEMPTY + i), 2);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(bar(B_PVDONE + i), 1);
            mbar_init(bar(B_SFULL + i), 1);
            mbar_init(bar(B_PREADY + i), 32 * kSoftmaxWarps / 2);
        }
        mbar_init(bar(B_FIN), 2);
        for (int s = 0; s < NST; ++s) {
            mbar_init(bar(B_KFULL + s), 1);
            mbar_init(bar(B_KEMPTY + s), 2);
            mbar_init(bar(B_VFULL + s), 1);
            mbar_init(bar(B_VEMPTY + s), 2);
        }
        *abort_flag = 0;
        *err_sh = 0;
        fence_mbar_init();
        tma_prefetch_desc(&mQ);
        tma_prefetch_desc(&mKc);
        tma_prefetch_desc(&mVc);
        tma_prefetch_desc(&mKn);
        tma_prefetch_desc(&mVn);
    }

    // ---------------------------------------------------------------- plan
    // total units, then the sequence that this CTA's run starts in
    int64_t *plan = reinterpret_cast<int64_t *>(ctl + kOffPlan);                // units before the first sequence, its index
    Seq *plan_seq = reinterpret_cast<Seq *>(plan + 2);
    int64_t *wsum = reinterpret_cast<int64_t *>(ctl + kOffXch);                 // [11], where no copy (async proxy) ever lands
    static_assert(16 + sizeof(Seq) <= kOffPar - kOffPlan, "plan area");
    static_assert(kOffXch % 8 == 0 && 8 * kThreads / 32 <= kCtlBytes - kOffXch, "scratch of the plan");
    int64_t W = 0, w0 = 0, w1 = 0;
    const bool one_pass = p.num_seqs <= kThreads;
    if (!one_pass) {   // the total first
        for (int b = tid; b < p.num_seqs; b += kThreads) W += load_seq<ROWS>(p, b).work(p.Hkv);
#pragma unroll
        for (int o = 16; o; o >>= 1) W += __shfl_xor_sync(kAll, W, o);
        if (lane == 0) wsum[warp] = W;
        __syncthreads();
        W = 0;
        for (int i = 0; i < kThreads / 32; ++i) W += wsum[i];
    }
    auto my_run = [&] {
        const int runs = (int)min((int64_t)gridDim.x, W);   // no run is empty
        w0 = w1 = W;
        if (cta < runs) {
            const Cut cut(W, runs);
            w0 = cut.start(cta);
            w1 = cut.start(cta + 1);
        }
    };
    if (!one_pass) my_run();
    int64_t carry = 0;
    for (int b0 = 0; b0 < p.num_seqs && (carry <= w0 || cta == 0); b0 += kThreads) {
        const int b = b0 + tid;
        Seq s;
        int64_t mine = 0;
        if (b < p.num_seqs) {
            s = load_seq<ROWS>(p, b);
            mine = s.work(p.Hkv);
        }
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
        for (int i = 0; i < kThreads / 32; ++i) {
            if (i < warp) before += wsum[i];
            carry += wsum[i];
        }
        if (one_pass) {
            W = carry;
            my_run();
        }
        const int64_t start = before + incl - mine;
        if (mine > 0 && start <= w0 && w0 < start + mine) {
            plan[0] = start;
            plan[1] = b;
            *plan_seq = s;
        }
        if (cta == 0 && b < p.num_seqs) p.prefix[b] = start;
    }
    if (cta == 0 && tid == 0) p.prefix[p.num_seqs] = W;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = *tmem_slot;
    const uint64_t lim = p.timeout_ns, drain = p.drain_ns;
    if (w0 < w1) {
    Walk<ROWS> seg(p, w0, w1, (int)plan[1], plan[0], *plan_seq);

    if (warp == kProducerWarp) {
        // ------------------------------------------------------------ TMA producer
        if (lane == 0) {
            int used = 0, segs = 0;   // key blocks and segments so far
            int issued_k[NST] = {}, issued_v[NST] = {}, issued_q[2] = {};
            const uint32_t qbytes = 2u * 128u * (uint32_t)(p.group * p.box_nodes);
            bool ok = true;
            for (; ok && seg.next(); ++segs) {
                const int tiles = seg.tiles(), qb = segs % p.q_bufs;
                if (segs >= p.q_bufs && !wait_phase(bar(B_QEMPTY + qb), (segs / p.q_bufs - 1) & 1, lim, abort_flag)) { fail(81); break; }
                mbar_arrive_expect_tx(bar(B_QFULL + qb), tiles * qbytes);
                for (int x = 0; x < tiles; ++x) {
                    const int row = (int)(seg.s.bos + (ROWS ? 2 * seg.it + x : 0) * p.tile_nodes);
                    const uint32_t at = smem_u32(sm + C::kQ + x * kBlk) + qb * (kHalf / 2);
                    tma_load_3d(at, &mQ, 0, seg.h * p.group, row, bar(B_QFULL + qb));
                    tma_load_3d(at + kHalf, &mQ, 64, seg.h * p.group, row, bar(B_QFULL + qb));
                }
                ++issued_q[qb];
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
                    if (used >= NST && !wait_phase(bar(B_KEMPTY + s), ph, lim, abort_flag)) { fail(82); ok = false; break; }
                    copy(C::kK + s * kBlk, &mKc, &mKn, bar(B_KFULL + s));
                    ++issued_k[s];
                    if (used >= NST && !wait_phase(bar(B_VEMPTY + s), ph, lim, abort_flag)) { fail(83); ok = false; break; }
                    copy(C::kV + s * kBlk, &mVc, &mVn, bar(B_VFULL + s));
                    ++issued_v[s];
                }
            }
            const int zero = 0;   // no copy may still be landing in shared memory at exit
            for (int s = 0; s < 2; ++s)
                if (issued_q[s]) wait_phase(bar(B_QFULL + s), (issued_q[s] - 1) & 1, drain, &zero);
            for (int s = 0; s < NST; ++s) {
                if (issued_k[s]) wait_phase(bar(B_KFULL + s), (issued_k[s] - 1) & 1, drain, &zero);
                if (issued_v[s]) wait_phase(bar(B_VFULL + s), (issued_v[s] - 1) & 1, drain, &zero);
            }
        }
    } else if (warp >= kMmaWarp) {
        // ------------------------------------------------------------ MMA issuers, one warp per stream
        // Both release every stage, whether they had a product on it or not.
        const int x = warp - kMmaWarp;
        constexpr uint32_t id_s = idesc_bf16(kBM, kSub, false, false);  // Q (K-major) x K (K-major)
        constexpr uint32_t id_o = idesc_bf16(kBM, kD, false, true);     // P (TMEM) x V (MN-major)
        const uint64_t dKm = desc_sw128(smem_u32(sm), 16, 1024);
        const uint64_t dMN = desc_sw128(smem_u32(sm), kHalf, 1024);
        int used = 0, segs = 0;
        int qks = 0, pvs = 0;   // score and output products issued
        bool ok = true;
        auto wait = [&](int b, uint32_t parity, int code) {
            if (!__all_sync(kAll, wait_phase(bar(b), parity, lim, abort_flag))) {
                fail(code);
                ok = false;
            }
            return ok;
        };
        for (; ok && seg.next(); ++segs) {
            const int qb = segs % p.q_bufs;
            if (!wait(B_QFULL + qb, (segs / p.q_bufs) & 1, 84)) break;
            const uint64_t qd = dKm + ((C::kQ + (ROWS ? x * kBlk : qb * (kHalf / 2))) >> 4);
            // S = Q K^T of half block `a`, into the buffer whose P the product
            // before last has read
            auto scores = [&](const Halves<ROWS> &a) {
                const int at = used + a.j - seg.blk0, s = at % NST;
                if (a.h == 0 && !wait(B_KFULL + s, (at / NST) & 1, 85)) return;
                if (a.has(seg, x)) {
                    const int n = qks;
                    if (n >= 2 && !wait(B_PVDONE + 2 * x + (n & 1), ((n - 2) >> 1) & 1, 86)) return;
                    tc_fence_after();
                    const uint64_t kd = dKm + ((C::kK + s * kBlk + a.half(x) * (kHalf / 2)) >> 4);
                    const uint32_t d = tm + TM_S + x * 128 + (n & 1) * kSub;
                    if (elect_one()) {
#pragma unroll
                        for (int ks = 0; ks < kD / 16; ++ks) {
                            const uint32_t off = ((ks >> 2) * kHalf + (ks & 3) * 32) >> 4;
                            mma_bf16_ss(d, qd + off, kd + off, id_s, ks > 0);
                        }
                        mma_commit(bar(B_SFULL + 2 * x + (n & 1)));
                    }
                    __syncwarp();
                    ++qks;
                }
                if (a.last(seg) && elect_one()) {
                    mma_commit(bar(B_KEMPTY + s));
                    if (a.j == seg.blk1 - 1) mma_commit(bar(B_QEMPTY + qb));
                }
                __syncwarp();
            };
            Halves<ROWS> a{seg.blk0, 0}, c{seg.blk0, 0};   // next scores, next outputs
            for (int i = 0; ok && i < 2 && !a.done(seg); ++i, a.step(seg)) scores(a);
            uint32_t more = 0;
            for (; ok && !c.done(seg); c.step(seg)) {
                const int at = used + c.j - seg.blk0, s = at % NST, h = c.half(x);
                if (c.h == 0 && !wait(B_VFULL + s, (at / NST) & 1, 88)) break;
                if (c.has(seg, x)) {
                    const int n = pvs;
                    if (!wait(B_PREADY + 2 * x + (n & 1), (n >> 1) & 1, 87)) break;
                    tc_fence_after();
                    // O (+)= P V, over the keys that count (P is zero beyond them)
                    const int steps = (min(kSub, seg.valid(c.j) - kSub * h) + 15) / 16;
                    const uint64_t vd = dMN + ((C::kV + s * kBlk + h * (kHalf / 2)) >> 4);
                    const uint32_t pa = tm + TM_S + x * 128 + (n & 1) * kSub;
                    if (elect_one()) {
#pragma unroll
                        for (int ks = 0; ks < kSub / 16; ++ks)
                            if (ks < steps) mma_bf16_ts(tm + TM_O + x * kD, pa + ks * 8, vd + ks * (2048 >> 4), id_o, ks > 0 ? 1u : more);
                        mma_commit(bar(B_PVDONE + 2 * x + (n & 1)));
                    }
                    __syncwarp();
                    more = 1;
                    ++pvs;
                }
                if (c.last(seg) && elect_one()) mma_commit(bar(B_VEMPTY + s));
                __syncwarp();
                if (!a.done(seg)) {
                    scores(a);
                    a.step(seg);
                }
            }
            used += seg.blk1 - seg.blk0;
        }
        if (elect_one()) mma_commit(bar(B_FIN));   // every issued MMA completes before TMEM is released
        __syncwarp();
        const int zero = 0;
        wait_phase(bar(B_FIN), 0, drain, &zero);
    } else {
        // ------------------------------------------------------------ softmax (warps 0-7)
        // A wait that gives up does not leave the loops (others could be
        // waiting at an exchange): with the abort flag set the remaining waits
        // return at once and nothing is stored.
        const int x = warp >> 2, gtid = tid & 127;
        const int r = gtid;                      // row of the tile = TMEM lane
        const uint32_t lane_off = static_cast<uint32_t>(32 * (warp & 3)) << 16;
        const uint32_t oa = tm + lane_off + TM_O + x * kD;
        const float c = p.c;
        float2 *xch = reinterpret_cast<float2 *>(ctl + kOffXch);          // [stream][128 rows]
        int8_t *par = reinterpret_cast<int8_t *>(ctl + kOffPar) + x * 64;
        const int bar_group = 1 + x, bar_both = 3;
        int used = 0, cnt = 0;                   // key blocks so far; half blocks of this stream so far
        bool ok = true;
        auto wait = [&](int b, uint32_t parity, int code) {
            if (!__all_sync(kAll, wait_phase(bar(b), parity, lim, abort_flag))) {
                fail(code);
                ok = false;
            }
        };
        auto wait_pv = [&](int n, int code) { wait(B_PVDONE + 2 * x + (n & 1), (n >> 1) & 1, code); };   // P V of half block n
        while (seg.next()) {
            const int tile = ROWS ? 2 * seg.it + x : 0;
            if (ROWS && tile >= seg.s.tiles) {   // an odd tile count leaves stream 1 without rows
                used += seg.blk1 - seg.blk0;
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
                named_bar_sync(bar_group, 128);
                if (gtid < seg.s.n) par[gtid] = (int8_t)tree_parent(p.parents, seg.s.bos, gtid);
                named_bar_sync(bar_group, 128);
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
            const int top = p.window ? __reduce_max_sync(kAll, vrow ? far : INT32_MIN) : 0;   // the warp's last masked position
            // half blocks with all 64 keys, which come first, need no care; the last
            // block of the cache and the tree's own go through `a`
            const int full = min(seg.blk1 - seg.blk0, max(0, (seg.s.len - seg.s.kstart) / kBN - seg.blk0));
            const int plain = ROWS ? 2 * full : full;
            Halves<ROWS> a{seg.blk0 + full, 0};
            int k0 = seg.key0(seg.blk0) + (ROWS ? 0 : kSub * x);   // first slot of the half block
            constexpr int kStep = ROWS ? kSub : kBN;
            // positions of a half block's keys, two a lane, fetched ahead
            int p0 = INT32_MAX, p1 = INT32_MAX;
            auto fetch_pos = [&](int k) {
                p0 = k + lane < seg.s.len ? pos[k + lane] : INT32_MAX;
                p1 = k + 32 + lane < seg.s.len ? pos[k + 32 + lane] : INT32_MAX;
            };
            const bool by_pos = pos && work;
            if (by_pos) fetch_pos(k0);
            float m = -INFINITY, l = 0.f;
            const int cnt0 = cnt;
            for (int u = 0;; ++u, k0 += kStep) {
                const bool special = u >= plain;
                bool masked = false;
                uint64_t vis = ~0ull;            // which of the 64 keys the row sees
                int valid = kSub, j = 0, h = 0;
                if (special) {
                    while (!a.done(seg) && !a.has(seg, x)) a.step(seg);   // by keys, short blocks have nothing for stream 1
                    if (a.done(seg)) break;
                    j = a.j;
                    h = a.half(x);
                    valid = min(kSub, seg.valid(j) - kSub * h);
                    vis = seg.draft(j) ? anc : valid >= kSub ? ~0ull : (1ull << valid) - 1;
                    masked = true;
                }
                if (p.window && work && !(special && seg.draft(j))) {
                    if (pos) {
                        if (__reduce_min_sync(kAll, min(p0, p1)) <= top) {
                            uint32_t lo = 0, hi = 0;
                            for (int i = 0; i < 32; ++i) {
                                if (__shfl_sync(kAll, p0, i) > far) lo |= 1u << i;
                                if (__shfl_sync(kAll, p1, i) > far) hi |= 1u << i;
                            }
                            vis &= (uint64_t)hi << 32 | lo;
                            masked = true;
                        }
                    } else if (k0 <= top) {
                        const int skip = far + 1 - k0;   // keys of this half before the window
                        if (skip > 0) vis &= skip >= kSub ? 0 : ~0ull << skip;
                        masked = true;
                    }
                }
                if (by_pos) fetch_pos(k0 + kStep);
                const int buf = cnt & 1;
                const uint32_t sa = tm + lane_off + TM_S + x * 128 + buf * kSub;
                wait(B_SFULL + 2 * x + buf, (cnt >> 1) & 1, 89);
                tc_fence_after();
                if (work) {
                    float v[64];
                    tmem_ld64(sa, v);
                    if (masked) {
                        const uint32_t lo = (uint32_t)vis, hi = (uint32_t)(vis >> 32);
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            if (!(lo >> i & 1)) v[i] = -INFINITY;
                            if (!(hi >> i & 1)) v[32 + i] = -INFINITY;
                        }
                    }
                    float mx[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
                    for (int i = 4; i < 60; i += 8)
#pragma unroll
                        for (int e = 0; e < 4; ++e) mx[e] = fmaxf(fmaxf(mx[e], v[i + e]), v[i + 4 + e]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) mx[e] = fmaxf(mx[e], v[60 + e]);
                    const float mb = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;
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
                    const uint64_t cc = pack_f32x2(c, c), mm = pack_f32x2(-msub, -msub);
                    uint64_t sum[4] = {0, 0, 0, 0};
                    uint32_t pk[32];
#pragma unroll
                    for (int i = 0; i < 64; i += 2) {
                        float e0, e1;
                        unpack_f32x2(fma_f32x2(pack_f32x2(v[i], v[i + 1]), cc, mm), e0, e1);
                        e0 = ex2_approx(e0);
                        e1 = ex2_approx(e1);
                        sum[(i >> 1) & 3] = add_f32x2(sum[(i >> 1) & 3], pack_f32x2(e0, e1));
                        pk[i >> 1] = pack_bf16(e0, e1);
                    }
                    tmem_st32u(sa, pk);
                    float s0, s1;
                    unpack_f32x2(add_f32x2(add_f32x2(sum[0], sum[1]), add_f32x2(sum[2], sum[3])), s0, s1);
                    l = fmaf(l, alpha, s0 + s1);
                    if (__any_sync(kAll, rescale)) {    // once P V of the half block before has completed
                        if (cnt > cnt0) wait_pv(cnt - 1, 90);
                        tc_fence_after();
#pragma unroll 1
                        for (int c4 = 0; c4 < 4; ++c4) {
                            float o[32];
                            tmem_ld32(oa + 32 * c4, o);
#pragma unroll
                            for (int i = 0; i < 32; ++i) o[i] *= alpha;
                            tmem_st32(oa + 32 * c4, o);
                        }
                    }
                }
                if (special) {
                    // V rows behind the last key, up to the 16 of a product step, may hold
                    // anything; P is zero there and the rows are cleared (by rows both
                    // streams write the same zeros, each before its own product)
                    const int behind = (16 - valid % 16) % 16, at = used + j - seg.blk0;
                    if (behind) {
                        const int s = at % NST;
                        wait(B_VFULL + s, (at / NST) & 1, 91);
                        for (int e = gtid; e < behind * 16; e += 128) {
                            const int row = kSub * h + valid + e / 16, ch = e % 16;
                            st_shared_v4(smem_u32(sm + C::kV + s * kBlk + (ch >> 3) * kHalf + row * 128 + (ch & 7) * 16), 0, 0, 0, 0);
                        }
                        fence_proxy_async_smem();
                    }
                    a.step(seg);
                }
                ++cnt;
                tc_fence_before();
                mbar_arrive(bar(B_PREADY + 2 * x + buf));
            }
            used += seg.blk1 - seg.blk0;
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
            if (cnt > cnt0) wait_pv(cnt - 1, 92);
            if (ROWS) {
                tc_fence_after();
                if (work) {
                    const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll 1
                    for (int c4 = 0; c4 < 4; ++c4) {
                        float v[32];
                        tmem_ld32(oa + 32 * c4, v);
                        if (vrow && ok) store(32 * c4, v, inv);
                    }
                    if (vrow && ok) store_ml(m, l);
                }
            } else {
                // merge the streams; each writes 64 columns
                xch[x * 128 + r] = make_float2(m, l);             // a stream without keys: m = -inf, l = 0
                tc_fence_before();
                named_bar_sync(bar_both, 32 * kSoftmaxWarps);     // both streams' products have completed
                tc_fence_after();
                if (work) {
                    const float2 s0 = xch[r], s1 = xch[128 + r];
                    const float mm = fmaxf(s0.x, s1.x);
                    const float f0 = s0.x == -INFINITY ? 0.f : ex2_approx(s0.x - mm), f1 = s1.x == -INFINITY ? 0.f : ex2_approx(s1.x - mm);
                    const float ll = f0 * s0.y + f1 * s1.y, inv = ll > 0.f ? 1.f / ll : 0.f;
                    // a stream that had no half block in this segment has no accumulator
                    const bool two = seg.valid(seg.blk0) > kSub;   // full blocks come first
#pragma unroll 1
                    for (int c4 = 0; c4 < 2; ++c4) {
                        float v[32];
                        tmem_ld32(tm + lane_off + TM_O + 64 * x + 32 * c4, v);
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] *= f0;
                        if (two) {
                            float u[32];
                            tmem_ld32(tm + lane_off + TM_O + kD + 64 * x + 32 * c4, u);
#pragma unroll
                            for (int i = 0; i < 32; ++i) v[i] = fmaf(u[i], f1, v[i]);
                        }
                        if (vrow && ok) store(64 * x + 32 * c4, v, inv);
                    }
                    if (vrow && ok && x == 0) store_ml(mm, ll);
                }
                tc_fence_before();
                named_bar_sync(bar_both, 32 * kSoftmaxWarps);   // both accumulators read, the exchange free
            }
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
        const int64_t start = p.prefix[b] + ((int64_t)h * s.items + it) * s.cost() + kItemCost, last = start + s.blocks - 1;
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
    // trees of at most half a tile leave room for the next item's Q beside this
    // one's (a token of 64 sequences: 56.9 against 58.3 us)
    p.box_nodes = ROWS ? nodes : L.max_nodes;
    p.q_bufs = !ROWS && group * L.max_nodes <= kBM / 2 ? 2 : 1;
    CUtensorMap mq, mkc, mvc, mkn, mvn;
    const int64_t rows = (int64_t)L.num_seqs * L.capacity;
    bool ok = make_rows_map(&mq, L.q, L.total_nodes, L.Hq, group, p.box_nodes) && make_rows_map(&mkn, L.k, L.total_nodes, L.Hkv, 1, kBox) &&
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
    // Few items are cut many times: then a whole block joins a row.  A warp and a
    // block a row: 30.7 and 16.5 us for one token at 8192 slots, 108 and 83 for 24
    // nodes at 262144; 169 and 270 for 32 trees of 64 nodes, of two parts each.
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
