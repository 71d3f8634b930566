// Attention weight that the newest tokens of a sequence lay on every slot of
// its cache and on one another, added up per key.
//
//   w[s] += sum over queries i and the heads of the group of 2^(c q_i . k_s - lse_i log2(e)),  c = scale log2(e)
//
// The log-sum-exp is known, so no row statistics are needed and the sum runs
// over the rows, not the keys.  The keys are therefore the M side of the
// product, 128 a block: S^T = K Q^T in tensor memory has a key per lane, and a
// thread adds up its key's columns without talking to another.  Every key
// belongs to one CTA and its sum runs in a fixed order: results repeat.
//
// What bounds it: K is read once, 256 bytes a key and key/value head, for
// R = queries x Hq / Hkv rows of 256 flops and one exponential each.  Memory up
// to about R = 100; beyond, the special-function unit (16 exponentials a clock
// and SM against 32 keys' worth of tensor work).
//
// Bf16, 16 query and 2 key/value heads: 5 queries of each of 32 sequences over 0 to
// 8192 slots take 28.9 us (3.6 TB/s), 64 queries over the 32768 tokens of a prompt
// 22.8 (8.5 us of exponentials at 16 a clock).
//
// All (sequence, key/value head, key block) units are laid end to end, each
// weighted by its row chunks, and cut evenly over one persistent CTA per SM.
// Four groups of 4 warps take the key blocks in turn, each with its own 128
// columns of tensor memory, so that a block's sums need no exchange and the groups'
// special-function work fills the gaps of one another.  Up to two chunks of 128 query
// rows stay in shared memory for a whole item; longer query lists stream through
// the same slots, once for four blocks.
//   warps 0-15  sums: group w / 4, the keys of TMEM lane quarter w % 4
//   warp 16     TMA producer
//   warp 17     MMA issuer
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

constexpr int kD = 128, kKeys = 128, kRows = 128;
constexpr uint32_t kHalf = 16384, kBlk = 2 * kHalf;
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kKStages = 4, kQSlots = 2;
constexpr int kGroups = 4;
constexpr int kSumWarps = 16, kProducerWarp = 16, kMmaWarp = 17, kThreads = 32 * 18;

constexpr uint32_t SM_K = 0, SM_Q = kKStages * kBlk, SM_CTL = SM_Q + kQSlots * kBlk;
enum : int { B_KFULL = 0, B_KEMPTY = B_KFULL + kKStages, B_QFULL = B_KEMPTY + kKStages, B_QEMPTY = B_QFULL + kQSlots,
             B_SFULL = B_QEMPTY + kQSlots, B_SEMPTY = B_SFULL + 4, B_FIN = B_SEMPTY + 4, B_NUM };
constexpr uint32_t kOffTmem = 8 * B_NUM, kOffAbort = kOffTmem + 4, kOffErr = kOffTmem + 8, kOffPlan = 192;   // units, index, Seq
constexpr uint32_t kOffLse = 256;                              // [groups][slots][128] fp32: lse log2(e)
constexpr uint32_t kOffPos = kOffLse + kGroups * kQSlots * 512;   // the same, int32: positions of the rows' queries
constexpr size_t kSmem = SM_CTL + kOffPos + kGroups * kQSlots * 512 + 1024;
static_assert(kOffErr + 4 <= kOffPlan, "barrier area");
static_assert(kSmem <= 232448, "shared memory");
constexpr uint32_t kTmemCols = 512;

struct Params {
    const float *lse, *w_in;
    float *w_out, *w_new;
    const int32_t *cuq, *cut, *lens, *pos, *seen;
    int64_t uq, ut, total_q, total_t, capacity;
    int num_seqs, Hq, Hkv, group, chunk_q;   // chunk_q: queries of a chunk of rows
    int window;                              // INT32_MAX: none
    float c;
    int *status;                             // cleared before the launch
    uint64_t timeout_ns, drain_ns;
};

struct Seq {
    int64_t q0, t0;
    int nq, m, len, old_blocks, blocks, chunks, cost;   // cost of a key block
    __device__ __forceinline__ int64_t work(int Hkv) const { return (int64_t)Hkv * blocks * cost; }
};

__device__ __forceinline__ Seq load_seq(const Params &p, int b) {
    Seq s;
    s.nq = seq_rows(p.cuq, p.uq, p.total_q, b, INT32_MAX, s.q0);
    s.m = seq_rows(p.cut, p.ut, p.total_t, b, INT32_MAX, s.t0);
    if (s.nq > s.m) {
        s.q0 += s.nq - s.m;
        s.nq = s.m;
    }
    s.len = cached_slots(p.lens, p.capacity, b);
    s.old_blocks = (s.len + kKeys - 1) / kKeys;
    s.blocks = s.old_blocks + (s.m + kKeys - 1) / kKeys;
    s.chunks = (s.nq + p.chunk_q - 1) / p.chunk_q;
    s.cost = max(1, s.chunks);
    return s;
}

// A CTA's run of work, cut into segments of key blocks [blk0, blk1) of one
// (sequence, key/value head).  A block belongs to the run that its first unit is in.
struct Walk {
    const Params &p;
    int64_t w, end, base;
    int b;
    Seq s;
    int h, blk0, blk1;
    __device__ Walk(const Params &p_, int64_t w_, int64_t end_, int b_, int64_t base_, const Seq &s_)
        : p(p_), w(w_), end(end_), base(base_), b(b_), s(s_) {}
    __device__ __forceinline__ bool next() {
        while (w < end) {
            int64_t share;
            while (w >= base + (share = s.work(p.Hkv))) {
                base += share;
                s = load_seq(p, ++b);
            }
            const int64_t head = (int64_t)s.blocks * s.cost, off = w - base;
            h = head <= INT32_MAX && off <= INT32_MAX ? (int)((uint32_t)off / (uint32_t)head) : (int)(off / head);
            const int64_t at = off - h * head, upto = min(head, at + (end - w));
            if (s.cost == 1) {
                blk0 = (int)at;
                blk1 = (int)upto;
            } else {
                blk0 = (int)((at + s.cost - 1) / s.cost);
                blk1 = (int)((upto + s.cost - 1) / s.cost);
            }
            w += upto - at;
            if (blk0 < blk1) return true;
        }
        return false;
    }
    __device__ __forceinline__ bool old(int j) const { return j < s.old_blocks; }
    __device__ __forceinline__ int key0(int j) const { return (old(j) ? j : j - s.old_blocks) * kKeys; }
    __device__ __forceinline__ int valid(int j) const { return min(kKeys, (old(j) ? s.len : s.m) - key0(j)); }
    // rows of chunk c that exist
    __device__ __forceinline__ int rows(int c) const { return min(p.chunk_q, s.nq - c * p.chunk_q) * p.group; }
    // whether no query of chunk c sees a key of block j: later tokens, or, by the
    // order of the new tokens, ones before the window
    __device__ __forceinline__ bool skip(int j, int c) const {
        if (old(j)) return false;
        const int q_first = s.m - s.nq + c * p.chunk_q, q_last = min(s.m - 1, q_first + p.chunk_q - 1);
        return key0(j) > q_last || q_first - (key0(j) + kKeys - 1) >= p.window;
    }
};

__global__ void __launch_bounds__(kThreads, 1)
    cache_weights_kernel(const __grid_constant__ CUtensorMap mQ, const __grid_constant__ CUtensorMap mKc,
                         const __grid_constant__ CUtensorMap mKn, const Params p) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t pad = (1024u - (smem_u32(smem_raw) & 1023u)) & 1023u;
    uint8_t *sm = smem_raw + pad, *ctl = sm + SM_CTL;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, cta = blockIdx.x;
    constexpr unsigned kAll = 0xffffffffu;
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
        tma_prefetch_desc(&mQ);
        tma_prefetch_desc(&mKc);
        tma_prefetch_desc(&mKn);
        for (int s = 0; s < kKStages; ++s) {
            mbar_init(bar(B_KFULL + s), 1);
            mbar_init(bar(B_KEMPTY + s), 1);
        }
        for (int s = 0; s < kQSlots; ++s) {
            mbar_init(bar(B_QFULL + s), 1);
            mbar_init(bar(B_QEMPTY + s), 1);
        }
        for (int s = 0; s < 4; ++s) {
            mbar_init(bar(B_SFULL + s), 1);
            mbar_init(bar(B_SEMPTY + s), 32 * kSumWarps / kGroups);
        }
        mbar_init(bar(B_FIN), 1);
        *abort_flag = 0;
        *err_sh = 0;
        fence_mbar_init();
    }

    // ---------------------------------------------------------------- plan (as in tree_attention.cu)
    int64_t *plan = reinterpret_cast<int64_t *>(ctl + kOffPlan);                // units before the first sequence, its index
    Seq *plan_seq = reinterpret_cast<Seq *>(plan + 2);
    static_assert(16 + sizeof(Seq) <= kOffLse - kOffPlan, "plan area");
    int64_t *wsum = reinterpret_cast<int64_t *>(ctl + kOffLse);                 // [18], where no copy (async proxy) ever lands
    static_assert(kOffLse % 8 == 0 && 8 * kThreads / 32 <= kGroups * kQSlots * 512, "scratch of the plan");
    int64_t W = 0, w0 = 0, w1 = 0;
    const bool one_pass = p.num_seqs <= kThreads;
    if (!one_pass) {   // the total first
        for (int b = tid; b < p.num_seqs; b += kThreads) W += load_seq(p, b).work(p.Hkv);
#pragma unroll
        for (int o = 16; o; o >>= 1) W += __shfl_xor_sync(kAll, W, o);
        if (lane == 0) wsum[warp] = W;
        __syncthreads();
        W = 0;
        for (int i = 0; i < kThreads / 32; ++i) W += wsum[i];
    }
    auto my_run = [&] {
        const Cut cut(W, gridDim.x);
        w0 = cut.start(cta);
        w1 = cut.start(cta + 1);
    };
    if (!one_pass) my_run();
    int64_t carry = 0;
    for (int b0 = 0; b0 < p.num_seqs && carry <= w0; b0 += kThreads) {
        const int b = b0 + tid;
        Seq s;
        int64_t mine = 0;
        if (b < p.num_seqs) {
            s = load_seq(p, b);
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
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = *tmem_slot;
    const uint64_t lim = p.timeout_ns, drain = p.drain_ns;
    if (w0 < w1) {
    Walk seg(p, w0, w1, (int)plan[1], plan[0], *plan_seq);

    if (warp == kProducerWarp) {
        // ------------------------------------------------------------ TMA producer
        if (lane == 0) {
            int keys = 0, loads = 0;   // key blocks and row chunks so far
            int issued_k[kKStages] = {}, issued_q[kQSlots] = {};
            const uint32_t qbytes = 2u * 128u * (uint32_t)(p.group * p.chunk_q);
            bool ok = true;
            auto load_q = [&](int c) -> bool {
                const int s = loads % kQSlots;
                if (loads >= kQSlots && !wait_phase(bar(B_QEMPTY + s), ((loads - kQSlots) / kQSlots) & 1, lim, abort_flag)) {
                    fail(101);
                    return false;
                }
                mbar_arrive_expect_tx(bar(B_QFULL + s), qbytes);
                const int row = (int)seg.s.q0 + c * p.chunk_q;
                tma_load_3d(smem_u32(sm + SM_Q + s * kBlk), &mQ, 0, seg.h * p.group, row, bar(B_QFULL + s));
                tma_load_3d(smem_u32(sm + SM_Q + s * kBlk + kHalf), &mQ, 64, seg.h * p.group, row, bar(B_QFULL + s));
                ++issued_q[s];
                ++loads;
                return true;
            };
            while (ok && seg.next()) {
                const int chunks = seg.s.chunks;
                if (chunks == 0) continue;
                const bool resident = chunks <= kQSlots;
                for (int j = seg.blk0; ok && j < seg.blk1; j += kGroups) {
                    if (resident && j == seg.blk0)
                        for (int c = 0; ok && c < chunks; ++c) ok = load_q(c);
                    for (int x = 0; x < kGroups && j + x < seg.blk1; ++x, ++keys) {
                        const int s = keys % kKStages;
                        if (keys >= kKStages && !wait_phase(bar(B_KEMPTY + s), ((keys - kKStages) / kKStages) & 1, lim, abort_flag)) {
                            fail(102);
                            ok = false;
                            break;
                        }
                        const bool old = seg.old(j + x);
                        const int row = (int)((old ? seg.b * p.capacity : seg.s.t0) + seg.key0(j + x));
                        const CUtensorMap *m = old ? &mKc : &mKn;
                        mbar_arrive_expect_tx(bar(B_KFULL + s), kBlk);
                        tma_load_3d(smem_u32(sm + SM_K + s * kBlk), m, 0, seg.h, row, bar(B_KFULL + s));
                        tma_load_3d(smem_u32(sm + SM_K + s * kBlk + kHalf), m, 64, seg.h, row, bar(B_KFULL + s));
                        ++issued_k[s];
                    }
                    if (!resident)
                        for (int c = 0; ok && c < chunks; ++c) ok = load_q(c);
                }
            }
            const int zero = 0;   // no copy may still be landing in shared memory at exit
            for (int s = 0; s < kKStages; ++s)
                if (issued_k[s]) wait_phase(bar(B_KFULL + s), (issued_k[s] - 1) & 1, drain, &zero);
            for (int s = 0; s < kQSlots; ++s)
                if (issued_q[s]) wait_phase(bar(B_QFULL + s), (issued_q[s] - 1) & 1, drain, &zero);
        }
    } else if (warp == kMmaWarp) {
        // ------------------------------------------------------------ MMA issuer
        const uint64_t dKm = desc_sw128(smem_u32(sm), 16, 1024);
        int keys = 0, loads = 0, blocks = 0, cnt[kGroups] = {0, 0, 0, 0};   // cnt: products per group
        bool ok = true;
        auto wait = [&](int b, uint32_t parity, int code) {
            if (!__all_sync(kAll, wait_phase(bar(b), parity, lim, abort_flag))) {
                fail(code);
                ok = false;
            }
            return ok;
        };
        // S^T = K Q^T of the block in K stage `key` and the chunk in slot `slot`, for group g
        auto product = [&](int g, int key, int slot, int rows) {
            int n = 0;   // products of this group so far (no dynamic indexing of registers)
#pragma unroll
            for (int i = 0; i < kGroups; ++i)
                if (i == g) n = cnt[i]++;
            if (n && !wait(B_SEMPTY + g, (n - 1) & 1, 105)) return;
            tc_fence_after();
            const uint32_t id = idesc_bf16(kKeys, min(kRows, (rows + 15) & ~15), false, false);
            const uint64_t kd = dKm + ((SM_K + key * kBlk) >> 4), qd = dKm + ((SM_Q + slot * kBlk) >> 4);
            if (elect_one()) {
#pragma unroll
                for (int ks = 0; ks < kD / 16; ++ks) {
                    const uint32_t off = ((ks >> 2) * kHalf + (ks & 3) * 32) >> 4;
                    mma_bf16_ss(tm + g * kRows, kd + off, qd + off, id, ks > 0);
                }
                mma_commit(bar(B_SFULL + g));
            }
            __syncwarp();
        };
        auto free_stage = [&](int b) {
            if (elect_one()) mma_commit(bar(b));
            __syncwarp();
        };
        while (ok && seg.next()) {
            const int chunks = seg.s.chunks, nblk = seg.blk1 - seg.blk0;
            if (chunks == 0) {
                blocks += nblk;
                continue;
            }
            if (chunks <= kQSlots) {   // all chunks stay
                for (int c = 0; ok && c < chunks; ++c) wait(B_QFULL + (loads + c) % kQSlots, ((loads + c) / kQSlots) & 1, 104);
                for (int j = seg.blk0; ok && j < seg.blk1; ++j, ++keys, ++blocks) {
                    if (!wait(B_KFULL + keys % kKStages, (keys / kKStages) & 1, 103)) break;
                    for (int c = 0; ok && c < chunks; ++c)
                        if (!seg.skip(j, c)) product(blocks % kGroups, keys % kKStages, (loads + c) % kQSlots, seg.rows(c));
                    free_stage(B_KEMPTY + keys % kKStages);
                }
                for (int c = 0; c < chunks; ++c) free_stage(B_QEMPTY + (loads + c) % kQSlots);
                loads += chunks;
            } else {
                for (int j = seg.blk0; ok && j < seg.blk1; j += kGroups) {
                    const int many = min(kGroups, seg.blk1 - j);
                    for (int x = 0; ok && x < many; ++x) wait(B_KFULL + (keys + x) % kKStages, ((keys + x) / kKStages) & 1, 103);
                    for (int c = 0; ok && c < chunks; ++c, ++loads) {
                        if (!wait(B_QFULL + loads % kQSlots, (loads / kQSlots) & 1, 104)) break;
                        for (int x = 0; ok && x < many; ++x)
                            if (!seg.skip(j + x, c)) product((blocks + x) % kGroups, (keys + x) % kKStages, loads % kQSlots, seg.rows(c));
                        free_stage(B_QEMPTY + loads % kQSlots);
                    }
                    for (int x = 0; x < many; ++x) free_stage(B_KEMPTY + (keys + x) % kKStages);
                    keys += many;
                    blocks += many;
                }
            }
        }
        free_stage(B_FIN);   // every issued MMA completes before TMEM is released
        const int zero = 0;
        wait_phase(bar(B_FIN), 0, drain, &zero);
    } else {
        // ------------------------------------------------------------ sums (warps 0-15)
        // As in tree_attention.cu, a wait that gives up does not leave the loops.
        const int grp = warp >> 2, gtid = tid & 127;
        const int r = gtid;   // the key of this thread = TMEM lane
        const uint32_t sa = tm + (static_cast<uint32_t>(32 * (warp & 3)) << 16) + grp * kRows;
        float *lse_sh = reinterpret_cast<float *>(ctl + kOffLse) + grp * kQSlots * kRows;
        int *pos_sh = reinterpret_cast<int *>(ctl + kOffPos) + grp * kQSlots * kRows;
        const int bar_group = 1 + grp;
        const float c2 = p.c;
        bool ok = true;
        int cnt = 0, blocks = 0;
        while (seg.next()) {
            const Seq &s = seg.s;
            const int chunks = s.chunks;
            const bool resident = chunks <= kQSlots;
            // positions count from the first new token
            const int64_t seen = p.pos ? p.seen[seg.b] : s.len;
            auto fetch = [&](int c) {   // lse and position of row gtid of chunk c, into its slot
                float l = INFINITY;
                if (gtid < seg.rows(c)) {
                    const int64_t row = (s.q0 + c * p.chunk_q + gtid / p.group) * p.Hq + (int64_t)seg.h * p.group + gtid % p.group;
                    l = p.lse[row];
                    l = l == -INFINITY ? INFINITY : l * kLog2e;
                }
                lse_sh[(c % kQSlots) * kRows + gtid] = l;
                pos_sh[(c % kQSlots) * kRows + gtid] = s.m - s.nq + c * p.chunk_q + gtid / p.group;
            };
            if (resident) {
                named_bar_sync(bar_group, 128);
                for (int c = 0; c < chunks; ++c) fetch(c);
                named_bar_sync(bar_group, 128);
            }
            for (int j = seg.blk0 + (grp - blocks % kGroups + kGroups) % kGroups; j < seg.blk1; j += kGroups) {
                const bool old = seg.old(j), mine = r < seg.valid(j);
                const int key = seg.key0(j) + r;
                const int64_t slot = ((int64_t)seg.b * p.Hkv + seg.h) * p.capacity + key;
                float before = 0.f;
                if (old && mine) before = p.w_in[slot];
                // a slot's position, seen from the first new token; never behind the first query
                int kp = 0;
                bool all = true;   // whether every row sees every key of the warp
                if (!old || p.window != INT32_MAX) {
                    if (mine) {
                        if (!old) kp = key;
                        else
                            kp = (int)max((int64_t)INT32_MIN, min((int64_t)(s.m - s.nq), (p.pos ? (int64_t)p.pos[slot] : key) - seen));
                    }
                    all = false;
                }
                const int kmin = all ? 0 : __reduce_min_sync(kAll, mine ? kp : INT32_MAX);
                const int kmax = all ? 0 : __reduce_max_sync(kAll, mine ? kp : INT32_MIN);
                float sum = 0.f;
                for (int c = 0; c < chunks; ++c) {
                    if (!resident) {
                        named_bar_sync(bar_group, 128);
                        fetch(c);
                        named_bar_sync(bar_group, 128);
                    }
                    if (seg.skip(j, c)) continue;
                    const int rows = seg.rows(c);
                    const float *ls = lse_sh + (c % kQSlots) * kRows;
                    const int *ps = pos_sh + (c % kQSlots) * kRows;
                    const int first = s.m - s.nq + c * p.chunk_q, last = first + rows / p.group - 1;
                    const bool open = all || ((old || kmax <= first) && (p.window == INT32_MAX || (int64_t)last - kmin < p.window));
                    if (!__all_sync(kAll, wait_phase(bar(B_SFULL + grp), cnt & 1, lim, abort_flag))) {
                        fail(106);
                        ok = false;
                    }
                    ++cnt;
                    tc_fence_after();
#pragma unroll 1
                    for (int c0 = 0; c0 < rows; c0 += 32) {
                        float v[32];
                        tmem_ld32(sa + c0, v);
                        if (c0 + 32 >= rows) {   // the last of them: the columns may be written again
                            tc_fence_before();
                            mbar_arrive(bar(B_SEMPTY + grp));
                            if (c0 + 32 > rows)
#pragma unroll
                                for (int i = 0; i < 32; ++i) v[i] = c0 + i < rows ? v[i] : 0.f;   // lse is infinite there
                        }
                        float a[4] = {0.f, 0.f, 0.f, 0.f};
                        if (open) {
#pragma unroll
                            for (int i = 0; i < 32; i += 4) {
                                const float4 l4 = *reinterpret_cast<const float4 *>(ls + c0 + i);
                                a[0] += ex2_approx(fmaf(v[i], c2, -l4.x));
                                a[1] += ex2_approx(fmaf(v[i + 1], c2, -l4.y));
                                a[2] += ex2_approx(fmaf(v[i + 2], c2, -l4.z));
                                a[3] += ex2_approx(fmaf(v[i + 3], c2, -l4.w));
                            }
                        } else {
#pragma unroll
                            for (int i = 0; i < 32; ++i) {
                                const float e = ex2_approx(fmaf(v[i], c2, -ls[c0 + i]));
                                a[i & 3] += (uint32_t)ps[c0 + i] - (uint32_t)kp < (uint32_t)p.window ? e : 0.f;   // a distance below 0 is above 2^31
                            }
                        }
                        sum += (a[0] + a[1]) + (a[2] + a[3]);
                    }
                }
                if (mine && ok) {
                    if (old) p.w_out[slot] = before + sum;
                    else p.w_new[(s.t0 + key) * p.Hkv + seg.h] = sum;
                }
            }
            blocks += seg.blk1 - seg.blk0;
        }
    }
    }
    tc_fence_before();
    __syncthreads();
    if (tid == 0 && *err_sh) atomicCAS(p.status, 0, *err_sh);
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tm, kTmemCols);
    }
}

}  // namespace

size_t cache_weights_workspace() { return 256; }

cudaError_t launch_cache_weights(const CacheWeightsLaunch &L, cudaStream_t stream) {
    static bool done[64] = {false};
    static int sms[64] = {0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!done[dev]) {
        e = cudaFuncSetAttribute(cache_weights_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
        if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms[dev], cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return e;
        done[dev] = true;
    }
    Params p;
    p.lse = L.lse; p.w_in = L.w_in; p.w_out = L.w_out; p.w_new = L.w_new;
    p.cuq = L.cu_queries; p.cut = L.cu_tokens; p.lens = L.cache_lens;
    p.pos = L.window ? L.cache_pos : nullptr; p.seen = L.seen;
    p.uq = L.cu_queries ? 0 : L.total_queries / L.num_seqs;
    p.ut = L.cu_tokens ? 0 : L.total_tokens / L.num_seqs;
    p.total_q = L.total_queries; p.total_t = L.total_tokens; p.capacity = L.capacity;
    p.num_seqs = L.num_seqs; p.Hq = L.Hq; p.Hkv = L.Hkv;
    p.group = L.Hq / L.Hkv;
    p.chunk_q = kRows / p.group;
    p.window = L.window ? L.window : INT32_MAX;
    p.c = L.scale * kLog2e;
    p.status = static_cast<int *>(L.workspace);
    p.timeout_ns = L.timeout_ns; p.drain_ns = L.drain_ns;
    CUtensorMap mq, mkc, mkn;
    const int64_t rows = (int64_t)L.num_seqs * L.capacity;
    bool ok = true, any = false;
    if (rows > 0) ok = make_rows_map(&mkc, L.k_cache, rows, L.Hkv, 1, kKeys), any = true;
    if (L.total_tokens > 0) ok = ok && make_rows_map(&mkn, L.k, L.total_tokens, L.Hkv, 1, kKeys);
    else mkn = mkc;
    if (!any) mkc = mkn;   // a map without a tensor is never read
    if (L.total_queries > 0) ok = ok && make_rows_map(&mq, L.q, L.total_queries, L.Hq, p.group, p.chunk_q);
    else mq = mkn;
    if (!ok) return cudaErrorInvalidValue;
    cache_weights_kernel<<<sms[dev], kThreads, kSmem, stream>>>(mq, mkc, mkn, p);
    return cudaGetLastError();
}

}  // namespace gdn
