// Attention of a tree of drafts on the 5th-generation tensor cores.
//
//   out[i] = sum_t softmax_t(scale <q_i, k_t>) v_t
// over the prefix and the entries of the tree in node i's mask, one pass over
// K and V with a running maximum and sum per row (a row: one node and one
// query head of the kv head's group).
//
// Work split.  A unit is one (request, kv head); its context is cut into
// blocks of BK keys.  The blocks of all units, laid end to end, are dealt out
// in equal contiguous ranges to the G groups of CTAs of a grid that fills the
// GPU once, so every SM reads the same amount of K and V whatever the batch
// and the lengths.  A group walks its range unit by unit (a segment each).  A
// unit that lies in one range is finished there; one that spans several
// leaves a partial (m, l, o) per range, joined by tree_join_kernel.  A range
// holds at most two partial segments (its first and its last), so the
// workspace does not grow with the context.
//
// Tiles.  Rows are cut into tiles of 128 (one MMA's M).  One tile: CTAs of
// one tile, two to an SM, which overlap each other's S / softmax / P V chain.
// Two and three: CTAs of two and three tiles, one to an SM, whose tiles take
// turns on the tensor core.  Four: groups of two CTAs, two tiles each, on the
// same range in step, so the second CTA finds K and V in L2.  (Three tiles as
// a launch of two and one of one read K and V twice: 320 rows at 131072 keys
// 728 us instead of 613.)
//
// A CTA: a producer warp that fills a ring of K and V blocks by TMA (one
// 16-row x 64-channel box per page and 128-byte column), a warp that issues
// the tcgen05.mma of all tiles, and four softmax warps per tile (a thread owns
// a row = TMEM lane).  Step i is block i / tiles, tile i % tiles.  Its S goes to
// S buffer i % NBUF, its P (bf16) overwrites that S, and behind P V (i) the
// issue warp sends S (i + NBUF) into the buffer: the tensor core runs them in
// order, so the buffer is free by then.  With no more buffers than tiles a
// finished S also says that O is at rest and may be rescaled; with more, the
// softmax warps wait for the P V before (rare: only when the maximum grows).
//
// Barriers are waited for by parity, which tells only the current phase from
// the one before.  So a barrier's waiter must know that the phase before the
// one it waits for is over: S barriers go by buffer where NBUF >= tiles (the
// waiter has seen S (i - tiles), which came after S (i - NBUF)), else by tile;
// P V barriers by tile (S (i) was issued behind P V (i - NBUF), and NBUF <= 2
// tiles), the end of a segment has one of its own.
//
// The tree's own entries.  In blocks that reach into the tree a row's bits
// pick the scores that count.  A V row that some nodes do not see must not
// reach them as 0 * infinity: the producer warp clears non-finite values from
// the tree's V rows (and all of the rows behind the request) once such a block
// has arrived, before it is handed on, and notes the nodes; rows that do see
// one of those end as NaN.
//
// Rounding.  P enters the second product in bf16, whatever the output's type:
// an MMA takes operands of one type, and V is bf16 (P as a sum of two bf16
// numbers would double the products of P V).  Each probability is off by at
// most half a step, 2^-8 of itself; together that is 0.0012 (64 keys) to 0.0017
// (4096 and more) of a result's norm, as much as a bf16 output's own rounding,
// and 0.0023 with it.  Scores, maxima, sums and O are fp32; the sum takes P as
// it is before rounding.
//
// Every wait is bounded.  A timeout is reported and the CTA drains: its rows of
// one range are zeros, and so are those joined with one of its partials.
#pragma once

#include "verify_tc.cuh"

namespace vc {
namespace tree {

using vtc::kTileRows;
constexpr int kSMs = 152;
constexpr int kBadRing = 16;  // segments whose cleared V rows are noted (more than the ring holds blocks)

struct Args {
    CUtensorMap kmap, vmap;
    const uint16_t *q;  // [B][n_q][Hq][D]
    int64_t n_pages;
    const int32_t *table, *lens;
    const unsigned long long *mask;  // [B][n_q]
    int batch, maxb, n_q, hq, hkv, grp, max_len;
    int rows;    // of a unit
    int lanes;   // CTAs per group
    int groups;  // G
    float scale_log2;
    float *ws_o;   // [CTA][2][rows of a CTA][D]
    float *ws_ml;  // [CTA][2][rows of a CTA][2]
    void *out;
    int out_bf16;
    int32_t *status;
    uint64_t wait_ns;
    int skip_copies;
};

template <int D, int QT>
struct Cfg {
    static constexpr int NC = D / 64;        // 128-byte columns of a row
    // Keys per block, S buffers.  An instruction of S (M 128, N = BK, K 16) takes
    // about 64 cycles for its A operand whatever N is, and the math of N = 128
    // 68: 128 keys where TMEM holds a buffer of that for each tile (256 rows at
    // 131072 keys, head_dim 128: 397 us; 64 keys with four buffers: 450).  A
    // third buffer for two tiles takes 64-channel heads from 172 to 154 us (256
    // rows at 8 x 32768 keys), four for three tiles from 274 to 213.  One-tile
    // CTAs, which memory bounds, take 64 keys, so that two fit an SM.
    static constexpr int BK = QT == 2 ? 128 : 64;
    static constexpr int NBUF = QT == 1 ? (D == 64 ? 2 : 1) : QT == 2 ? (D == 64 ? 3 : 2) : D == 64 ? 4 : 2;
    static constexpr bool AHEAD = NBUF > QT;
    static_assert(NBUF <= 2 * QT, "phases that a parity tells apart");
    static constexpr int PG = BK / kPage;    // pages of a block
    static constexpr int SLOT = BK * D * 2;  // one block of K or of V
    static constexpr bool QTM = QT == 1;     // Q in TMEM
    static constexpr int QTILE = kTileRows * D * 2;
    static constexpr int OFF_KV = QTM ? 0 : QT * QTILE;
    // where a softmax warp turns rows round (32 rows x 128 bytes each); with Q
    // in shared memory the warp's own rows of Q, which are done with by then
    static constexpr int STAGE = QTM ? 4 * 4096 : 0;
    static constexpr int FIT = ((QT == 1 ? 113 : 225) * 1024 - 512 - OFF_KV - STAGE) / SLOT;
    static constexpr int SLOTS = FIT < 14 ? FIT : 14;
    static_assert(SLOTS >= 5 && SLOTS / 2 + 2 <= kBadRing, "ring depth");
    static constexpr int OFF_STAGE = OFF_KV + SLOTS * SLOT;
    static constexpr int OFF_BAR = OFF_STAGE + STAGE;
    static constexpr int NS = NBUF < QT ? QT : NBUF;  // S barriers: by buffer, or by tile
    static constexpr int NBAR = 3 * QT + NS + NBUF + 2 * SLOTS + 2;  // q, o, pv per tile; s; p per buffer; full, empty; tail, idle
    static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
    static constexpr int SMEM = OFF_MISC + kBadRing * 8 + 16;
    static_assert(SMEM <= (QT == 1 ? 113 : 227) * 1024, "shared memory of the CTAs an SM holds");
    // TMEM columns: S (then P) and O of each tile, Q (bf16 pairs)
    static constexpr int O_COL0 = NBUF * BK;
    static constexpr int Q_COL0 = O_COL0 + QT * D;
    static constexpr int TMEM_USED = Q_COL0 + (QTM ? D / 2 : 0);
    static constexpr int TMEM_COLS = TMEM_USED <= 256 ? 256 : 512;
    static_assert(TMEM_USED <= (QT == 1 ? 256 : 512), "TMEM columns");
    static constexpr int SM_WARPS = QT * 4;  // softmax warps
    // CTAs of more than one tile: the last warpgroup (producer, MMA issue, two idle
    // warps) gives registers up for the softmax warps, which hold BK scores each
    // (2 x 128 x 216 + 128 x 72 = 384 x 168; 3 x 128 x 136 + 128 x 96 = 64512 <= 512 x 128)
    static constexpr int WARPS = QT == 1 ? 6 : 4 * QT + 4;
    static constexpr int REGS_SOFTMAX = QT == 2 ? 216 : 136, REGS_OTHER = QT == 2 ? 72 : 96;
    static constexpr int THREADS = WARPS * 32;
    static constexpr int MIN_CTAS = QT == 1 ? 2 : 1;
    static constexpr int ROWS = QT * kTileRows;
};

// Blocks of a request's context: 0 for one that is refused.
template <int BK, class A>
__device__ inline int blocks_of(const A &a, int b) {
    const int len = a.lens[b];
    return len >= a.n_q && len <= a.max_len ? ceil_div(len, BK) : 0;
}

// How the blocks of all units, laid end to end, are dealt out: T = q G + r,
// the first r groups take q + 1 blocks and the others q.  (T is below 2^31:
// K and V of 2^31 blocks would fill 70 TB.)
struct Deal {
    int q, r;
    __device__ Deal(int total, int groups) : q(total / groups), r(total % groups) {}
    __device__ int start(int g) const { return g * q + min(g, r); }
    __device__ int group_of(int block) const {
        const int split = r * (q + 1);
        return block < split ? block / (q + 1) : r + (block - split) / q;
    }
};

// Blocks (of one kv head) of all requests and of those before request
// `until`: every warp adds them up for itself, a lane per request.
template <int BK, class A>
__device__ inline void sum_blocks(const A &a, int until, int lane, int &total, int &before) {
    total = before = 0;
    for (int b = lane; b < a.batch; b += 32) {
        const int n = blocks_of<BK>(a, b);
        total += n;
        before += b < until ? n : 0;
    }
    for (int o = 16; o > 0; o >>= 1) {
        total += __shfl_xor_sync(0xffffffffu, total, o);
        before += __shfl_xor_sync(0xffffffffu, before, o);
    }
}

// The request that holds block f of the blocks laid end to end, and the block's
// place among that request's (all kv heads); by a warp.
template <int BK, class A>
__device__ inline void find_block(const A &a, int f, int lane, int &b, int &rest) {
    int before = 0;
    for (int b0 = 0;; b0 += 32) {
        const int n = b0 + lane < a.batch ? blocks_of<BK>(a, b0 + lane) * a.hkv : 0;
        int upto = n;
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += v;
        }
        const unsigned here = __ballot_sync(0xffffffffu, f < before + upto);
        if (here) {
            const int first = __ffs(here) - 1;
            b = b0 + first;
            rest = f - before - __shfl_sync(0xffffffffu, upto - n, first);
            return;
        }
        before += __shfl_sync(0xffffffffu, upto, 31);
    }
}

// A group's walk through its range.
template <int BK>
struct Walk {
    int b, kvh, blk, nblk, len;
    int left;
    bool first;
    // the current segment
    int seg_b, seg_kvh, seg_len, seg_blk, seg_n;
    bool whole, at_start;

    template <class A>
    __device__ void begin(const A &a, int b_, int rest, int left_) {
        b = b_;
        left = left_;
        first = true;
        if (left > 0) {
            nblk = blocks_of<BK>(a, b);
            len = a.lens[b];
            kvh = rest / nblk;
            blk = rest % nblk;
        }
    }
    // The next segment.
    template <class A>
    __device__ bool next(const A &a) {
        if (left <= 0) return false;
        while (blk >= nblk) {  // the next unit that has blocks
            blk = 0;
            if (++kvh == a.hkv) {
                kvh = 0;
                ++b;
                nblk = blocks_of<BK>(a, b);
                len = a.lens[b];
            }
        }
        seg_n = min(nblk - blk, left);
        whole = seg_n == nblk;
        at_start = first;
        seg_b = b;
        seg_kvh = kvh;
        seg_len = len;
        seg_blk = blk;
        first = false;
        left -= seg_n;
        blk += seg_n;
        return true;
    }
};

// tcgen05.mma and commit by one elected thread of a warp that runs in step.
__device__ inline void umma(uint32_t tmem_d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|q, 0xffffffff;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc));
}
__device__ inline void umma_ta(uint32_t tmem_d, uint32_t tmem_a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|q, 0xffffffff;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(tmem_d),
        "r"(tmem_a), "l"(b), "r"(idesc), "r"(acc));
}
__device__ inline void umma_commit(uint64_t *bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar))
        : "memory");
}

// Two values in one packed instruction, each rounded as its scalar form.
__device__ inline void fma2(float &d0, float &d1, float a0, float a1, float b, float c) {
    asm("{\n\t.reg .b64 ra, rb, rc;\n\t"
        "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %4};\n\tmov.b64 rc, {%5, %5};\n\t"
        "fma.rn.f32x2 ra, ra, rb, rc;\n\tmov.b64 {%0, %1}, ra;\n\t}"
        : "=f"(d0), "=f"(d1)
        : "f"(a0), "f"(a1), "f"(b), "f"(c));
}
__device__ inline void add2(float &d0, float &d1, float a0, float a1) {
    asm("{\n\t.reg .b64 ra, rd;\n\t"
        "mov.b64 ra, {%2, %3};\n\tmov.b64 rd, {%0, %1};\n\t"
        "add.rn.f32x2 rd, rd, ra;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "+f"(d0), "+f"(d1)
        : "f"(a0), "f"(a1));
}
__device__ inline float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
// max of N values: four chains of three-input maxima (exact in any order)
template <int N>
__device__ inline float max_of(const float (&v)[N]) {
    float m[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
    for (int i = 4; i < N; i += 8)
#pragma unroll
        for (int k = 0; k < 4; ++k) m[k] = i + 4 + k < N ? max3(m[k], v[i + k], v[i + 4 + k]) : fmaxf(m[k], v[i + k]);
    return fmaxf(max3(m[0], m[1], m[2]), m[3]);
}

// Which of two bf16 values are infinite or NaN (the exponent all ones: 1 more
// carries into the sign's place): bits 15 and 31.
__device__ inline uint32_t non_finite(uint32_t w) { return ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u; }
// 16 bytes of bf16 without them (set to 0); whether there were any.
__device__ inline bool clear_non_finite(uint4 &u) {
    if (!(non_finite(u.x) | non_finite(u.y) | non_finite(u.z) | non_finite(u.w))) return false;
    uint32_t *w = reinterpret_cast<uint32_t *>(&u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t f = non_finite(w[i]);
        if (f & 0x8000u) w[i] &= 0xffff0000u;
        if (f & 0x80000000u) w[i] &= 0x0000ffffu;
    }
    return true;
}

// Row rg's bits of the block of keys [key0, key0 + 64): which of them count.
__device__ inline unsigned long long seen_bits(unsigned long long mask, int key0, int base) {
    const int sh = key0 - base;  // place in the tree of the first key
    if (sh <= -64) return ~0ull;
    if (sh < 0) return (mask << -sh) | ((1ull << -sh) - 1);
    return sh >= 64 ? 0ull : mask >> sh;
}

template <int D, int QT>
__device__ __forceinline__ void tree_cta(const Args &a, uint8_t *smem) {
    using C = Cfg<D, QT>;
    constexpr int BK = C::BK, PG = C::PG;
    if (smem_u32(smem) & 1023u) {  // (the swizzled tiles start on 1024-byte boundaries: the array is declared so)
        if (threadIdx.x == 0) report(a.status, VC_ERR_UNSUPPORTED);
        return;
    }
    uint8_t *sq = smem;
    uint64_t *q_ready = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);  // [QT]
    uint64_t *s_ready = q_ready + QT, *p_ready = s_ready + C::NS, *o_done = p_ready + C::NBUF, *pv_done = o_done + QT;
    uint64_t *full = pv_done + QT, *empty = full + C::SLOTS, *tail = empty + C::SLOTS;
    uint64_t *idle = tail + 1;
    unsigned long long *bad = reinterpret_cast<unsigned long long *>(smem + C::OFF_MISC);  // [kBadRing]
    uint32_t *tslot = reinterpret_cast<uint32_t *>(bad + kBadRing);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int grp_id = blockIdx.x / a.lanes, glane = blockIdx.x % a.lanes;
    const int tile0 = QT * glane;  // this CTA's tiles: QT from there

    uint8_t *skv = smem + C::OFF_KV;

    // ---- set-up ----
    if (tid == 0) {
        for (int t = 0; t < QT; ++t) {
            mbar_init(&q_ready[t], 4);
            mbar_init(&o_done[t], 1);
            mbar_init(&pv_done[t], 1);
        }
        for (int i = 0; i < C::NS; ++i) mbar_init(&s_ready[i], 1);
        for (int i = 0; i < C::NBUF; ++i) mbar_init(&p_ready[i], 4);
        for (int i = 0; i < C::SLOTS; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        mbar_init(tail, 1);
        mbar_init(idle, 1);
        fence_mbar_init();
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tslot)),
                     "r"(C::TMEM_COLS));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    vtc::tc_fence_before();
    // this group's range, by every warp for itself
    int total, before, b0 = 0, rest = 0;
    sum_blocks<BK>(a, 0, lane, total, before);
    const Deal deal(total * a.hkv, a.groups);
    const int f0 = deal.start(grp_id), mine = deal.start(grp_id + 1) - f0;
    if (mine > 0) find_block<BK>(a, f0, lane, b0, rest);
    Walk<BK> w;
    w.begin(a, b0, rest, mine);
    __syncthreads();
    vtc::tc_fence_after();
    const uint32_t tmem = *tslot;

    constexpr uint32_t IQK = vtc::idesc_bf16(128, BK, false);
    constexpr uint32_t IPV = vtc::idesc_bf16(128, D, true);
    bool alive = true;

    if (warp == C::SM_WARPS) {
        // ================= producer =================
        if constexpr (QT > 1) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::REGS_OTHER));
        if (!block_skips(a.skip_copies)) {
            uint32_t seq = 0;   // copies into the ring so far
            int seg = 0;
            uint32_t tails = 0;
            // V blocks of the tree that are under way, oldest first
            struct Pend { int slot, key0, len, seg; } pend{};
            bool pending = false;
            int lost = -1;  // slot of a tree block whose copy did not arrive in time
            // wait for the pending V block, clear what must not be read, hand it on
            auto flush = [&]() {
                if (!pending) return;
                pending = false;
                alive = __all_sync(0xffffffffu, mbar_wait(tail, tails & 1, a.status, a.wait_ns));
                ++tails;
                if (!alive) {
                    lost = pend.slot;
                    return;
                }
                const int base = pend.len - a.n_q;
                uint8_t *vt = skv + pend.slot * C::SLOT;
                unsigned long long found = 0;
                const int r0 = max(0, base - pend.key0);
                for (int e = lane; e < (BK - r0) * (D / 8); e += 32) {
                    const int r = r0 + e / (D / 8), c = e % (D / 8);
                    uint4 *p = reinterpret_cast<uint4 *>(vt + vtc::sw128(r, c, BK));
                    const int node = pend.key0 + r - base;
                    if (node >= a.n_q) {
                        *p = make_uint4(0, 0, 0, 0);
                    } else {
                        uint4 u = *p;
                        if (clear_non_finite(u)) {
                            found |= 1ull << node;
                            *p = u;
                        }
                    }
                }
                if (found) atomicOr(&bad[pend.seg % kBadRing], found);
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive(&full[pend.slot]);
            };
            while (alive && w.next(a)) {
                const int32_t *trow = a.table + (int64_t)w.seg_b * a.maxb;
                const int npages = ceil_div(w.seg_len, kPage);
                if (lane == 0) bad[seg % kBadRing] = 0;
                __syncwarp();
                // page ids, 32 at a time, one batch ahead (pages behind the
                // request's end: any valid page, masked and cleared)
                constexpr int NB = 32 / PG;
                auto load_ids = [&](int i0) {
                    const int i = i0 + lane / PG;
                    int id = 0;
                    if (i < w.seg_n) {
                        const int pidx = (w.seg_blk + i) * PG + lane % PG;
                        if (pidx < npages) {
                            id = pidx < a.maxb ? trow[pidx] : -1;
                            if (id < 0 || id >= a.n_pages) {
                                report(a.status, VC_ERR_BAD_INDEX);
                                id = 0;
                            }
                        }
                    }
                    return id;
                };
                // copies of this lane: page lane / NC, column lane % NC
                const int off = (lane % C::NC) * (BK * 128) + (lane / C::NC) * (kPage * 128);
                auto copy = [&](int i, int ids, const CUtensorMap *map, bool is_v) {
                    const int id = __shfl_sync(0xffffffffu, ids, (i % NB) * PG + (lane / C::NC) % PG);
                    const int y = (id * a.hkv + w.seg_kvh) * kPage;
                    const int key0 = (w.seg_blk + i) * BK;
                    const int slot = seq % C::SLOTS;
                    const uint32_t use = seq / C::SLOTS;
                    if (use > 0 && !__all_sync(0xffffffffu, mbar_try_wait(&empty[slot], (use - 1) & 1))) {
                        // (the ring cannot drain past a V block that was not handed on)
                        flush();
                        alive = alive &&
                                __all_sync(0xffffffffu, mbar_wait(&empty[slot], (use - 1) & 1, a.status, a.wait_ns));
                    }
                    const bool clean = is_v && key0 + BK > w.seg_len - a.n_q;
                    if (clean) flush();  // one at a time
                    if (!alive) return;
                    uint64_t *bar = clean ? tail : &full[slot];
                    if (lane == 0) mbar_arrive_expect_tx(bar, C::SLOT);
                    __syncwarp();
                    if (lane < PG * C::NC) vtc::tma2d(skv + slot * C::SLOT + off, map, (lane % C::NC) * 64, y, bar);
                    if (clean) {
                        pend = {slot, key0, w.seg_len, seg};
                        pending = true;
                    }
                    ++seq;
                };
                int cur = 0, nxt = load_ids(0);
                for (int i = 0; i < w.seg_n && alive; ++i) {
                    if (i % NB == 0) {
                        cur = nxt;
                        nxt = load_ids(i + NB);
                    }
                    copy(i, cur, &a.kmap, false);
                    if (alive) copy(i, cur, &a.vmap, true);
                    // the last segment's end, now that its copy has had the time of
                    // this one's first
                    if (pending && pend.seg != seg) flush();
                }
                ++seg;
            }
            flush();
            // no copy may be under way when the CTA ends (however short the limit of
            // the waits before)
            for (uint32_t q = seq > C::SLOTS ? seq - C::SLOTS : 0; q < seq; ++q)
                if ((int)(q % C::SLOTS) != lost && !mbar_wait(&full[q % C::SLOTS], (q / C::SLOTS) & 1, a.status, kWaitNs))
                    break;
            if (lost >= 0) mbar_wait(tail, (tails - 1) & 1, a.status, kWaitNs);
        }
    } else if (warp == C::SM_WARPS + 1) {
        // ================= MMA issue (the warp in step, one elected thread) =================
        if constexpr (QT > 1) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::REGS_OTHER));
        // (a descriptor's address field counts 16 bytes: steps are added to it)
        const uint64_t qd0 = vtc::sdesc(smem_u32(sq), 16, 1024);
        const uint64_t kd0 = vtc::sdesc(smem_u32(skv), 16, 1024), vd0 = vtc::sdesc(smem_u32(skv), BK * 128, 1024);
        auto issue_s = [&](int t, uint32_t buf, uint32_t slot) {
            const uint64_t kd = kd0 + slot * (C::SLOT / 16), qd = qd0 + t * (C::QTILE / 16);
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
                const uint64_t ko = ((ks >> 2) * (BK * 128) + (ks & 3) * 32) / 16;
                if constexpr (C::QTM)
                    umma_ta(tmem + buf * BK, tmem + C::Q_COL0 + ks * 8, kd + ko, IQK, ks > 0);
                else
                    umma(tmem + buf * BK, qd + ((ks >> 2) * (kTileRows * 128) + (ks & 3) * 32) / 16, kd + ko, IQK, ks > 0);
            }
            umma_commit(&s_ready[C::NBUF < QT ? t : buf]);
        };
        auto issue_pv = [&](int t, uint32_t buf, uint32_t slot, bool add) {
            const uint64_t vd = vd0 + slot * (C::SLOT / 16);
#pragma unroll
            for (int kk = 0; kk < BK / 16; ++kk)
                umma_ta(tmem + C::O_COL0 + t * D, tmem + buf * BK + kk * 8, vd + kk * 16 * 128 / 16, IPV, add || kk > 0);
        };
        // places in the ring (K and V of a block lie side by side, so each steps by
        // two) and among the S buffers, with the parity of the phase waited for there
        struct Place {
            uint32_t i, par;
            __device__ void step(uint32_t by, uint32_t of) {
                if ((i += by) >= of) {
                    i -= of;
                    par ^= 1;
                }
            }
        } kp{0, 0}, vp{1, 0}, pp{0, 0};
        uint32_t sb = 0, seg = 0;
        // What a step needs before its P V and the S ahead of it: its P, its V, that
        // S's K and Q.  All first: a wait between P V and S lets the tensor core run
        // dry (256 rows at 131072 keys: 453 instead of 421 us).
        auto wait1 = [&](uint64_t *bar, uint32_t par) {
            alive = __all_sync(0xffffffffu, mbar_wait(bar, par, a.status, a.wait_ns));
            return alive;
        };
        auto wait = [&](bool p, bool v, bool k, int q) {
            if (p && !wait1(&p_ready[pp.i], pp.par)) return false;
            if (v && !wait1(&full[vp.i], vp.par)) return false;
            if (k && !wait1(&full[kp.i], kp.par)) return false;
            if (q >= 0 && !wait1(&q_ready[q], seg & 1)) return false;
            vtc::tc_fence_after();
            return true;
        };
        // S of the next step, which is one of tile t
        auto next_s = [&](int t) {
            issue_s(t, sb, kp.i);
            if (++sb == C::NBUF) sb = 0;
            if (t == QT - 1) {
                umma_commit(&empty[kp.i]);
                kp.step(2, C::SLOTS);
            }
        };
        for (;; ++seg) {
            // (by shuffle, so that the compiler knows it, and with it the loops' state,
            // to be uniform: what the tensor core's instructions take is then not
            // moved there one by one; 64-key blocks, 256 rows: 450 instead of 632 us)
            const bool any = alive && w.next(a);
            const int n = __shfl_sync(0xffffffffu, any ? w.seg_n : 0, 0);
            if (n == 0) break;
#pragma unroll
            for (int i = 0; i < C::NBUF; ++i) {
                if (i / QT >= n) break;
                if (!wait(false, false, i % QT == 0, i < QT ? i : -1)) break;
                next_s(i % QT);
            }
            for (int j = 0; j < n && alive; ++j) {
#pragma unroll
                for (int t = 0; t < QT; ++t) {
                    const int t2 = (t + C::NBUF) % QT;  // tile of the step that is NBUF ahead
                    const bool more = j + (t + C::NBUF) / QT < n;
                    if (!wait(true, t == 0, more && t2 == 0, t + C::NBUF < QT && j == 0 ? t2 : -1)) break;
                    issue_pv(t, pp.i, vp.i, j > 0);
                    pp.step(1, C::NBUF);
                    if (C::AHEAD) umma_commit(&pv_done[t]);
                    if (more) next_s(t2);
                    if (j + 1 == n) umma_commit(&o_done[t]);
                }
                if (!alive) break;
                umma_commit(&empty[vp.i]);
                vp.step(2, C::SLOTS);
            }
        }
        // nor may a product be: TMEM is freed behind it
        umma_commit(idle);
        mbar_wait(idle, 0, a.status, kWaitNs);
    } else if (QT > 1 && warp >= C::SM_WARPS) {
        // (idle warps of that warpgroup)
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::REGS_OTHER));
    } else {
        // ================= softmax: one thread per row =================
        if constexpr (QT > 1) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::REGS_SOFTMAX));
        const int t = warp >> 2;
        const int r = (warp & 3) * 32 + lane;  // row within the tile = TMEM lane
        const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t t_o = tmem + lane_base + C::O_COL0 + t * D;
        const int rg = (tile0 + t) * kTileRows + r;
        const bool rvalid = rg < a.rows;
        const int qi = rvalid ? rg / a.grp : 0, qn = rvalid ? rg % a.grp : 0;
        // the warp's 32 rows x 8 pieces of 16 bytes, on their way between a
        // thread's own row and eight neighbouring lanes a row (whole lines of
        // global memory; a thread by itself would touch 32 of them at a time)
        uint4 *stage = reinterpret_cast<uint4 *>(C::QTM ? smem + C::OFF_STAGE + warp * 4096
                                                        : sq + t * C::QTILE + (warp & 3) * 4096);
        const int srow = lane >> 3, spc = lane & 7;  // row (of 4 at a time) and piece
        auto at = [&](int row, int piece) { return stage + row * 8 + (piece ^ (row & 7)); };
        uint32_t it = 0, seg = 0;  // blocks and segments of this chain
        for (; w.next(a); ++seg) {
            const int base = w.seg_len - a.n_q;
            const int64_t orow = ((int64_t)w.seg_b * a.n_q + qi) * a.hq + (int64_t)w.seg_kvh * a.grp + qn;
            unsigned long long mask = 0;
            if (alive) {
                if (rvalid) mask = a.mask[(int64_t)w.seg_b * a.n_q + qi] & (~0ull >> (64 - a.n_q));
                // the warp's rows of Q, 64 channels at a time
                uint4 u[D / 64][8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int64_t ro = __shfl_sync(0xffffffffu, rvalid ? orow : (int64_t)-1, i * 4 + srow);
                    const uint4 *src = reinterpret_cast<const uint4 *>(a.q + ro * D) + spc;
#pragma unroll
                    for (int h = 0; h < D / 64; ++h) u[h][i] = ro >= 0 ? src[h * 8] : make_uint4(0, 0, 0, 0);
                }
#pragma unroll
                for (int h = 0; h < D / 64; ++h) {
                    if constexpr (C::QTM) {  // to TMEM, bf16 pairs
#pragma unroll
                        for (int i = 0; i < 8; ++i) *at(i * 4 + srow, spc) = u[h][i];
                        __syncwarp();
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            float v[16];
#pragma unroll
                            for (int j = 0; j < 4; ++j) *reinterpret_cast<uint4 *>(v + 4 * j) = *at(lane, c * 4 + j);
                            vtc::tmem_st16_nowait(tmem + lane_base + C::Q_COL0 + h * 32 + c * 16, v);
                        }
                        __syncwarp();
                    } else {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            *reinterpret_cast<uint4 *>(
                                sq + t * C::QTILE + vtc::sw128((warp & 3) * 32 + i * 4 + srow, h * 8 + spc, kTileRows)) = u[h][i];
                    }
                }
                if constexpr (C::QTM)
                    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                else
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                vtc::tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&q_ready[t]);
            }
            float m_used = -INFINITY, l = 0.0f;
            // tcgen05.ld / st are warp-collective: every lane runs them together
            for (int j = 0; j < w.seg_n && alive; ++j, ++it) {
                const uint32_t step = it * QT + t, buf = step % C::NBUF, t_s = tmem + lane_base + buf * BK;
                alive = __all_sync(0xffffffffu, mbar_wait(&s_ready[C::NBUF < QT ? t : buf], (C::NBUF < QT ? it : step / C::NBUF) & 1, a.status,
                                                             a.wait_ns));
                if (!alive) break;
                vtc::tc_fence_after();
                float s[BK];
#pragma unroll
                for (int h = 0; h < BK / 64; ++h)
                    vtc::tmem_ld_row<64>(t_s + 64 * h, *reinterpret_cast<float(*)[64]>(&s[64 * h]));
                const int key0 = (w.seg_blk + j) * BK;
                if (key0 + BK > base) {
#pragma unroll
                    for (int h = 0; h < BK / 64; ++h) {
                        const unsigned long long seen = seen_bits(mask, key0 + 64 * h, base);
#pragma unroll
                        for (int c = 0; c < 64; ++c)
                            if (!((seen >> c) & 1)) s[64 * h + c] = -INFINITY;
                    }
                }
                const float mb = max_of<BK>(s) * a.scale_log2;
                // the reference maximum follows only rises of more than 2^8
                // (rare after the first block): then O is rescaled
                const bool grow = mb > m_used + 8.0f;
                if (__any_sync(0xffffffffu, grow) && j > 0) {
                    if constexpr (C::AHEAD) {
                        alive = __all_sync(0xffffffffu, mbar_wait(&pv_done[t], (it - 1) & 1, a.status, a.wait_ns));
                        if (!alive) break;
                        vtc::tc_fence_after();
                    }
                    const float f = grow ? (m_used == -INFINITY ? 0.0f : ex2(m_used - mb)) : 1.0f;
#pragma unroll 1
                    for (int c0 = 0; c0 < D; c0 += 16) {
                        float v[16];
                        vtc::tmem_ld16(t_o + c0, v);
#pragma unroll
                        for (int i = 0; i < 16; ++i) v[i] *= f;
                        vtc::tmem_st16(t_o + c0, v);
                    }
                    l *= f;
                }
                if (grow) m_used = mb;
                const float nms = m_used == -INFINITY ? 0.0f : -m_used;
                float ls[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int h = 0; h < BK / 32; ++h) {
                    float pk[16];
#pragma unroll
                    for (int c = 0; c < 16; ++c) {
                        float p0, p1;
                        fma2(p0, p1, s[h * 32 + 2 * c], s[h * 32 + 2 * c + 1], a.scale_log2, nms);
                        p0 = ex2(p0);
                        p1 = ex2(p1);
                        add2(ls[(2 * c) & 2], ls[((2 * c) & 2) + 1], p0, p1);
                        pk[c] = __uint_as_float(pack_bf16(p0, p1));
                    }
                    vtc::tmem_st16_nowait(t_s + h * 16, pk);
                }
                asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                vtc::tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_ready[buf]);
                l += (ls[0] + ls[1]) + (ls[2] + ls[3]);
            }
            if (alive)
                alive = __all_sync(0xffffffffu, mbar_wait(&o_done[t], seg & 1, a.status, a.wait_ns));
            // ---- the segment's result ----
            if (alive) {
                vtc::tc_fence_after();
                if (mask & *(volatile unsigned long long *)&bad[seg % kBadRing]) l = __int_as_float(0x7fffffff);
            } else {
                m_used = -INFINITY;
                l = 0.0f;
            }
            // a row that is left out or saw no key: zeros (m = -infinity); one
            // that met a NaN: NaN (m = +infinity, which no other range outweighs);
            // one whose keys did not all come in time: zeros, and l = -1, which
            // makes zeros of what it is joined with
            const bool zero = mask == 0 || (m_used == -INFINITY && l == 0.0f);
            const int64_t prow = ((int64_t)blockIdx.x * 2 + !w.at_start) * C::ROWS + t * kTileRows + r;
            const float f = zero ? 0.0f : w.whole ? 1.0f / l : 1.0f;
            const int64_t drow = !rvalid ? -1 : w.whole ? orow : prow;  // the row's place
            const bool half = w.whole && a.out_bf16;
            uint8_t *base8 = static_cast<uint8_t *>(w.whole ? a.out : a.ws_o);
            int64_t to[8];  // the rows that this lane writes a piece of
#pragma unroll
            for (int i = 0; i < 8; ++i) to[i] = __shfl_sync(0xffffffffu, drow, i * 4 + srow);
            // 128 bytes of every row at a time, all eight pieces under way together
            auto put = [&](int part, int parts) {
                __syncwarp();
                uint4 u[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) u[i] = *at(i * 4 + srow, spc);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (to[i] >= 0) *reinterpret_cast<uint4 *>(base8 + (to[i] * parts + part) * 128 + spc * 16) = u[i];
                __syncwarp();
            };
#pragma unroll 1
            for (int c0 = 0; c0 < D; c0 += 32) {
                float v[32];
                if (alive) vtc::tmem_ld_row<32>(t_o + c0, v);
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = zero ? 0.0f : v[i] * f;
                if (half) {
                    const int j0 = (c0 / 32 & 1) * 4;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        *at(lane, j0 + j) = make_uint4(pack_bf16(v[8 * j], v[8 * j + 1]), pack_bf16(v[8 * j + 2], v[8 * j + 3]),
                                                       pack_bf16(v[8 * j + 4], v[8 * j + 5]), pack_bf16(v[8 * j + 6], v[8 * j + 7]));
                    if (j0) put(c0 / 64, D / 64);
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) *at(lane, j) = *reinterpret_cast<uint4 *>(v + 4 * j);
                    put(c0 / 32, D / 32);
                }
            }
            if (rvalid && !w.whole) {
                a.ws_ml[prow * 2] = zero ? -INFINITY : l != l ? INFINITY : m_used;
                a.ws_ml[prow * 2 + 1] = !alive ? -1.0f : zero ? 0.0f : l;
            }
            vtc::tc_fence_before();
        }
        pdl_trigger();
    }
    vtc::tc_fence_before();
    __syncthreads();
    vtc::tc_fence_after();
    if (warp == 0)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::TMEM_COLS));
}

// Join the partials of units that span several ranges, and write zeros for
// requests that are refused.  One block per (unit, kJoinWarps / W rows): W warps
// share a row and take every W-th range each (a running maximum and sum, eight
// partials read at once), in an order that the lengths alone fix.
constexpr int kJoinWarps = 8;
template <int D, int QT>
__device__ __forceinline__ void tree_join_block(const Args &a, int W) {
    using C = Cfg<D, QT>;
    constexpr int BK = C::BK, E = D / 32, U = 8;
    __shared__ float part[kJoinWarps][E + 2][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int unit = blockIdx.x, b = unit / a.hkv, kvh = unit % a.hkv;
    const int nblk = blocks_of<BK>(a, b);
    if (nblk == 0 && threadIdx.x == 0 && kvh == 0 && blockIdx.y == 0) report(a.status, VC_ERR_BAD_INDEX);
    int total, before;
    sum_blocks<BK>(a, b, lane, total, before);
    const Deal deal(total * a.hkv, a.groups);
    const int u0 = before * a.hkv + kvh * nblk;
    // groups whose ranges hold the unit's first and last block
    const int g0 = nblk > 0 ? deal.group_of(u0) : 0, g1 = nblk > 0 ? deal.group_of(u0 + nblk - 1) : -1;
    if (nblk > 0 && g0 == g1) return;  // finished there
    const int rg = blockIdx.y * (kJoinWarps / W) + warp / W;
    const bool row_ok = rg < a.rows;
    const int cta = rg / C::ROWS, trow = rg % C::ROWS;
    float M = -INFINITY, L = 0.0f, acc[E];
    bool lost = false;  // a partial that did not come in time is among them
#pragma unroll
    for (int i = 0; i < E; ++i) acc[i] = 0.0f;
    if (row_ok) {
        for (int gb = g0 + warp % W; gb <= g1; gb += U * W) {
            float m[U], l[U], o[U][E];
#pragma unroll
            for (int k = 0; k < U; ++k) {
                const int g = gb + k * W;
                m[k] = -INFINITY;
                l[k] = 0.0f;
#pragma unroll
                for (int i = 0; i < E; ++i) o[k][i] = 0.0f;
                if (g <= g1) {
                    // (ranges between the first and the last are never empty)
                    const int64_t pr = ((int64_t)(g * a.lanes + cta) * 2 + (u0 > deal.start(g))) * C::ROWS + trow;
                    const float2 ml = *reinterpret_cast<const float2 *>(a.ws_ml + pr * 2);
                    m[k] = ml.x;
                    l[k] = ml.y;
                    const float *src = a.ws_o + pr * D + lane * E;
                    if constexpr (E == 4) {
                        const float4 q = *reinterpret_cast<const float4 *>(src);
                        o[k][0] = q.x; o[k][1] = q.y; o[k][2] = q.z; o[k][3] = q.w;
                    } else {
                        const float2 q = *reinterpret_cast<const float2 *>(src);
                        o[k][0] = q.x; o[k][1] = q.y;
                    }
                }
            }
            float mx = M;
#pragma unroll
            for (int k = 0; k < U; ++k) {
                mx = fmaxf(mx, m[k]);
                lost |= l[k] < 0.0f;
            }
            if (mx == -INFINITY) continue;
            const float f = ex2(M - mx);
            M = mx;
            L *= f;
#pragma unroll
            for (int i = 0; i < E; ++i) acc[i] *= f;
#pragma unroll
            for (int k = 0; k < U; ++k) {
                if (m[k] == -INFINITY) continue;  // (such a partial's sums are not to be used)
                const float wk = ex2(m[k] - mx);
                L = fmaf(wk, l[k], L);
#pragma unroll
                for (int i = 0; i < E; ++i) acc[i] = fmaf(wk, o[k][i], acc[i]);
            }
        }
    }
    if (W > 1) {
        part[warp][0][lane] = M;
        part[warp][1][lane] = lost ? -1.0f : L;
#pragma unroll
        for (int i = 0; i < E; ++i) part[warp][2 + i][lane] = acc[i];
        __syncthreads();
        if (warp % W) return;
        for (int k = 1; k < W; ++k) {
            const float m = part[warp + k][0][lane], mx = fmaxf(M, m);
            lost |= part[warp + k][1][lane] < 0.0f;
            if (m == -INFINITY) continue;
            const float f = ex2(M - mx), wk = ex2(m - mx);
            M = mx;
            L = L * f + part[warp + k][1][lane] * wk;
#pragma unroll
            for (int i = 0; i < E; ++i) acc[i] = acc[i] * f + part[warp + k][2 + i][lane] * wk;
        }
    }
    if (!row_ok) return;
    const int64_t orow = ((int64_t)b * a.n_q + rg / a.grp) * a.hq + (int64_t)kvh * a.grp + rg % a.grp;
    const bool zero = lost || M == -INFINITY;
    const float f = zero ? 0.0f : 1.0f / L;
#pragma unroll
    for (int i = 0; i < E; ++i) acc[i] = zero ? 0.0f : acc[i] * f;
    if (a.out_bf16) {
        uint32_t *dst = reinterpret_cast<uint32_t *>((uint16_t *)a.out + orow * D + lane * E);
#pragma unroll
        for (int i = 0; i < E / 2; ++i) dst[i] = pack_bf16(acc[2 * i], acc[2 * i + 1]);
    } else {
#pragma unroll
        for (int i = 0; i < E; ++i) ((float *)a.out)[orow * D + lane * E + i] = acc[i];
    }
}

}  // namespace tree
}  // namespace vc
