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
// More: CTAs of two tiles, one to an SM, whose tiles take turns on the tensor
// core.  Four tiles: groups of two CTAs, two tiles each, on the same range in
// step, so the second CTA finds K and V in L2.  Three tiles: groups of three
// CTAs -- two share tiles 0 and 1 and take every other block, the third has
// tile 2 and all blocks -- which keeps the three in step.
//
// A CTA: a producer warp that fills a ring of K and V blocks by TMA (one
// 16-row x 64-channel box per page and 128-byte column), one thread that
// issues the tcgen05.mma of all tiles in the order  P V (j), S (j + 1)  tile
// by tile, and four softmax warps per tile (a thread owns a row = TMEM lane).
// P (bf16) overwrites the S it came from.  S (j + 1) is issued behind P V (j),
// so a finished S also says that O is at rest and may be rescaled.
//
// The tree's own entries.  In blocks that reach into the tree a row's bits
// pick the scores that count.  A V row that some nodes do not see must not
// reach them as 0 * infinity: the producer warp clears non-finite values from
// the tree's V rows (and all of the rows behind the request) once such a block
// has arrived, before it is handed on, and notes the nodes; rows that do see
// one of those end as NaN.
//
// Every wait is bounded; a timeout is reported and the CTA drains.
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
    int lanes;   // CTAs per group
    int tiles;   // 128-row tiles of a unit
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
    static constexpr int NC = D / 64;           // 128-byte columns of a row
    static constexpr int BK = QT == 1 ? 64 : 128;
    static constexpr bool QTM = QT == 1;        // Q in TMEM beside S and O (else in shared memory)
    static constexpr int QTILE = kTileRows * D * 2;
    static constexpr int SLOT = BK * D * 2;     // one block of K or of V
    static constexpr int OFF_KV = QTM ? 0 : QT * QTILE;
    static constexpr int FIT = ((QT == 1 ? 100 : 225) * 1024 - OFF_KV) / SLOT;
    static constexpr int SLOTS = FIT < 12 ? FIT : 12;
    static_assert(SLOTS >= 4 && SLOTS / 2 + 2 <= kBadRing, "ring depth");
    static constexpr int OFF_BAR = OFF_KV + SLOTS * SLOT;
    static constexpr int NBAR = 4 * QT + 2 * SLOTS + 1;  // q, s, p, o per tile; full, empty; tail
    static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
    static constexpr int SMEM = OFF_MISC + kBadRing * 8 + 64 * 4 + 1024;
    static constexpr int O_COL0 = QT * BK;
    static constexpr int Q_COL0 = O_COL0 + QT * D;
    static constexpr int TMEM_USED = Q_COL0 + (QTM ? D / 2 : 0);
    static constexpr int TMEM_COLS = TMEM_USED <= 256 ? 256 : 512;
    static_assert(TMEM_USED <= (QT == 1 ? 256 : 512), "TMEM columns");
    static constexpr int WARPS = QT * 4 + 2;
    static constexpr int THREADS = WARPS * 32;
    static constexpr int MIN_CTAS = QT == 1 ? 2 : 1;
    static constexpr int ROWS = QT * kTileRows;
};

// Blocks of a request's context: 0 for one that is refused.
template <int BK>
__device__ inline int blocks_of(const Args &a, int b) {
    const int len = a.lens[b];
    return len >= a.n_q && len <= a.max_len ? ceil_div(len, BK) : 0;
}

// Sums over the batch in one go: the blocks of all requests and those of the
// requests before b_until; a thread takes a run of `per` requests, and `mine`
// / `before` are its run's blocks and those before its run.
struct Sums {
    int64_t total, before, mine;
    int b0, b1;
};
template <int BK>
__device__ inline Sums sum_blocks(const Args &a, int64_t *sh, int tid, int nthreads) {
    Sums s;
    const int per = ceil_div(a.batch, nthreads), lane = tid & 31, warp = tid >> 5;
    s.b0 = min(a.batch, tid * per);
    s.b1 = min(a.batch, s.b0 + per);
    s.mine = 0;
    for (int b = s.b0; b < s.b1; ++b) s.mine += blocks_of<BK>(a, b);
    int64_t inc = s.mine;
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
    }
    if (lane == 31) sh[warp] = inc;
    __syncthreads();
    s.before = inc - s.mine;
    s.total = 0;
    for (int w = 0; w < nthreads / 32; ++w) {
        if (w < warp) s.before += sh[w];
        s.total += sh[w];
    }
    return s;
}

// The range of group g among G: blocks [g T / G, (g + 1) T / G) of T.
__host__ __device__ inline int64_t range_start(int64_t total, int g, int groups) { return total * g / groups; }

// Which blocks of a segment [b0, b0 + n) a CTA of lane `lane` takes: every
// `step`-th from `first`, `count` of them.  whole: the segment is the unit.
struct Share {
    int first, step, count;
};
__device__ inline Share share_of(int lanes, int lane, int64_t unit, int b0, int n, bool whole) {
    if (lanes < 3 || lane == 2) return {b0, 1, n};
    if (whole) return {b0, 1, (int)(unit & 1) == lane ? n : 0};
    const int first = b0 + ((b0 ^ lane) & 1), end = b0 + n;
    return {first, 2, first < end ? (end - first + 1) / 2 : 0};
}

// A group's walk through its range.
template <int BK>
struct Walk {
    int b, kvh, blk, nblk, len;
    int64_t left;
    bool first;
    // the current segment
    int seg_b, seg_kvh, seg_len, seg_blk;
    Share sh;
    bool whole, at_start;

    __device__ void begin(const Args &a, int b_, int kvh_, int blk_, int64_t left_) {
        b = b_;
        kvh = kvh_;
        blk = blk_;
        left = left_;
        first = true;
        if (left > 0) {
            nblk = blocks_of<BK>(a, b);
            len = a.lens[b];
        }
    }
    // The next segment in which this CTA has blocks.
    __device__ bool next(const Args &a, int lane) {
        while (left > 0) {
            while (blk >= nblk) {  // the next unit that has blocks
                blk = 0;
                if (++kvh == a.hkv) {
                    kvh = 0;
                    ++b;
                    nblk = blocks_of<BK>(a, b);
                    len = a.lens[b];
                }
            }
            const int n = (int)min((int64_t)(nblk - blk), left);
            whole = n == nblk;
            at_start = first;
            sh = share_of(a.lanes, lane, (int64_t)b * a.hkv + kvh, blk, n, whole);
            seg_b = b;
            seg_kvh = kvh;
            seg_len = len;
            seg_blk = blk;
            first = false;
            left -= n;
            blk += n;
            if (sh.count > 0) return true;
        }
        return false;
    }
};

// 128 consecutive columns of this thread's lane: one load, one wait
__device__ inline void tmem_ld128(uint32_t taddr, float (&v)[128]) {
    uint32_t r[128];
#define VC_R8(i) "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3]), "=r"(r[i + 4]), "=r"(r[i + 5]), "=r"(r[i + 6]), "=r"(r[i + 7])
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x128.b32 {"
        "%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,"
        "%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
        "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63,"
        "%64,%65,%66,%67,%68,%69,%70,%71,%72,%73,%74,%75,%76,%77,%78,%79,"
        "%80,%81,%82,%83,%84,%85,%86,%87,%88,%89,%90,%91,%92,%93,%94,%95,"
        "%96,%97,%98,%99,%100,%101,%102,%103,%104,%105,%106,%107,%108,%109,%110,%111,"
        "%112,%113,%114,%115,%116,%117,%118,%119,%120,%121,%122,%123,%124,%125,%126,%127"
        "}, [%128];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : VC_R8(0), VC_R8(8), VC_R8(16), VC_R8(24), VC_R8(32), VC_R8(40), VC_R8(48), VC_R8(56), VC_R8(64), VC_R8(72),
          VC_R8(80), VC_R8(88), VC_R8(96), VC_R8(104), VC_R8(112), VC_R8(120)
        : "r"(taddr)
        : "memory");
#undef VC_R8
#pragma unroll
    for (int i = 0; i < 128; ++i) v[i] = __uint_as_float(r[i]);
}
template <int N>
__device__ inline void tmem_ld_block(uint32_t taddr, float (&v)[N]) {
    if constexpr (N == 128)
        tmem_ld128(taddr, v);
    else
        vtc::tmem_ld_row<N>(taddr, v);
}

// 16 bytes of bf16 without their infinities and NaN (set to 0); whether there were any.
__device__ inline bool clear_non_finite(uint4 &u) {
    bool any = false;
    uint32_t *w = reinterpret_cast<uint32_t *>(&u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if ((w[i] & 0x7f80u) == 0x7f80u) {
            w[i] &= 0xffff0000u;
            any = true;
        }
        if ((w[i] & 0x7f800000u) == 0x7f800000u) {
            w[i] &= 0x0000ffffu;
            any = true;
        }
    }
    return any;
}

// Row rg's bits of the block of keys [key0, key0 + 64): which of them count.
__device__ inline unsigned long long seen_bits(unsigned long long mask, int key0, int base) {
    const int sh = key0 - base;  // place in the tree of the first key
    if (sh <= -64) return ~0ull;
    if (sh < 0) return (mask << -sh) | ((1ull << -sh) - 1);
    return sh >= 64 ? 0ull : mask >> sh;
}

// One row's result: the final value of a finished unit, in out's type.
template <int D>
__device__ inline void store_out16(const Args &a, int64_t orow, int c0, const float (&v)[16], float f, bool zero) {
    float y[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) y[i] = zero ? 0.0f : v[i] * f;
    if (a.out_bf16) {
        uint4 *dst = reinterpret_cast<uint4 *>((uint16_t *)a.out + orow * D + c0);
        dst[0] = make_uint4(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]), pack_bf16(y[4], y[5]), pack_bf16(y[6], y[7]));
        dst[1] = make_uint4(pack_bf16(y[8], y[9]), pack_bf16(y[10], y[11]), pack_bf16(y[12], y[13]),
                            pack_bf16(y[14], y[15]));
    } else {
        float4 *dst = reinterpret_cast<float4 *>((float *)a.out + orow * D + c0);
#pragma unroll
        for (int i = 0; i < 4; ++i) dst[i] = make_float4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
    }
}

template <int D, int QT>
__device__ __forceinline__ void tree_cta(const Args &a, uint8_t *smem_raw) {
    using C = Cfg<D, QT>;
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t *smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);  // 1024-byte aligned
    uint8_t *sq = smem;
    uint8_t *skv = smem + C::OFF_KV;
    uint64_t *q_ready = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);  // [QT]
    uint64_t *s_ready = q_ready + QT, *p_ready = s_ready + QT, *o_done = p_ready + QT;
    uint64_t *full = o_done + QT, *empty = full + C::SLOTS, *tail = empty + C::SLOTS;
    unsigned long long *bad = reinterpret_cast<unsigned long long *>(smem + C::OFF_MISC);  // [kBadRing]
    int32_t *misc = reinterpret_cast<int32_t *>(bad + kBadRing);  // 64 words
    uint32_t *tslot = reinterpret_cast<uint32_t *>(misc);
    int *where = misc + 2;                                        // first request, kv head, block
    int64_t *sums = reinterpret_cast<int64_t *>(misc + 8);        // one per warp

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int grp_id = blockIdx.x / a.lanes, glane = blockIdx.x % a.lanes;
    // this CTA's tiles: all of one tile; or 0, 1 | 2, 3; of three, lane 2 has the last alone
    const int tile0 = QT == 1 ? 0 : a.lanes == 3 ? (glane == 2 ? 2 : 0) : 2 * glane;
    const int nt = QT == 1 ? 1 : a.lanes == 3 && glane == 2 ? 1 : min(QT, a.tiles - tile0);

    // ---- set-up ----
    if (tid == 0) {
        for (int t = 0; t < QT; ++t) {
            mbar_init(&q_ready[t], kTileRows);
            mbar_init(&s_ready[t], 1);
            mbar_init(&p_ready[t], kTileRows);
            mbar_init(&o_done[t], 1);
        }
        for (int i = 0; i < C::SLOTS; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        mbar_init(tail, 1);
        fence_mbar_init();
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tslot)),
                     "r"(C::TMEM_COLS));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    vtc::tc_fence_before();
    const Sums sm = sum_blocks<C::BK>(a, sums, tid, C::THREADS);  // (holds a __syncthreads)
    const int64_t total = sm.total * a.hkv;
    const int64_t f0 = range_start(total, grp_id, a.groups), f1 = range_start(total, grp_id + 1, a.groups);
    if (f0 < f1 && f0 >= sm.before * a.hkv && f0 < (sm.before + sm.mine) * a.hkv) {
        int64_t rem = f0 - sm.before * a.hkv;
        int b = sm.b0, n = blocks_of<C::BK>(a, b);
        while (rem >= (int64_t)n * a.hkv) {
            rem -= (int64_t)n * a.hkv;
            n = blocks_of<C::BK>(a, ++b);
        }
        where[0] = b;
        where[1] = (int)(rem / n);
        where[2] = (int)(rem % n);
    }
    __syncthreads();
    vtc::tc_fence_after();
    const uint32_t tmem = *tslot;
    Walk<C::BK> w;
    w.begin(a, f0 < f1 ? where[0] : 0, f0 < f1 ? where[1] : 0, f0 < f1 ? where[2] : 0, f1 - f0);

    constexpr uint32_t IQK = vtc::idesc_bf16(128, C::BK, false);
    constexpr uint32_t IPV = vtc::idesc_bf16(128, D, true);
    constexpr int PG = C::BK / kPage;  // pages of a block
    bool alive = true;

    if (warp == QT * 4) {
        // ================= producer =================
        if (!a.skip_copies) {
            uint32_t seq = 0;   // copies into the ring so far
            int seg = 0;
            uint32_t tails = 0;
            // V blocks of the tree that are under way, oldest first
            struct Pend { uint32_t seq; int key0, len, seg; } pend{};
            bool pending = false;
            int64_t lost = -1;  // a tree block whose copy did not arrive in time
            // wait for the pending V block, clear what must not be read, hand it on
            auto flush = [&]() {
                if (!pending) return;
                pending = false;
                alive = __all_sync(0xffffffffu, mbar_wait(tail, tails & 1, a.status, a.wait_ns));
                ++tails;
                if (!alive) {
                    lost = pend.seq;
                    return;
                }
                const int slot = pend.seq % C::SLOTS, base = pend.len - a.n_q;
                uint8_t *vt = skv + slot * C::SLOT;
                unsigned long long found = 0;
                const int r0 = max(0, base - pend.key0);
                for (int e = lane; e < (C::BK - r0) * (D / 8); e += 32) {
                    const int r = r0 + e / (D / 8), c = e % (D / 8);
                    uint4 *p = reinterpret_cast<uint4 *>(vt + vtc::sw128(r, c, C::BK));
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
                if (lane == 0) mbar_arrive(&full[slot]);
            };
            while (alive && w.next(a, glane)) {
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
                    if (i < w.sh.count) {
                        const int pidx = (w.sh.first + i * w.sh.step) * PG + lane % PG;
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
                int cur = 0, nxt = load_ids(0);
                for (int i = 0; i < w.sh.count && alive; ++i) {
                    if (i % NB == 0) {
                        cur = nxt;
                        nxt = load_ids(i + NB);
                    }
                    // copies of this lane: page lane / NC, column lane % NC
                    const int id = __shfl_sync(0xffffffffu, cur, (i % NB) * PG + (lane / C::NC) % PG);
                    const int y = (id * a.hkv + w.seg_kvh) * kPage;
                    const int off = (lane % C::NC) * (C::BK * 128) + (lane / C::NC) * (kPage * 128);
                    const int key0 = (w.sh.first + i * w.sh.step) * C::BK;
                    const bool in_tree = key0 + C::BK > w.seg_len - a.n_q;
#pragma unroll
                    for (int kv = 0; kv < 2; ++kv) {
                        const int slot = seq % C::SLOTS;
                        const uint32_t use = seq / C::SLOTS;
                        if (use > 0 && !__all_sync(0xffffffffu, mbar_try_wait(&empty[slot], (use - 1) & 1))) {
                            // (the ring cannot drain past a V block that was not handed on)
                            flush();
                            alive = alive && __all_sync(0xffffffffu, mbar_wait(&empty[slot], (use - 1) & 1, a.status,
                                                                               a.wait_ns));
                        }
                        if (!alive) break;
                        const bool clean = kv == 1 && in_tree;
                        if (clean) flush();  // one at a time
                        if (!alive) break;
                        uint64_t *bar = clean ? tail : &full[slot];
                        if (lane == 0) mbar_arrive_expect_tx(bar, C::SLOT);
                        __syncwarp();
                        if (lane < PG * C::NC)
                            vtc::tma2d(skv + slot * C::SLOT + off, kv ? &a.vmap : &a.kmap, (lane % C::NC) * 64, y, bar);
                        if (clean) {
                            pend = {seq, key0, w.seg_len, seg};
                            pending = true;
                        }
                        ++seq;
                    }
                }
                ++seg;
            }
            flush();
            // no copy may be under way when the CTA ends
            for (uint32_t s = seq > C::SLOTS ? seq - C::SLOTS : 0; s < seq; ++s)
                if ((int64_t)s != lost && !mbar_wait(&full[s % C::SLOTS], (s / C::SLOTS) & 1, a.status, a.wait_ns))
                    break;
        }
    } else if (warp == QT * 4 + 1) {
        // ================= MMA issue (one thread) =================
        if (lane == 0) {
            uint32_t it = 0;
            int seg = 0;
            auto wait = [&](uint64_t *bar, uint32_t parity) {
                alive = alive && mbar_wait(bar, parity, a.status, a.wait_ns);
                vtc::tc_fence_after();
                return alive;
            };
            auto k_seq = [](uint32_t n) { return 2 * n; };
            auto issue_s = [&](uint32_t n, int t) {
                const uint8_t *kt = skv + (k_seq(n) % C::SLOTS) * C::SLOT;
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                    const uint64_t kd = vtc::sdesc(smem_u32(kt) + (ks >> 2) * (C::BK * 128) + (ks & 3) * 32, 16, 1024);
                    if constexpr (C::QTM) {
                        vtc::umma_ta(tmem + t * C::BK, tmem + C::Q_COL0 + ks * 8, kd, IQK, ks > 0);
                    } else {
                        const uint64_t qd = vtc::sdesc(
                            smem_u32(sq + t * C::QTILE) + (ks >> 2) * (kTileRows * 128) + (ks & 3) * 32, 16, 1024);
                        vtc::umma(tmem + t * C::BK, qd, kd, IQK, ks > 0);
                    }
                }
                vtc::umma_commit(&s_ready[t]);
            };
            auto issue_pv = [&](uint32_t n, int t, bool add) {
                const uint8_t *vt = skv + ((k_seq(n) + 1) % C::SLOTS) * C::SLOT;
#pragma unroll
                for (int kk = 0; kk < C::BK / 16; ++kk)
                    vtc::umma_ta(tmem + C::O_COL0 + t * D, tmem + t * C::BK + kk * 8,
                                 vtc::sdesc(smem_u32(vt) + kk * 16 * 128, C::BK * 128, 1024), IPV, add || kk > 0);
            };
            while (alive && w.next(a, glane)) {
                const int n = w.sh.count;
                if (!wait(&full[k_seq(it) % C::SLOTS], (k_seq(it) / C::SLOTS) & 1)) break;
                for (int t = 0; t < nt && alive; ++t)
                    if (wait(&q_ready[t], seg & 1)) issue_s(it, t);
                if (!alive) break;
                vtc::umma_commit(&empty[k_seq(it) % C::SLOTS]);
                for (int j = 0; j < n && alive; ++j, ++it) {
                    const uint32_t vs = k_seq(it) + 1, kn = k_seq(it + 1);
                    const bool more = j + 1 < n;
                    if (!wait(&full[vs % C::SLOTS], (vs / C::SLOTS) & 1)) break;
                    for (int t = 0; t < nt && alive; ++t) {
                        if (!wait(&p_ready[t], it & 1)) break;
                        issue_pv(it, t, j > 0);
                        if (more) {
                            if (t == 0 && !wait(&full[kn % C::SLOTS], (kn / C::SLOTS) & 1)) break;
                            issue_s(it + 1, t);
                        } else {
                            vtc::umma_commit(&o_done[t]);
                        }
                    }
                    if (!alive) break;
                    vtc::umma_commit(&empty[vs % C::SLOTS]);
                    if (more) vtc::umma_commit(&empty[kn % C::SLOTS]);
                }
                ++seg;
            }
        }
    } else if ((warp >> 2) < nt) {
        // ================= softmax: one thread per row =================
        const int t = warp >> 2;
        const int r = (warp & 3) * 32 + lane;  // row within the tile = TMEM lane
        const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t t_s = tmem + lane_base + t * C::BK, t_o = tmem + lane_base + C::O_COL0 + t * D;
        const int rg = (tile0 + t) * kTileRows + r;
        const bool rvalid = rg < a.n_q * a.grp;
        const int qi = rvalid ? rg / a.grp : 0, qn = rvalid ? rg % a.grp : 0;
        uint32_t it = 0;
        int seg = 0;
        while (w.next(a, glane)) {
            const int base = w.seg_len - a.n_q;
            const int64_t orow = ((int64_t)w.seg_b * a.n_q + qi) * a.hq + (int64_t)w.seg_kvh * a.grp + qn;
            unsigned long long mask = 0;
            if (alive) {
                // this row of Q, to TMEM (as bf16 pairs) or to shared memory
                uint4 u[D / 8];
                const uint4 *src = reinterpret_cast<const uint4 *>(a.q + orow * D);
#pragma unroll
                for (int j = 0; j < D / 8; ++j) u[j] = rvalid ? src[j] : make_uint4(0, 0, 0, 0);
                if (rvalid) mask = a.mask[(int64_t)w.seg_b * a.n_q + qi] & (~0ull >> (64 - a.n_q));
                if constexpr (C::QTM) {
#pragma unroll
                    for (int c0 = 0; c0 < D / 2; c0 += 16) {
                        float v[16];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            v[4 * j] = __uint_as_float(u[c0 / 4 + j].x);
                            v[4 * j + 1] = __uint_as_float(u[c0 / 4 + j].y);
                            v[4 * j + 2] = __uint_as_float(u[c0 / 4 + j].z);
                            v[4 * j + 3] = __uint_as_float(u[c0 / 4 + j].w);
                        }
                        vtc::tmem_st16_nowait(tmem + lane_base + C::Q_COL0 + c0, v);
                    }
                    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                } else {
#pragma unroll
                    for (int j = 0; j < D / 8; ++j)
                        *reinterpret_cast<uint4 *>(sq + t * C::QTILE + vtc::sw128(r, j, kTileRows)) = u[j];
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                }
                vtc::tc_fence_before();
                mbar_arrive(&q_ready[t]);
            }
            float m_used = -INFINITY, l = 0.0f;
            // tcgen05.ld / st are warp-collective: every lane runs them together
            for (int j = 0; j < w.sh.count && alive; ++j, ++it) {
                alive = __all_sync(0xffffffffu, mbar_wait(&s_ready[t], it & 1, a.status, a.wait_ns));
                if (!alive) break;
                vtc::tc_fence_after();
                float s[C::BK];
                tmem_ld_block<C::BK>(t_s, s);
                const int key0 = (w.sh.first + j * w.sh.step) * C::BK;
                if (key0 + C::BK > base) {
#pragma unroll
                    for (int h = 0; h < C::BK / 64; ++h) {
                        const unsigned long long seen = seen_bits(mask, key0 + 64 * h, base);
#pragma unroll
                        for (int c = 0; c < 64; ++c)
                            if (!((seen >> c) & 1)) s[64 * h + c] = -INFINITY;
                    }
                }
                const float mb = vtc::max_tree<C::BK>(s) * a.scale_log2;
                // the reference maximum follows only rises of more than 2^8
                // (rare after the first block): then O is rescaled
                const bool grow = mb > m_used + 8.0f;
                if (__any_sync(0xffffffffu, grow) && j > 0) {
                    const float f = grow ? (m_used == -INFINITY ? 0.0f : ex2(m_used - mb)) : 1.0f;
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
                for (int h = 0; h < C::BK / 32; ++h) {
                    float pk[16];
#pragma unroll
                    for (int c = 0; c < 16; ++c) {
                        const float p0 = ex2(fmaf(s[h * 32 + 2 * c], a.scale_log2, nms));
                        const float p1 = ex2(fmaf(s[h * 32 + 2 * c + 1], a.scale_log2, nms));
                        ls[(2 * c) & 3] += p0;
                        ls[(2 * c + 1) & 3] += p1;
                        pk[c] = __uint_as_float(pack_bf16(p0, p1));
                    }
                    vtc::tmem_st16_nowait(t_s + h * 16, pk);
                }
                asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                l += (ls[0] + ls[1]) + (ls[2] + ls[3]);
                vtc::tc_fence_before();
                mbar_arrive(&p_ready[t]);
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
            // that met a NaN: NaN (m = +infinity, which no other range outweighs)
            const bool zero = mask == 0 || (m_used == -INFINITY && l == 0.0f);
            const int64_t prow = ((int64_t)blockIdx.x * 2 + !w.at_start) * C::ROWS + t * kTileRows + r;
            const float f = 1.0f / l;
            for (int c0 = 0; c0 < D; c0 += 16) {
                float v[16];
                if (alive) {
                    vtc::tmem_ld16(t_o + c0, v);
                } else {
#pragma unroll
                    for (int i = 0; i < 16; ++i) v[i] = 0.0f;
                }
                if (!rvalid) continue;
                if (w.whole) {
                    store_out16<D>(a, orow, c0, v, f, zero);
                } else {
#pragma unroll
                    for (int i = 0; i < 16; i += 4)
                        *reinterpret_cast<float4 *>(a.ws_o + prow * D + c0 + i) =
                            make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
                }
            }
            if (rvalid && !w.whole) {
                a.ws_ml[prow * 2] = zero ? -INFINITY : l != l ? INFINITY : m_used;
                a.ws_ml[prow * 2 + 1] = zero ? 0.0f : l;
            }
            vtc::tc_fence_before();
            ++seg;
        }
        pdl_trigger();
    }
    vtc::tc_fence_before();
    __syncthreads();
    vtc::tc_fence_after();
    if (warp == 0)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::TMEM_COLS));
}

// Join the partials of units that span several ranges, in range order, and
// write zeros for requests that are refused.  One block per (unit, kJoinRows
// rows), one warp per row in turn.
constexpr int kJoinRows = 8;
template <int D, int QT>
__device__ __forceinline__ void tree_join_block(const Args &a) {
    using C = Cfg<D, QT>;
    constexpr int E = D / 32;
    __shared__ int64_t sums[4];
    __shared__ int64_t before_s;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int unit = blockIdx.x, b = unit / a.hkv, kvh = unit % a.hkv;
    const int nblk = blocks_of<C::BK>(a, b);
    if (nblk == 0 && tid == 0 && kvh == 0 && blockIdx.y == 0) report(a.status, VC_ERR_BAD_INDEX);
    const Sums sm = sum_blocks<C::BK>(a, sums, tid, 128);
    if (b >= sm.b0 && b < sm.b1) {
        int64_t p = sm.before;
        for (int i = sm.b0; i < b; ++i) p += blocks_of<C::BK>(a, i);
        before_s = p;
    }
    __syncthreads();
    const int64_t total = sm.total * a.hkv, u0 = before_s * a.hkv + (int64_t)kvh * nblk, u1 = u0 + nblk;
    // groups whose ranges hold the unit's first and last block
    int g0 = 0, g1 = -1;
    if (nblk > 0) {
        g0 = (int)(((u0 + 1) * a.groups - 1) / total);
        g1 = (int)((u1 * a.groups - 1) / total);
        if (g0 == g1) return;  // finished there
    }
    for (int k = warp; k < kJoinRows; k += 4) {
        const int rg = blockIdx.y * kJoinRows + k;
        if (rg >= a.n_q * a.grp) return;
        const int64_t orow = ((int64_t)b * a.n_q + rg / a.grp) * a.hq + (int64_t)kvh * a.grp + rg % a.grp;
        const int tile = rg / kTileRows;
        // the CTAs of a group that hold this tile
        const bool pair = QT == 2 && a.lanes == 3 && tile < 2;
        const int lane0 = QT == 1 || pair ? 0 : a.lanes == 3 ? 2 : tile / 2;
        const int trow = (QT == 1 ? 0 : a.lanes == 3 && tile == 2 ? 0 : (tile & 1)) * kTileRows + rg % kTileRows;
        float M = -INFINITY, L = 0.0f, acc[E];
#pragma unroll
        for (int i = 0; i < E; ++i) acc[i] = 0.0f;
        for (int g = g0; g <= g1; ++g) {
            const int64_t s0 = range_start(total, g, a.groups), s1 = range_start(total, g + 1, a.groups);
            const int64_t lo = max(u0, s0), hi = min(u1, s1);
            for (int ln = 0; ln < (pair ? 2 : 1); ++ln) {
                if (share_of(a.lanes, lane0 + ln, unit, (int)(lo - u0), (int)(hi - lo), false).count == 0) continue;
                const int64_t prow =
                    (((int64_t)g * a.lanes + lane0 + ln) * 2 + (lo != s0)) * C::ROWS + trow;
                const float m = a.ws_ml[prow * 2], l = a.ws_ml[prow * 2 + 1];
                const float mn = fmaxf(M, m);
                if (mn == -INFINITY) continue;
                const float fo = ex2(M - mn), fn = ex2(m - mn);
                M = mn;
                L = L * fo + l * fn;
                const float *o = a.ws_o + prow * D + lane * E;
#pragma unroll
                for (int i = 0; i < E; ++i) acc[i] = acc[i] * fo + o[i] * fn;
            }
        }
        const float f = M == -INFINITY ? 0.0f : 1.0f / L;
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const float y = M == -INFINITY ? 0.0f : acc[i] * f;
            if (a.out_bf16)
                ((uint16_t *)a.out)[orow * D + lane * E + i] = __bfloat16_as_ushort(__float2bfloat16_rn(y));
            else
                ((float *)a.out)[orow * D + lane * E + i] = y;
        }
    }
}

}  // namespace tree
}  // namespace vc
