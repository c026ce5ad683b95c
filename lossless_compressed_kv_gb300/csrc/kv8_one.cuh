// Attention over an 8-bit cache for up to 128 rows, on the 5th-generation
// tensor cores.  Codes become fp16 in shared memory as in kv8_tc.cuh, here by
// seven warps that fetch them by asynchronous copies; S runs NBUF blocks of 64
// keys ahead, and two groups of softmax warps take blocks in turn, each with a
// maximum, a sum and an O of its own for the same rows: at a segment's end the
// two are put together.
//
// 8 x 32768 keys, 8 heads of 128, 128 rows: 168 us, 80 of which HBM needs; of
// 4 rows it would take 155.  By clock reads a block of 64 keys takes a CTA 1250
// cycles (head_dim 64: 1040), all roles' beginnings and ends of segments dealt out
// to the blocks.  The warp that issues products works for 770 of them (590): P V
// 185 (215), S with two commits 480 (300), two commits 105 (75); it waits 190
// (200) and spends the rest, 290 (250), at segments' ends.  The tensor pipe works a
// third of the time; a softmax group 1300 of 2530 cycles for a block of its own, a
// converter 2000 of 4280 for an item.  ptxas spills 280 bytes a thread with 128
// channels, 8 with 64.  Measured against it: two CTAs an SM with a chain of one S
// buffer each 178 us; codes through a ring filled by TMA 230; S and P V issued by
// a warp each, which must then wait for one another's products, 222 (head_dim 64:
// 129, where this takes 131).
//
// Steps are blocks: step i uses S buffer i % NBUF and O i % 2.  A finished
// S (i) was issued behind P V (i - NBUF): the P V before of the same O, step
// i - 2, has a barrier of its own for the (rare) rescaling.
#pragma once

#include "kv8_tc.cuh"

namespace vc {
namespace kv8 {

template <int D>
struct One {
    static constexpr int BK = 64;
    static constexpr int NBUF = D == 64 ? 4 : 3;
    static_assert(NBUF > 2 && NBUF <= 4, "phases that a parity tells apart");
    static constexpr int PG = BK / kPage;
    static constexpr int SLOT = BK * D * 2;
    static constexpr int LAG = NBUF;  // S runs NBUF blocks ahead of P V
    static constexpr int STAGE = 8 * 4096;
    static constexpr int LIMIT = 226 * 1024;
    static constexpr int CONVERTERS = 7, CODES = BK * D;  // each one's codes under way
    static constexpr int FIT = (LIMIT - 8192 - STAGE - CONVERTERS * CODES) / SLOT;
    static constexpr int SLOTS = FIT < 16 ? FIT : 16;
    static_assert(SLOTS / 2 + LAG + 1 <= kScaleRing, "ring depth");
    static constexpr int OFF_CODES = SLOTS * SLOT, OFF_STAGE = OFF_CODES + CONVERTERS * CODES;
    static constexpr int OFF_SC = OFF_STAGE + STAGE;
    static constexpr int OFF_STATE = OFF_SC + kScaleRing * PG * 8;  // (m, l, vref, alive) of each group's rows
    static constexpr int OFF_BAR = OFF_STATE + 2 * kTileRows * 16;
    static constexpr int NBAR = 1 + 2 * NBUF + 2 + 1 + 2 * SLOTS + 1;
    static constexpr int SMEM = OFF_BAR + NBAR * 8 + 16;
    static_assert(SMEM <= LIMIT, "shared memory");
    static constexpr int O_COL0 = NBUF * BK, Q_COL0 = O_COL0 + 2 * D;
    static_assert(Q_COL0 + D / 2 <= 512, "TMEM columns");
    // two groups of softmax warps; MMA issue and seven converters.
    // (2 x 128 x 160 + 2 x 128 x 96 = 512 x 128 registers)
    static constexpr int SM_WARPS = 8, WARPS = 16, THREADS = WARPS * 32;
    static_assert(SM_WARPS + 1 + CONVERTERS == WARPS, "roles");
    static constexpr int REGS_SOFTMAX = 160, REGS_OTHER = 96;
    static constexpr int ROWS = kTileRows;
};

// The order of a range's blocks in the ring: within a segment V runs LAG
// blocks behind K, as the products that read them do; they are done with in
// this order as well.
template <int BK, int LAG>
struct Items {
    tree::Walk<BK> w;
    int i = 0, n = 0;   // step of the segment's n + LAG; v: its V was the last item
    bool v = true;
    int k0 = 0;         // blocks of the segments before
    // the item: a block of its segment
    int at = 0;
    bool is_v = false;
    __device__ bool next(const Args &a) {
        for (;;) {
            if (v) {  // the next step
                v = false;
                if (n == 0 || ++i == n + LAG) {
                    k0 += n;
                    i = n = 0;
                    if (!w.next(a)) {
                        v = true;
                        return false;
                    }
                    n = w.seg_n;
                }
                if (i < n) {
                    at = i;
                    is_v = false;
                    return true;
                }
            }
            v = true;
            if (i >= LAG) {
                at = i - LAG;
                is_v = true;
                return true;
            }
        }
    }
    // The item `by` further on.
    __device__ bool skip(const Args &a, int by) {
        const int q = 2 * i + v + by;
        if (i >= LAG && q >> 1 < n) {  // (where K and V alternate)
            i = q >> 1;
            v = is_v = q & 1;
            at = i - (v ? LAG : 0);
            return true;
        }
        while (--by > 0)
            if (!next(a)) return false;
        return next(a);
    }
};

// Converter warp `part` of C::CONVERTERS: every so many-th block from codes in
// global memory to fp16 in the ring.  A block's pages are under way by
// asynchronous copies, each lane's pieces for itself alone.  (The SM's TMA unit
// takes copies of a head block too slowly: 8 x 32768 keys 230 us; in registers
// they spill.)  The warp of a block of K leaves the block's scales beside it.
template <class C, int D, bool E4M3>
__device__ __forceinline__ void convert(const Args &a, const tree::Walk<C::BK> &w, int part, uint8_t *skv, uint8_t *codes,
                                        float2 *scales, uint64_t *full, uint64_t *empty) {
    constexpr int BK = C::BK, PG = C::PG, IT = D / 64, U = 2 * IT;  // pieces of a page that a lane holds
    const int lane = threadIdx.x & 31;
    if (block_skips(a.skip_copies)) return;
    Items<BK, C::LAG> it;
    it.w = w;
    uint32_t seq = part;  // this warp's item in the order
    struct Item {
        bool there, is_v;
        bool page;   // lane p: page p holds tokens
        int rows;    // rows that hold tokens
        int id;      // lane p: page p
        float2 sc;   // lane p: its scales (of a block of K)
        int k, kvh;  // block of the range
    };
    // this warp's item `by` further on, its page ids on their way; a turn later they
    // are looked at and the scales set off, and used another turn later
    bool more = true;
    auto fetch = [&](int by) {
        Item m;
        more = more && it.skip(a, by);
        m.there = more;
        m.page = m.is_v = false;
        m.id = m.rows = m.kvh = m.k = 0;
        m.sc = make_float2(1.0f, 0.0f);
        if (more) {
            const int blk = it.w.seg_blk + it.at, pidx = blk * PG + lane;
            m.is_v = it.is_v;
            m.k = it.k0 + it.at;
            m.rows = it.w.seg_len - blk * BK;
            m.kvh = it.w.seg_kvh;
            // (pages behind the request's end: any valid page, masked and cleared)
            m.page = lane < PG && pidx * kPage < it.w.seg_len;
            if (m.page) m.id = pidx < a.maxb ? a.table[(int64_t)it.w.seg_b * a.maxb + pidx] : -1;
        }
        return m;
    };
    auto look = [&](Item &m) {
        if (m.id < 0 || m.id >= a.n_pages) {
            report(a.status, VC_ERR_BAD_INDEX);
            m.id = 0;
        }
        if (m.page && !m.is_v) {
            const int64_t x = (int64_t)m.id * a.hkv + m.kvh;
            m.sc = make_float2(a.ks[x], a.vs[x]);
        }
    };
    // a lane's pieces of a page: row r0 (and r0 + 8), piece c0 (and, with 128-byte
    // rows, c1): eight lanes read whole sectors and write different banks, half of
    // one row and the other half of the next
    const int r0 = lane >> 2, c0 = D == 128 ? (lane & 3) + 4 * (r0 & 1) : lane & 3, c1 = c0 ^ 4;
    uint4 *mine = reinterpret_cast<uint4 *>(codes) + lane;  // [PG][U][32]
    auto copy = [&](const Item &m, int page) {
        const int id = __shfl_sync(0xffffffffu, m.id, page);
        const uint8_t *src = (m.is_v ? a.vc : a.kc) + ((int64_t)id * a.hkv + m.kvh) * (kPage * D) + r0 * D;
#pragma unroll
        for (int k = 0; k < U; ++k)
            cp_async16(mine + (page * U + k) * 32, src + k / IT * 8 * D + (IT == 2 && k % 2 ? c1 : c0) * 16);
    };
    // where the halves of piece c of row r0 go
    auto place = [&](int c, int h) { return (c >> 2) * (BK * 128) + r0 * 128 + (((2 * c + h) & 7) ^ r0) * 16; };
    const int to[2][2] = {{place(c0, 0), place(c0, 1)}, {place(c1, 0), place(c1, 1)}};
    Item cur = fetch(part + 1), nxt = fetch(C::CONVERTERS), after = fetch(C::CONVERTERS);
    look(cur);
    look(nxt);
    if (cur.there) {
#pragma unroll
        for (int p = 0; p < PG; ++p) {
            copy(cur, p);
            cp_async_commit();
        }
    }
    for (; cur.there; seq += C::CONVERTERS) {
        const uint32_t slot = seq % C::SLOTS, use = seq / C::SLOTS;
        // (parity: this warp's last block had its place, so the one SLOTS before that is used up)
        static_assert(C::CONVERTERS <= C::SLOTS, "phases that a parity tells apart");
        if (use > 0 && !__all_sync(0xffffffffu, mbar_wait(&empty[slot], (use - 1) & 1, a.status, a.wait_ns))) break;
        uint8_t *dst = skv + slot * C::SLOT;
        if (!cur.is_v && lane < PG)
            scales[cur.k % kScaleRing * PG + lane] = make_float2(scale_of(cur.sc.x), scale_of(cur.sc.y));
#pragma unroll
        for (int p = 0; p < PG; ++p) {
            cp_async_wait<PG - 1>();
            uint4 u[U];
#pragma unroll
            for (int k = 0; k < U; ++k) u[k] = mine[(p * U + k) * 32];
            // (a group each time, so that what is under way is counted in pages)
            if (nxt.there) copy(nxt, p);
            cp_async_commit();
#pragma unroll
            for (int k = 0; k < U; ++k) {
                const int r = p * kPage + k / IT * 8;
                uint4 lo, hi;
                widen<E4M3>(u[k], lo, hi);
                // V behind the request's end: whatever it holds, 0 times it is to be 0
                if (cur.is_v && r + r0 >= cur.rows) lo = hi = make_uint4(0, 0, 0, 0);
                *reinterpret_cast<uint4 *>(dst + to[IT == 2 && k % 2][0] + r * 128) = lo;
                *reinterpret_cast<uint4 *>(dst + to[IT == 2 && k % 2][1] + r * 128) = hi;
            }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[slot]);
        cur = nxt;
        nxt = after;
        look(nxt);
        after = fetch(C::CONVERTERS);
    }
    cp_async_wait<0>();
}

template <int D, bool E4M3>
__device__ __forceinline__ void one_cta(const Args &a, uint8_t *smem) {
    using C = One<D>;
    constexpr int BK = C::BK, PG = C::PG;
    if (smem_u32(smem) & 1023u) {  // (the swizzled tiles start on 1024-byte boundaries: the array is declared so)
        if (threadIdx.x == 0) report(a.status, VC_ERR_UNSUPPORTED);
        return;
    }
    uint8_t *skv = smem;
    float2 *scales = reinterpret_cast<float2 *>(smem + C::OFF_SC);    // [kScaleRing][PG]
    float4 *states = reinterpret_cast<float4 *>(smem + C::OFF_STATE);  // [2][rows]
    uint64_t *q_ready = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);
    uint64_t *s_ready = q_ready + 1, *p_ready = s_ready + C::NBUF, *pv_done = p_ready + C::NBUF, *o_done = pv_done + 2;
    uint64_t *full = o_done + 1, *empty = full + C::SLOTS, *idle = empty + C::SLOTS;
    uint32_t *tslot = reinterpret_cast<uint32_t *>(idle + 1);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    // ---- set-up ----
    if (tid == 0) {
        mbar_init(q_ready, 8);
        for (int i = 0; i < C::NBUF; ++i) {
            mbar_init(&s_ready[i], 1);
            mbar_init(&p_ready[i], 4);
        }
        mbar_init(&pv_done[0], 1);
        mbar_init(&pv_done[1], 1);
        mbar_init(o_done, 1);
        for (int i = 0; i < C::SLOTS; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        mbar_init(idle, 1);
        fence_mbar_init();
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tslot)), "r"(512));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    vtc::tc_fence_before();
    int total, before, b0 = 0, rest = 0;
    tree::sum_blocks<BK>(a, 0, lane, total, before);
    const tree::Deal deal(total * a.hkv, a.groups);
    const int f0 = deal.start(blockIdx.x), mine = deal.start(blockIdx.x + 1) - f0;
    if (mine > 0) tree::find_block<BK>(a, f0, lane, b0, rest);
    tree::Walk<BK> w;
    w.begin(a, b0, rest, mine);
    __syncthreads();
    vtc::tc_fence_after();
    const uint32_t tmem = *tslot;

    constexpr uint32_t IQK = idesc_f16(128, BK, false);
    constexpr uint32_t IPV = idesc_f16(128, D, true);
    bool alive = true;

    if (warp >= C::SM_WARPS) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::REGS_OTHER));
    if (warp == C::SM_WARPS) {
        // ================= MMA issue (the warp in step, one elected thread; see tree_tc.cuh) =================
        const uint64_t kd0 = vtc::sdesc(smem_u32(skv), 16, 1024), vd0 = vtc::sdesc(smem_u32(skv), BK * 128, 1024);
        // places in the ring and among the S buffers, with the parity of the phase waited for there
        struct Place {
            uint32_t i, par;
            __device__ void step(uint32_t by, uint32_t of) {
                if ((i += by) >= of) {
                    i -= of;
                    par ^= 1;
                }
            }
        } kp{0, 0}, vp{0, 0}, pp{0, 0};
        uint32_t sb = 0, chain = 0, seg = 0;
        int kt = 0;  // blocks of K behind kp
        auto wait1 = [&](uint64_t *bar, uint32_t par) {
            alive = __all_sync(0xffffffffu, mbar_wait(bar, par, a.status, a.wait_ns));
            return alive;
        };
        auto next_s = [&]() {
            const uint64_t kd = kd0 + kp.i * (C::SLOT / 16);
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks)
                tree::umma_ta(tmem + sb * BK, tmem + C::Q_COL0 + ks * 8, kd + ((ks >> 2) * (BK * 128) + (ks & 3) * 32) / 16, IQK,
                              ks > 0);
            tree::umma_commit(&s_ready[sb]);
            tree::umma_commit(&empty[kp.i]);
            if (++sb == C::NBUF) sb = 0;
            kp.step(kt++ < C::LAG ? 1 : 2, C::SLOTS);
        };
        for (;; ++seg) {
            // (by shuffle, so that the compiler knows the loops' state to be uniform)
            const bool any = alive && w.next(a);
            const int n = __shfl_sync(0xffffffffu, any ? w.seg_n : 0, 0);
            if (n == 0) break;
            kp = vp;  // (places in the ring follow the order of Items)
            kt = 0;
            vp.step(min(C::LAG + 1, n), C::SLOTS);
            if (!wait1(q_ready, seg & 1)) break;
#pragma unroll
            for (int i = 0; i < C::NBUF; ++i) {
                if (i >= n) break;
                if (!wait1(&full[kp.i], kp.par)) break;
                vtc::tc_fence_after();
                next_s();
            }
            for (int j = 0; j < n && alive; ++j) {
                const bool more = j + C::NBUF < n;
                if (!__all_sync(0xffffffffu, ready3(&p_ready[pp.i], pp.par, &full[vp.i], vp.par, more ? &full[kp.i] : &full[vp.i],
                                                    more ? kp.par : vp.par))) {
                    if (!wait1(&p_ready[pp.i], pp.par)) break;
                    if (!wait1(&full[vp.i], vp.par)) break;
                    if (more && !wait1(&full[kp.i], kp.par)) break;
                }
                vtc::tc_fence_after();
                const uint64_t vd = vd0 + vp.i * (C::SLOT / 16);
#pragma unroll
                for (int kk = 0; kk < BK / 16; ++kk)
                    tree::umma_ta(tmem + C::O_COL0 + chain * D, tmem + pp.i * BK + kk * 8, vd + kk * 16 * 128 / 16, IPV,
                                  j > 1 || kk > 0);
                tree::umma_commit(&pv_done[chain]);
                if (more) next_s();
                tree::umma_commit(&empty[vp.i]);  // (in the order of Items)
                pp.step(1, C::NBUF);
                vp.step(j + 1 + C::LAG < n ? 2 : 1, C::SLOTS);
                chain ^= 1;
            }
            if (!alive) break;
            tree::umma_commit(o_done);
        }
        // no product may be under way when TMEM is freed
        tree::umma_commit(idle);
        mbar_wait(idle, 0, a.status, kWaitNs);
    } else if (warp > C::SM_WARPS) {
        convert<C, D, E4M3>(a, w, warp - C::SM_WARPS - 1, skv, smem + C::OFF_CODES + (warp - C::SM_WARPS - 1) * C::CODES, scales, full,
                            empty);
    } else {
        // ================= softmax: a thread of each group per row =================
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::REGS_SOFTMAX));
        const int grp = warp >> 2;             // takes the steps of its parity
        const int r = (warp & 3) * 32 + lane;  // row = TMEM lane
        const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t t_o = tmem + lane_base + C::O_COL0;
        const bool rvalid = r < a.rows;
        const bool any_row = (warp & 3) * 32 < a.rows;  // of the warp's
        const int qi = rvalid ? r / a.grp : 0, qn = rvalid ? r % a.grp : 0;
        // the warp's 32 rows x 8 pieces of 16 bytes, on their way between a thread's
        // own row and eight neighbouring lanes a row
        uint4 *stage = reinterpret_cast<uint4 *>(smem + C::OFF_STAGE + warp * 4096);
        const int srow = lane >> 3, spc = lane & 7;  // row (of 4 at a time) and piece
        auto at = [&](int row, int piece) { return stage + row * 8 + (piece ^ (row & 7)); };
        uint32_t it0 = 0, seg = 0;  // steps before this segment, segments
        for (; w.next(a); ++seg, it0 += w.seg_n) {
            const int base = w.seg_len - a.n_q;
            const int64_t orow = ((int64_t)w.seg_b * a.n_q + qi) * a.hq + (int64_t)w.seg_kvh * a.grp + qn;
            const unsigned long long mask = rvalid ? mask_of(a, w.seg_b, qi) : 0;
            float rf = 0.0f;  // this row's factor beside K's scale
            if (alive) {
                // the warp's rows of Q to TMEM: each group looks at all channels and
                // stores 64 of them (the first group those of head_dim 64)
                uint4 u[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int64_t ro = __shfl_sync(0xffffffffu, rvalid ? orow : (int64_t)-1, i * 4 + srow);
                    const uint4 *src = reinterpret_cast<const uint4 *>(a.q + ro * D) + spc;
                    uint32_t mx = 0;
#pragma unroll
                    for (int h = 0; h < D / 64; ++h) {
                        const uint4 x = ro >= 0 ? src[h * 8] : make_uint4(0, 0, 0, 0);
                        if (D == 64 || h == grp) u[i] = x;
                        mx = __vmaxu2(mx, __vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu));
                        mx = __vmaxu2(mx, __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu));
                    }
                    mx = max(mx & 0xffffu, mx >> 16);
#pragma unroll
                    for (int o = 1; o < 8; o <<= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                    const int e = q_exponent(bf16_bits_to_f32((uint16_t)mx));
                    const float up = exp2i(e);
                    uint32_t *x = reinterpret_cast<uint32_t *>(&u[i]);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        x[j] = pack_f16(__uint_as_float(x[j] << 16) * up, __uint_as_float(x[j] & 0xffff0000u) * up);
                    const int mine_e = __shfl_sync(0xffffffffu, e, (lane & 3) * 8);
                    if (lane >> 2 == i) rf = a.scale_log2 * exp2i(-mine_e);
                }
                if (D == 128 || grp == 0) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) *at(i * 4 + srow, spc) = u[i];
                    __syncwarp();
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float v[16];
#pragma unroll
                        for (int j = 0; j < 4; ++j) *reinterpret_cast<uint4 *>(v + 4 * j) = *at(lane, c * 4 + j);
                        vtc::tmem_st16_nowait(tmem + lane_base + C::Q_COL0 + grp * 32 + c * 16, v);
                    }
                    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                }
                vtc::tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(q_ready);
            }
            float m_used = -INFINITY, l = 0.0f, vref = 0.0f, inv_vref = 0.0f;
            // tcgen05.ld / st are warp-collective: every lane runs them together
            bool first = true;
            for (int j = (it0 ^ grp) & 1; j < w.seg_n && alive; j += 2) {
                const uint32_t step = it0 + j, buf = step % C::NBUF, t_s = tmem + lane_base + buf * BK;
                alive = __all_sync(0xffffffffu, mbar_wait(&s_ready[buf], (step / C::NBUF) & 1, a.status, a.wait_ns));
                if (!alive) break;
                if (!any_row) {  // (what P holds in rows that are not there goes nowhere)
                    if (lane == 0) mbar_arrive(&p_ready[buf]);
                    continue;
                }
                vtc::tc_fence_after();
                float s[BK];
                vtc::tmem_ld_row<64>(t_s, s);
                const int key0 = (w.seg_blk + j) * BK;
                if (key0 + BK > base) {
                    const unsigned long long seen = tree::seen_bits(mask, key0, base);
#pragma unroll
                    for (int c = 0; c < 64; ++c)
                        if (!((seen >> c) & 1)) s[c] = -INFINITY;
                }
                const float2 *sc = scales + step % kScaleRing * PG;
                float mb = -INFINITY, vtop = 0.0f, kf[PG], vw[PG];
#pragma unroll
                for (int p = 0; p < PG; ++p) {
                    const float2 f = sc[p];
                    kf[p] = factor_of(f.x, rf);
                    vw[p] = f.y;
                    mb = fmaxf(mb, tree::max_of<16>(*reinterpret_cast<float(*)[16]>(&s[16 * p])) * kf[p]);
                    vtop = fmaxf(vtop, f.y);
                }
                // the reference of a row's maximum follows only rises beyond kRise, V's
                // is twice the largest scale so far; then O is rescaled
                const bool grow = mb > m_used + kRise, more = vtop > vref;
                if (__any_sync(0xffffffffu, grow || more)) {
                    float f = grow ? (m_used == -INFINITY ? 0.0f : ex2(m_used - (mb - kBelow))) : 1.0f;
                    l *= f;
                    if (more) {
                        inv_vref = 0.5f / vtop;
                        f *= vref * inv_vref;
                        vref = 2.0f * vtop;
                    }
                    if (!first) {
                        alive = __all_sync(0xffffffffu, mbar_wait(&pv_done[grp], ((step >> 1) - 1) & 1, a.status, a.wait_ns));
                        if (!alive) break;
                        vtc::tc_fence_after();
#pragma unroll 1
                        for (int c0 = 0; c0 < D; c0 += 16) {
                            float v[16];
                            vtc::tmem_ld16(t_o + grp * D + c0, v);
#pragma unroll
                            for (int i = 0; i < 16; ++i) v[i] *= f;
                            vtc::tmem_st16(t_o + grp * D + c0, v);
                        }
                    }
                }
                first = false;
                if (grow) m_used = mb - kBelow;
                const float nms = m_used == -INFINITY ? 0.0f : -m_used;
                float ls[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int h = 0; h < BK / 32; ++h) {
                    float pk[16];
#pragma unroll
                    for (int p = 0; p < 2; ++p) {
                        const float v = vw[2 * h + p] * inv_vref;
#pragma unroll
                        for (int c = 8 * p; c < 8 * p + 8; ++c) {
                            float p0, p1;
                            tree::fma2(p0, p1, s[h * 32 + 2 * c], s[h * 32 + 2 * c + 1], kf[2 * h + p], nms);
                            p0 = ex2(p0);
                            p1 = ex2(p1);
                            tree::add2(ls[(2 * c) & 2], ls[((2 * c) & 2) + 1], p0, p1);
                            mul2(p0, p1, v);
                            pk[c] = __uint_as_float(pack_f16(p0, p1));
                        }
                    }
                    vtc::tmem_st16_nowait(t_s + h * 16, pk);
                }
                asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                vtc::tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_ready[buf]);
                l += (ls[0] + ls[1]) + (ls[2] + ls[3]);
            }
            if (alive) alive = __all_sync(0xffffffffu, mbar_wait(o_done, seg & 1, a.status, a.wait_ns));
            // ---- the segment's result: the groups' two put together (rows' states as in kv8_few.cuh) ----
            states[grp * kTileRows + r] = make_float4(m_used, l, vref, alive ? 1.0f : 0.0f);
            asm volatile("bar.sync 1, 256;" ::: "memory");
            const float4 other = states[(grp ^ 1) * kTileRows + r];
            alive = alive && __all_sync(0xffffffffu, other.w != 0.0f);
            vtc::tc_fence_after();
            const float4 s0 = grp ? other : make_float4(m_used, l, vref, 0.0f), s1 = grp ? make_float4(m_used, l, vref, 0.0f) : other;
            const float m = fmaxf(s0.x, s1.x);
            const float w0 = s0.x == -INFINITY ? 0.0f : ex2(s0.x - m), w1 = s1.x == -INFINITY ? 0.0f : ex2(s1.x - m);
            // (a sum that is not a number is one beside any other)
            const float ls = s0.y != s0.y || s1.y != s1.y ? __int_as_float(0x7fffffff) : s0.y * w0 + s1.y * w1;
            const bool zero = !alive || mask == 0 || (m == -INFINITY && ls == 0.0f);
            const float f0 = zero ? 0.0f : w0 / ls * s0.z, f1 = zero ? 0.0f : w1 / ls * s1.z;
            // (a segment of one block leaves one O as it was)
            const bool two = w.seg_n > 1;
            const int only = it0 & 1;
            const int64_t prow = ((int64_t)blockIdx.x * 2 + !w.at_start) * C::ROWS + r;
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
            if (any_row && (D == 128 || grp == 0)) {
#pragma unroll 1
                for (int c0 = grp * 64; c0 < grp * 64 + 64; c0 += 32) {
                    float v[32];
                    if (alive) {
                        vtc::tmem_ld_row<32>(t_o + (two ? 0 : only * D) + c0, v);
                        const float fa = two || !only ? f0 : f1;
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] *= fa;
                        if (two) {
                            float x[32];
                            vtc::tmem_ld_row<32>(t_o + D + c0, x);
#pragma unroll
                            for (int i = 0; i < 32; ++i) v[i] = fmaf(x[i], f1, v[i]);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = zero ? 0.0f : v[i];
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
            }
            if (rvalid && !w.whole && grp == 0) {
                a.ws_ml[prow * 2] = zero ? -INFINITY : ls != ls ? INFINITY : m;
                a.ws_ml[prow * 2 + 1] = !alive ? -1.0f : zero ? 0.0f : ls;
            }
            // both have read both before O, Q and the states are written again
            vtc::tc_fence_before();
            asm volatile("bar.sync 1, 256;" ::: "memory");
        }
        pdl_trigger();
    }
    vtc::tc_fence_before();
    __syncthreads();
    vtc::tc_fence_after();
    if (warp == 0) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
}

}  // namespace kv8
}  // namespace vc
