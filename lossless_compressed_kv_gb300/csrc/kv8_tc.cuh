// Attention over an 8-bit cache for more than 128 rows, on the 5th-generation
// tensor cores: the kernel of tree_tc.cuh (its work split, tiles, S buffers, barriers
// by parity and bounded waits) with codes instead of bf16 rows.
//
// tcgen05 takes both operands of one type, and whole numbers are not among
// them: two warps turn blocks of codes (a ring filled by TMA) into fp16 in a
// second ring, which the products read.  The conversion is exact, so Q and P
// in fp16 are all that is rounded; e4m3 products of Q and P split in two would
// need as many instructions and more softmax arithmetic, and not serve int8.
// What it costs is shared memory: 32 KB of codes (128 keys, head_dim 128) are
// written, read, written again as 64 KB and read by each tile, with Q: 320 KB for
// two tiles, 2500 cycles where the products take 2180.
// 8 x 32768 keys, 256 rows 283 us (970 TFLOP/s of products), 320 rows 407 (ptxas
// spills 160 to 194 bytes a thread); seven
// warps that fetch codes themselves, as in kv8_one.cuh, took 360 and 448 (the
// ring of fp16 blocks is then too short, and the softmax warps spill).
//
// K's scales join the softmax scale, a factor a page; V's go with the
// probabilities, relative to a reference (kv8.cuh) that moves like the running
// maximum: rarely, with O rescaled.  The producer leaves each block's scales
// beside its copies.
#pragma once

#include "kv8_few.cuh"

namespace vc {
namespace kv8 {

using vtc::kTileRows;
constexpr int kScaleRing = 16;  // blocks whose scales are held (more than are under way)

template <int D, int QT>
struct Tc {
    // Keys per block and S buffers as in tree_tc.cuh.
    static constexpr int BK = QT == 2 ? 128 : 64;
    static constexpr int NBUF = QT == 2 ? (D == 64 ? 3 : 2) : D == 64 ? 4 : 2;
    static constexpr bool AHEAD = NBUF > QT;
    static_assert(NBUF <= 2 * QT, "phases that a parity tells apart");
    static constexpr int PG = BK / kPage;
    static constexpr int SLOT = BK * D * 2;   // a block in fp16
    static constexpr int SLOT8 = BK * D;      // a block of codes
    static constexpr int QTILE = kTileRows * D * 2;
    static constexpr int OFF_KV = QT * QTILE;
    static constexpr int LIMIT = 226 * 1024;
    static constexpr int SLOTS = D == 128 && QT < 3 ? 3 : 4;
    static constexpr int FIT = (LIMIT - 2048 - OFF_KV - SLOTS * SLOT) / SLOT8;
    static constexpr int SLOTS8 = FIT < 12 ? FIT : 12;
    static_assert(SLOTS8 >= 4 && SLOTS8 / 2 + SLOTS / 2 + NBUF + 3 <= kScaleRing, "ring depths");
    static constexpr int OFF_CODES = OFF_KV + SLOTS * SLOT;
    static constexpr int OFF_SC = OFF_CODES + SLOTS8 * SLOT8;
    static constexpr int OFF_BAR = OFF_SC + kScaleRing * PG * 8;
    static constexpr int NS = NBUF < QT ? QT : NBUF;
    static constexpr int NBAR = 3 * QT + NS + NBUF + 2 * SLOTS + 2 * SLOTS8 + 1;
    static constexpr int SMEM = OFF_BAR + NBAR * 8 + 16;
    static_assert(SMEM <= LIMIT, "shared memory of the CTAs an SM holds");
    static constexpr int O_COL0 = NBUF * BK;
    static_assert(O_COL0 + QT * D <= 512, "TMEM columns");
    static constexpr int SM_WARPS = QT * 4;
    // the last warpgroup: producer, MMA issue, two converters; it gives registers
    // up for the softmax warps (2 x 128 x 216 + 128 x 72 <= 384 x 168; 3 x 128 x 136
    // + 128 x 96 <= 512 x 128)
    static constexpr int WARPS = 4 * QT + 4;
    static constexpr int REGS_SOFTMAX = QT == 2 ? 216 : 136, REGS_OTHER = QT == 2 ? 72 : 96;
    static constexpr int THREADS = WARPS * 32;
    static constexpr int ROWS = QT * kTileRows;
};

// Instruction descriptor, kind::f16: fp32 accumulate, fp16 A and B, A K-major.
__host__ __device__ constexpr uint32_t idesc_f16(int m, int n, bool b_mn_major) {
    return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// 16 codes as fp16.
template <bool E4M3>
__device__ __forceinline__ void widen(const uint4 &u, uint4 &lo, uint4 &hi) {
    const uint32_t x = raw<E4M3>(u.x), y = raw<E4M3>(u.y), z = raw<E4M3>(u.z), w = raw<E4M3>(u.w);
    lo = make_uint4(to_f16_lo<E4M3>(x), to_f16_hi<E4M3>(x), to_f16_lo<E4M3>(y), to_f16_hi<E4M3>(y));
    hi = make_uint4(to_f16_lo<E4M3>(z), to_f16_hi<E4M3>(z), to_f16_lo<E4M3>(w), to_f16_hi<E4M3>(w));
}

// Whether three phases are over, asked for at once: one after another a wait takes
// the warp that issues products 130 cycles each, ready or not.
__device__ __forceinline__ bool ready3(uint64_t *a, uint32_t pa, uint64_t *b, uint32_t pb, uint64_t *c, uint32_t pc) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p, q, r;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 q, [%3], %4;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 r, [%5], %6;\n\t"
        "and.pred p, p, q;\n\tand.pred p, p, r;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(a)), "r"(pa), "r"(smem_u32(b)), "r"(pb), "r"(smem_u32(c)), "r"(pc)
        : "memory");
    return ok != 0;
}

__device__ __forceinline__ void mul2(float &d0, float &d1, float b) {
    asm("{\n\t.reg .b64 ra, rb;\n\t"
        "mov.b64 ra, {%0, %1};\n\tmov.b64 rb, {%2, %2};\n\t"
        "mul.rn.f32x2 ra, ra, rb;\n\tmov.b64 {%0, %1}, ra;\n\t}"
        : "+f"(d0), "+f"(d1)
        : "f"(b));
}

template <int D, int QT, bool E4M3>
__device__ __forceinline__ void tc_cta(const Args &a, uint8_t *smem) {
    using C = Tc<D, QT>;
    constexpr int BK = C::BK, PG = C::PG;
    if (smem_u32(smem) & 1023u) {  // (the swizzled tiles start on 1024-byte boundaries: the array is declared so)
        if (threadIdx.x == 0) report(a.status, VC_ERR_UNSUPPORTED);
        return;
    }
    uint8_t *sq = smem, *skv = smem + C::OFF_KV, *scodes = smem + C::OFF_CODES;
    float2 *scales = reinterpret_cast<float2 *>(smem + C::OFF_SC);  // [kScaleRing][PG]
    uint64_t *q_ready = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);  // [QT]
    uint64_t *s_ready = q_ready + QT, *p_ready = s_ready + C::NS, *o_done = p_ready + C::NBUF, *pv_done = o_done + QT;
    uint64_t *full = pv_done + QT, *empty = full + C::SLOTS;           // blocks in fp16
    uint64_t *full8 = empty + C::SLOTS, *empty8 = full8 + C::SLOTS8;   // blocks of codes
    uint64_t *idle = empty8 + C::SLOTS8;
    uint32_t *tslot = reinterpret_cast<uint32_t *>(idle + 1);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int grp_id = blockIdx.x / a.lanes, glane = blockIdx.x % a.lanes;
    const int tile0 = QT * glane;  // this CTA's tiles: QT from there

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
            mbar_init(&full[i], 2);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < C::SLOTS8; ++i) {
            mbar_init(&full8[i], 1);
            mbar_init(&empty8[i], 2);
        }
        mbar_init(idle, 1);
        fence_mbar_init();
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tslot)),
                     "r"(512));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    vtc::tc_fence_before();
    // this group's range, by every warp for itself
    int total, before, b0 = 0, rest = 0;
    tree::sum_blocks<BK>(a, 0, lane, total, before);
    const tree::Deal deal(total * a.hkv, a.groups);
    const int f0 = deal.start(grp_id), mine = deal.start(grp_id + 1) - f0;
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
        // ================= producer =================
        if (!block_skips(a.skip_copies)) {
            uint32_t seq = 0;   // copies into the ring so far
            uint32_t blocks = 0;
            while (alive && w.next(a)) {
                const int32_t *trow = a.table + (int64_t)w.seg_b * a.maxb;
                const int npages = ceil_div(w.seg_len, kPage);
                // page ids, 32 at a time, one batch ahead; their scales half a batch later
                // (pages behind the request's end: any valid page, masked and cleared)
                constexpr int NB = 32 / PG;
                bool nthere = false;
                auto load_ids = [&](int i0) {
                    const int i = i0 + lane / PG;
                    int id = 0;
                    nthere = false;
                    if (i < w.seg_n) {
                        const int pidx = (w.seg_blk + i) * PG + lane % PG;
                        if (pidx < npages) {
                            id = pidx < a.maxb ? trow[pidx] : -1;
                            if (id < 0 || id >= a.n_pages) {
                                report(a.status, VC_ERR_BAD_INDEX);
                                id = 0;
                            }
                            nthere = true;
                        }
                    }
                    return id;
                };
                auto load_scales = [&](int id) {
                    const int64_t at = (int64_t)id * a.hkv + w.seg_kvh;
                    return nthere ? make_float2(a.ks[at], a.vs[at]) : make_float2(1.0f, 0.0f);
                };
                auto copy = [&](int i, int ids, const CUtensorMap *map) {
                    const int id = __shfl_sync(0xffffffffu, ids, (i % NB) * PG + lane % PG);
                    const int y = (id * a.hkv + w.seg_kvh) * kPage;
                    const int slot = seq % C::SLOTS8;
                    const uint32_t use = seq / C::SLOTS8;
                    if (use > 0)
                        alive = __all_sync(0xffffffffu, mbar_wait(&empty8[slot], (use - 1) & 1, a.status, a.wait_ns));
                    if (!alive) return;
                    if (lane == 0) mbar_arrive_expect_tx(&full8[slot], C::SLOT8);
                    __syncwarp();
                    if (lane < PG) vtc::tma2d(scodes + slot * C::SLOT8 + lane * kPage * D, map, 0, y, &full8[slot]);
                    ++seq;
                };
                int cur = 0, nxt = load_ids(0);
                float2 sc{}, nsc = load_scales(nxt);
                for (int i = 0; i < w.seg_n && alive; ++i, ++blocks) {
                    if (i % NB == 0) {
                        cur = nxt;
                        sc = nsc;
                        nxt = load_ids(i + NB);
                    } else if (i % NB == NB / 2) {
                        nsc = load_scales(nxt);
                    }
                    const int from = (i % NB) * PG + lane % PG;
                    const float pk = __shfl_sync(0xffffffffu, sc.x, from), pv = __shfl_sync(0xffffffffu, sc.y, from);
                    if (lane < PG) scales[blocks % kScaleRing * PG + lane] = make_float2(scale_of(pk), scale_of(pv));
                    __syncwarp();
                    copy(i, cur, &a.kmap);
                    if (alive) copy(i, cur, &a.vmap);
                }
            }
            // no copy may be under way when the CTA ends
            for (uint32_t q = seq > C::SLOTS8 ? seq - C::SLOTS8 : 0; q < seq; ++q)
                if (!mbar_wait(&full8[q % C::SLOTS8], (q / C::SLOTS8) & 1, a.status, kWaitNs)) break;
        }
    } else if (warp == C::SM_WARPS + 1) {
        // ================= MMA issue (the warp in step, one elected thread; see tree_tc.cuh) =================
        const uint64_t qd0 = vtc::sdesc(smem_u32(sq), 16, 1024);
        const uint64_t kd0 = vtc::sdesc(smem_u32(skv), 16, 1024), vd0 = vtc::sdesc(smem_u32(skv), BK * 128, 1024);
        auto issue_s = [&](int t, uint32_t buf, uint32_t slot) {
            const uint64_t kd = kd0 + slot * (C::SLOT / 16), qd = qd0 + t * (C::QTILE / 16);
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
                const uint64_t ko = ((ks >> 2) * (BK * 128) + (ks & 3) * 32) / 16;
                tree::umma(tmem + buf * BK, qd + ((ks >> 2) * (kTileRows * 128) + (ks & 3) * 32) / 16, kd + ko, IQK, ks > 0);
            }
            tree::umma_commit(&s_ready[C::NBUF < QT ? t : buf]);
        };
        auto issue_pv = [&](int t, uint32_t buf, uint32_t slot, bool add) {
            const uint64_t vd = vd0 + slot * (C::SLOT / 16);
#pragma unroll
            for (int kk = 0; kk < BK / 16; ++kk)
                tree::umma_ta(tmem + C::O_COL0 + t * D, tmem + buf * BK + kk * 8, vd + kk * 16 * 128 / 16, IPV, add || kk > 0);
        };
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
        auto wait1 = [&](uint64_t *bar, uint32_t par) {
            alive = __all_sync(0xffffffffu, mbar_wait(bar, par, a.status, a.wait_ns));
            return alive;
        };
        auto wait = [&](bool p, bool v, bool k, int q) {
            if (p && q < 0 &&
                __all_sync(0xffffffffu, ready3(&p_ready[pp.i], pp.par, v ? &full[vp.i] : &p_ready[pp.i], v ? vp.par : pp.par,
                                               k ? &full[kp.i] : &p_ready[pp.i], k ? kp.par : pp.par))) {
                vtc::tc_fence_after();
                return true;
            }
            if (p && !wait1(&p_ready[pp.i], pp.par)) return false;
            if (v && !wait1(&full[vp.i], vp.par)) return false;
            if (k && !wait1(&full[kp.i], kp.par)) return false;
            if (q >= 0 && !wait1(&q_ready[q], seg & 1)) return false;
            vtc::tc_fence_after();
            return true;
        };
        auto next_s = [&](int t) {
            issue_s(t, sb, kp.i);
            if (++sb == C::NBUF) sb = 0;
            if (t == QT - 1) {
                tree::umma_commit(&empty[kp.i]);
                kp.step(2, C::SLOTS);
            }
        };
        for (;; ++seg) {
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
                    if (C::AHEAD) tree::umma_commit(&pv_done[t]);
                    if (more) next_s(t2);
                    if (j + 1 == n) tree::umma_commit(&o_done[t]);
                }
                if (!alive) break;
                tree::umma_commit(&empty[vp.i]);
                vp.step(2, C::SLOTS);
            }
        }
        // nor may a product be: TMEM is freed behind it
        tree::umma_commit(idle);
        mbar_wait(idle, 0, a.status, kWaitNs);
    } else if (warp >= C::SM_WARPS + 2) {
        // ================= conversion: half a block's rows each =================
        const int half = warp - (C::SM_WARPS + 2);
        uint32_t seq = 0;
        while (alive && w.next(a)) {
            for (int i = 0; i < 2 * w.seg_n && alive; ++i, ++seq) {
                const int slot = seq % C::SLOTS, slot8 = seq % C::SLOTS8;
                alive = __all_sync(0xffffffffu, mbar_wait(&full8[slot8], (seq / C::SLOTS8) & 1, a.status, a.wait_ns));
                if (alive && seq >= C::SLOTS)
                    alive = __all_sync(0xffffffffu, mbar_wait(&empty[slot], (seq / C::SLOTS - 1) & 1, a.status, a.wait_ns));
                if (!alive) break;
                const uint8_t *src = scodes + slot8 * C::SLOT8;
                uint8_t *dst = skv + slot * C::SLOT;
                // rows of V behind the request's end: whatever they hold, 0 times it is to be 0
                const int rows = i & 1 ? w.seg_len - (w.seg_blk + i / 2) * BK : BK;
                // eight lanes read and write different banks: with 128-byte rows of codes
                // half of one row and the other half of the next
                constexpr int IT = D / 64, U = 4;  // passes over eight rows; pieces under way
                constexpr int N = BK / 2 / 8 * IT;
                auto place = [&](int k, int &r, int &c) {
                    r = half * (BK / 2) + k / IT * 8 + (lane >> 2);
                    c = D == 128 ? (lane & 3) + 4 * ((r & 1) ^ (k & 1)) : lane & 3;
                };
#pragma unroll 1
                for (int k0 = 0; k0 < N; k0 += U) {
                    uint4 u[U];
#pragma unroll
                    for (int k = 0; k < U; ++k) {
                        int r, c;
                        place(k0 + k, r, c);
                        u[k] = *reinterpret_cast<const uint4 *>(src + piece_at<D>(r, c));
                    }
#pragma unroll
                    for (int k = 0; k < U; ++k) {
                        int r, c;
                        place(k0 + k, r, c);
                        uint4 lo, hi;
                        widen<E4M3>(u[k], lo, hi);
                        if (r >= rows) lo = hi = make_uint4(0, 0, 0, 0);
                        *reinterpret_cast<uint4 *>(dst + vtc::sw128(r, 2 * c, BK)) = lo;
                        *reinterpret_cast<uint4 *>(dst + vtc::sw128(r, 2 * c + 1, BK)) = hi;
                    }
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&full[slot]);
                    mbar_arrive(&empty8[slot8]);
                }
            }
        }
    } else {
        // ================= softmax: one thread per row =================
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::REGS_SOFTMAX));
        const int t = warp >> 2;
        const int r = (warp & 3) * 32 + lane;  // row within the tile = TMEM lane
        const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t t_o = tmem + lane_base + C::O_COL0 + t * D;
        const int rg = (tile0 + t) * kTileRows + r;
        const bool rvalid = rg < a.rows;
        const bool any_row = (tile0 + t) * kTileRows + (warp & 3) * 32 < a.rows;  // of the warp's
        const int qi = rvalid ? rg / a.grp : 0, qn = rvalid ? rg % a.grp : 0;
        // the warp's 32 rows x 8 pieces of 16 bytes, on their way between a thread's
        // own row and eight neighbouring lanes a row: the warp's own rows of Q, which
        // are done with by then
        uint4 *stage = reinterpret_cast<uint4 *>(sq + t * C::QTILE + (warp & 3) * 4096);
        const int srow = lane >> 3, spc = lane & 7;  // row (of 4 at a time) and piece
        auto at = [&](int row, int piece) { return stage + row * 8 + (piece ^ (row & 7)); };
        uint32_t it = 0, seg = 0;  // blocks and segments of this chain
        for (; w.next(a); ++seg) {
            const int base = w.seg_len - a.n_q;
            const int64_t orow = ((int64_t)w.seg_b * a.n_q + qi) * a.hq + (int64_t)w.seg_kvh * a.grp + qn;
            const unsigned long long mask = rvalid ? mask_of(a, w.seg_b, qi) : 0;
            float rf = 0.0f;  // this row's factor beside K's scale
            if (alive) {
                // the warp's rows of Q, 64 channels at a time
                uint4 u[D / 64][8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int64_t ro = __shfl_sync(0xffffffffu, rvalid ? orow : (int64_t)-1, i * 4 + srow);
                    const uint4 *src = reinterpret_cast<const uint4 *>(a.q + ro * D) + spc;
                    uint32_t mx = 0;
#pragma unroll
                    for (int h = 0; h < D / 64; ++h) {
                        u[h][i] = ro >= 0 ? src[h * 8] : make_uint4(0, 0, 0, 0);
                        mx = __vmaxu2(mx, __vmaxu2(u[h][i].x & 0x7fff7fffu, u[h][i].y & 0x7fff7fffu));
                        mx = __vmaxu2(mx, __vmaxu2(u[h][i].z & 0x7fff7fffu, u[h][i].w & 0x7fff7fffu));
                    }
                    mx = max(mx & 0xffffu, mx >> 16);
#pragma unroll
                    for (int o = 1; o < 8; o <<= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                    const int e = q_exponent(bf16_bits_to_f32((uint16_t)mx));
                    const float up = exp2i(e);
#pragma unroll
                    for (int h = 0; h < D / 64; ++h) {
                        uint32_t *x = reinterpret_cast<uint32_t *>(&u[h][i]);
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            x[j] = pack_f16(__uint_as_float(x[j] << 16) * up, __uint_as_float(x[j] & 0xffff0000u) * up);
                    }
                    const int mine_e = __shfl_sync(0xffffffffu, e, (lane & 3) * 8);
                    if (lane >> 2 == i) rf = a.scale_log2 * exp2i(-mine_e);
                }
#pragma unroll
                for (int h = 0; h < D / 64; ++h) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        *reinterpret_cast<uint4 *>(
                            sq + t * C::QTILE + vtc::sw128((warp & 3) * 32 + i * 4 + srow, h * 8 + spc, kTileRows)) = u[h][i];
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                vtc::tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&q_ready[t]);
            }
            float m_used = -INFINITY, l = 0.0f, vref = 0.0f, inv_vref = 0.0f;
            // tcgen05.ld / st are warp-collective: every lane runs them together
            for (int j = 0; j < w.seg_n && alive; ++j, ++it) {
                const uint32_t step = it * QT + t, buf = step % C::NBUF, t_s = tmem + lane_base + buf * BK;
                alive = __all_sync(0xffffffffu, mbar_wait(&s_ready[C::NBUF < QT ? t : buf],
                                                          (C::NBUF < QT ? it : step / C::NBUF) & 1, a.status, a.wait_ns));
                if (!alive) break;
                if (!any_row) {  // (what P holds in rows that are not there goes nowhere)
                    if (lane == 0) mbar_arrive(&p_ready[buf]);
                    continue;
                }
                vtc::tc_fence_after();
                float s[BK];
#pragma unroll
                for (int h = 0; h < BK / 64; ++h)
                    vtc::tmem_ld_row<64>(t_s + 64 * h, *reinterpret_cast<float(*)[64]>(&s[64 * h]));
                const int key0 = (w.seg_blk + j) * BK;
                if (key0 + BK > base) {
#pragma unroll
                    for (int h = 0; h < BK / 64; ++h) {
                        const unsigned long long seen = tree::seen_bits(mask, key0 + 64 * h, base);
#pragma unroll
                        for (int c = 0; c < 64; ++c)
                            if (!((seen >> c) & 1)) s[64 * h + c] = -INFINITY;
                    }
                }
                const float2 *sc = scales + it % kScaleRing * PG;
                float mb = -INFINITY, vtop = 0.0f;
#pragma unroll
                for (int p = 0; p < PG; ++p) {
                    const float2 f = sc[p];
                    const float kf = factor_of(f.x, rf);
                    mb = fmaxf(mb, tree::max_of<16>(*reinterpret_cast<float(*)[16]>(&s[16 * p])) * kf);
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
                    if (j > 0) {
                        if constexpr (C::AHEAD) {
                            alive = __all_sync(0xffffffffu, mbar_wait(&pv_done[t], (it - 1) & 1, a.status, a.wait_ns));
                            if (!alive) break;
                            vtc::tc_fence_after();
                        }
#pragma unroll 1
                        for (int c0 = 0; c0 < D; c0 += 16) {
                            float v[16];
                            vtc::tmem_ld16(t_o + c0, v);
#pragma unroll
                            for (int i = 0; i < 16; ++i) v[i] *= f;
                            vtc::tmem_st16(t_o + c0, v);
                        }
                    }
                }
                if (grow) m_used = mb - kBelow;
                const float nms = m_used == -INFINITY ? 0.0f : -m_used;
                float ls[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int h = 0; h < BK / 32; ++h) {
                    float pk[16];
#pragma unroll
                    for (int p = 0; p < 2; ++p) {
                        const float2 f = sc[2 * h + p];
                        const float kf = factor_of(f.x, rf), vw = f.y * inv_vref;
#pragma unroll
                        for (int c = 8 * p; c < 8 * p + 8; ++c) {
                            float p0, p1;
                            tree::fma2(p0, p1, s[h * 32 + 2 * c], s[h * 32 + 2 * c + 1], kf, nms);
                            p0 = ex2(p0);
                            p1 = ex2(p1);
                            tree::add2(ls[(2 * c) & 2], ls[((2 * c) & 2) + 1], p0, p1);
                            mul2(p0, p1, vw);
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
            if (alive)
                alive = __all_sync(0xffffffffu, mbar_wait(&o_done[t], seg & 1, a.status, a.wait_ns));
            // ---- the segment's result (the rows' states as in kv8_few.cuh) ----
            if (alive) vtc::tc_fence_after();
            const bool zero = !alive || mask == 0 || (m_used == -INFINITY && l == 0.0f);
            const int64_t prow = ((int64_t)blockIdx.x * 2 + !w.at_start) * C::ROWS + t * kTileRows + r;
            const float f = zero ? 0.0f : vref / l;
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
            if (any_row) {
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
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
}

}  // namespace kv8
}  // namespace vc
