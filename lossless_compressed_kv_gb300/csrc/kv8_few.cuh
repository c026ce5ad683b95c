// Attention over an 8-bit cache for few rows (a row: one query token and one
// query head of the kv head's group): drafting steps and short blocks, which
// the cache's bytes bound.
//
// Every warp walks a range of its own, page by page, through a ring of pages
// that it fills itself by asynchronous copies of 16 bytes a lane: no barrier
// joins warps, so their loads, products and exponentials overlap freely.  (By
// TMA, a head block of a page a copy, 8 x 32768 keys took 98 us, and 60 with
// head_dim 64: the SM's TMA unit takes such small copies too slowly.)
// Per page, on mma.sync with 16 keys or channels as M:
//   S^T = K Q^T      16 keys x 8 rows, D / 16 steps
//   O^T += V^T P^T   D / 16 tiles of 16 channels x 8 rows
// With few rows the 128-row instructions of tcgen05 would spend their time on
// rows that are not there (kv8_one.cuh takes 155 us for four rows), while these
// spend an instruction on 128 codes.
// 8 x 32768 keys, 8 heads of 128: 4 rows 98 us (0.81 of measured HBM), 16 rows
// 112; 4 x 131072 keys, 8 rows 181 (0.88).  Chains of shared-memory loads,
// products and conversions bound it: a scheduler's four warps issue in 0.45 of the
// cycles.
//
// A product of K and Q may take channels in any order, if both take the same:
// a lane reads 16-byte pieces of a key's row and feeds four channels of them
// to a step as they lie.  For V^T a lane holds two (and two) keys' pieces and
// pairs them up byte by byte before the conversion.  The pieces that eight
// lanes read together lie in different banks (the swizzle moves a row's pieces
// by the row's number).
#pragma once

#include "kv8.cuh"

namespace vc {
namespace kv8 {

template <int D, int NT>
struct Few {
    static constexpr int WARPS = 4;                 // of a CTA
    static constexpr int CTAS = NT == 1 ? 4 : NT == 2 ? 3 : 2;  // an SM holds
    static constexpr int TILE = kPage * D;          // a head block of codes
    static constexpr int STAGE = 2 * TILE;
    static constexpr int ROOM = (228 * 1024 / CTAS - 1024) / WARPS / (STAGE + 8);
    static constexpr int STAGES = ROOM < 8 ? ROOM : 8;
    static_assert(STAGES >= 3, "ring depth");
    static constexpr int OFF_SC = WARPS * STAGES * STAGE;
    static constexpr int SMEM = OFF_SC + WARPS * STAGES * 8;
    static_assert(CTAS * (SMEM + 1024) <= 228 * 1024, "shared memory of the CTAs an SM holds");
    static constexpr int ROWS = 8 * NT;
    static constexpr int THREADS = WARPS * 32;
};

// The 16-byte piece c of a block's row r, as the copy places it.
template <int D>
__device__ __forceinline__ int piece_at(int r, int c) {
    return D == 128 ? r * 128 + ((c ^ (r & 7)) << 4) : r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}

template <int D, int NT, bool E4M3>
__device__ __forceinline__ void few_warp(const Args &a, uint8_t *smem) {
    using F = Few<D, NT>;
    constexpr int KS = D / 16;       // steps of S, tiles of O
    constexpr int BK = kPage;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int range = blockIdx.x * F::WARPS + warp;
    uint8_t *ring = smem + warp * F::STAGES * F::STAGE;
    float2 *scales = reinterpret_cast<float2 *>(smem + F::OFF_SC) + warp * F::STAGES;
    if (range >= a.groups) return;
    int total, before, b0 = 0, rest = 0;
    tree::sum_blocks<BK>(a, 0, lane, total, before);
    const tree::Deal deal(total * a.hkv, a.groups);
    const int f0 = deal.start(range), mine = deal.start(range + 1) - f0;
    if (mine <= 0) return;
    tree::find_block<BK>(a, f0, lane, b0, rest);

    // ---- the copies, STAGES pages ahead ----
    tree::Walk<BK> iw;
    iw.begin(a, b0, rest, mine);
    int fill = 0, use = 0;  // stages next filled and used
    int ii = 0, in = 0;  // place in the segment whose pages are being issued
    // ids and scales of 32 pages, a lane each; the ids are read a batch ahead
    int id_next = 0, id = 0;
    float ks = 0.0f, vs = 0.0f;
    auto load_ids = [&](int i0) {
        const int i = i0 + lane, pidx = iw.seg_blk + i;
        int p = 0;
        if (i < iw.seg_n) {
            p = pidx < a.maxb ? a.table[(int64_t)iw.seg_b * a.maxb + pidx] : -1;
            if (p < 0 || p >= a.n_pages) {
                report(a.status, VC_ERR_BAD_INDEX);
                p = 0;
            }
        }
        return p;
    };
    // (a group of copies each time, so that what is under way is counted in pages)
    auto issue = [&]() {
        if (ii < in || iw.next(a)) {
            if (ii == in) {
                ii = 0;
                in = iw.seg_n;
                id_next = load_ids(0);
            }
            if (ii % 32 == 0) {
                id = id_next;
                const int64_t at = (int64_t)id * a.hkv + iw.seg_kvh;
                ks = a.ks[at];
                vs = a.vs[at];
                id_next = load_ids(ii + 32);
            }
            const int p = __shfl_sync(0xffffffffu, id, ii % 32);
            const float pk = __shfl_sync(0xffffffffu, ks, ii % 32), pv = __shfl_sync(0xffffffffu, vs, ii % 32);
            ++ii;
            if (lane == 0) scales[fill] = make_float2(scale_of(pk), scale_of(pv));
            const int64_t from = ((int64_t)p * a.hkv + iw.seg_kvh) * F::TILE;
            uint8_t *to = ring + fill * F::STAGE;
#pragma unroll
            for (int e = lane; e < F::TILE / 16; e += 32) {
                const int off = piece_at<D>(e / (D / 16), e % (D / 16));
                cp_async16(to + off, a.kc + from + e * 16);
                cp_async16(to + F::TILE + off, a.vc + from + e * 16);
            }
            if (++fill == F::STAGES) fill = 0;
        }
        cp_async_commit();
    };
#pragma unroll 1
    for (int i = 0; i < F::STAGES; ++i) issue();

    tree::Walk<BK> w;
    w.begin(a, b0, rest, mine);
    while (w.next(a)) {
        const int base = w.seg_len - a.n_q;
        // ---- the unit's rows: this lane's share of Q, as the second operand's fragments ----
        uint32_t qf[NT][KS][2];
        float rf[NT][2], m[NT][2], l[NT][2], acc[NT][KS][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int r = n * 8 + g;
            uint32_t u[KS * 2];
            if (r < a.rows) {
                const int64_t row = ((int64_t)w.seg_b * a.n_q + r / a.grp) * a.hq + w.seg_kvh * a.grp + r % a.grp;
                const uint4 *src = reinterpret_cast<const uint4 *>(a.q + row * D + t * (D / 4));
#pragma unroll
                for (int j = 0; j < KS / 2; ++j) *reinterpret_cast<uint4 *>(&u[4 * j]) = src[j];
            } else {
#pragma unroll
                for (int j = 0; j < KS * 2; ++j) u[j] = 0;
            }
            uint32_t mx = 0;  // (magnitudes of bf16 compare as whole numbers)
#pragma unroll
            for (int j = 0; j < KS * 2; ++j) mx = __vmaxu2(mx, u[j] & 0x7fff7fffu);
            mx = max(mx & 0xffffu, mx >> 16);
            mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            const int e = q_exponent(bf16_bits_to_f32((uint16_t)mx));
            const float up = exp2i(e);
#pragma unroll
            for (int j = 0; j < KS * 2; ++j)
                qf[n][j / 2][j % 2] = pack_f16(__uint_as_float(u[j] << 16) * up, __uint_as_float(u[j] & 0xffff0000u) * up);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                rf[n][c] = a.scale_log2 * exp2i(-__shfl_sync(0xffffffffu, e, 8 * t + 4 * c));
                m[n][c] = -INFINITY;
                l[n][c] = 0.0f;
            }
#pragma unroll
            for (int j = 0; j < KS; ++j)
#pragma unroll
                for (int c = 0; c < 4; ++c) acc[n][j][c] = 0.0f;
        }
        float vref = 0.0f, inv_vref = 0.0f;
#pragma unroll 1
        for (int i = 0; i < w.seg_n; ++i) {
            cp_async_wait<F::STAGES - 1>();
            __syncwarp();
            uint8_t *kt = ring + use * F::STAGE, *vt = kt + F::TILE;
            const float2 sc2 = scales[use];
            if (++use == F::STAGES) use = 0;
            const int key0 = (w.seg_blk + i) * BK;
            // rows of V behind the request's end: whatever they hold, 0 times it is to be 0
            const bool ends = key0 + BK > w.seg_len;
            if (ends) {
                for (int e = lane + (w.seg_len - key0) * (D / 16); e < kPage * (D / 16); e += 32)
                    *reinterpret_cast<uint4 *>(vt + e * 16) = make_uint4(0, 0, 0, 0);  // (a row's pieces stay in the row)
                __syncwarp();
            }
            // ---- S^T ----
            float x[NT][4];
            {
                uint32_t ka[2][KS];  // keys g and g + 8: four channels a step
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int c = 0; c < D / 64; ++c) {
                        const uint4 u = *reinterpret_cast<const uint4 *>(kt + piece_at<D>(g + 8 * h, t * (D / 64) + c));
                        ka[h][4 * c] = raw<E4M3>(u.x);
                        ka[h][4 * c + 1] = raw<E4M3>(u.y);
                        ka[h][4 * c + 2] = raw<E4M3>(u.z);
                        ka[h][4 * c + 3] = raw<E4M3>(u.w);
                    }
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int c = 0; c < 4; ++c) x[n][c] = 0.0f;
#pragma unroll
                for (int j = 0; j < KS; ++j) {
                    const uint32_t f[4] = {to_f16_lo<E4M3>(ka[0][j]), to_f16_lo<E4M3>(ka[1][j]), to_f16_hi<E4M3>(ka[0][j]),
                                           to_f16_hi<E4M3>(ka[1][j])};
#pragma unroll
                    for (int n = 0; n < NT; ++n) mma_f16(x[n], f, qf[n][j][0], qf[n][j][1]);
                }
            }
            // ---- softmax: rows 2t, 2t + 1 of each eight, keys g and g + 8 ----
            bool grow = sc2.y > vref;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int c = 0; c < 4; ++c) x[n][c] *= factor_of(sc2.x, rf[n][c & 1]);
            if (key0 + BK > base) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const int r = n * 8 + 2 * t + c;
                        const unsigned long long seen =
                            r < a.rows ? tree::seen_bits(mask_of(a, w.seg_b, r / a.grp), key0, base) : 0ull;
                        if (!((seen >> g) & 1)) x[n][c] = -INFINITY;
                        if (!((seen >> (g + 8)) & 1)) x[n][c + 2] = -INFINITY;
                    }
            }
            // (the reference of a row's maximum follows only rises beyond kRise)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int c = 0; c < 4; ++c) grow |= x[n][c] > m[n][c & 1] + kRise;
            if (__any_sync(0xffffffffu, grow)) {
                // V's reference: twice the largest scale so far
                float fv = 1.0f;
                if (sc2.y > vref) {
                    inv_vref = 0.5f / sc2.y;
                    fv = vref * inv_vref;
                    vref = 2.0f * sc2.y;
                }
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float mx = fmaxf(x[n][c], x[n][c + 2]);
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                        float f = 1.0f;
                        if (mx > m[n][c] + kRise) {
                            mx -= kBelow;
                            f = ex2(m[n][c] - mx);
                            m[n][c] = mx;
                        }
                        l[n][c] *= f;
                        f *= fv;
#pragma unroll
                        for (int j = 0; j < KS; ++j) {
                            acc[n][j][c] *= f;
                            acc[n][j][c + 2] *= f;
                        }
                    }
            }
            const float vw = sc2.y * inv_vref;
            uint32_t pf[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float p[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) p[c] = ex2(x[n][c] - (m[n][c & 1] == -INFINITY ? 0.0f : m[n][c & 1]));
                l[n][0] += p[0] + p[2];
                l[n][1] += p[1] + p[3];
                pf[n][0] = movmatrix_t(pack_f16(p[0] * vw, p[1] * vw));
                pf[n][1] = movmatrix_t(pack_f16(p[2] * vw, p[3] * vw));
            }
            // ---- O^T: this lane's D / 8 channels of keys 2t, 2t + 1 and 8 behind ----
            {
                constexpr int W = D / 32;  // words of a row
                uint32_t va[4][W];
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    const int r = 2 * t + (h & 1) + 8 * (h >> 1);
                    if constexpr (D == 128) {
                        const uint4 u = *reinterpret_cast<const uint4 *>(vt + piece_at<D>(r, g));
                        va[h][0] = u.x; va[h][1] = u.y; va[h][2] = u.z; va[h][3] = u.w;
                    } else {
                        const uint2 u = *reinterpret_cast<const uint2 *>(vt + piece_at<D>(r, g >> 1) + (g & 1) * 8);
                        va[h][0] = u.x; va[h][1] = u.y;
                    }
                }
#pragma unroll
                for (int j = 0; j < W; ++j) {
                    // pairs of keys, channels 4j and 4j + 1, then 4j + 2 and 4j + 3
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const uint32_t lo = raw<E4M3>(__byte_perm(va[0][j], va[1][j], c ? 0x7362 : 0x5140));
                        const uint32_t hi = raw<E4M3>(__byte_perm(va[2][j], va[3][j], c ? 0x7362 : 0x5140));
                        const uint32_t f[4] = {to_f16_lo<E4M3>(lo), to_f16_hi<E4M3>(lo), to_f16_lo<E4M3>(hi),
                                               to_f16_hi<E4M3>(hi)};
#pragma unroll
                        for (int n = 0; n < NT; ++n) mma_f16(acc[n][2 * j + c], f, pf[n][0], pf[n][1]);
                    }
                }
            }
            __syncwarp();
            issue();
        }
        // ---- the segment's result ----
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float ls = l[n][c];
                ls += __shfl_xor_sync(0xffffffffu, ls, 4);
                ls += __shfl_xor_sync(0xffffffffu, ls, 8);
                ls += __shfl_xor_sync(0xffffffffu, ls, 16);
                const int r = n * 8 + 2 * t + c;
                if (r >= a.rows) continue;
                // a row that is left out or saw no key: zeros (m = -infinity); one
                // that met a NaN: NaN (m = +infinity, which no other range outweighs)
                const bool zero = mask_of(a, w.seg_b, r / a.grp) == 0 || (m[n][c] == -INFINITY && ls == 0.0f);
                const float f = zero ? 0.0f : vref / ls;
                const int64_t orow = ((int64_t)w.seg_b * a.n_q + r / a.grp) * a.hq + w.seg_kvh * a.grp + r % a.grp;
                const int64_t prow = ((int64_t)range * 2 + !w.at_start) * F::ROWS + r;
                float o[D / 8];
#pragma unroll
                for (int j = 0; j < KS; ++j) {
                    o[2 * j] = zero ? 0.0f : acc[n][j][c] * f;
                    o[2 * j + 1] = zero ? 0.0f : acc[n][j][c + 2] * f;
                }
                if (w.whole && a.out_bf16) {
                    uint4 *dst = reinterpret_cast<uint4 *>((uint16_t *)a.out + orow * D + g * (D / 8));
#pragma unroll
                    for (int j = 0; j < D / 64; ++j)
                        dst[j] = make_uint4(pack_bf16(o[8 * j], o[8 * j + 1]), pack_bf16(o[8 * j + 2], o[8 * j + 3]),
                                            pack_bf16(o[8 * j + 4], o[8 * j + 5]), pack_bf16(o[8 * j + 6], o[8 * j + 7]));
                } else {
                    float4 *dst = reinterpret_cast<float4 *>((w.whole ? (float *)a.out + orow * D : a.ws_o + prow * D) + g * (D / 8));
#pragma unroll
                    for (int j = 0; j < D / 32; ++j) dst[j] = make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
                }
                if (!w.whole && g == 0) {
                    a.ws_ml[prow * 2] = zero ? -INFINITY : ls != ls ? INFINITY : m[n][c];
                    a.ws_ml[prow * 2 + 1] = zero ? 0.0f : ls;
                }
            }
    }
    cp_async_wait<0>();
}

}  // namespace kv8
}  // namespace vc
