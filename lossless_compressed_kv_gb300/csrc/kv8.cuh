// What the kernels over an 8-bit cache share: arguments, codes as fp16, the
// join of partial results.
//
//   out[i] = sum_t softmax_t(scale <q_i, sk_t ck_t>) sv_t cv_t
// Both codes are exact in fp16 (e4m3 by definition, whole numbers up to 127),
// so the products run on codes and the scales stand outside: K's beside the
// softmax scale, a factor a page, and V's beside the probability.  A
// probability times V's scale goes to fp16 relative to a reference that is
// twice the largest scale met so far, and the probability relative to one that
// lies 2^8 to 2^16 below the largest (kBelow, kRise): stored values reach 2^15,
// of fp16's 2^16, and the largest is at least 2^7, so one of which that is off by
// half the smallest step, 2^-25, is off by at most 2^-32 of the largest beside
// V's largest scale.  Q is bf16 and goes to
// fp16 by a power of two that puts a row's largest value at 2^8: what lies
// within 2^25 of it keeps all its bits.
//
// Work split: as in tree_tc.cuh, the blocks of all units (request, kv head)
// laid end to end and dealt out in equal ranges.  A unit that lies in one
// range is finished there, one that spans several leaves a partial (m, l,
// o / l) in each: at most two a range, its first and its last.
#pragma once

#include "tree_tc.cuh"

namespace vc {
namespace kv8 {

struct Args {
    const uint8_t *kc, *vc;  // codes [pages][kv heads][16][D]
    CUtensorMap kmap, vmap;  // the same for the TMA unit, a head block of a page a box (more than 128 rows)
    const float *ks, *vs;    // [pages][kv heads]
    const uint16_t *q;     // [B][n_q][Hq][D]
    int64_t n_pages;
    const int32_t *table, *lens;
    const unsigned long long *mask;  // [B][n_q] or null: causal
    int batch, maxb, n_q, hq, hkv, grp, max_len;
    int rows;    // of a unit
    int lanes;   // row chunks: each walks all ranges
    int groups;  // ranges
    float scale_log2;
    float *ws_o;   // [range][lane][2][rows of a lane][D]
    float *ws_ml;  // [range][lane][2][rows of a lane][2]
    void *out;
    int out_bf16;
    int32_t *status;
    uint64_t wait_ns;
    int skip_copies;
};

// Two codes (the low or the high half of a register) as fp16 pairs.
template <bool E4M3>
__device__ __forceinline__ uint32_t to_f16_lo(uint32_t w) {
    uint32_t d;
    if constexpr (E4M3) {
        asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(d) : "r"(w));
    } else {  // (w holds codes + 128: 1024 + 128 + code, less 1152)
        d = __byte_perm(w, 0x64646464u, 0x5140);
        asm("sub.f16x2 %0, %0, %1;" : "+r"(d) : "r"(0x64806480u));
    }
    return d;
}
template <bool E4M3>
__device__ __forceinline__ uint32_t to_f16_hi(uint32_t w) {
    uint32_t d;
    if constexpr (E4M3) {
        asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}" : "=r"(d) : "r"(w));
    } else {
        d = __byte_perm(w, 0x64646464u, 0x5342);
        asm("sub.f16x2 %0, %0, %1;" : "+r"(d) : "r"(0x64806480u));
    }
    return d;
}
// Codes as to_f16_lo / hi take them.
template <bool E4M3>
__device__ __forceinline__ uint32_t raw(uint32_t w) {
    return E4M3 ? w : w ^ 0x80808080u;
}

// A row's reference for its probabilities 2^(score - reference): set kBelow below
// the largest score met, and again once one lies kRise above it.
constexpr float kBelow = 8.0f, kRise = 16.0f;

// A scale, or the nearer end of what scales may be (NaN: the lower).
__device__ __forceinline__ float scale_of(float s) { return fminf(fmaxf(s, 0x1p-126f), 0x1p122f); }

// A row's factor beside K's scale, kept finite (a score of 0 stays 0) and not 0
// (it meets the masked scores' infinity; 2^-126 more moves no score by 2^-100).
__device__ __forceinline__ float factor_of(float k_scale, float rf) { return fminf(fmaf(k_scale, rf, 0x1p-126f), 0x1p127f); }

// The power of two that takes a row whose largest magnitude is `amax` to 2^8.
__device__ __forceinline__ int q_exponent(float amax) {
    const int e = (int)(__float_as_uint(amax) >> 23 & 255) - 127;
    return 8 - max(e, -110);
}
__device__ __forceinline__ float exp2i(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// Row i's bits of the block.
__device__ __forceinline__ unsigned long long mask_of(const Args &a, int b, int i) {
    return a.mask ? a.mask[(int64_t)b * a.n_q + i] & (~0ull >> (64 - a.n_q)) : ~0ull >> (63 - i);
}

// Warps that share a row of a unit of so many ranges: one reads eight at once.
__host__ __device__ inline int join_warps(int ranges) { return ranges < 8 ? 1 : ranges < 16 ? 2 : ranges < 32 ? 4 : 8; }

// Join the partials of units that span several ranges, and write zeros for
// requests that are refused.  A unit's blocks (gridDim.y) go through its rows,
// W warps to a row, each of which takes every W-th range, eight partials read
// at once.  W follows from the unit's own ranges, so the order of the sums is
// fixed by the lengths alone: not by the bound that the call is given for
// them, from which the grid follows.
constexpr int kJoinWarps = 8;
template <int D, int BK>
__device__ __forceinline__ void join_block(const Args &a, int lane_rows) {
    constexpr int E = D / 32, U = 8;
    __shared__ float part[kJoinWarps][E + 2][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int unit = blockIdx.x, b = unit / a.hkv, kvh = unit % a.hkv;
    const int nblk = tree::blocks_of<BK>(a, b);
    if (nblk == 0 && threadIdx.x == 0 && kvh == 0 && blockIdx.y == 0 && a.lens[b] != 0)
        report(a.status, VC_ERR_BAD_INDEX);
    int total, before;
    tree::sum_blocks<BK>(a, b, lane, total, before);
    const tree::Deal deal(total * a.hkv, a.groups);
    const int u0 = before * a.hkv + kvh * nblk;
    const int g0 = nblk > 0 ? deal.group_of(u0) : 0, g1 = nblk > 0 ? deal.group_of(u0 + nblk - 1) : -1;
    if (nblk > 0 && g0 == g1) return;  // finished there
    const int W = join_warps(g1 - g0 + 1), per = kJoinWarps / W;
#pragma unroll 1
    for (int row0 = blockIdx.y * per; row0 < a.rows; row0 += gridDim.y * per) {
        const int rg = row0 + warp / W;
        const bool row_ok = rg < a.rows;
        const int rlane = rg / lane_rows, trow = rg % lane_rows;
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
                        const int64_t pr = ((int64_t)(g * a.lanes + rlane) * 2 + (u0 > deal.start(g))) * lane_rows + trow;
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
                    if (m[k] == -INFINITY) continue;  // (nothing seen there)
                    const float wk = ex2(m[k] - mx) * l[k];
                    L += wk;
#pragma unroll
                    for (int i = 0; i < E; ++i) acc[i] = fmaf(wk, o[k][i], acc[i]);
                }
            }
        }
        if (W > 1) {
            __syncthreads();  // (the rows before have been read)
            part[warp][0][lane] = M;
            part[warp][1][lane] = lost ? -1.0f : L;
#pragma unroll
            for (int i = 0; i < E; ++i) part[warp][2 + i][lane] = acc[i];
            __syncthreads();
            if (warp % W) continue;
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
        if (!row_ok) continue;
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
}

}  // namespace kv8
}  // namespace vc
