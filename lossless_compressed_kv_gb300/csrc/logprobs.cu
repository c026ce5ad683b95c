// vc_token_logprobs: log probabilities of given tokens, entropy and the most
// probable alternatives of rows of logits.
//
//   y_v = (x_v - M) / tau,  M = max x
//   log p_v = y_v - log S,  entropy = log S - (sum_v y_v e^y_v) / S
// with S = c + R: c the number of logits equal to the maximum (each adds
// exactly 1), R the sum of the others, log S = log c + log1p(R / c).
#include <cmath>

#include "vc_internal.cuh"

namespace vc {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

// 16 bytes of logits: VEC of them, as they lie in memory.
template <typename T>
struct Pack;
template <>
struct Pack<float> {
    static constexpr int VEC = 4;
    using Word = uint32_t;
    static constexpr uint32_t kNone = 0xff800000u;  // words of -infinity
    __device__ static float one(const float *p) { return *p; }
    __device__ static float of(Word w) { return __uint_as_float(w); }
    __device__ static void unpack(const uint4 &u, float (&v)[4]) {
        v[0] = __uint_as_float(u.x); v[1] = __uint_as_float(u.y);
        v[2] = __uint_as_float(u.z); v[3] = __uint_as_float(u.w);
    }
    __device__ static float max_of(const uint4 &u);
};
// (NaN wins)
__device__ inline float max_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}
__device__ inline float max_nan(float a, float b, float c) {
    float d;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ inline float Pack<float>::max_of(const uint4 &u) {
    return max_nan(max_nan(__uint_as_float(u.x), __uint_as_float(u.y), __uint_as_float(u.z)), __uint_as_float(u.w));
}
template <>
struct Pack<__nv_bfloat16> {
    static constexpr int VEC = 8;
    using Word = uint16_t;
    static constexpr uint32_t kNone = 0xff80ff80u;
    __device__ static float one(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
    __device__ static float of(Word w) { return __uint_as_float((uint32_t)w << 16); }
    __device__ static void unpack(const uint4 &u, float (&v)[8]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    __device__ static float max_of(const uint4 &u) {
        uint32_t a;
        asm("{\n\t.reg .b32 p, q;\n\tmax.NaN.bf16x2 p, %1, %2;\n\tmax.NaN.bf16x2 q, %3, %4;\n\t"
            "max.NaN.bf16x2 %0, p, q;\n\t}"
            : "=r"(a)
            : "r"(u.x), "r"(u.y), "r"(u.z), "r"(u.w));
        return max_nan(__uint_as_float(a << 16), __uint_as_float(a & 0xffff0000u));
    }
};
template <>
struct Pack<__half> {
    static constexpr int VEC = 8;
    using Word = uint16_t;
    static constexpr uint32_t kNone = 0xfc00fc00u;
    __device__ static float one(const __half *p) { return __half2float(*p); }
    __device__ static float of(Word w) { return __half2float(__ushort_as_half(w)); }
    __device__ static void unpack(const uint4 &u, float (&v)[8]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    }
    __device__ static float max_of(const uint4 &u) {
        uint32_t a;
        asm("{\n\t.reg .b32 p, q;\n\tmax.NaN.f16x2 p, %1, %2;\n\tmax.NaN.f16x2 q, %3, %4;\n\t"
            "max.NaN.f16x2 %0, p, q;\n\t}"
            : "=r"(a)
            : "r"(u.x), "r"(u.y), "r"(u.z), "r"(u.w));
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&a));
        return max_nan(f.x, f.y);
    }
};

// Order-preserving key: value bits mapped to an unsigned order in the high
// word (-0 folded onto +0 first), the complement of the id in the low word.
__device__ inline uint32_t order_bits(float v) {
    const uint32_t b = __float_as_uint(v + 0.0f);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ inline float order_value(uint32_t o) {
    return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}
__device__ inline unsigned long long order_key(float v, int id) {
    return ((unsigned long long)order_bits(v) << 32) | (uint32_t)~(uint32_t)id;
}
// Two values in one packed instruction, each rounded as its scalar form.
__device__ inline void fma2(float &d0, float &d1, float a0, float a1, float b, float c) {  // a b + c
    asm("{\n\t.reg .b64 ra, rb, rc;\n\t"
        "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %4};\n\tmov.b64 rc, {%5, %5};\n\t"
        "fma.rn.f32x2 ra, ra, rb, rc;\n\tmov.b64 {%0, %1}, ra;\n\t}"
        : "=f"(d0), "=f"(d1)
        : "f"(a0), "f"(a1), "f"(b), "f"(c));
}
__device__ inline void acc2(float &d0, float &d1, float a0, float a1) {  // d + a
    asm("{\n\t.reg .b64 ra, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rd, {%0, %1};\n\t"
        "add.rn.f32x2 rd, rd, ra;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "+f"(d0), "+f"(d1)
        : "f"(a0), "f"(a1));
}
__device__ inline void facc2(float &d0, float &d1, float a0, float a1, float b0, float b1) {  // d + a b
    asm("{\n\t.reg .b64 ra, rb, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\tmov.b64 rd, {%0, %1};\n\t"
        "fma.rn.f32x2 rd, ra, rb, rd;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "+f"(d0), "+f"(d1)
        : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}

struct LpArgs {
    const void *x;
    int64_t stride;
    int rows, vocab;
    int parts, part_len;  // a row in parts of part_len logits (a multiple of a pack)
    unsigned long long *ws;  // parts > 1: per part {m, c}, {r, t}, number of keys, the keys
    const int32_t *ids;
    int n_ids, k;
    float inv_tau;
    float *lp, *ent;
    int32_t *top_ids;
    float *top_lp;
    int32_t *status;
    uint64_t wait_ns;
    int skip_copies;
};

// What a row's logits amount to: the maximum, how many logits equal it, the
// sum of the others' e^y, and the sum of y e^y.
struct Stats {
    float m, c, r, t;
};

// Outputs of row `row`, given its statistics and its `have` largest keys, by
// one warp.  The first 32 tokens asked for and their logits come in registers.
template <typename T>
__device__ void finish_row(const LpArgs &a, int64_t row, Stats s, const unsigned long long *top, int have, int lane,
                           int id, typename Pack<T>::Word raw) {
    float logit = Pack<T>::of(raw);
    const bool none = s.m == -INFINITY, bad = s.m == INFINITY || s.m != s.m;
    const float nan = __int_as_float(0x7fffffff);
    const float log_s = none || bad ? 0.0f : logf(s.c) + log1pf(s.r / s.c);
    for (int i = lane; i < a.n_ids; i += 32) {
        if (i >= 32) {
            id = a.ids[row * a.n_ids + i];
            if (id >= 0 && id < a.vocab) logit = Pack<T>::one(reinterpret_cast<const T *>(a.x) + row * a.stride + id);
        }
        float v = 0.0f;
        if (id >= 0 && id < a.vocab)
            v = bad ? nan : none ? -INFINITY : (logit - s.m) * a.inv_tau - log_s;
        else if (id != -1)
            report(a.status, VC_ERR_BAD_INDEX);
        a.lp[row * a.n_ids + i] = v;
    }
    if (lane == 0 && a.ent) a.ent[row] = bad ? nan : none ? 0.0f : log_s - s.t / (s.c + s.r);
    for (int j = lane; j < a.k; j += 32) {
        const bool in = !bad && j < have;
        a.top_ids[row * a.k + j] = in ? (int32_t)~(uint32_t)top[j] : -1;
        a.top_lp[row * a.k + j] =
            bad ? nan : in ? (order_value((uint32_t)(top[j] >> 32)) - s.m) * a.inv_tau - log_s : -INFINITY;
    }
}
// ... which these load, early, so that the loads' latency is not met at the end.
__device__ inline int asked_id(const LpArgs &a, int64_t row, int lane) {
    return lane < a.n_ids ? a.ids[row * a.n_ids + lane] : -1;
}
template <typename T>
__device__ inline typename Pack<T>::Word asked_logit(const LpArgs &a, int64_t row, int id) {  // (as it lies in memory)
    using W = typename Pack<T>::Word;
    return id >= 0 && id < a.vocab ? reinterpret_cast<const W *>(a.x)[row * a.stride + id] : (W)0;
}

__device__ inline float warp_max_nan(float v) {
    float d;
    asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(d) : "f"(v));
    return d;
}
// Sums of two values over a warp: u's in lanes 0 to 15, v's in the others (each
// half of the lanes adds up one of them).
__device__ inline float warp_sum2(float u, float v, int lane) {
    const bool hi = lane & 16;
    float s = (hi ? v : u) + __shfl_xor_sync(0xffffffffu, hi ? u : v, 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}

// Puts n keys in order, by one warp: each one's place is the number of larger ones.
__device__ inline void order_keys(const unsigned long long *cand, int n, int k, unsigned long long *top, int lane) {
    for (int i = lane; i < n; i += 32) {
        const unsigned long long key = cand[i];
        int rank = 0;
#pragma unroll 8
        for (int q = 0; q < n; ++q) rank += cand[q] > key;
        if (rank < k) top[rank] = key;
    }
    __syncwarp();
}

// The `have` largest keys of a part (at most k), in order, where too many
// logits are not below the bound for the lists, by one warp that reads the part
// again: those above the bound, then, equal to it, the first ones.  Should the
// former be too many as well, the largest key below the last one, k times.
template <typename T>
__device__ int order_again(const T *x, int v0, int n, int k, float lo, unsigned long long *cand, int cands,
                           unsigned long long *top, int lane) {
    int above = 0;
    for (int i0 = 0; i0 < n; i0 += 32) {
        const int i = i0 + lane;
        const float v = i < n ? Pack<T>::one(x + i) : -INFINITY;
        const unsigned in = __ballot_sync(0xffffffffu, v > lo);
        const int at = above + __popc(in & ((1u << lane) - 1));
        if (v > lo && at < cands) cand[at] = order_key(v, v0 + i);
        above += __popc(in);
    }
    __syncwarp();
    if (above <= cands) {
        order_keys(cand, above, k, top, lane);
        int have = min(above, k);
        if (lo > -INFINITY)
            for (int i0 = 0; i0 < n && have < k; i0 += 32) {
                const int i = i0 + lane;
                const bool eq = i < n && Pack<T>::one(x + i) == lo;
                const unsigned in = __ballot_sync(0xffffffffu, eq);
                const int at = have + __popc(in & ((1u << lane) - 1));
                if (eq && at < k) top[at] = order_key(lo, v0 + i);
                have = min(k, have + __popc(in));
            }
        __syncwarp();
        return have;
    }
    unsigned long long last = ~0ull;
    for (int have = 0; have < k; ++have) {
        unsigned long long best = 0;
        for (int i = lane; i < n; i += 32) {
            const float v = Pack<T>::one(x + i);
            const unsigned long long key = order_key(v, v0 + i);
            if (v > lo && key < last && key > best) best = key;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const unsigned long long q = __shfl_xor_sync(0xffffffffu, best, o);
            best = q > best ? q : best;
        }
        last = best;  // (more than `cands` >= k of them)
        if (lane == 0) top[have] = last;
    }
    __syncwarp();
    return k;
}

// Statistics of two sets of logits together.
__device__ inline Stats join_stats(Stats a, Stats b, float inv_tau) {
    if (b.m > a.m) {
        const Stats s = a;
        a = b;
        b = s;
    }
    if (b.m == -INFINITY || !(a.m < INFINITY)) return a;
    if (a.m == b.m) return {a.m, a.c + b.c, a.r + b.r, a.t + b.t};
    // b's sums relative to a's maximum: e^d each, and y gains d
    const float d = fmaxf((b.m - a.m) * inv_tau, -10000.0f), f = ex2(d * kLog2e);
    return {a.m, a.c, a.r + f * (b.c + b.r), a.t + f * (b.t + d * (b.c + b.r))};
}

// The sums of a thread's packs relative to `m`, every term added (the maximum's
// too): r in units, t in units of log 2; those of packs that a thread holds.
// y = scale (v - m) takes one multiply-add, scale v - h with h = scale m rounded:
// every y is then too large by the same d = scale m - h, which is known and
// comes off at the end (e^y by 2^-d, y e^y by d e^y as well).  t is NaN where
// that cannot be done: -infinity among the logits, h or d out of range.  Packs
// in `skip` are left out.
template <typename T, int NV>
__device__ inline void sums_of(const uint4 (&x)[NV], int held, float m, float scale, float &r, float &t, uint32_t skip = 0) {
    using P = Pack<T>;
    constexpr int VEC = P::VEC;
    float r2[2] = {0.0f, 0.0f}, t2[2] = {0.0f, 0.0f};
    const float h = __fmul_rn(scale, m);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        if (j >= held) break;
        if (skip >> j & 1) continue;
        float v[VEC];
        P::unpack(x[j], v);
#pragma unroll
        for (int e = 0; e < VEC; e += 2) {
            float y[2], p[2];
            fma2(y[0], y[1], v[e], v[e + 1], scale, -h);
            p[0] = ex2(y[0]);
            p[1] = ex2(y[1]);
            acc2(r2[0], r2[1], p[0], p[1]);
            facc2(t2[0], t2[1], p[0], p[1], y[0], y[1]);
        }
    }
    const float d = __fmaf_rn(scale, m, -h), f = ex2(-d);
    r = r2[0] + r2[1];
    t = f * __fmaf_rn(-d, r, t2[0] + t2[1]);
    r *= f;
    // (from |h| = 2^30 on, d may reach sizes whose 2^d leaves fp32's range)
    if (!(fabsf(d) < 64.0f)) t = __int_as_float(0x7fffffff);
}
// The same where -infinity may be among them (0 times infinity above; here a
// bound keeps it out of y e^y: e^y is 0 long before) or the maximum, which is
// counted and not added.
template <typename T>
__device__ inline void careful_sums(uint4 u, float m, float scale, float &r, float &t, int &c) {
    float v[Pack<T>::VEC];
    Pack<T>::unpack(u, v);
#pragma unroll
    for (int e = 0; e < Pack<T>::VEC; ++e) {
        const float y = fmaxf((v[e] - m) * scale, -10000.0f), p = ex2(y);
        c += v[e] == m;
        r += v[e] == m ? 0.0f : p;
        t = fmaf(p, y, t);
    }
}

// ---------------------------------------------------------------------------
// Long rows: a block streams parts of rows through shared memory.
//
// A producer warp keeps STAGES parts under way, one bulk copy of the whole packs
// of 16 bytes each; the few logits at a part's ends that share a pack with
// something else are the finisher's (padded with -infinity they would send two
// main warps through the careful sums in every row: 4096 rows of 32001 bf16
// logits 97 instead of 55 us).  16 main warps, in groups of GW that take a part
// each, go through it once: a thread takes up to 8 packs, their maximum, and the
// sums relative to that; the warp's sums relative to the warp's maximum.  They
// never meet.  A finishing warp joins the group's sums, goes again through the
// threads' packs that hold the maximum to count it apart, takes the k-th largest
// of 32 or 64 groups' maxima as a bound (k logits at least are not below it),
// collects the logits not below it from the threads whose maximum is not, puts
// them in order and writes the results, while the others work on later parts.
// GW is the least whose threads hold a part (8, 16, 32 or 64 KB of it): with 16
// warps to every part their fixed cost bounds (16384 bf16 rows of 4000 logits 89
// instead of 55 us, of 15000 150 instead of 95).
// Bound by memory for no or one alternative (16384 x 32000 bf16: 162 and 167 us,
// 0.95 and 0.93 of a copy's rate; 8192 x 32000 fp32 157 us, 0.98); beyond by how
// long a finisher holds its stage (20 alternatives: 243 us): three stages of 64 KB
// fit.
// ---------------------------------------------------------------------------
constexpr int kMainWarps = 16, kPacks = 8;  // warps, packs a thread holds

template <int GW>
struct Hand {  // from the main warps of a part to a finisher
    float m[GW], t[GW];
    float r[GW], top[GW];  // r apart: of the threads whose maximum is the warp's
    float tmax[GW * 32];
};
template <int GW>
struct Ring {
    static constexpr int N = GW * 32, GROUPS = kMainWarps / GW;
    static constexpr int STAGE = N * kPacks * 16, STAGES = GW == 16 ? 3 : GW == 8 ? 6 : 8;
    static constexpr int FIN = GW == 16 ? 4 : GW == 8 ? 7 : 8;  // finishing warps
    // Logits not below the bound.  Should there be more, the finisher reads the part
    // again, once for those above the bound and, if they are too many too, once for
    // each alternative: what a top 64 of 32 KB parts, 300 candidates on average,
    // comes to in a third of the rows (16384 x 16000 bf16: top 50 219 us, top 64
    // 15.5 ms).
    static constexpr int CANDS = GW == 8 ? 320 : 512;
    static constexpr int THREADS = 32 * (kMainWarps + FIN + 1);
    static constexpr int OFF_HAND = STAGE * STAGES;
    static constexpr int OFF_CAND = OFF_HAND + FIN * (int)sizeof(Hand<GW>);
    static constexpr int OFF_TOP = OFF_CAND + FIN * CANDS * 8;
    static constexpr int OFF_GRP = OFF_TOP + FIN * VC_MAX_TOP * 8;
    static constexpr int OFF_LIST = OFF_GRP + FIN * 32 * 4;
    static constexpr int OFF_COUNT = OFF_LIST + FIN * N * 2;
    static constexpr int OFF_META = OFF_COUNT + FIN * 8;
    static constexpr int OFF_BAR = OFF_META + 64;
    static_assert(STAGES * 4 <= 64, "packs of a stage");
    // (the part FIN behind another is loaded after that one's stage, and with it
    // its finisher's Hand, came free)
    static_assert(STAGES <= FIN, "a Hand is written once it has been read");
    // (copies land in any order, and a parity tells two phases apart: who waits for
    // a phase must have seen the one before)
    static_assert(STAGES % GROUPS == 0, "a stage's parts go to one group");
    static constexpr int SMEM = OFF_BAR + (2 * STAGES + FIN) * 8;
    static_assert(SMEM <= 227 * 1024, "shared memory");
};

template <typename T, int GW>
__global__ void __launch_bounds__(Ring<GW>::THREADS, 1) logprobs_ring_kernel(const __grid_constant__ LpArgs a) {
    pdl_wait();
    using P = Pack<T>;
    using R = Ring<GW>;
    constexpr int VEC = P::VEC, N = R::N, NV = kPacks;
    extern __shared__ __align__(128) uint8_t smem[];
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + R::OFF_BAR), *empty = full + R::STAGES, *ready = empty + R::STAGES;
    int *packs_of = reinterpret_cast<int *>(smem + R::OFF_META);  // of a stage
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t items = (int64_t)a.rows * a.parts;
    const float scale = a.inv_tau * kLog2e;
    bool alive = true;
    if (tid == 0) {
        for (int i = 0; i < R::STAGES; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < R::FIN; ++i) mbar_init(&ready[i], GW);
        fence_mbar_init();
    }
    __syncthreads();
    // part `item`: its first logit, its place in the row, how many; the logits
    // before its first whole pack, and the whole packs
    struct Part {
        const T *p;
        int64_t row;
        int v0, n, head, packs;
    };
    auto part_of = [&](int64_t item) {
        Part q;
        q.row = a.parts == 1 ? item : item / a.parts;
        q.v0 = (int)(item - q.row * a.parts) * a.part_len;
        q.p = reinterpret_cast<const T *>(a.x) + q.row * a.stride + q.v0;
        q.n = min(a.part_len, a.vocab - q.v0);
        const int skew = (int)((uintptr_t)q.p & 15) / (int)sizeof(T);
        q.head = min(q.n, skew ? VEC - skew : 0);
        q.packs = (q.n - q.head) / VEC;
        return q;
    };
    if (warp == kMainWarps + R::FIN) {
        // ---- producer ----
        int stage = 0, parity = 0;
        int64_t sent = 0;
        for (int64_t item = block_skips(a.skip_copies) ? items : blockIdx.x; item < items && alive;
             item += gridDim.x, ++sent) {
            const Part q = part_of(item);
            if (sent >= R::STAGES)
                alive = __all_sync(0xffffffffu, mbar_wait(&empty[stage], parity ^ 1, a.status, a.wait_ns));
            if (!alive) break;
            if (lane == 0) {
                *(volatile int *)&packs_of[stage] = q.packs;
                if (q.packs > 0) {
                    mbar_arrive_expect_tx(&full[stage], q.packs * 16);
                    bulk_g2s(smem + stage * R::STAGE, q.p + q.head, q.packs * 16, &full[stage]);
                } else {
                    mbar_arrive(&full[stage]);
                }
            }
            if (++stage == R::STAGES) {
                stage = 0;
                parity ^= 1;
            }
        }
        pdl_trigger();
        // no copy may be under way when the block ends (however short the waits' limit)
        for (int i = 0; i < R::STAGES && i < sent; ++i) {
            const int64_t uses = (sent - 1 - i) / R::STAGES;  // copies into slot i before its last one
            if (!mbar_wait(&full[i], uses & 1, a.status, kWaitNs)) break;
        }
        return;
    }
    if (warp < kMainWarps) {
        // ---- main warps ----
        const int gt = tid % N, gw = warp % GW;  // place in the group
        for (uint32_t k = warp / GW; blockIdx.x + (int64_t)k * gridDim.x < items; k += R::GROUPS) {
            const int stage = k % R::STAGES, f = k % R::FIN;
            const uint8_t *src = smem + stage * R::STAGE + gt * 16;
            if (!__all_sync(0xffffffffu, mbar_wait(&full[stage], k / R::STAGES & 1, a.status, a.wait_ns))) break;
            // packs of this thread
            const int packs = *(volatile int *)&packs_of[stage];
            const int held = packs > gt ? min(NV, (packs - gt + N - 1) / N) : 0;
            uint4 x[NV];
            float mine = -INFINITY;
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                if (j >= held) break;
                x[j] = *reinterpret_cast<const uint4 *>(src + j * (N * 16));
                mine = max_nan(mine, P::max_of(x[j]));
            }
            const float wm = warp_max_nan(mine);
            float r = 0.0f, t = 0.0f;
            if (mine > -INFINITY && mine < INFINITY && wm < INFINITY) {
                sums_of<T, NV>(x, held, mine, scale, r, t);
                if (!(t <= 0.0f)) {  // -infinity is among them, or h is out of range
                    int c = 0;
                    r = t = 0.0f;
#pragma unroll
                    for (int j = 0; j < NV; ++j)
                        if (j < held) careful_sums<T>(x[j], mine, scale, r, t, c);
                    r += (float)c;
                }
                const float d = fmaxf((mine - wm) * scale, -10000.0f), g = ex2(d);
                t = g * fmaf(d, r, t);
                r *= g;
            }
            const bool holds_top = mine == wm;
            const unsigned tops = __ballot_sync(0xffffffffu, holds_top);
            float r_top = r;
            if (tops & (tops - 1)) {  // (several: rare)
                r_top = holds_top ? r : 0.0f;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) r_top += __shfl_xor_sync(0xffffffffu, r_top, o);
            }
            const float rt = warp_sum2(holds_top ? 0.0f : r, t, lane);
            Hand<GW> &h = reinterpret_cast<Hand<GW> *>(smem + R::OFF_HAND)[f];
            h.tmax[gt] = mine;
            if (holds_top) h.top[gw] = r_top;
            if (lane == 0) {
                h.m[gw] = wm;
                h.r[gw] = rt;
            }
            if (lane == 16) h.t[gw] = rt;
            __syncwarp();
            if (lane == 0) mbar_arrive(&ready[f]);
        }
        return;
    }
    // ---- finishing warps ----
    const int f = warp - kMainWarps;
    const Hand<GW> &h = reinterpret_cast<const Hand<GW> *>(smem + R::OFF_HAND)[f];
    unsigned long long *cand = reinterpret_cast<unsigned long long *>(smem + R::OFF_CAND) + f * R::CANDS;
    unsigned long long *top = reinterpret_cast<unsigned long long *>(smem + R::OFF_TOP) + f * VC_MAX_TOP;
    float *grp = reinterpret_cast<float *>(smem + R::OFF_GRP) + f * 32;
    int16_t *list = reinterpret_cast<int16_t *>(smem + R::OFF_LIST) + f * N;
    int *count = reinterpret_cast<int *>(smem + R::OFF_COUNT) + f * 2;
    int stage = f % R::STAGES, parity = 0;
    int id_next = -1;
    if (a.parts == 1 && blockIdx.x + (int64_t)f * gridDim.x < items)
        id_next = asked_id(a, blockIdx.x + (int64_t)f * gridDim.x, lane);
    for (int64_t item = blockIdx.x + (int64_t)f * gridDim.x; item < items; item += (int64_t)R::FIN * gridDim.x) {
        const Part q = part_of(item);
        const uint8_t *src = smem + stage * R::STAGE;
        const int id = id_next;
        typename P::Word logit = 0;
        if (a.parts == 1) {
            logit = asked_logit<T>(a, q.row, id);
            const int64_t later = item + (int64_t)R::FIN * gridDim.x;
            id_next = later < items ? asked_id(a, later, lane) : -1;
        }
        // a logit at an end of the part, beside the whole packs (at most 14)
        const int loose_i = lane < q.head ? lane : lane >= 8 && lane < 16 ? q.head + q.packs * VEC + lane - 8 : -1;
        typename P::Word loose_w = 0;
        const bool has_loose = loose_i >= 0 && loose_i < q.n;
        if (has_loose) loose_w = reinterpret_cast<const typename P::Word *>(q.p)[loose_i];
        // once a wait has run out, this part and the warp's later ones end as if a
        // NaN were among their logits: no row keeps what its outputs held before
        alive = alive && __all_sync(0xffffffffu, mbar_wait(&ready[f], parity, a.status, a.wait_ns));
        parity ^= 1;
        const float loose = has_loose ? P::of(loose_w) : -INFINITY;
        Stats s;
        const float wm = lane < GW ? h.m[lane] : -INFINITY;
        s.m = alive ? warp_max_nan(max_nan(wm, loose)) : __int_as_float(0x7fffffff);
        s.c = s.r = s.t = 0.0f;
        const bool sound = s.m > -INFINITY && s.m < INFINITY;
        int have = 0, n = 0;
        float lo = s.m;
        if (sound) {
            float tm[GW];  // maxima of the threads w * 32 + lane
#pragma unroll
            for (int w = 0; w < GW; ++w) tm[w] = h.tmax[w * 32 + lane];
            // the packs of `threads` listed threads, 32 at a time
            auto for_packs = [&](int threads, auto fn) {
                for (int i0 = 0; i0 < threads * NV; i0 += 32) {
                    const int i = i0 + lane;
                    int pk = i < threads * NV ? (i % NV) * N + list[i / NV] : -1;
                    if (pk >= q.packs) pk = -1;
                    fn(pk);
                }
                __syncwarp();
            };
            float r = 0.0f, t = 0.0f;
            if (wm > -INFINITY) {
                const float d = fmaxf((wm - s.m) * scale, -10000.0f), g = ex2(d);
                const float all = h.r[lane] + h.top[lane];
                t = g * fmaf(d, all, h.t[lane]);
                r = wm == s.m ? h.r[lane] : g * all;
            }
            // the threads that hold the maximum (listed in order: sums must not
            // depend on chance): their terms again, it counted apart
            int c = loose == s.m, threads = 0;
            float unused = 0.0f;
            if (loose > -INFINITY && loose < s.m) {
                const float y = fmaxf((loose - s.m) * scale, -10000.0f), p = ex2(y);
                r += p;
                t = fmaf(p, y, t);
            }
#pragma unroll
            for (int w = 0; w < GW; ++w) {
                const unsigned who = __ballot_sync(0xffffffffu, tm[w] == s.m);
                if (!who) continue;
                if (tm[w] == s.m) list[threads + __popc(who & ((1u << lane) - 1))] = (int16_t)(w * 32 + lane);
                threads += __popc(who);
            }
            __syncwarp();
            uint32_t first = loose == s.m ? q.v0 + loose_i : ~0u;  // id of a maximum: for k = 1 all that is asked
            for_packs(threads, [&](int pk) {
                if (pk < 0) return;
                const uint4 u = *reinterpret_cast<const uint4 *>(src + pk * 16);
                careful_sums<T>(u, s.m, scale, r, unused, c);
                if (a.k == 1) {
                    float v[VEC];
                    P::unpack(u, v);
#pragma unroll
                    for (int e = VEC - 1; e >= 0; --e)
                        if (v[e] == s.m) first = min(first, (uint32_t)(q.v0 + q.head + pk * VEC + e));
                }
            });
            if (a.k == 1) {
                first = __reduce_min_sync(0xffffffffu, first);
                if (lane == 0) top[0] = order_key(s.m, first);
                have = 1;
            }
            const float both = warp_sum2(r, t, lane);
            s.r = __shfl_sync(0xffffffffu, both, 0);
            s.t = __shfl_sync(0xffffffffu, both, 16) * 0.6931471805599453f;
            s.c = (float)__reduce_add_sync(0xffffffffu, c);
            if (a.k > 1) {
                // 32 groups of threads, for a larger k 64 (two a lane): the
                // smallest maximum that fewer than k exceed
                float g[2] = {-INFINITY, -INFINITY};
#pragma unroll
                for (int w = 0; w < GW; ++w) g[w & 1] = fmaxf(g[w & 1], tm[w]);
                const bool two = a.k > 24;
                if (!two) g[0] = fmaxf(g[0], g[1]);
                int above[2] = {0, 0};
                for (int w = 0; w <= (int)two; ++w) {
                    grp[lane] = w ? g[1] : g[0];
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 32; i += 4) {
                        const float4 o = *reinterpret_cast<const float4 *>(grp + i);
                        above[0] += (o.x > g[0]) + (o.y > g[0]) + (o.z > g[0]) + (o.w > g[0]);
                        if (two) above[1] += (o.x > g[1]) + (o.y > g[1]) + (o.z > g[1]) + (o.w > g[1]);
                    }
                    __syncwarp();
                }
                float least = above[0] < a.k ? g[0] : INFINITY;
                if (two && above[1] < a.k) least = fminf(least, g[1]);
                lo = -warp_max_nan(-least);
                // the logits not below it (and not -infinity), from the threads whose
                // maximum is not, in an order left to chance (what follows is not)
                const float floor = fmaxf(lo, -3.402823466e38f);
                if (lane == 0) count[0] = count[1] = 0;
                __syncwarp();
                if (loose >= floor) {
                    const int at = atomicAdd(&count[1], 1);  // (the first: there is room)
                    cand[at] = order_key(loose, q.v0 + loose_i);
                }
                uint32_t mine = 0;
#pragma unroll
                for (int w = 0; w < GW; ++w) mine |= tm[w] >= floor ? 1u << w : 0u;
                if (mine)
                    for (int at = atomicAdd(&count[0], __popc(mine)); mine; mine &= mine - 1, ++at)
                        list[at] = (int16_t)((__ffs(mine) - 1) * 32 + lane);
                __syncwarp();
                // four packs a lane at a time: which of their logits, then one count
                // for all of them (most lanes have none)
                const int packs = count[0] * NV;
                for (int i0 = lane; i0 < packs; i0 += 128) {
                    auto pack_of = [&](int k) {
                        const int i = i0 + 32 * k;
                        const int pk = i < packs ? (i % NV) * N + list[i / NV] : q.packs;
                        return pk < q.packs ? pk : -1;
                    };
                    uint32_t in = 0;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int pk = pack_of(k);
                        if (pk < 0) continue;
                        float v[VEC];
                        P::unpack(*reinterpret_cast<const uint4 *>(src + pk * 16), v);
#pragma unroll
                        for (int e = 0; e < VEC; ++e) in |= v[e] >= floor ? 1u << (8 * k + e) : 0u;
                    }
                    if (in)
                        for (int at = atomicAdd(&count[1], __popc(in)); in && at < R::CANDS; in &= in - 1, ++at) {
                            const int bit = __ffs(in) - 1, pk = pack_of(bit / 8), e = bit % 8;
                            cand[at] = order_key(P::one(reinterpret_cast<const T *>(src + pk * 16) + e),
                                                 q.v0 + q.head + pk * VEC + e);
                        }
                }
                __syncwarp();
                n = count[1];
            }
        }
        // stage and hand-over are free again
        __syncwarp();
        if (lane == 0 && alive) mbar_arrive(&empty[stage]);
        stage = (stage + R::FIN) % R::STAGES;
        if (a.k > 1 && sound) {
            if (n <= R::CANDS) {
                order_keys(cand, n, a.k, top, lane);
                have = min(a.k, n);
            } else {
                have = order_again<T>(q.p, q.v0, q.n, a.k, lo, cand, R::CANDS, top, lane);
            }
        }
        if (a.parts == 1) {
            finish_row<T>(a, q.row, s, top, have, lane, id, logit);
        } else {
            unsigned long long *w = a.ws + item * (3 + a.k);
            if (lane == 0) {
                reinterpret_cast<float2 *>(w)[0] = make_float2(s.m, s.c);
                reinterpret_cast<float2 *>(w)[1] = make_float2(s.r, s.t);
                w[2] = have;
            }
            for (int i = lane; i < have; i += 32) w[3 + i] = top[i];
        }
        __syncwarp();
    }
}

// ---------------------------------------------------------------------------
// Short rows: a warp each, the row in registers (NV packs a lane).  Bound by
// instructions, some hundreds a row, and with alternatives by the ranking of the
// candidates (16384 x 1000 bf16: none 15 us, top 5 31, top 20 45, top 32 153, for
// 4.8 us of bytes).  The bound for the alternatives is the k-th largest of 32
// lanes' maxima: from k = 33 on there is none, every logit is a candidate, and a
// row of more than kShortCands of them is read once for each alternative (top 33
// 577 us, top 64 1058).
// ---------------------------------------------------------------------------
constexpr int kShortWarps = 4, kShortPacks = 8, kShortCands = 256;

// TOP: no alternative, one, or more (registers for each by itself: 16384 rows of
// 1000 bf16 logits, top 5, 33 us in one kernel for all)
template <typename T, int TOP>
__global__ void __launch_bounds__(kShortWarps * 32, 8) logprobs_short_kernel(const __grid_constant__ LpArgs a) {
    pdl_begin();
    using P = Pack<T>;
    constexpr int VEC = P::VEC, NV = kShortPacks;
    __shared__ unsigned long long cands[kShortWarps][kShortCands], tops[kShortWarps][VC_MAX_TOP];
    __shared__ int counts[kShortWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    unsigned long long *cand = cands[warp], *top = tops[warp];
    const float scale = a.inv_tau * kLog2e;
    const int64_t step = (int64_t)gridDim.x * kShortWarps;
    int64_t row = (int64_t)blockIdx.x * kShortWarps + warp;
    int id_next = row < a.rows ? asked_id(a, row, lane) : -1;
    for (; row < a.rows; row += step) {
        const T *p = reinterpret_cast<const T *>(a.x) + row * a.stride;
        const int skew = (int)((uintptr_t)p & 15) / (int)sizeof(T), n = a.vocab, packs = ceil_div(n + skew, VEC);
        const int held = packs > lane ? min(NV, (packs - lane + 31) / 32) : 0;
        uint4 x[NV];
        float mine = -INFINITY;
        uint32_t apart = 0;  // packs that hold the maximum or an end of the row
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int i0 = (j * 32 + lane) * VEC - skew;
            if (i0 >= 0 && i0 + VEC <= n) {
                x[j] = __ldcs(reinterpret_cast<const uint4 *>(p + i0));
            } else {  // an end of the row, or behind it
                uint32_t w[4] = {P::kNone, P::kNone, P::kNone, P::kNone};
                if (j < held) {
                    apart |= 1u << j;
#pragma unroll
                    for (int e = 0; e < VEC; ++e)
                        if (i0 + e >= 0 && i0 + e < n) {
                            const uint32_t v = reinterpret_cast<const typename P::Word *>(p)[i0 + e];
                            if constexpr (VEC == 4)
                                w[e] = v;
                            else
                                w[e / 2] = e % 2 ? (w[e / 2] & 0xffffu) | v << 16 : (w[e / 2] & 0xffff0000u) | v;
                        }
                }
                x[j] = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
        const int id = id_next;
        const auto logit = asked_logit<T>(a, row, id);
        if (row + step < a.rows) {  // what comes next: its tokens, and its logits into L2
            id_next = asked_id(a, row + step, lane);
            const int64_t ahead = (int64_t)lane * 128 / (int)sizeof(T);
            if (ahead < n) asm volatile("prefetch.global.L2 [%0];" ::"l"(p + step * a.stride + ahead));
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) mine = max_nan(mine, P::max_of(x[j]));
        Stats s{warp_max_nan(mine), 0.0f, 0.0f, 0.0f};
        const bool sound = s.m > -INFINITY && s.m < INFINITY;
        int have = 0;
        if (sound) {
            // the maximum counted apart, -infinity (behind an end, or of tokens ruled
            // out) kept out of y e^y: such packs one by one, the others together (a
            // thread's packs all one by one if one is: 16384 rows of 1000 bf16
            // logits, top 5, 41 instead of 31 us)
            float r = 0.0f, t = 0.0f, r1 = 0.0f, t1 = 0.0f;
            int c = 0;
            if (mine == s.m) {
#pragma unroll
                for (int j = 0; j < NV; ++j)
                    if (P::max_of(x[j]) == s.m) apart |= 1u << j;
            }
            sums_of<T, NV>(x, held, s.m, scale, r, t, apart);
            if (!(t <= 0.0f)) {
                r = t = 0.0f;
                apart = ~0u;
            }
#pragma unroll
            for (int j = 0; j < NV; ++j)
                if (j < held && (apart >> j & 1)) careful_sums<T>(x[j], s.m, scale, r1, t1, c);
            r += r1;
            t += t1;
            __syncwarp();
            const float both = warp_sum2(r, t, lane);
            s.r = __shfl_sync(0xffffffffu, both, 0);
            s.t = __shfl_sync(0xffffffffu, both, 16) * 0.6931471805599453f;
            s.c = (float)__reduce_add_sync(0xffffffffu, c);
            if constexpr (TOP == 1) {  // the first that equals the maximum
                uint32_t first = ~0u;
                if (mine == s.m) {
#pragma unroll
                    for (int j = NV - 1; j >= 0; --j) {
                        if (P::max_of(x[j]) != s.m) continue;
                        float v[VEC];
                        P::unpack(x[j], v);
#pragma unroll
                        for (int e = VEC - 1; e >= 0; --e)
                            if (v[e] == s.m) first = (uint32_t)((j * 32 + lane) * VEC - skew + e);
                    }
                }
                first = __reduce_min_sync(0xffffffffu, first);
                if (lane == 0) top[0] = order_key(s.m, first);
                __syncwarp();
                have = 1;
            } else if constexpr (TOP > 1) {
                // the k-th largest of the lanes' maxima is a bound
                float lo;
                float left = mine;
                for (int above = 0;;) {  // (a lane at least drops out each time)
                    lo = warp_max_nan(left);
                    above += __popc(__ballot_sync(0xffffffffu, left == lo));
                    if (above >= a.k || lo == -INFINITY) break;
                    if (left == lo) left = -INFINITY;
                }
                if (lane == 0) counts[warp] = 0;
                __syncwarp();
                if (mine >= lo && mine > -INFINITY) {
#pragma unroll
                    for (int j = 0; j < NV; ++j) {
                        const float pm = P::max_of(x[j]);
                        if (!(pm >= lo && pm > -INFINITY)) continue;
                        float v[VEC];
                        P::unpack(x[j], v);
#pragma unroll
                        for (int e = 0; e < VEC; ++e)
                            if (v[e] >= lo && v[e] > -INFINITY) {
                                const int at = atomicAdd(&counts[warp], 1);
                                if (at < kShortCands) cand[at] = order_key(v[e], (j * 32 + lane) * VEC - skew + e);
                            }
                    }
                }
                __syncwarp();
                const int nc = counts[warp];
                if (nc <= kShortCands) {
                    order_keys(cand, nc, a.k, top, lane);
                    have = min(a.k, nc);
                } else {
                    have = order_again<T>(p, 0, n, a.k, lo, cand, kShortCands, top, lane);
                }
            }
        }
        finish_row<T>(a, row, s, top, have, lane, id, logit);
        __syncwarp();
    }
}

// Rows of several parts: one block joins a row's statistics and alternatives.
// Bound by latency: everything is asked for at once, a lane per part (4 rows of
// 131072 fp32 logits, a loop over the parts: 9.7 instead of 8.4 us).
constexpr int kJoinKeys = 1024, kJoinThreads = 128;
template <typename T>
__global__ void __launch_bounds__(kJoinThreads) logprobs_join_kernel(const __grid_constant__ LpArgs a) {
    pdl_begin();
    __shared__ unsigned long long top[VC_MAX_TOP], keys[kJoinKeys];
    const int64_t row = blockIdx.x;
    const int size = 3 + a.k, tid = threadIdx.x, lane = tid & 31, all = a.parts * a.k;
    const unsigned long long *w = a.ws + row * a.parts * size;
    auto keys_of = [&](int p) { return (int)min(w[p * size + 2], (unsigned long long)a.k); };
    const int id = asked_id(a, row, lane);
    const auto logit = asked_logit<T>(a, row, id);
    // a key's place is the number of larger ones: among all of them in shared
    // memory, or, where they are many, its place in its own part and the larger
    // ones of the others
    if (all <= kJoinKeys) {
        for (int i = tid; i < all; i += kJoinThreads) {
            const int p = i / a.k, j = i % a.k;
            const unsigned long long key = w[p * size + 3 + j];  // (in the workspace, if not a key)
            keys[i] = j < keys_of(p) ? key : 0;
        }
    }
    Stats s{-INFINITY, 0.0f, 0.0f, 0.0f};
    int n = 0;
    if (tid < 32) {
        bool nan = false;
        for (int p = lane; p < a.parts; p += 32) {
            const float2 mc = *reinterpret_cast<const float2 *>(w + p * size);
            const float2 rt = *reinterpret_cast<const float2 *>(w + p * size + 1);
            n += keys_of(p);
            if (mc.x != mc.x)
                nan = true;
            else
                s = join_stats(s, {mc.x, mc.y, rt.x, rt.y}, a.inv_tau);
        }
        auto from = [&](int l) {
            return Stats{__shfl_sync(0xffffffffu, s.m, l), __shfl_sync(0xffffffffu, s.c, l),
                         __shfl_sync(0xffffffffu, s.r, l), __shfl_sync(0xffffffffu, s.t, l)};
        };
        for (int o = 1; o < min(a.parts, 32); o *= 2) s = join_stats(s, from(lane ^ o), a.inv_tau);
        s = from(0);
        n = __reduce_add_sync(0xffffffffu, n);
        if (__any_sync(0xffffffffu, nan)) s.m = __int_as_float(0x7fffffff);
    }
    __syncthreads();
    if (all <= kJoinKeys) {
        for (int i = tid; i < all; i += kJoinThreads) {
            const unsigned long long key = keys[i];
            int rank = 0;
#pragma unroll 8
            for (int q = 0; q < all; ++q) rank += keys[q] > key;
            if (key && rank < a.k) top[rank] = key;
        }
    } else {
        for (int i = tid; i < all; i += kJoinThreads) {
            const int p = i / a.k, j = i % a.k;
            if (j >= keys_of(p)) continue;
            const unsigned long long key = w[p * size + 3 + j];
            int rank = j;
            for (int o = 0; o < a.parts; ++o) {
                if (o == p) continue;
                const int no = keys_of(o);
                for (int q = 0; q < no && w[o * size + 3 + q] > key; ++q) ++rank;
            }
            if (rank < a.k) top[rank] = key;
        }
    }
    __syncthreads();
    if (tid < 32) finish_row<T>(a, row, s, top, min(n, a.k), lane, id, logit);
}

// Parts of a row: packs of at most 64 KB, of one size, a multiple of 8 logits.
constexpr int kVocabMax = 1 << 22;
void split(int vocab, int dtype, int &parts, int &len) {
    const int most = (kMainWarps * 32 * kPacks - 1) * (dtype == VC_F32 ? 4 : 8) / 8 * 8;  // (wherever it starts in its first pack)
    parts = ceil_div(vocab, most);
    len = parts == 1 ? vocab : ceil_div(ceil_div(vocab, parts), 8) * 8;
    parts = ceil_div(vocab, len);
}

template <typename T, int GW>
cudaError_t launch_ring(const LpArgs &a, cudaStream_t st) {
    const cudaError_t e = set_smem_limit((const void *)logprobs_ring_kernel<T, GW>, Ring<GW>::SMEM);
    if (e != cudaSuccess) return e;
    const int64_t items = (int64_t)a.rows * a.parts;
    return launch_pdl(logprobs_ring_kernel<T, GW>, dim3((unsigned)(items < 152 ? items : 152)), Ring<GW>::THREADS,
                      Ring<GW>::SMEM, st, a);
}

template <typename T>
cudaError_t launch(LpArgs a, int dtype, cudaStream_t st) {
    constexpr int VEC = Pack<T>::VEC;
    split(a.vocab, dtype, a.parts, a.part_len);
    const int packs = ceil_div(a.part_len + VEC - 1, VEC);  // wherever the row starts
    if (packs <= 32 * kShortPacks) {
        const int64_t blocks = ((int64_t)a.rows + kShortWarps - 1) / kShortWarps, most = 152 * 8;
        const dim3 grid((unsigned)(blocks < most ? blocks : most));
        return a.k == 0   ? launch_pdl(logprobs_short_kernel<T, 0>, grid, kShortWarps * 32, 0, st, a)
               : a.k == 1 ? launch_pdl(logprobs_short_kernel<T, 1>, grid, kShortWarps * 32, 0, st, a)
                          : launch_pdl(logprobs_short_kernel<T, 2>, grid, kShortWarps * 32, 0, st, a);
    }
    cudaError_t e = packs <= 2 * 32 * kPacks   ? launch_ring<T, 2>(a, st)
                    : packs <= 4 * 32 * kPacks ? launch_ring<T, 4>(a, st)
                    : packs <= 8 * 32 * kPacks ? launch_ring<T, 8>(a, st)
                                               : launch_ring<T, 16>(a, st);
    if (e == cudaSuccess && a.parts > 1) e = launch_pdl(logprobs_join_kernel<T>, a.rows, kJoinThreads, 0, st, a);
    return e;
}

}  // namespace
}  // namespace vc

using namespace vc;

extern "C" {

size_t vc_token_logprobs_workspace_bytes(int32_t rows, int32_t vocab, int32_t top_k) {
    if (rows < 0 || vocab < 1 || vocab > kVocabMax || top_k < 0 || top_k > VC_MAX_TOP) return 0;
    int parts, len;
    split(vocab, VC_F32, parts, len);  // (fp32 logits take the most parts)
    return parts == 1 ? 8 : (size_t)rows * parts * (3 + top_k) * 8;
}

vc_status vc_token_logprobs(const void *logits, int32_t dtype, int32_t rows, int32_t vocab, int64_t row_stride,
                            const int32_t *ids, int32_t n_ids, float temperature, int32_t top_k, float *logprobs,
                            float *entropy, int32_t *top_ids, float *top_logprobs, void *workspace,
                            size_t workspace_bytes, int32_t *dev_status, vc_stream_t stream) {
    if (rows < 0 || vocab < 1 || row_stride < vocab || n_ids < 0 || top_k < 0 || !(temperature > 0.0f) ||
        !std::isfinite(temperature))
        return VC_ERR_INVALID_ARG;
    const int bytes = dtype_bytes(dtype);
    const float inv_tau = 1.0f / temperature;
    if (bytes == 0 || top_k > VC_MAX_TOP || vocab > kVocabMax || !std::isfinite(inv_tau * kLog2e))
        return VC_ERR_UNSUPPORTED;
    if (rows == 0) return VC_OK;
    if (!logits || (uintptr_t)logits % bytes || (n_ids > 0 && (!ids || !logprobs)) || (top_k > 0 && (!top_ids || !top_logprobs)))
        return VC_ERR_INVALID_ARG;
    if ((uintptr_t)workspace & 7) return VC_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < vc_token_logprobs_workspace_bytes(rows, vocab, top_k))
        return VC_ERR_WORKSPACE;
    LpArgs a;
    a.x = logits;
    a.stride = row_stride;
    a.rows = rows;
    a.vocab = vocab;
    a.ws = (unsigned long long *)workspace;
    a.ids = ids;
    a.n_ids = n_ids;
    a.k = top_k;
    a.inv_tau = inv_tau;
    a.lp = logprobs;
    a.ent = entropy;
    a.top_ids = top_ids;
    a.top_lp = top_logprobs;
    a.status = dev_status;
    a.wait_ns = wait_fault().wait_ns;
    a.skip_copies = wait_fault().skip_copies;
    const cudaStream_t st = (cudaStream_t)stream;
    const cudaError_t e = dtype == VC_F32    ? launch<float>(a, dtype, st)
                          : dtype == VC_BF16 ? launch<__nv_bfloat16>(a, dtype, st)
                                             : launch<__half>(a, dtype, st);
    return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? VC_OK : VC_ERR_CUDA;
}

}  // extern "C"
