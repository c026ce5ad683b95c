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
    static constexpr uint32_t kNone = 0xff800000u;  // words of -infinity
    __device__ static float one(const float *p) { return *p; }
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
    static constexpr uint32_t kNone = 0xff80ff80u;
    __device__ static float one(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
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
    static constexpr uint32_t kNone = 0xfc00fc00u;
    __device__ static float one(const __half *p) { return __half2float(*p); }
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
__device__ inline void sub_mul2(float &d0, float &d1, float a0, float a1, float b, float c) {  // (a - b) c
    asm("{\n\t.reg .b64 ra, rb, rc;\n\t.reg .f32 nb;\n\tneg.f32 nb, %4;\n\t"
        "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {nb, nb};\n\tmov.b64 rc, {%5, %5};\n\t"
        "add.rn.f32x2 ra, ra, rb;\n\tmul.rn.f32x2 ra, ra, rc;\n\tmov.b64 {%0, %1}, ra;\n\t}"
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
};

// What a row's logits amount to: the maximum, how many logits equal it, the
// sum of the others' e^y, and the sum of y e^y.
struct Stats {
    float m, c, r, t;
};

// Outputs of row `row`, given its statistics and its `have` largest keys.
template <typename T>
__device__ void finish_row(const LpArgs &a, int64_t row, Stats s, const unsigned long long *top, int have, int tid,
                           int nthreads) {
    const bool none = s.m == -INFINITY, bad = s.m == INFINITY || s.m != s.m;
    const float nan = __int_as_float(0x7fffffff);
    const float log_s = none || bad ? 0.0f : logf(s.c) + log1pf(s.r / s.c);
    const T *x = reinterpret_cast<const T *>(a.x) + row * a.stride;
    for (int i = tid; i < a.n_ids; i += nthreads) {
        const int id = a.ids[row * a.n_ids + i];
        float v = 0.0f;
        if (id >= 0 && id < a.vocab)
            v = bad ? nan : none ? -INFINITY : (Pack<T>::one(x + id) - s.m) * a.inv_tau - log_s;
        else if (id != -1)
            report(a.status, VC_ERR_BAD_INDEX);
        a.lp[row * a.n_ids + i] = v;
    }
    if (tid == 0 && a.ent) a.ent[row] = bad ? nan : none ? 0.0f : log_s - s.t / (s.c + s.r);
    for (int j = tid; j < a.k; j += nthreads) {
        const bool in = !bad && j < have;
        a.top_ids[row * a.k + j] = in ? (int32_t)~(uint32_t)top[j] : -1;
        a.top_lp[row * a.k + j] =
            bad ? nan : in ? (order_value((uint32_t)(top[j] >> 32)) - s.m) * a.inv_tau - log_s : -INFINITY;
    }
}

// A part of a row in registers, NV packs a thread; pack j of thread t is pack
// j * THREADS + t of the part (counted from the 16-byte boundary at or before
// its first logit), so loads are whole and a run of neighbours is spread over
// the threads.
template <typename T, int THREADS, int NV>
struct Chunk {
    using P = Pack<T>;
    static constexpr int VEC = P::VEC;
    uint4 x[NV];
    int skew, packs, n;  // logits before the part in its first pack; packs; logits

    // first logit's index (in the part) of this thread's pack j
    __device__ int index(int j) const { return (j * THREADS + (int)threadIdx.x) * VEC - skew; }
    __device__ bool holds(int j) const { return j * THREADS + (int)threadIdx.x < packs; }

    // The packs are read anew: what was unpacked of them is not kept in registers.
    __device__ void again() {
#pragma unroll
        for (int j = 0; j < NV; ++j) asm volatile("" : "+r"(x[j].x), "+r"(x[j].y), "+r"(x[j].z), "+r"(x[j].w));
    }

    __device__ void load(const T *p, int n_) {
        n = n_;
        skew = (int)((uintptr_t)p & 15) / (int)sizeof(T);
        packs = ceil_div(n + skew, VEC);
        const uint4 *base = reinterpret_cast<const uint4 *>(p - skew);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int i0 = index(j);
            if (i0 >= 0 && i0 + VEC <= n) {
                x[j] = __ldcs(base + j * THREADS + threadIdx.x);
            } else {  // an end of the part, or behind it: its logits one by one, -infinity beside them
                uint32_t w[4] = {P::kNone, P::kNone, P::kNone, P::kNone};
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    if (i0 + e >= 0 && i0 + e < n) {
                        if constexpr (sizeof(T) == 4) {
                            w[e] = reinterpret_cast<const uint32_t *>(p)[i0 + e];
                        } else {
                            const uint32_t v = reinterpret_cast<const uint16_t *>(p)[i0 + e];
                            w[e / 2] = e % 2 ? (w[e / 2] & 0xffffu) | v << 16 : (w[e / 2] & 0xffff0000u) | v;
                        }
                    }
                x[j] = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
    }
};

constexpr int kGroups = 64;   // groups of threads whose maxima bound the k-th largest logit
constexpr int kCands = 2048;  // logits above that bound (more: one alternative at a time)

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

// One block per part of a row, in turn over the parts it owns.  The part stays
// in registers; the block meets four times: for the maximum (and the groups'
// maxima), for the sums (and the bound), for the logits above the bound, for
// their order.  Memory bounds it (64 KB of bf16 at an SM's share of the
// bandwidth take 1.4 us), so what comes next is asked into L2 before the
// arithmetic begins, and the arithmetic is packed: maxima of 8 logits in 4
// instructions, two logits' differences, products and sums in one.
template <typename T, int THREADS, int NV, int MIN_CTAS>
__global__ void __launch_bounds__(THREADS, MIN_CTAS) logprobs_kernel(const __grid_constant__ LpArgs a) {
    pdl_begin();
    using P = Pack<T>;
    constexpr int VEC = P::VEC, WARPS = THREADS / 32, PER = THREADS / kGroups;
    __shared__ float wmax[WARPS], wsum[3][WARPS], gmax[kGroups], bound;
    __shared__ int n_cand;
    __shared__ unsigned long long cand[kCands], top[VC_MAX_TOP], wkey[WARPS];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int items = a.rows * a.parts;
    const float scale = a.inv_tau * kLog2e;
    for (int item = blockIdx.x; item < items; item += gridDim.x) {
        const int64_t row = item / a.parts;
        const int part = item % a.parts, v0 = part * a.part_len;
        Chunk<T, THREADS, NV> ch;
        ch.load(reinterpret_cast<const T *>(a.x) + row * a.stride + v0, min(a.part_len, a.vocab - v0));
        if (tid == 0 && item + (int)gridDim.x < items) {  // the next part: whole 16-byte pieces within it
            const int ni = item + gridDim.x, nv0 = ni % a.parts * a.part_len;
            const T *np = reinterpret_cast<const T *>(a.x) + (ni / a.parts) * a.stride + nv0;
            const uintptr_t lo = ((uintptr_t)np + 15) & ~(uintptr_t)15;
            const uintptr_t hi = (uintptr_t)(np + min(a.part_len, a.vocab - nv0)) & ~(uintptr_t)15;
            if (hi > lo)
                asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(lo), "r"((uint32_t)(hi - lo)) : "memory");
        }
        // ---- maxima ----
        float g = -INFINITY;
#pragma unroll
        for (int j = 0; j < NV; ++j) g = max_nan(g, P::max_of(ch.x[j]));
#pragma unroll
        for (int o = 1; o < PER; o <<= 1) g = max_nan(g, __shfl_xor_sync(0xffffffffu, g, o));
        if (tid % PER == 0) gmax[tid / PER] = g;
#pragma unroll
        for (int o = PER; o < 32; o <<= 1) g = max_nan(g, __shfl_xor_sync(0xffffffffu, g, o));
        if (lane == 0) wmax[warp] = g;
        if (tid == 0) {
            n_cand = 0;
            bound = -INFINITY;
        }
        __syncthreads();
        Stats s{-INFINITY, 0.0f, 0.0f, 0.0f};
        s.m = wmax[lane % WARPS];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s.m = max_nan(s.m, __shfl_xor_sync(0xffffffffu, s.m, o));
        const bool sound = s.m > -INFINITY && s.m < INFINITY;
        // ---- the bound: the k-th largest of the groups' maxima (k logits at least are not below it) ----
        if (a.k > 0 && warp >= WARPS - 2) {
            const int i = tid - (THREADS - 64);
            const float mine = gmax[i];
            int rank = 0;
#pragma unroll 16
            for (int q = 0; q < kGroups; ++q) rank += gmax[q] > mine || (gmax[q] == mine && q < i);
            if (rank == a.k - 1) bound = mine;
        }
        // ---- sums ----
        if (sound) {
            float r2[2] = {0.0f, 0.0f}, t2[2] = {0.0f, 0.0f};  // t in units of log 2
            ch.again();
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                if (!ch.holds(j)) continue;
                float v[VEC], rv[2] = {0.0f, 0.0f}, tv[2] = {0.0f, 0.0f};
                P::unpack(ch.x[j], v);
#pragma unroll
                for (int e = 0; e < VEC; e += 2) {
                    float y[2], p[2];
                    sub_mul2(y[0], y[1], v[e], v[e + 1], s.m, scale);
                    p[0] = ex2(y[0]);
                    p[1] = ex2(y[1]);
                    acc2(rv[0], rv[1], p[0], p[1]);
                    facc2(tv[0], tv[1], p[0], p[1], y[0], y[1]);
                }
                const float check = tv[0] + tv[1];
                if (rv[0] + rv[1] >= 1.0f || check != check) {
                    // a pack that may hold the maximum (which is counted, not
                    // added), or -infinity (the bound keeps it out of y e^y: e^y
                    // is 0 long before)
                    rv[0] = rv[1] = tv[0] = tv[1] = 0.0f;
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        const float y = fmaxf((v[e] - s.m) * scale, -10000.0f), p = ex2(y);
                        if (v[e] == s.m)
                            s.c += 1.0f;
                        else
                            rv[0] += p;
                        tv[0] = fmaf(p, y, tv[0]);
                    }
                }
                acc2(r2[0], r2[1], rv[0], rv[1]);
                acc2(t2[0], t2[1], tv[0], tv[1]);
            }
            s.r = r2[0] + r2[1];
            s.t = (t2[0] + t2[1]) * 0.6931471805599453f;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            s.c += __shfl_xor_sync(0xffffffffu, s.c, o);
            s.r += __shfl_xor_sync(0xffffffffu, s.r, o);
            s.t += __shfl_xor_sync(0xffffffffu, s.t, o);
        }
        if (lane == 0) {
            wsum[0][warp] = s.c;
            wsum[1][warp] = s.r;
            wsum[2][warp] = s.t;
        }
        __syncthreads();
        s.c = lane < WARPS ? wsum[0][lane] : 0.0f;
        s.r = lane < WARPS ? wsum[1][lane] : 0.0f;
        s.t = lane < WARPS ? wsum[2][lane] : 0.0f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            s.c += __shfl_xor_sync(0xffffffffu, s.c, o);
            s.r += __shfl_xor_sync(0xffffffffu, s.r, o);
            s.t += __shfl_xor_sync(0xffffffffu, s.t, o);
        }
        // ---- alternatives ----
        int have = 0;
        if (a.k > 0 && sound) {
            const float lo = bound;
            ch.again();
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                if (!(P::max_of(ch.x[j]) >= lo)) continue;
                float v[VEC];
                P::unpack(ch.x[j], v);
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    if (v[e] >= lo && v[e] > -INFINITY) {
                        const int at = atomicAdd(&n_cand, 1);
                        if (at < kCands) cand[at] = order_key(v[e], v0 + ch.index(j) + e);
                    }
            }
            __syncthreads();
            const int n = n_cand;
            have = min(a.k, n);
            if (n <= kCands) {
                // each one's place among them (their order in memory is left to chance, this is not)
                for (int i = tid; i < n; i += THREADS) {
                    const unsigned long long key = cand[i];
                    int rank = 0;
                    for (int q = 0; q < n; ++q) rank += cand[q] > key;
                    if (rank < a.k) top[rank] = key;
                }
            } else {
                // too many (equal or sorted logits): the largest key below the last one, k times
                unsigned long long last = ~0ull;
                for (int i = 0; i < have; ++i) {
                    unsigned long long best = 0;
                    ch.again();
#pragma unroll
                    for (int j = 0; j < NV; ++j) {
                        if (!(P::max_of(ch.x[j]) >= lo)) continue;
                        float v[VEC];
                        P::unpack(ch.x[j], v);
#pragma unroll
                        for (int e = 0; e < VEC; ++e) {
                            const unsigned long long key = order_key(v[e], v0 + ch.index(j) + e);
                            if (v[e] > -INFINITY && key < last && key > best) best = key;
                        }
                    }
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) {
                        const unsigned long long q = __shfl_xor_sync(0xffffffffu, best, o);
                        best = q > best ? q : best;
                    }
                    if (lane == 0) wkey[warp] = best;
                    __syncthreads();
                    last = wkey[0];
                    for (int q = 1; q < WARPS; ++q) last = wkey[q] > last ? wkey[q] : last;
                    if (tid == 0) top[i] = last;
                    __syncthreads();
                }
            }
            __syncthreads();
        }
        if (a.parts == 1) {
            finish_row<T>(a, row, s, top, have, tid, THREADS);
        } else {
            unsigned long long *w = a.ws + (int64_t)item * (3 + a.k);
            if (tid == 0) {
                reinterpret_cast<float2 *>(w)[0] = make_float2(s.m, s.c);
                reinterpret_cast<float2 *>(w)[1] = make_float2(s.r, s.t);
                w[2] = have;
            }
            for (int i = tid; i < have; i += THREADS) w[3 + i] = top[i];
        }
        __syncthreads();  // the shared arrays are written again
    }
}

// Rows of several parts: one block joins a row's statistics and alternatives.
template <typename T>
__global__ void __launch_bounds__(128) logprobs_join_kernel(const __grid_constant__ LpArgs a) {
    pdl_begin();
    __shared__ unsigned long long top[VC_MAX_TOP];
    const int64_t row = blockIdx.x;
    const int size = 3 + a.k;
    const unsigned long long *w = a.ws + row * a.parts * size;
    Stats s{-INFINITY, 0.0f, 0.0f, 0.0f};
    int n = 0;
    bool nan = false;
    for (int p = 0; p < a.parts; ++p) {
        const float2 mc = *reinterpret_cast<const float2 *>(w + p * size);
        const float2 rt = *reinterpret_cast<const float2 *>(w + p * size + 1);
        nan = nan || mc.x != mc.x;
        s = join_stats(s, {mc.x, mc.y, rt.x, rt.y}, a.inv_tau);
        n += (int)w[p * size + 2];
    }
    if (nan) s.m = __int_as_float(0x7fffffff);
    // a key's place: its place in its own part, and the larger ones of the others
    for (int i = threadIdx.x; i < a.parts * a.k; i += blockDim.x) {
        const int p = i / a.k, j = i % a.k;
        if (j >= (int)w[p * size + 2]) continue;
        const unsigned long long key = w[p * size + 3 + j];
        int rank = j;
        for (int o = 0; o < a.parts; ++o) {
            if (o == p) continue;
            const int no = (int)w[o * size + 2];
            for (int q = 0; q < no && w[o * size + 3 + q] > key; ++q) ++rank;
        }
        if (rank < a.k) top[rank] = key;
    }
    __syncthreads();
    finish_row<T>(a, row, s, top, min(n, a.k), threadIdx.x, blockDim.x);
}

// Parts of a row: at most what the largest block holds, of one size.
constexpr int kPartMax = 32768 - 8;  // (a part may start anywhere in its first pack)
int parts_of(int vocab) { return ceil_div(vocab, kPartMax); }

template <typename T>
cudaError_t launch(LpArgs a, cudaStream_t st) {
    constexpr int VEC = Pack<T>::VEC;
    a.parts = parts_of(a.vocab);
    a.part_len = a.parts == 1 ? a.vocab : ceil_div(ceil_div(a.vocab, a.parts), VEC) * VEC;
    const int64_t items = (int64_t)a.rows * a.parts;
    // blocks of a size that holds the part, as many as are resident at once
    auto go = [&](auto kernel, int threads, int per_sm) {
        const int64_t most = (int64_t)152 * per_sm;
        return launch_pdl(kernel, dim3((unsigned)(items < most ? items : most)), threads, 0, st, a);
    };
    constexpr int F = sizeof(T) / 2;  // packs a thread, relative to 16-bit logits
    const int len = a.part_len + VEC - 1;
    cudaError_t e;
    if (len <= 1024)
        e = go(logprobs_kernel<T, 128, F, 8>, 128, 8);
    else if (len <= 4096)
        e = go(logprobs_kernel<T, 128, 4 * F, 8>, 128, 8);
    else if (len <= 16384)
        e = go(logprobs_kernel<T, 512, 4 * F, 2>, 512, 2);
    else if constexpr (F == 1)
        e = go(logprobs_kernel<T, 512, 8, 2>, 512, 2);
    else
        e = go(logprobs_kernel<T, 1024, 8, 1>, 1024, 1);
    if (e == cudaSuccess && a.parts > 1) e = launch_pdl(logprobs_join_kernel<T>, a.rows, 128, 0, st, a);
    return e;
}

}  // namespace
}  // namespace vc

using namespace vc;

extern "C" {

size_t vc_token_logprobs_workspace_bytes(int32_t rows, int32_t vocab, int32_t top_k) {
    if (rows < 0 || vocab < 1 || top_k < 0 || top_k > VC_MAX_TOP) return 0;
    const int parts = parts_of(vocab);
    return parts == 1 ? 8 : (size_t)rows * parts * (3 + top_k) * 8;
}

vc_status vc_token_logprobs(const void *logits, int32_t dtype, int32_t rows, int32_t vocab, int64_t row_stride,
                            const int32_t *ids, int32_t n_ids, float temperature, int32_t top_k, float *logprobs,
                            float *entropy, int32_t *top_ids, float *top_logprobs, void *workspace,
                            size_t workspace_bytes, int32_t *dev_status, vc_stream_t stream) {
    if (rows < 0 || vocab < 1 || row_stride < vocab || n_ids < 0 || top_k < 0 || !(temperature > 0.0f) ||
        !std::isfinite(temperature))
        return VC_ERR_INVALID_ARG;
    if (dtype_bytes(dtype) == 0 || top_k > VC_MAX_TOP) return VC_ERR_UNSUPPORTED;
    if (rows == 0) return VC_OK;
    if (!logits || (n_ids > 0 && (!ids || !logprobs)) || (top_k > 0 && (!top_ids || !top_logprobs)))
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
    a.inv_tau = 1.0f / temperature;
    a.lp = logprobs;
    a.ent = entropy;
    a.top_ids = top_ids;
    a.top_lp = top_logprobs;
    a.status = dev_status;
    const cudaStream_t st = (cudaStream_t)stream;
    const cudaError_t e = dtype == VC_F32    ? launch<float>(a, st)
                          : dtype == VC_BF16 ? launch<__nv_bfloat16>(a, st)
                                             : launch<__half>(a, st);
    return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? VC_OK : VC_ERR_CUDA;
}

}  // extern "C"
