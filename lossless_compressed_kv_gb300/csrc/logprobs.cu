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

// Outputs of row `row`, given its statistics and its `have` largest keys, by
// one warp.  The first 32 tokens asked for and their logits come in registers.
template <typename T>
__device__ void finish_row(const LpArgs &a, int64_t row, Stats s, const unsigned long long *top, int have, int lane,
                           int id, float logit) {
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
// ... which this loads, early, so that the loads' latency is not met at the end.
template <typename T>
__device__ inline int asked(const LpArgs &a, int64_t row, int lane, float &logit) {
    int id = -1;
    logit = 0.0f;
    if (lane < a.n_ids) {
        id = a.ids[row * a.n_ids + lane];
        if (id >= 0 && id < a.vocab) logit = Pack<T>::one(reinterpret_cast<const T *>(a.x) + row * a.stride + id);
    }
    return id;
}

// A part of a row in registers, NV packs a thread; pack j of thread t is pack
// j * THREADS + t of the part (counted from the 16-byte boundary at or before
// its first logit), so loads are whole and a run of neighbours is spread over
// the threads.  Packs behind the part hold -infinity.
template <typename T, int THREADS, int NV>
struct Chunk {
    using P = Pack<T>;
    static constexpr int VEC = P::VEC;
    uint4 x[NV];
    int skew, packs;  // logits before the part in its first pack; packs

    // place (in the part) of the first logit of this thread's pack j
    __device__ int index(int j) const { return (j * THREADS + (int)threadIdx.x) * VEC - skew; }
    __device__ bool holds(int j) const { return j * THREADS + (int)threadIdx.x < packs; }
    __device__ void load(const T *p, int n) {
        skew = (int)((uintptr_t)p & 15) / (int)sizeof(T);
        packs = ceil_div(n + skew, VEC);
        const uint4 *base = reinterpret_cast<const uint4 *>(p - skew) + threadIdx.x;
        const uint4 none = make_uint4(P::kNone, P::kNone, P::kNone, P::kNone);
        // whole packs: [first, last)
        const int first = skew > 0, last = (n + skew) / VEC;
        // an end within a pack: its logits one by one, -infinity beside them
        auto edge = [&](int q) {
            uint32_t w[4] = {P::kNone, P::kNone, P::kNone, P::kNone};
#pragma unroll 1
            for (int e = 0; e < VEC; ++e) {
                const int i = q * VEC - skew + e;
                if (i < 0 || i >= n) continue;
                uint32_t bits, keep, at;
                if constexpr (sizeof(T) == 4) {
                    bits = reinterpret_cast<const uint32_t *>(p)[i];
                    keep = 0;
                    at = e;
                } else {
                    bits = (uint32_t) reinterpret_cast<const uint16_t *>(p)[i] << (16 * (e & 1));
                    keep = e & 1 ? 0xffffu : 0xffff0000u;
                    at = e >> 1;
                }
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (at == k) w[k] = (w[k] & keep) | bits;
            }
            return make_uint4(w[0], w[1], w[2], w[3]);
        };
        const bool cut = last < packs && last >= first;  // the last pack is not whole
        uint4 head = none, end = none;
        if (first && threadIdx.x == 0) head = edge(0);
        if (cut && last % THREADS == threadIdx.x) end = edge(last);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int q = j * THREADS + threadIdx.x;
            if ((j > 0 || first == 0) && (j + 1) * THREADS <= last)  // whole for all threads
                x[j] = __ldcs(base + j * THREADS);
            else
                x[j] = q >= first && q < last ? __ldcs(base + j * THREADS) : cut && q == last ? end : none;
        }
        if (first && threadIdx.x == 0) x[0] = head;
    }
    // The packs are read anew: what was unpacked of them is not kept in registers.
    __device__ void again() {
#pragma unroll
        for (int j = 0; j < NV; ++j) asm volatile("" : "+r"(x[j].x), "+r"(x[j].y), "+r"(x[j].z), "+r"(x[j].w));
    }
};

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

constexpr int kPacks = 256;  // packs with logits not below the bound that are kept (more: the row is read again)

// A kernel's blocks: MAIN threads that go through the logits, NV packs each,
// and one more warp that puts the alternatives in order and writes results.
template <typename T, int MAIN_, int NV_, int MIN_CTAS_>
struct Shape {
    static constexpr int MAIN = MAIN_, NV = NV_, MIN_CTAS = MIN_CTAS_, THREADS = MAIN + 32, WARPS = MAIN / 32;
    static constexpr int CANDS = MAIN >= 64 ? 2048 : 1024;  // logits not below the bound that are put in order
    static constexpr int CAP = MAIN * NV * Pack<T>::VEC - (Pack<T>::VEC - 1);  // logits of a part, wherever it starts
};
__device__ inline void bar_sync(int id, int n) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory"); }
__device__ inline void bar_arrive(int id, int n) { asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(n) : "memory"); }

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
        for (int i = lane; i < above; i += 32) {
            const unsigned long long key = cand[i];
            int rank = 0;
            for (int q = 0; q < above; ++q) rank += cand[q] > key;
            if (rank < k) top[rank] = key;
        }
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

// One block per part of a row, in turn over the parts it owns.  The part stays
// in registers; the main warps meet twice, for the maximum (and the groups'
// maxima) and for the bound, and leave what is left to the last warp, which
// finishes a part while they are at the next.  Memory bounds it at best (64 KB
// of bf16 at an SM's share of the bandwidth take 1.4 us, 2600 cycles), with the
// instructions close behind, so what comes next is asked into L2 before the
// arithmetic begins, and the arithmetic is packed: maxima of 8 logits in 4
// instructions, two logits' differences, products and sums in one; what the
// maximum itself and -infinity need is done by the warps that meet them.
template <typename T, typename S>
__global__ void __launch_bounds__(S::THREADS, S::MIN_CTAS) logprobs_kernel(const __grid_constant__ LpArgs a) {
    pdl_begin();
    using P = Pack<T>;
    constexpr int VEC = P::VEC, NV = S::NV, WARPS = S::WARPS;
    constexpr int GROUPS = S::MAIN < 128 ? S::MAIN : 128;  // at most
    // between the main warps (by turns where one may be at the next part already)
    __shared__ float wmax[2][WARPS], bound_s[2];
    __shared__ float gmax[GROUPS];
    // from them to the last warp, by turns
    struct Hand {
        float m, lo, sum[2][WARPS];
        int n_max, n_pack;
        int at[kPacks];
    };
    __shared__ Hand hand[2];
    __shared__ uint4 pack[2][kPacks];
    // the last warp's own
    __shared__ unsigned long long cand[S::CANDS], top[VC_MAX_TOP];
    __shared__ int n_cand;
    constexpr int kMain = 1, kReady = 2, kFree = 4;  // named barriers; the latter two by turns
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t items = (int64_t)a.rows * a.parts;
    int turn = 0;
    if (warp == WARPS) {
        for (int64_t item = blockIdx.x; item < items; item += gridDim.x, turn ^= 1) {
            const int64_t row = a.parts == 1 ? item : item / a.parts;
            const int v0 = (int)(item - row * a.parts) * a.part_len;
            float logit = 0.0f;
            int id = -1;
            if (a.parts == 1) id = asked<T>(a, row, lane, logit);
            if (lane == 0) n_cand = 0;
            bar_sync(kReady + turn, S::THREADS);
            const Hand &h = hand[turn];
            Stats s{h.m, (float)h.n_max, 0.0f, 0.0f};
            const bool sound = s.m > -INFINITY && s.m < INFINITY;
            const float both =
                warp_sum2(lane < WARPS ? h.sum[0][lane] : 0.0f, lane < WARPS ? h.sum[1][lane] : 0.0f, lane);
            s.r = __shfl_sync(0xffffffffu, both, 0);
            s.t = __shfl_sync(0xffffffffu, both, 16) * 0.6931471805599453f;
            int have = 0;
            if (a.k > 0 && sound) {
                const float lo = h.lo;
                const int np = h.n_pack;
                int n = S::CANDS + 1;
                if (np <= kPacks) {
                    for (int i = lane; i < np; i += 32) {
                        float v[VEC];
                        P::unpack(pack[turn][i], v);
                        const int at_v = h.at[i];
#pragma unroll
                        for (int e = 0; e < VEC; ++e)
                            if (v[e] >= lo && v[e] > -INFINITY) {
                                const int at = atomicAdd(&n_cand, 1);
                                if (at < S::CANDS) cand[at] = order_key(v[e], at_v + e);
                            }
                    }
                    __syncwarp();
                    n = n_cand;
                }
                if (n <= S::CANDS) {
                    // each one's place among them (their order in memory is left to chance, this is not)
                    for (int i = lane; i < n; i += 32) {
                        const unsigned long long key = cand[i];
                        int rank = 0;
                        for (int q = 0; q < n; ++q) rank += cand[q] > key;
                        if (rank < a.k) top[rank] = key;
                    }
                    have = min(a.k, n);
                } else {
                    have = order_again<T>(reinterpret_cast<const T *>(a.x) + row * a.stride + v0, v0,
                                          min(a.part_len, a.vocab - v0), a.k, lo, cand, S::CANDS, top, lane);
                }
                __syncwarp();
            }
            if (item + 2 * (int64_t)gridDim.x < items) bar_arrive(kFree + turn, S::THREADS);
            if (a.parts == 1) {
                finish_row<T>(a, row, s, top, have, lane, id, logit);
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
        return;
    }
    const float scale = a.inv_tau * kLog2e;
    // groups of threads whose maxima bound the k-th largest logit: warps or equal
    // parts of warps, as many as it takes for k groups
    int per = 32;
    while (per > 1 && S::MAIN / per < a.k && 2 * (S::MAIN / per) <= GROUPS) per >>= 1;
    const int groups = S::MAIN / per;
    for (int64_t item = blockIdx.x; item < items; item += gridDim.x, turn ^= 1) {
        const int64_t row = a.parts == 1 ? item : item / a.parts;
        const int v0 = (int)(item - row * a.parts) * a.part_len;
        Chunk<T, S::MAIN, NV> ch;
        ch.load(reinterpret_cast<const T *>(a.x) + row * a.stride + v0, min(a.part_len, a.vocab - v0));
        if (tid == 0) {
            const int64_t ni = item + gridDim.x;
            if (ni < items) {  // the next part: whole 16-byte pieces within it
                const int64_t nr = a.parts == 1 ? ni : ni / a.parts;
                const int nv0 = (int)(ni - nr * a.parts) * a.part_len;
                const T *np = reinterpret_cast<const T *>(a.x) + nr * a.stride + nv0;
                const uintptr_t lo = ((uintptr_t)np + 15) & ~(uintptr_t)15;
                const uintptr_t hi = (uintptr_t)(np + min(a.part_len, a.vocab - nv0)) & ~(uintptr_t)15;
                if (hi > lo)
                    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(lo), "r"((uint32_t)(hi - lo))
                                 : "memory");
            }
        }
        // the hand-over two parts ago has been read
        if (item >= 2 * (int64_t)gridDim.x) bar_sync(kFree + turn, S::THREADS);
        Hand &h = hand[turn];
        if (tid == 0) {
            h.n_pack = h.n_max = 0;
            bound_s[turn] = -INFINITY;
        }
        // ---- maxima ----
        float mine = -INFINITY;  // this thread's maximum
#pragma unroll
        for (int j = 0; j < NV; ++j)
            mine = max_nan(mine, P::max_of(ch.x[j]));
        const float wm = warp_max_nan(mine);
        if (lane == 0) wmax[turn][warp] = wm;
        if (a.k > 1) {
            float g = mine;
            for (int o = 1; o < per; o <<= 1) g = max_nan(g, __shfl_xor_sync(0xffffffffu, g, o));
            if (tid % per == 0) gmax[tid / per] = g;
        }
        bar_sync(kMain, S::MAIN);
        const float m = warp_max_nan(lane < WARPS ? wmax[turn][lane] : -INFINITY);
        const bool sound = m > -INFINITY && m < INFINITY;
        // ---- the bound: the k-th largest of the groups' maxima (k logits at
        // least are not below it; with fewer groups than k: none), by one warp ----
        if (a.k > 1 && sound && warp == WARPS - 1)
            for (int i = lane; i < groups; i += 32) {
                const float own = gmax[i];
                int rank = 0;
                for (int q = 0; q < groups; ++q) {
                    const float o = gmax[q];
                    rank += o > own || (o == own && q < i);
                }
                if (rank == a.k - 1) bound_s[turn] = own;
            }
        // ---- sums ----
        float r2[2] = {0.0f, 0.0f}, t2[2] = {0.0f, 0.0f};  // t in units of log 2
        if (sound) {
            bool careful = wm == m;  // a warp that holds the maximum
            if (!careful) {
                ch.again();
#pragma unroll
                for (int j = 0; j < NV; ++j) {
                    if (!ch.holds(j)) continue;
                    float v[VEC];
                    P::unpack(ch.x[j], v);
#pragma unroll
                    for (int e = 0; e < VEC; e += 2) {
                        float y[2], p[2];
                        sub_mul2(y[0], y[1], v[e], v[e + 1], m, scale);
                        p[0] = ex2(y[0]);
                        p[1] = ex2(y[1]);
                        acc2(r2[0], r2[1], p[0], p[1]);
                        facc2(t2[0], t2[1], p[0], p[1], y[0], y[1]);
                    }
                }
                careful = __any_sync(0xffffffffu, !(t2[0] + t2[1] <= 0.0f));  // -infinity: 0 times infinity
            }
            if (careful) {
                r2[0] = r2[1] = t2[0] = t2[1] = 0.0f;
                ch.again();
#pragma unroll
                for (int j = 0; j < NV; ++j) {
                    if (!ch.holds(j)) continue;
                    float v[VEC], rv[2] = {0.0f, 0.0f}, tv[2] = {0.0f, 0.0f};
                    P::unpack(ch.x[j], v);
#pragma unroll
                    for (int e = 0; e < VEC; e += 2) {
                        float y[2], p[2];
                        sub_mul2(y[0], y[1], v[e], v[e + 1], m, scale);
                        p[0] = ex2(y[0]);
                        p[1] = ex2(y[1]);
                        acc2(rv[0], rv[1], p[0], p[1]);
                        facc2(tv[0], tv[1], p[0], p[1], y[0], y[1]);
                    }
                    if (!(rv[0] + rv[1] < 1.0f && tv[0] + tv[1] <= 0.0f)) {
                        // it may hold the maximum (a term of 1), which is counted
                        // and not added, or -infinity, which the bound keeps out of
                        // y e^y: e^y is 0 long before
                        int c = 0;
                        rv[0] = rv[1] = tv[0] = tv[1] = 0.0f;
#pragma unroll
                        for (int e = 0; e < VEC; ++e) {
                            const float y = fmaxf((v[e] - m) * scale, -10000.0f), p = ex2(y);
                            c += v[e] == m;
                            rv[0] += v[e] == m ? 0.0f : p;
                            tv[0] = fmaf(p, y, tv[0]);
                        }
                        if (c) atomicAdd(&h.n_max, c);
                    }
                    acc2(r2[0], r2[1], rv[0], rv[1]);
                    acc2(t2[0], t2[1], tv[0], tv[1]);
                }
            }
        }
        const float rt = warp_sum2(r2[0] + r2[1], t2[0] + t2[1], lane);
        if ((lane & 15) == 0) h.sum[lane >> 4][warp] = rt;
        // ---- packs with alternatives ----
        float lo = m;
        if (a.k > 1) {
            bar_sync(kMain, S::MAIN);
            lo = bound_s[turn];
        }
        if (a.k > 0 && sound && mine >= lo && mine > -INFINITY) {
            ch.again();
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const float pm = P::max_of(ch.x[j]);
                if (pm >= lo && pm > -INFINITY) {
                    const int at = atomicAdd(&h.n_pack, 1);
                    if (at < kPacks) {
                        pack[turn][at] = ch.x[j];
                        h.at[at] = v0 + ch.index(j);
                    }
                }
            }
        }
        if (tid == 0) {
            h.m = m;
            h.lo = lo;
        }
        bar_arrive(kReady + turn, S::THREADS);
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
    float logit;
    const int id = asked<T>(a, row, threadIdx.x & 31, logit);
    __syncthreads();
    if (threadIdx.x < 32) finish_row<T>(a, row, s, top, min(n, a.k), threadIdx.x, id, logit);
}

// Parts of a row, of one size: what a block of the largest shape holds.
template <typename T>
struct Shapes {
    static constexpr int F = sizeof(T) / 2;  // packs are half as long in fp32
    using Tiny = Shape<T, 32, 4 * F + 1, 12>;
    using Small = Shape<T, 96, 6 * F, 6>;
    using Middle = Shape<T, 480, 5 * F, 2>;
    using Large = Shape<T, 480, 9 * F, 2 / F>;
};
constexpr int kPartMax = Shapes<float>::Large::CAP < Shapes<__half>::Large::CAP ? Shapes<float>::Large::CAP
                                                                                : Shapes<__half>::Large::CAP;
constexpr int kVocabMax = 1 << 22;
void split(int vocab, int &parts, int &len) {
    parts = ceil_div(vocab, kPartMax / 8 * 8);
    len = parts == 1 ? vocab : ceil_div(ceil_div(vocab, parts), 8) * 8;
    parts = ceil_div(vocab, len);
}

template <typename T, typename S>
cudaError_t launch_shape(const LpArgs &a, cudaStream_t st) {
    // as many blocks as are resident at once
    const int64_t items = (int64_t)a.rows * a.parts, most = (int64_t)152 * S::MIN_CTAS;
    return launch_pdl(logprobs_kernel<T, S>, dim3((unsigned)(items < most ? items : most)), S::THREADS, 0, st, a);
}

template <typename T>
cudaError_t launch(LpArgs a, cudaStream_t st) {
    using H = Shapes<T>;
    split(a.vocab, a.parts, a.part_len);
    const int n = a.part_len;
    cudaError_t e = n <= H::Tiny::CAP     ? launch_shape<T, typename H::Tiny>(a, st)
                    : n <= H::Small::CAP  ? launch_shape<T, typename H::Small>(a, st)
                    : n <= H::Middle::CAP ? launch_shape<T, typename H::Middle>(a, st)
                                          : launch_shape<T, typename H::Large>(a, st);
    if (e == cudaSuccess && a.parts > 1) e = launch_pdl(logprobs_join_kernel<T>, a.rows, 128, 0, st, a);
    return e;
}

}  // namespace
}  // namespace vc

using namespace vc;

extern "C" {

size_t vc_token_logprobs_workspace_bytes(int32_t rows, int32_t vocab, int32_t top_k) {
    if (rows < 0 || vocab < 1 || vocab > kVocabMax || top_k < 0 || top_k > VC_MAX_TOP) return 0;
    int parts, len;
    split(vocab, parts, len);
    return parts == 1 ? 8 : (size_t)rows * parts * (3 + top_k) * 8;
}

vc_status vc_token_logprobs(const void *logits, int32_t dtype, int32_t rows, int32_t vocab, int64_t row_stride,
                            const int32_t *ids, int32_t n_ids, float temperature, int32_t top_k, float *logprobs,
                            float *entropy, int32_t *top_ids, float *top_logprobs, void *workspace,
                            size_t workspace_bytes, int32_t *dev_status, vc_stream_t stream) {
    if (rows < 0 || vocab < 1 || row_stride < vocab || n_ids < 0 || top_k < 0 || !(temperature > 0.0f) ||
        !std::isfinite(temperature))
        return VC_ERR_INVALID_ARG;
    if (dtype_bytes(dtype) == 0 || top_k > VC_MAX_TOP || vocab > kVocabMax) return VC_ERR_UNSUPPORTED;
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
