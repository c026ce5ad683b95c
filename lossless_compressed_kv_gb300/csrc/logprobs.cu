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

template <typename T>
__device__ inline float logit(T v);
template <>
__device__ inline float logit<float>(float v) { return v; }
template <>
__device__ inline float logit<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ inline float logit<__half>(__half v) { return __half2float(v); }

// Order-preserving key: value bits mapped to an unsigned order in the high
// word (-0 folded onto +0 first), the complement of the id in the low word;
// every key of a logit above -infinity is larger than key_floor().
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
__device__ inline unsigned long long key_floor() { return ((unsigned long long)0x007fffffu << 32) | 0xffffffffu; }

struct LpArgs {
    const void *x;
    int64_t stride;
    int vocab;
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
            v = bad ? nan : none ? -INFINITY : (logit<T>(x[id]) - s.m) * a.inv_tau - log_s;
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

template <typename V, typename F>
__device__ V block_reduce(V v, V *sh, F f) {
    for (int o = 16; o > 0; o >>= 1) v = f(v, __shfl_xor_sync(0xffffffffu, v, o));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
    __syncthreads();
    v = sh[0];
    for (int w = 1; w < (int)blockDim.x / 32; ++w) v = f(v, sh[w]);
    return v;
}

// One block per row: a pass for the maximum, one for the sums, and one for
// each alternative (the largest key below the last one).
template <typename T>
__global__ void __launch_bounds__(256) logprobs_row_kernel(LpArgs a) {
    pdl_begin();
    __shared__ float fs[8];
    __shared__ unsigned long long ks[8], top[VC_MAX_TOP];
    const int64_t row = blockIdx.x;
    const T *x = reinterpret_cast<const T *>(a.x) + row * a.stride;
    auto add = [](float p, float q) { return p + q; };
    // a NaN stays: fmaxf would drop it
    auto larger = [](float p, float q) { return p != p || p > q ? p : q; };
    Stats s{-INFINITY, 0.0f, 0.0f, 0.0f};
    for (int v = threadIdx.x; v < a.vocab; v += blockDim.x) s.m = larger(s.m, logit<T>(x[v]));
    s.m = block_reduce(s.m, fs, larger);
    if (s.m > -INFINITY && s.m < INFINITY) {
        for (int v = threadIdx.x; v < a.vocab; v += blockDim.x) {
            const float l = logit<T>(x[v]);
            // (e^-10000 is 0: the bound keeps -infinity out of y e^y)
            const float y = fmaxf((l - s.m) * a.inv_tau, -10000.0f), e = ex2(y * kLog2e);
            if (l == s.m)
                s.c += 1.0f;
            else
                s.r += e;
            s.t += y * e;
        }
        s.c = block_reduce(s.c, fs, add);
        s.r = block_reduce(s.r, fs, add);
        s.t = block_reduce(s.t, fs, add);
    }
    int have = 0;
    unsigned long long last = ~0ull;
    auto larger_key = [](unsigned long long p, unsigned long long q) { return p > q ? p : q; };
    for (; have < a.k; ++have) {
        unsigned long long best = 0;
        for (int v = threadIdx.x; v < a.vocab; v += blockDim.x) {
            const unsigned long long key = order_key(logit<T>(x[v]), v);
            if (key < last && key > best) best = key;
        }
        last = block_reduce(best, ks, larger_key);
        if (last <= key_floor()) break;
        if (threadIdx.x == 0) top[have] = last;
    }
    __syncthreads();
    finish_row<T>(a, row, s, top, have, threadIdx.x, blockDim.x);
}

}  // namespace
}  // namespace vc

using namespace vc;

extern "C" {

size_t vc_token_logprobs_workspace_bytes(int32_t rows, int32_t vocab, int32_t top_k) {
    if (rows < 0 || vocab < 1 || top_k < 0 || top_k > VC_MAX_TOP) return 0;
    return 8;
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
    if (!workspace || workspace_bytes < vc_token_logprobs_workspace_bytes(rows, vocab, top_k))
        return VC_ERR_WORKSPACE;
    LpArgs a;
    a.x = logits;
    a.stride = row_stride;
    a.vocab = vocab;
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
    cudaError_t e;
    if (dtype == VC_F32)
        e = launch_pdl(logprobs_row_kernel<float>, rows, 256, 0, st, a);
    else if (dtype == VC_BF16)
        e = launch_pdl(logprobs_row_kernel<__nv_bfloat16>, rows, 256, 0, st, a);
    else
        e = launch_pdl(logprobs_row_kernel<__half>, rows, 256, 0, st, a);
    return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? VC_OK : VC_ERR_CUDA;
}

}  // extern "C"
