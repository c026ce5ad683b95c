// vc_tree_attn: attention of a tree of drafted tokens over KV_full.
//
//   out[i] = sum_t softmax_t(scale <q_i, k_t>) v_t   over the prefix and the
//   entries of the tree whose bit is set in node i's mask.
#include <cmath>

#include "vc_internal.cuh"

namespace vc {
bool verify_supported(const vc_kv_format &f, int hq, int n_q);
namespace {

struct TreeArgs {
    const uint16_t *q;
    const uint16_t *kp, *vp;
    int64_t n_pages;
    const int32_t *table, *lens;
    const unsigned long long *mask;
    int batch, maxb, n_q, hq, hkv, max_len;
    float scale_log2;
    void *out;
    int out_bf16;
    int32_t *status;
};

// One warp per (node, query head): 32 keys at a time, lane = key for the
// scores, lane = channels for the sum over V.
template <int D>
__global__ void __launch_bounds__(128) tree_rows_kernel(TreeArgs a) {
    pdl_begin();
    constexpr int C = D / 32;
    const int lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int rows = a.n_q * a.hq;
    const int b = (int)(row / rows);
    if (b >= a.batch) return;
    const int i = (int)(row % rows) / a.hq, h = (int)(row % a.hq), kvh = h / (a.hq / a.hkv);
    const int len = a.lens[b], base = len - a.n_q;
    const bool ok = base >= 0 && len <= a.max_len;
    if (!ok && lane == 0) report(a.status, VC_ERR_BAD_INDEX);
    const unsigned long long mask = a.mask[(int64_t)b * a.n_q + i] & (~0ull >> (64 - a.n_q));
    const uint16_t *q = a.q + row * D;
    float o[C] = {}, m = -INFINITY, l = 0.0f;
    const int n = ok && mask ? len : 0;
    for (int t0 = 0; t0 < n; t0 += 32) {
        const int t = t0 + lane;
        const bool seen = t < base || (t < len && ((mask >> (t - base)) & 1));
        int64_t off = -1;
        float s = -INFINITY;
        if (seen) {
            const int pg = t / kPage < a.maxb ? a.table[(int64_t)b * a.maxb + t / kPage] : -1;
            if (pg < 0 || pg >= a.n_pages) {
                report(a.status, VC_ERR_BAD_INDEX);
            } else {
                off = (((int64_t)pg * a.hkv + kvh) * kPage + t % kPage) * D;
                s = 0.0f;
                for (int c = 0; c < D; ++c) s = fmaf(bf16_bits_to_f32(q[c]), bf16_bits_to_f32(a.kp[off + c]), s);
                s *= a.scale_log2;
            }
        }
        float mx = s;
        for (int w = 16; w > 0; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
        const float mn = fmaxf(m, mx);
        if (mn == -INFINITY) continue;
        const float f = ex2(m - mn), p = ex2(s - mn);
        m = mn;
        l = l * f + p;
        for (int c = 0; c < C; ++c) o[c] *= f;
        for (int j = 0; j < 32; ++j) {
            const float pj = __shfl_sync(0xffffffffu, p, j);
            const int64_t oj = __shfl_sync(0xffffffffu, off, j);
            if (oj >= 0)
                for (int c = 0; c < C; ++c) o[c] = fmaf(pj, bf16_bits_to_f32(a.vp[oj + lane * C + c]), o[c]);
        }
    }
    for (int w = 16; w > 0; w >>= 1) l += __shfl_xor_sync(0xffffffffu, l, w);
    for (int c = 0; c < C; ++c) {
        const float v = m == -INFINITY ? 0.0f : o[c] / l;
        if (a.out_bf16)
            ((uint16_t *)a.out)[row * D + lane * C + c] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
        else
            ((float *)a.out)[row * D + lane * C + c] = v;
    }
}

}  // namespace
}  // namespace vc

using namespace vc;

extern "C" {

size_t vc_tree_workspace_bytes(const vc_paged_kv *full, int32_t n_q, int32_t num_q_heads, int32_t max_seq_len) {
    if (!full || full->batch < 0 || max_seq_len < 0 || !verify_supported(full->fmt, num_q_heads, n_q)) return 0;
    return 16;
}

vc_status vc_tree_attn(const void *q, int32_t n_q, int32_t num_q_heads, const vc_paged_kv *full,
                       const uint64_t *mask, float softmax_scale, void *out, int32_t out_dtype, int32_t max_seq_len,
                       void *workspace, size_t workspace_bytes, int32_t *dev_status, vc_stream_t stream) {
    if (!paged_fmt_ok(full) || max_seq_len < 0 || n_q < 1 || !(softmax_scale > 0.0f) || !std::isfinite(softmax_scale))
        return VC_ERR_INVALID_ARG;
    if (!verify_supported(full->fmt, num_q_heads, n_q) || (out_dtype != VC_F32 && out_dtype != VC_BF16))
        return VC_ERR_UNSUPPORTED;
    if (full->batch == 0) return VC_OK;
    if (!q || !mask || !out || !paged_ok(full) || ((uintptr_t)q & 15) || ((uintptr_t)out & 15) ||
        ((uintptr_t)full->k_pages & 15) || ((uintptr_t)full->v_pages & 15))
        return VC_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < vc_tree_workspace_bytes(full, n_q, num_q_heads, max_seq_len))
        return VC_ERR_WORKSPACE;
    TreeArgs a;
    a.q = (const uint16_t *)q;
    a.kp = (const uint16_t *)full->k_pages;
    a.vp = (const uint16_t *)full->v_pages;
    a.n_pages = full->num_pages;
    a.table = full->block_table;
    a.lens = full->seq_lens;
    a.mask = (const unsigned long long *)mask;
    a.batch = full->batch;
    a.maxb = full->max_blocks;
    a.n_q = n_q;
    a.hq = num_q_heads;
    a.hkv = full->fmt.num_kv_heads;
    a.max_len = max_seq_len;
    a.scale_log2 = softmax_scale * 1.4426950408889634f;
    a.out = out;
    a.out_bf16 = out_dtype == VC_BF16;
    a.status = dev_status;
    const int64_t rows = (int64_t)full->batch * n_q * num_q_heads;
    const unsigned grid = (unsigned)((rows + 3) / 4);
    const cudaError_t e = full->fmt.head_dim == 64
                              ? launch_pdl(tree_rows_kernel<64>, grid, 128, 0, (cudaStream_t)stream, a)
                              : launch_pdl(tree_rows_kernel<128>, grid, 128, 0, (cudaStream_t)stream, a);
    return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? VC_OK : VC_ERR_CUDA;
}

}  // extern "C"
