// vc_tree_attn: the verification pass of a tree of drafts over KV_full (see
// tree_tc.cuh for the design).
#include <cmath>

#include "tree_tc.cuh"

namespace vc {
bool verify_supported(const vc_kv_format &f, int hq, int n_q);
bool encode_pool(CUtensorMap *m, const void *pool, int64_t n_pages, int hkv, int d);
namespace {

template <int D, int QT>
__global__ void __launch_bounds__(tree::Cfg<D, QT>::THREADS, tree::Cfg<D, QT>::MIN_CTAS)
    tree_kernel(const __grid_constant__ tree::Args a) {
    pdl_wait();
    extern __shared__ __align__(1024) uint8_t smem[];
    tree::tree_cta<D, QT>(a, smem);
}

template <int D, int QT>
__global__ void __launch_bounds__(tree::kJoinWarps * 32)
    tree_join_kernel(const __grid_constant__ tree::Args a, int warps_per_row) {
    pdl_begin();
    tree::tree_join_block<D, QT>(a, warps_per_row);
}

// How a call is laid out over the GPU (see tree_tc.cuh).
struct Plan {
    int tiles, lanes, groups;  // tiles of a CTA, CTAs per group, groups
    int64_t slots() const { return (int64_t)groups * lanes * 2 * tiles * tree::kTileRows; }  // partial rows
};
Plan plan_of(const vc_paged_kv &f, int n_q, int hq, int max_seq_len) {
    const int tiles = ceil_div(n_q * (hq / f.fmt.num_kv_heads), tree::kTileRows), lanes = tiles == 4 ? 2 : 1;
    constexpr int BK = tree::Cfg<128, 1>::BK;
    const int64_t blocks = (int64_t)f.batch * f.fmt.num_kv_heads * (((int64_t)max_seq_len + BK - 1) / BK);
    const int most = (tiles == 1 ? 2 * tree::kSMs : tree::kSMs) / lanes;
    return {tiles / lanes, lanes, (int)(blocks < 1 ? 1 : blocks < most ? blocks : most)};
}
size_t workspace_of(const Plan &p, int d) { return (size_t)p.slots() * (d + 2) * sizeof(float); }

template <int D, int QT>
cudaError_t launch(const tree::Args &a, cudaStream_t st) {
    using C = tree::Cfg<D, QT>;
    cudaError_t e = set_smem_limit((const void *)tree_kernel<D, QT>, C::SMEM);
    if (e != cudaSuccess) return e;
    e = launch_pdl(tree_kernel<D, QT>, a.groups * a.lanes, C::THREADS, C::SMEM, st, a);
    if (e != cudaSuccess) return e;
    // ranges that a unit spans, were the lengths alike: a warp reads eight at once
    const int ranges = a.groups / (a.batch * a.hkv), W = ranges < 8 ? 1 : ranges < 16 ? 2 : ranges < 32 ? 4 : 8;
    const dim3 grid(a.batch * a.hkv, ceil_div(a.rows, tree::kJoinWarps / W));
    e = launch_pdl(tree_join_kernel<D, QT>, grid, tree::kJoinWarps * 32, 0, st, a, W);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace
}  // namespace vc

using namespace vc;

extern "C" {

size_t vc_tree_workspace_bytes(const vc_paged_kv *full, int32_t n_q, int32_t num_q_heads, int32_t max_seq_len) {
    if (!full || full->batch < 0 || max_seq_len < 0 || n_q < 1 || !verify_supported(full->fmt, num_q_heads, n_q))
        return 0;
    return workspace_of(plan_of(*full, n_q, num_q_heads, max_seq_len), full->fmt.head_dim);
}

vc_status vc_tree_attn(const void *q, int32_t n_q, int32_t num_q_heads, const vc_paged_kv *full,
                       const uint64_t *mask, float softmax_scale, void *out, int32_t out_dtype, int32_t max_seq_len,
                       void *workspace, size_t workspace_bytes, int32_t *dev_status, vc_stream_t stream) {
    if (!paged_fmt_ok(full) || max_seq_len < 0 || n_q < 1 || !(softmax_scale > 0.0f) || !std::isfinite(softmax_scale))
        return VC_ERR_INVALID_ARG;
    const float scale_log2 = softmax_scale * 1.4426950408889634f;
    if (!verify_supported(full->fmt, num_q_heads, n_q) || (out_dtype != VC_F32 && out_dtype != VC_BF16) ||
        !std::isfinite(scale_log2))
        return VC_ERR_UNSUPPORTED;
    // (the kernel counts keys and blocks in 32 bits)
    const int64_t held = (int64_t)full->max_blocks * kPage, longest = held < max_seq_len ? held : max_seq_len;
    if (longest > INT32_MAX - 128 ||
        (longest / tree::Cfg<128, 1>::BK + 1) * full->batch * full->fmt.num_kv_heads > INT32_MAX)
        return VC_ERR_UNSUPPORTED;
    if (full->batch == 0) return VC_OK;
    if (!q || !mask || !out || !paged_ok(full) || ((uintptr_t)q & 15) || ((uintptr_t)out & 15) ||
        ((uintptr_t)full->k_pages & 15) || ((uintptr_t)full->v_pages & 15) || ((uintptr_t)workspace & 31))
        return VC_ERR_INVALID_ARG;
    const Plan p = plan_of(*full, n_q, num_q_heads, max_seq_len);
    const int d = full->fmt.head_dim;
    if (!workspace || workspace_bytes < workspace_of(p, d)) return VC_ERR_WORKSPACE;
    tree::Args a;
    a.q = (const uint16_t *)q;
    a.n_pages = full->num_pages;
    a.table = full->block_table;
    a.lens = full->seq_lens;
    a.mask = (const unsigned long long *)mask;
    a.batch = full->batch;
    a.maxb = full->max_blocks;
    a.n_q = n_q;
    a.hq = num_q_heads;
    a.hkv = full->fmt.num_kv_heads;
    a.grp = num_q_heads / a.hkv;
    a.max_len = (int)longest;
    a.scale_log2 = scale_log2;
    a.ws_o = (float *)workspace;
    a.out = out;
    a.out_bf16 = out_dtype == VC_BF16;
    a.status = dev_status;
    a.wait_ns = wait_fault().wait_ns;
    a.skip_copies = wait_fault().skip_copies;
    if (!encode_pool(&a.kmap, full->k_pages, full->num_pages, a.hkv, d) ||
        !encode_pool(&a.vmap, full->v_pages, full->num_pages, a.hkv, d))
        return VC_ERR_CUDA;
    a.rows = n_q * a.grp;
    a.lanes = p.lanes;
    a.groups = p.groups;
    a.ws_ml = a.ws_o + (size_t)p.slots() * d;
    const cudaStream_t st = (cudaStream_t)stream;
    cudaError_t e;
    if (d == 64)
        e = p.tiles == 1 ? launch<64, 1>(a, st) : p.tiles == 2 ? launch<64, 2>(a, st) : launch<64, 3>(a, st);
    else
        e = p.tiles == 1 ? launch<128, 1>(a, st) : p.tiles == 2 ? launch<128, 2>(a, st) : launch<128, 3>(a, st);
    return e == cudaSuccess ? VC_OK : VC_ERR_CUDA;
}

}  // extern "C"
