// vc_kv8_attn: attention over a cache held in 8 bits (see kv8.cuh).
#include <atomic>
#include <cmath>

#include "kv8_one.cuh"

namespace vc {
bool encode_pool8(CUtensorMap *m, const void *pool, int64_t n_pages, int hkv, int d);
namespace {

template <int D, int NT, bool E4M3>
__global__ void __launch_bounds__(kv8::Few<D, NT>::THREADS, kv8::Few<D, NT>::CTAS)
    kv8_few_kernel(const __grid_constant__ kv8::Args a) {
    pdl_wait();
    extern __shared__ __align__(1024) uint8_t smem[];
    kv8::few_warp<D, NT, E4M3>(a, smem);
    pdl_trigger();
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(kv8::One<D>::THREADS, 1) kv8_one_kernel(const __grid_constant__ kv8::Args a) {
    pdl_wait();
    extern __shared__ __align__(1024) uint8_t smem[];
    kv8::one_cta<D, E4M3>(a, smem);
}

template <int D, int QT, bool E4M3>
__global__ void __launch_bounds__(kv8::Tc<D, QT>::THREADS, 1) kv8_tc_kernel(const __grid_constant__ kv8::Args a) {
    pdl_wait();
    extern __shared__ __align__(1024) uint8_t smem[];
    kv8::tc_cta<D, QT, E4M3>(a, smem);
}

template <int D, int BK>
__global__ void __launch_bounds__(kv8::kJoinWarps * 32)
    kv8_join_kernel(const __grid_constant__ kv8::Args a, int lane_rows) {
    pdl_begin();
    kv8::join_block<D, BK>(a, lane_rows);
}

bool supported(const vc_paged_kv8 &kv, int n_q, int hq) {
    const int d = kv.head_dim, hkv = kv.num_kv_heads;
    return (kv.code == VC_E4M3 || kv.code == VC_INT8) && (d == 64 || d == 128) && hkv >= 1 && hq >= hkv &&
           hq % hkv == 0 && hq / hkv <= VC_MAX_GQA_GROUP && n_q >= 1 && n_q <= VC_MAX_VERIFY_QUERIES;
}

// Rows that go to kv8_few.cuh at most.  More go to kv8_one.cuh, whose time
// hardly depends on their number (8 x 32768 keys, head_dim 128: 16 rows 112 us
// in the first, 158 in the second; 20 rows 276 and 160: so many accumulators
// leave a scheduler two warps.  head_dim 64: 32 rows 104 and 125 us).
constexpr int few_rows(int d) { return d == 64 ? 32 : 16; }

// How a call is laid out over the GPU.
struct Plan {
    int nt, tiles;                  // kv8_few.cuh: eights of rows of a warp; else tiles of a CTA
    int lanes, lane_rows, groups;   // CTAs that share a range, the rows of one, ranges of the context
    int64_t slots() const { return (int64_t)groups * lanes * 2 * lane_rows; }  // partial rows
};
Plan plan_of(const vc_paged_kv8 &kv, int n_q, int hq, int max_seq_len) {
    const int rows = n_q * (hq / kv.num_kv_heads);
    Plan p{};
    int most, block;
    if (rows <= few_rows(kv.head_dim)) {
        p.nt = rows <= 8 ? 1 : rows <= 16 ? 2 : 4;
        p.lanes = 1;
        p.lane_rows = 8 * p.nt;
        most = tree::kSMs * 4 * (p.nt == 1 ? 4 : p.nt == 2 ? 3 : 2);
        block = kPage;
    } else {
        const int tiles = ceil_div(rows, kv8::kTileRows);
        p.lanes = tiles == 4 ? 2 : 1;
        p.tiles = tiles / p.lanes;
        p.lane_rows = p.tiles * kv8::kTileRows;
        most = tree::kSMs / p.lanes;
        block = kv8::One<128>::BK;
    }
    const int64_t blocks = (int64_t)kv.batch * kv.num_kv_heads * (((int64_t)max_seq_len + block - 1) / block);
    p.groups = (int)(blocks < 1 ? 1 : blocks < most ? blocks : most);
    return p;
}
size_t workspace_of(const Plan &p, int d) { return (size_t)p.slots() * (d + 2) * sizeof(float); }

template <int D, int BK>
cudaError_t launch_join(const kv8::Args &a, int lane_rows, cudaStream_t st) {
    // blocks for a go through all rows, were the lengths alike; a few more for a unit that
    // spans more ranges than the others
    const int W = kv8::join_warps(a.groups / (a.batch * a.hkv)), some = ceil_div(a.rows, kv8::kJoinWarps / W);
    const dim3 grid(a.batch * a.hkv, some < 4 ? (a.rows < 4 ? a.rows : 4) : some);
    const cudaError_t e = launch_pdl(kv8_join_kernel<D, BK>, grid, kv8::kJoinWarps * 32, 0, st, a, lane_rows);
    return e != cudaSuccess ? e : cudaGetLastError();
}
template <int D, int NT, bool E4M3>
cudaError_t launch_few(const kv8::Args &a, cudaStream_t st) {
    using F = kv8::Few<D, NT>;
    cudaError_t e = set_smem_limit((const void *)kv8_few_kernel<D, NT, E4M3>, F::SMEM);
    if (e != cudaSuccess) return e;
    e = launch_pdl(kv8_few_kernel<D, NT, E4M3>, ceil_div(a.groups, F::WARPS), F::THREADS, F::SMEM, st, a);
    return e != cudaSuccess ? e : launch_join<D, kPage>(a, F::ROWS, st);
}
// (C: One or Tc)
template <class C, int D, void (*kernel)(kv8::Args)>
cudaError_t launch_tiles(const kv8::Args &a, cudaStream_t st) {
    // the warps share out the registers that the block is launched with
    static std::atomic<int> known{0};
    int regs = known.load();
    if (regs == 0) {
        cudaFuncAttributes f;
        const cudaError_t e = cudaFuncGetAttributes(&f, kernel);
        if (e != cudaSuccess) return e;
        known.store(regs = f.numRegs);
    }
    if (regs * C::WARPS < C::REGS_SOFTMAX * C::SM_WARPS + C::REGS_OTHER * (C::WARPS - C::SM_WARPS))
        return cudaErrorInvalidConfiguration;
    cudaError_t e = set_smem_limit((const void *)kernel, C::SMEM);
    if (e != cudaSuccess) return e;
    e = launch_pdl(kernel, a.groups * a.lanes, C::THREADS, C::SMEM, st, a);
    return e != cudaSuccess ? e : launch_join<D, C::BK>(a, C::ROWS, st);
}
template <int D, bool E4M3>
cudaError_t launch(const Plan &p, const kv8::Args &a, cudaStream_t st) {
    if (p.nt == 1) return launch_few<D, 1, E4M3>(a, st);
    if (p.nt == 2) return launch_few<D, 2, E4M3>(a, st);
    if constexpr (few_rows(D) > 16)
        if (p.nt == 4) return launch_few<D, 4, E4M3>(a, st);
    return p.tiles == 1   ? launch_tiles<kv8::One<D>, D, kv8_one_kernel<D, E4M3>>(a, st)
           : p.tiles == 2 ? launch_tiles<kv8::Tc<D, 2>, D, kv8_tc_kernel<D, 2, E4M3>>(a, st)
                          : launch_tiles<kv8::Tc<D, 3>, D, kv8_tc_kernel<D, 3, E4M3>>(a, st);
}

}  // namespace

// The sizes of an 8-bit cache, and its pointers.
bool kv8_sizes_ok(const vc_paged_kv8 *p) {
    return p && p->batch >= 0 && p->num_kv_heads >= 1 && p->head_dim >= 1 && p->num_pages >= 0;
}
bool kv8_ok(const vc_paged_kv8 *p) {
    return p->k_codes && p->v_codes && p->k_scales && p->v_scales && p->block_table && p->max_blocks >= 1 &&
           p->num_pages >= 1 && !((uintptr_t)p->k_codes & 15) && !((uintptr_t)p->v_codes & 15) &&
           !((uintptr_t)p->k_scales & 3) && !((uintptr_t)p->v_scales & 3);
}

}  // namespace vc

using namespace vc;

extern "C" {

size_t vc_kv8_workspace_bytes(const vc_paged_kv8 *kv, int32_t n_q, int32_t num_q_heads, int32_t max_seq_len) {
    if (!kv8_sizes_ok(kv) || max_seq_len < 0 || !supported(*kv, n_q, num_q_heads)) return 0;
    return workspace_of(plan_of(*kv, n_q, num_q_heads, max_seq_len), kv->head_dim);
}

vc_status vc_kv8_attn(const void *q, int32_t n_q, int32_t num_q_heads, const vc_paged_kv8 *kv, const uint64_t *mask,
                      float softmax_scale, void *out, int32_t out_dtype, int32_t max_seq_len, void *workspace,
                      size_t workspace_bytes, int32_t *dev_status, vc_stream_t stream) {
    if (!kv8_sizes_ok(kv) || max_seq_len < 0 || n_q < 1 || !(softmax_scale > 0.0f) || !std::isfinite(softmax_scale))
        return VC_ERR_INVALID_ARG;
    const float scale_log2 = softmax_scale * 1.4426950408889634f;
    if (!supported(*kv, n_q, num_q_heads) || (out_dtype != VC_F32 && out_dtype != VC_BF16) || !std::isfinite(scale_log2))
        return VC_ERR_UNSUPPORTED;
    // (the kernels count keys, the pages of a call, and the rows of a pool, in 32 bits)
    const int64_t held = (int64_t)kv->max_blocks * kPage, longest = held < max_seq_len ? held : max_seq_len;
    if (longest > INT32_MAX - 128 || (longest / kPage + 1) * kv->batch * kv->num_kv_heads > INT32_MAX ||
        kv->num_pages > INT32_MAX / kPage / kv->num_kv_heads)
        return VC_ERR_UNSUPPORTED;
    if (kv->batch == 0) return VC_OK;
    if (!q || !out || !kv8_ok(kv) || !kv->seq_lens || ((uintptr_t)q & 15) || ((uintptr_t)out & 15) || ((uintptr_t)workspace & 31))
        return VC_ERR_INVALID_ARG;
    const Plan p = plan_of(*kv, n_q, num_q_heads, max_seq_len);
    const int d = kv->head_dim;
    if (!workspace || workspace_bytes < workspace_of(p, d)) return VC_ERR_WORKSPACE;
    kv8::Args a;
    a.kc = (const uint8_t *)kv->k_codes;
    a.vc = (const uint8_t *)kv->v_codes;
    a.ks = kv->k_scales;
    a.vs = kv->v_scales;
    a.q = (const uint16_t *)q;
    a.n_pages = kv->num_pages;
    a.table = kv->block_table;
    a.lens = kv->seq_lens;
    a.mask = (const unsigned long long *)mask;
    a.batch = kv->batch;
    a.maxb = kv->max_blocks;
    a.n_q = n_q;
    a.hq = num_q_heads;
    a.hkv = kv->num_kv_heads;
    a.grp = num_q_heads / a.hkv;
    a.max_len = (int)longest;
    a.rows = n_q * a.grp;
    a.lanes = p.lanes;
    a.groups = p.groups;
    a.scale_log2 = scale_log2;
    a.ws_o = (float *)workspace;
    a.ws_ml = a.ws_o + (size_t)p.slots() * d;
    a.out = out;
    a.out_bf16 = out_dtype == VC_BF16;
    a.status = dev_status;
    a.wait_ns = wait_fault().wait_ns;
    a.skip_copies = wait_fault().skip_copies;
    if (p.tiles > 1 && (!encode_pool8(&a.kmap, kv->k_codes, kv->num_pages, a.hkv, d) ||
                        !encode_pool8(&a.vmap, kv->v_codes, kv->num_pages, a.hkv, d)))
        return VC_ERR_CUDA;
    const cudaStream_t st = (cudaStream_t)stream;
    const bool e4m3 = kv->code == VC_E4M3;
    const cudaError_t e = d == 64 ? (e4m3 ? launch<64, true>(p, a, st) : launch<64, false>(p, a, st))
                                  : (e4m3 ? launch<128, true>(p, a, st) : launch<128, false>(p, a, st));
    return e == cudaSuccess ? VC_OK : VC_ERR_CUDA;
}

}  // extern "C"
