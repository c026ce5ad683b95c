// vc_tree_plan, vc_tree_accept, vc_tree_commit: the bookkeeping of a round
// that drafts a tree of at most 64 nodes.
//
// A node's mask is its own bit and its parent's mask.  Instead of walking up
// to 63 ancestors, every node folds in what its current ancestor has gathered
// and jumps to that one's: after k rounds a mask covers 2^k ancestors, so six
// rounds cover any tree.
#include "vc_internal.cuh"

namespace vc {
namespace {

constexpr int kNodes = VC_MAX_VERIFY_QUERIES;
constexpr int kAbsent = -2;

__global__ void __launch_bounds__(kNodes) tree_plan_kernel(const int32_t *parent, int n_q, const int32_t *lens,
                                                           unsigned long long *mask, int32_t *position,
                                                           int32_t *status) {
    pdl_begin();
    __shared__ unsigned long long ms[kNodes];
    __shared__ int up[kNodes];
    const int i = threadIdx.x;
    const int64_t row = (int64_t)blockIdx.x * n_q;
    const int base = lens[blockIdx.x] - n_q;
    int u = kAbsent;  // current ancestor; -1: none left; kAbsent: not in the tree
    unsigned long long m = 0;
    bool bad = false;
    if (i < n_q) {
        const int p = parent[row + i];
        u = p < -1 ? kAbsent : p;
        bad = base < 0 || u >= i;
        if (bad) u = kAbsent;
        if (u != kAbsent) m = 1ull << i;
    }
    const bool given = u != kAbsent;
    for (int k = 0; k < 6; ++k) {
        ms[i] = m;
        up[i] = u;
        __syncthreads();
        if (u >= 0) {
            m |= ms[u];
            u = up[u];
        }
        __syncthreads();
    }
    if (i >= n_q) return;
    if (u == kAbsent) m = 0;
    if (bad || (given && u == kAbsent)) report(status, VC_ERR_BAD_INDEX);
    mask[row + i] = m;
    position[row + i] = m ? base + __popcll(m) - 1 : -1;
}

// One block per request: every node that carries its parent's prediction
// offers itself as the parent's successor (the lowest index stays), then one
// thread follows the successors from node 0.
__global__ void __launch_bounds__(kNodes) tree_accept_kernel(const int32_t *parent, const int32_t *tokens,
                                                             const int32_t *verified, int n_q, int32_t *accept_len,
                                                             int32_t *path, int32_t *emitted) {
    pdl_begin();
    __shared__ int next[kNodes], walk[kNodes], len;
    const int i = threadIdx.x;
    const int64_t row = (int64_t)blockIdx.x * n_q;
    next[i] = kNodes;
    __syncthreads();
    if (i < n_q) {
        const int p = parent[row + i];
        if (p >= 0 && p < i && tokens[row + i] == verified[row + p]) atomicMin(&next[p], i);
    }
    __syncthreads();
    if (i == 0) {
        int a = -1;
        if (parent[row] == -1)
            for (int cur = 0; cur < kNodes; cur = next[cur]) walk[++a] = cur;
        len = a;
        accept_len[blockIdx.x] = a;
    }
    __syncthreads();
    if (i >= n_q) return;
    path[row + i] = i <= len ? walk[i] : -1;
    emitted[row + i] = i < len ? tokens[row + walk[i + 1]] : i == len ? verified[row + walk[i]] : -1;
}

constexpr int kLayersPerLaunch = 64;
struct CommitArgs {
    uint4 *pool[kLayersPerLaunch][2];
    int64_t n_pages;
    const int32_t *table, *lens, *accept_len, *path;
    int maxb, n_q, hkv, chunks;  // chunks: 16-byte pieces of a head's row
    int32_t *status;
};

// One block per (request, layer).  Each thread moves one 16-byte piece of
// every entry, in path order, four loads under way at a time: a target is not
// above its source and the sources ascend, so no target is a later source.
__global__ void __launch_bounds__(256) tree_commit_kernel(const __grid_constant__ CommitArgs a) {
    pdl_begin();
    __shared__ int64_t src[kNodes], dst[kNodes];  // 16-byte pieces from the pool's start, kv head 0
    __shared__ int broken;
    const int b = blockIdx.x, tid = threadIdx.x;
    const int len = a.accept_len[b], base = a.lens[b] - a.n_q;
    if (len <= 0) {
        if (len < -1 && tid == 0 && blockIdx.y == 0) report(a.status, VC_ERR_BAD_INDEX);
        return;
    }
    if (tid == 0) broken = len >= a.n_q || base < 0;
    __syncthreads();
    if (!broken && tid <= len) {
        const int32_t *p = a.path + (int64_t)b * a.n_q;
        const int from = p[tid];
        if (from >= a.n_q || (tid == 0 ? from != 0 : p[tid - 1] >= from)) broken = 1;
        const int32_t *row = a.table + (int64_t)b * a.maxb;
        auto piece = [&](int pos) -> int64_t {
            const int pg = pos / kPage < a.maxb ? row[pos / kPage] : -1;
            return pg < 0 || pg >= a.n_pages ? -1 : ((int64_t)pg * a.hkv * kPage + pos % kPage) * a.chunks;
        };
        src[tid] = piece(base + min(max(from, 0), a.n_q - 1));
        dst[tid] = piece(base + tid);
        if (src[tid] < 0 || dst[tid] < 0) {
            report(a.status, VC_ERR_BAD_INDEX);
            src[tid] = dst[tid] = -1;
        }
    }
    __syncthreads();
    if (broken) {
        if (tid == 0) report(a.status, VC_ERR_BAD_INDEX);
        return;
    }
    const int items = 2 * a.hkv * a.chunks;
    for (int e = tid; e < items; e += blockDim.x) {
        uint4 *pool = a.pool[blockIdx.y][e >= items / 2];
        const int r = e % (items / 2);
        const int64_t off = (int64_t)(r / a.chunks) * kPage * a.chunks + r % a.chunks;
        for (int j0 = 1; j0 <= len; j0 += 4) {
            uint4 u[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (j0 + k <= len && src[j0 + k] != dst[j0 + k]) u[k] = pool[src[j0 + k] + off];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (j0 + k <= len && src[j0 + k] != dst[j0 + k]) pool[dst[j0 + k] + off] = u[k];
        }
    }
}

}  // namespace
}  // namespace vc

using namespace vc;

extern "C" {

vc_status vc_tree_plan(const int32_t *parent, int32_t batch, int32_t n_q, const int32_t *seq_lens, uint64_t *mask,
                       int32_t *position, int32_t *dev_status, vc_stream_t stream) {
    if (batch < 0 || n_q < 1) return VC_ERR_INVALID_ARG;
    if (n_q > kNodes) return VC_ERR_UNSUPPORTED;
    if (batch == 0) return VC_OK;
    if (!parent || !seq_lens || !mask || !position) return VC_ERR_INVALID_ARG;
    const cudaError_t e = launch_pdl(tree_plan_kernel, batch, kNodes, 0, (cudaStream_t)stream, parent, n_q, seq_lens,
                                     (unsigned long long *)mask, position, dev_status);
    return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? VC_OK : VC_ERR_CUDA;
}

vc_status vc_tree_accept(const int32_t *parent, const int32_t *tokens, const int32_t *verified, int32_t batch,
                         int32_t n_q, int32_t *accept_len, int32_t *path, int32_t *emitted, vc_stream_t stream) {
    if (batch < 0 || n_q < 1) return VC_ERR_INVALID_ARG;
    if (n_q > kNodes) return VC_ERR_UNSUPPORTED;
    if (batch == 0) return VC_OK;
    if (!parent || !tokens || !verified || !accept_len || !path || !emitted) return VC_ERR_INVALID_ARG;
    const cudaError_t e = launch_pdl(tree_accept_kernel, batch, kNodes, 0, (cudaStream_t)stream, parent, tokens,
                                     verified, n_q, accept_len, path, emitted);
    return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? VC_OK : VC_ERR_CUDA;
}

vc_status vc_tree_commit(const vc_paged_kv *layers, int32_t n_layers, int32_t n_q, const int32_t *accept_len,
                         const int32_t *path, int32_t *dev_status, vc_stream_t stream) {
    if (n_layers < 0 || n_q < 1 || (n_layers > 0 && !layers)) return VC_ERR_INVALID_ARG;
    for (int i = 0; i < n_layers; ++i) {
        const vc_paged_kv &l = layers[i], &f = layers[0];
        if (!paged_fmt_ok(&l) || l.fmt.num_kv_heads != f.fmt.num_kv_heads || l.fmt.head_dim != f.fmt.head_dim ||
            l.fmt.bits != f.fmt.bits || l.batch != f.batch || l.max_blocks != f.max_blocks ||
            l.num_pages != f.num_pages || l.block_table != f.block_table || l.seq_lens != f.seq_lens)
            return VC_ERR_INVALID_ARG;
    }
    if (n_q > kNodes || (n_layers > 0 && layers[0].fmt.bits != 16)) return VC_ERR_UNSUPPORTED;
    if (n_layers == 0 || layers[0].batch == 0) return VC_OK;
    if (!accept_len || !path) return VC_ERR_INVALID_ARG;
    for (int i = 0; i < n_layers; ++i)
        if (!paged_ok(&layers[i]) || ((uintptr_t)layers[i].k_pages & 15) || ((uintptr_t)layers[i].v_pages & 15))
            return VC_ERR_INVALID_ARG;
    // a pool given twice would be moved twice at once
    for (int i = 0; i < 2 * n_layers; ++i)
        for (int j = 0; j < i; ++j) {
            auto pool = [&](int k) { return k % 2 ? layers[k / 2].v_pages : layers[k / 2].k_pages; };
            if (pool(i) == pool(j)) return VC_ERR_INVALID_ARG;
        }
    CommitArgs a;
    a.n_pages = layers[0].num_pages;
    a.table = layers[0].block_table;
    a.lens = layers[0].seq_lens;
    a.accept_len = accept_len;
    a.path = path;
    a.maxb = layers[0].max_blocks;
    a.n_q = n_q;
    a.hkv = layers[0].fmt.num_kv_heads;
    a.chunks = layers[0].fmt.head_dim / 8;
    a.status = dev_status;
    for (int l0 = 0; l0 < n_layers; l0 += kLayersPerLaunch) {
        const int n = n_layers - l0 < kLayersPerLaunch ? n_layers - l0 : kLayersPerLaunch;
        for (int i = 0; i < n; ++i) {
            a.pool[i][0] = (uint4 *)layers[l0 + i].k_pages;
            a.pool[i][1] = (uint4 *)layers[l0 + i].v_pages;
        }
        const cudaError_t e =
            launch_pdl(tree_commit_kernel, dim3(layers[0].batch, n), 256, 0, (cudaStream_t)stream, a);
        if (e != cudaSuccess || cudaGetLastError() != cudaSuccess) return VC_ERR_CUDA;
    }
    return VC_OK;
}

}  // extern "C"
