// vc_pages_*: which request holds which page of a pool.
//
// The state is three arrays in device memory that the attention calls read as
// they are: block tables, the pages each row holds, and a count of references
// for each page (0: free).  There is no list of free pages to keep in step:
// a page is free when nothing refers to it, and the lowest free ids are taken
// first, so the ids handed out follow from the state alone.
//
// The bookkeeping is latency: a block per row or pair, and one block of 1024
// threads for all rows that ask for pages (a scan of 32768 counts at a time).
// Copies are bound by HBM: 1854 pages of 32 KB in four pools 77 us, 0.94 of its
// measured rate.  A round of 56 forks with their copies takes 30 us, most of it the
// host's four calls.
#include "vc_internal.cuh"

namespace vc {
namespace {

struct Map {
    int32_t *table, *blocks, *refs;
    int64_t n_pages;
    int batch, maxb;
};

// Pages that n tokens take.
__device__ inline int pages_for(int n) { return n / kPage + (n % kPage != 0); }

// ---------------------------------------------------------------------------
// free: one block per row
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(256) pages_free_kernel(Map m, const int32_t *keep, int32_t *status) {
    pdl_begin();
    const int b = blockIdx.x, k = keep[b], have = min(m.blocks[b], m.maxb);
    if (k < 0) return;
    const int left = pages_for(k);
    int32_t *row = m.table + (int64_t)b * m.maxb;
    for (int j = left + threadIdx.x; j < have; j += blockDim.x) {
        const int p = row[j];
        row[j] = -1;
        if (p < 0 || p >= m.n_pages) {
            report(status, VC_ERR_BAD_INDEX);
        } else if (atomicSub(&m.refs[p], 1) <= 0) {  // (not held: put back)
            atomicAdd(&m.refs[p], 1);
            report(status, VC_ERR_BAD_INDEX);
        }
    }
    __syncthreads();
    if (threadIdx.x == 0 && left < have) m.blocks[b] = left;
}

// ---------------------------------------------------------------------------
// fork: one block per pair
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(256) pages_fork_kernel(Map m, int32_t *lens, const int32_t *src, const int32_t *dst,
                                                         int n, int32_t *status) {
    pdl_begin();
    const int i = blockIdx.x, s = src[i], d = dst[i];
    if (s == -1 && d == -1) return;  // no pair
    bool bad = s < 0 || s >= m.batch || d < 0 || d >= m.batch;
    // a row that is made by another pair too, or that another pair reads
    for (int j = threadIdx.x; j < n; j += blockDim.x) bad |= src[j] == d || (j != i && dst[j] == d);
    int have = 0;
    if (!__syncthreads_or(bad)) {
        const int len = lens[s];
        have = pages_for(max(len, 0));
        bad = len < 0 || have > m.blocks[s] || have > m.maxb || m.blocks[d] != 0;
        for (int j = threadIdx.x; j < have && !bad; j += blockDim.x) {
            const int p = m.table[(int64_t)s * m.maxb + j];
            // (other pairs add references meanwhile, but to pages that have some)
            bad = p < 0 || p >= m.n_pages || m.refs[p] <= 0;
        }
    }
    if (__syncthreads_or(bad)) {
        if (threadIdx.x == 0) report(status, VC_ERR_BAD_INDEX);
        return;
    }
    for (int j = threadIdx.x; j < have; j += blockDim.x) {
        const int p = m.table[(int64_t)s * m.maxb + j];
        m.table[(int64_t)d * m.maxb + j] = p;
        atomicAdd(&m.refs[p], 1);
    }
    if (threadIdx.x == 0) {
        m.blocks[d] = have;
        lens[d] = lens[s];
    }
}

// ---------------------------------------------------------------------------
// reserve: one block for all rows
// ---------------------------------------------------------------------------
constexpr int kThreads = 1024;

// Inclusive sum over the block's threads; `all` is the sum of all of them.
template <typename T>
__device__ inline T block_scan(T v, T *warps, T &all) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    for (int o = 1; o < 32; o <<= 1) {
        const T u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
    }
    __syncthreads();  // (the last call's sums have been read)
    if (lane == 31) warps[w] = v;
    __syncthreads();
    T x = lane < (int)blockDim.x / 32 ? warps[lane] : 0;
    for (int o = 1; o < 32; o <<= 1) {
        const T u = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += u;
    }
    all = __shfl_sync(0xffffffffu, x, 31);
    const T before = __shfl_sync(0xffffffffu, x, max(w - 1, 0));
    return v + (w ? before : 0);
}

struct Reserve {
    Map m;
    const int32_t *lens, *want;
    int32_t *granted, *copy_src, *copy_dst;
    int32_t *count, *last;  // [pages]: writers of a shared page, the last of them
    int32_t *fresh;         // [pages]: the free pages to be taken, lowest first
    int32_t *first;         // [batch + 1]: pages taken by the rows before
    int32_t *anew;          // [batch]: shared pages that the row replaces, or kRefused
    int32_t *status;
};

constexpr int kRefused = -1;

// The pages of a row that is to hold positions [len, want): j0 .. j1 - 1 are
// held already and written to, up to `goal` are needed.  ok: so far as the
// lengths tell.
struct Span {
    int j0, j1, have, goal;
    bool writes, ok;
};
__device__ inline Span span_of(const Reserve &a, int b) {
    const int len = a.lens[b], want = a.want[b], have = a.m.blocks[b];
    Span s{0, 0, have, have, want > len, true};
    if (!s.writes) return s;
    const int need = pages_for(want);
    s.ok = len >= 0 && have >= 0 && have <= a.m.maxb && need <= a.m.maxb && pages_for(len) <= have;
    if (!s.ok) return s;
    s.goal = max(have, need);
    s.j0 = len / kPage;
    s.j1 = min(have, need);
    return s;
}
// The same of a row that has been looked at: whether it is served was settled
// by the state that the call found, which handing out pages changes.
__device__ inline Span settled(const Reserve &a, int b) {
    Span s = span_of(a, b);
    if (a.anew[b] == kRefused) {
        s.ok = false;
        s.j1 = s.j0;
    }
    return s;
}
// Whether row b takes a new page in place of p, which others hold as well: not
// if all that hold it write to it now and b is the last of them.
__device__ inline bool replaces(const Reserve &a, int b, int p) {
    const int r = a.m.refs[p];
    return r > 1 && !(a.count[p] == r && a.last[p] == b);
}

__global__ void __launch_bounds__(kThreads) pages_reserve_kernel(const __grid_constant__ Reserve a) {
    pdl_begin();
    __shared__ int warps[32], upto_s;
    __shared__ int64_t wide[32];
    const Map &m = a.m;
    const int tid = threadIdx.x, lane = tid & 31;
    // ---- rows that are refused ----
    for (int b = tid; b < m.batch; b += kThreads) {
        Span s = span_of(a, b);
        for (int j = s.j0; j < s.j1; ++j) {
            const int p = m.table[(int64_t)b * m.maxb + j];
            s.ok &= p >= 0 && p < m.n_pages && m.refs[p] > 0;
        }
        if (!s.ok) report(a.status, VC_ERR_BAD_INDEX);
        a.anew[b] = s.ok ? 0 : kRefused;
    }
    // ---- the writers of each shared page ----
    for (int b = tid; b < m.batch; b += kThreads) {
        const Span s = settled(a, b);
        for (int j = s.j0; j < s.j1; ++j) {
            const int p = m.table[(int64_t)b * m.maxb + j];
            a.count[p] = 0;
            a.last[p] = -1;
        }
    }
    if (tid == 0) upto_s = 0;
    __syncthreads();
    for (int b = tid; b < m.batch; b += kThreads) {
        const Span s = settled(a, b);
        for (int j = s.j0; j < s.j1; ++j) {
            const int p = m.table[(int64_t)b * m.maxb + j];
            atomicAdd(&a.count[p], 1);
            atomicMax(&a.last[p], b);
        }
    }
    __syncthreads();
    // ---- pages that each row takes, and those taken by the rows before ----
    int64_t sum = 0;
    for (int b0 = 0; b0 < m.batch; b0 += kThreads) {
        const int b = b0 + tid;
        int64_t need = 0;
        if (b < m.batch) {
            const Span s = settled(a, b);
            if (s.ok) {
                int n = 0;
                for (int j = s.j0; j < s.j1; ++j) n += replaces(a, b, m.table[(int64_t)b * m.maxb + j]);
                a.anew[b] = n;
                need = n + s.goal - s.have;
            }
        }
        int64_t all;
        const int64_t upto = block_scan(need, wide, all);
        // (the pool's size stands for all that is beyond it)
        if (b < m.batch) a.first[b] = (int)min(sum + upto - need, m.n_pages + 1);
        sum += all;
    }
    const int asked = (int)min(sum, m.n_pages + 1);
    if (tid == 0) a.first[m.batch] = asked;
    // ---- the lowest free pages: a warp looks at 1024 at a time, a lane keeps 32 of them ----
    int found = 0;
    for (int64_t p0 = 0; p0 < m.n_pages && found < asked; p0 += kThreads * 32) {
        const int64_t w0 = p0 + (tid >> 5) * 1024;
        unsigned mine = 0;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            const int64_t p = w0 + i * 32 + lane;
            const unsigned f = __ballot_sync(0xffffffffu, p < m.n_pages && m.refs[p] == 0);
            if (i == lane) mine = f;
        }
        int all;
        int k = found + block_scan(__popc(mine), warps, all) - __popc(mine);
        found += all;
        for (; mine && k < asked; mine &= mine - 1, ++k) a.fresh[k] = (int)(w0 + lane * 32 + __ffs(mine) - 1);
    }
    __syncthreads();
    const int room = min(found, asked);
    // ---- the rows that find all of theirs: first the pages that they replace ----
    for (int b = tid; b < m.batch; b += kThreads) {
        const Span s = settled(a, b);
        const bool ok = s.ok && (!s.writes || a.first[b + 1] <= room);
        int from = -1, to = -1;
        if (ok && s.writes) {
            atomicMax(&upto_s, a.first[b + 1]);
            int32_t *take = a.fresh + a.first[b], *row = m.table + (int64_t)b * m.maxb;
            for (int j = s.j0; j < s.j1; ++j) {
                const int p = row[j];
                if (!replaces(a, b, p)) continue;
                const int page = *take;
                row[j] = page;
                m.refs[page] = 1;
                *take++ = p;  // given back below, once no row asks who holds it
                if (j == s.j0 && a.lens[b] % kPage) {
                    from = p;
                    to = page;
                }
            }
        }
        a.granted[b] = ok;
        a.copy_src[b] = from;
        a.copy_dst[b] = to;
    }
    __syncthreads();
    const int taken = upto_s;
    // ---- then those behind, and the shared pages given back ----
    for (int k = tid; k < taken; k += kThreads) {
        int lo = 0, hi = m.batch;  // first[lo] <= k < first[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (a.first[mid] <= k) lo = mid; else hi = mid;
        }
        const int i = k - a.first[lo] - a.anew[lo], p = a.fresh[k];
        if (i < 0) {
            if (atomicSub(&m.refs[p], 1) <= 0) {  // (more rows gave it up than held it: put back)
                atomicAdd(&m.refs[p], 1);
                report(a.status, VC_ERR_BAD_INDEX);
            }
        } else {
            m.table[(int64_t)lo * m.maxb + m.blocks[lo] + i] = p;
            m.refs[p] = 1;
        }
    }
    __syncthreads();
    for (int b = tid; b < m.batch; b += kThreads)
        if (a.granted[b] && a.want[b] > a.lens[b]) m.blocks[b] = max(m.blocks[b], pages_for(a.want[b]));
}

// ---------------------------------------------------------------------------
// compact: live pages to the lowest ids
// ---------------------------------------------------------------------------
constexpr int kChunk = 4096;  // pages of a block
struct Compact {
    Map m;
    int32_t *src, *dst, *moves, *remap;
    int32_t cap;
    int32_t *live;  // [chunks]: live pages of each
    int32_t *status;
};

__device__ inline int block_sum(int v, int *warps) {
    int all;
    block_scan(v, warps, all);
    return all;
}
__device__ inline int live_of(const Map &m, int64_t p, int64_t end) {
    int n = 0;
    for (int64_t i = p + threadIdx.x; i < end; i += blockDim.x) n += m.refs[i] > 0;
    return n;
}

__global__ void __launch_bounds__(kThreads) pages_count_kernel(const __grid_constant__ Compact a) {
    pdl_begin();
    __shared__ int warps[32];
    const int64_t p0 = (int64_t)blockIdx.x * kChunk;
    const int n = block_sum(live_of(a.m, p0, min(p0 + kChunk, a.m.n_pages)), warps);
    if (threadIdx.x == 0) a.live[blockIdx.x] = n;
}

// N live pages stay at or go to ids below N: the k-th hole there takes the
// k-th live page from N on.
__global__ void __launch_bounds__(kThreads) pages_rank_kernel(const __grid_constant__ Compact a) {
    pdl_begin();
    __shared__ int warps[32];
    const int tid = threadIdx.x;
    int all = 0, before = 0;
    for (int c = tid; c < (int)gridDim.x; c += kThreads) {
        const int n = a.live[c];
        all += n;
        before += c < (int)blockIdx.x ? n : 0;
    }
    const int N = block_sum(all, warps);
    before = block_sum(before, warps);
    // live pages below N
    const int64_t nc = N / kChunk;
    int low = 0;
    for (int c = tid; c < (int)nc; c += kThreads) low += a.live[c];
    low = block_sum(low + live_of(a.m, nc * kChunk, N), warps);
    if (blockIdx.x == 0) {
        if (tid == 0) *a.moves = N - low;
        for (int i = N - low + tid; i < a.cap; i += kThreads) a.src[i] = a.dst[i] = -1;
    }
    const int64_t p0 = (int64_t)blockIdx.x * kChunk;
    for (int i = 0; i < kChunk; i += kThreads) {
        const int64_t p = p0 + i + tid;
        const bool in = p < a.m.n_pages, live = in && a.m.refs[p] > 0;
        int n;
        const int rank = before + block_scan((int)live, warps, n) - live;  // live pages before p
        before += n;
        if (!in) continue;
        if (p < N && !live) a.dst[p - rank] = (int)p;
        if (p >= N && live) a.src[rank - low] = (int)p;
        a.remap[p] = live ? (int)p : -1;  // (of those that move: below)
    }
}

// The same by one block, the moves' marks included, for pools of up to
// kSmallPool pages, a third of them free: 1024 pages 5.0 us where three launches
// take 9.0, 4096 pages 7.4 and 10.8, 8192 pages 10.2 and 11.4, 12000 pages 13.6
// and 12.8, 16384 pages 16.0 and 12.3.
constexpr int kSmallPool = 8192;
__global__ void __launch_bounds__(kThreads) pages_rank_small_kernel(const __grid_constant__ Compact a) {
    pdl_begin();
    __shared__ int warps[32];
    const Map &m = a.m;
    const int tid = threadIdx.x, n = (int)m.n_pages;
    const int N = block_sum(live_of(m, 0, n), warps), low = block_sum(live_of(m, 0, N), warps), moves = N - low;
    int before = 0;
    for (int p0 = 0; p0 < n; p0 += kThreads) {
        const int p = p0 + tid;
        const bool live = p < n && m.refs[p] > 0;
        int all;
        const int rank = before + block_scan((int)live, warps, all) - live;  // live pages before p
        before += all;
        if (p >= n) continue;
        if (p < N && !live) a.dst[p - rank] = p;
        if (p >= N && live) a.src[rank - low] = p;
        a.remap[p] = live ? p : -1;
    }
    __syncthreads();
    for (int i = tid; i < a.cap; i += kThreads) {
        if (i >= moves) {
            a.src[i] = a.dst[i] = -1;
            continue;
        }
        const int s = a.src[i], d = a.dst[i];
        a.remap[s] = d;
        m.refs[d] = m.refs[s];
        m.refs[s] = 0;
    }
    if (tid == 0) *a.moves = moves;
}

__global__ void __launch_bounds__(256) pages_move_kernel(const __grid_constant__ Compact a) {
    pdl_begin();
    const int n = *a.moves;
    for (int i = blockIdx.x * 256 + threadIdx.x; i < n; i += gridDim.x * 256) {
        const int s = a.src[i], d = a.dst[i];
        a.remap[s] = d;
        a.m.refs[d] = a.m.refs[s];
        a.m.refs[s] = 0;
    }
}

// One block per row of the table.
__global__ void __launch_bounds__(256) pages_rename_kernel(const __grid_constant__ Compact a) {
    pdl_begin();
    const int b = blockIdx.x, have = min(a.m.blocks[b], a.m.maxb);
    int32_t *row = a.m.table + (int64_t)b * a.m.maxb;
    for (int j = threadIdx.x; j < have; j += 256) {
        const int p = row[j], to = p >= 0 && p < a.m.n_pages ? a.remap[p] : -1;
        if (to < 0) report(a.status, VC_ERR_BAD_INDEX);
        else row[j] = to;
    }
}

// ---------------------------------------------------------------------------
// copy
// ---------------------------------------------------------------------------
constexpr int kArrays = 64;  // of a launch
struct Copy {
    uint8_t *data[kArrays];
    int32_t pieces[kArrays];  // of a page
    int64_t n_pages;
    const int32_t *src, *dst, *count;
    int n;
    int32_t *status;
};

// Blocks of an array (blockIdx.y) go through its pages' pieces laid end to
// end, 32 KB in a row at a time, U pieces under way in a thread.  (Pieces a whole
// grid apart touch more rows of DRAM at once: 1854 pages of 32 KB in four
// pools 97 us instead of 77; 4 or 2 pieces a thread 79 and 76.)
template <typename T>
__global__ void __launch_bounds__(256) pages_copy_kernel(const __grid_constant__ Copy a) {
    pdl_begin();
    constexpr int U = 8;
    T *data = reinterpret_cast<T *>(a.data[blockIdx.y]);
    const int pieces = a.pieces[blockIdx.y];
    const int n = a.count ? min(max(*a.count, 0), a.n) : a.n;
    const int64_t all = (int64_t)n * pieces;
    for (int64_t e0 = (int64_t)blockIdx.x * (256 * U) + threadIdx.x; e0 < all; e0 += (int64_t)gridDim.x * (256 * U)) {
        T v[U];
        int64_t to[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t e = e0 + u * 256;
            to[u] = -1;
            if (e < all) {
                const int i = all <= INT32_MAX ? (int)((uint32_t)e / (uint32_t)pieces) : (int)(e / pieces);
                const int off = (int)(e - (int64_t)i * pieces), s = a.src[i], d = a.dst[i];
                if (s >= 0 && s < a.n_pages && d >= 0 && d < a.n_pages) {
                    v[u] = data[(int64_t)s * pieces + off];
                    to[u] = (int64_t)d * pieces + off;
                } else if (off == 0 && (s != -1 || d != -1)) {
                    report(a.status, VC_ERR_BAD_INDEX);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (to[u] >= 0) data[to[u]] = v[u];
    }
}

bool map_sizes_ok(const vc_page_map *m) {
    return m && m->batch >= 0 && m->max_blocks >= 0 && m->num_pages >= 0 && m->num_pages < INT32_MAX;
}
bool map_ok(const vc_page_map *m) {
    return m->table && m->blocks && m->refs && m->max_blocks >= 1 && m->num_pages >= 1;
}
Map map_of(const vc_page_map *m) {
    return {m->table, m->blocks, m->refs, m->num_pages, m->batch, m->max_blocks};
}
size_t workspace_of(const vc_page_map *m) {
    return ((size_t)m->num_pages * 3 + (size_t)m->batch * 2 + 1 + 3) / 4 * 16;
}
vc_status done(cudaError_t e) { return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? VC_OK : VC_ERR_CUDA; }

}  // namespace
}  // namespace vc

using namespace vc;

extern "C" {

size_t vc_pages_workspace_bytes(const vc_page_map *map) { return map_sizes_ok(map) ? workspace_of(map) : 0; }

vc_status vc_pages_free(const vc_page_map *map, const int32_t *keep, int32_t *dev_status, vc_stream_t stream) {
    if (!map_sizes_ok(map)) return VC_ERR_INVALID_ARG;
    if (map->batch == 0) return VC_OK;
    if (!map_ok(map) || !keep) return VC_ERR_INVALID_ARG;
    return done(launch_pdl(pages_free_kernel, map->batch, 256, 0, (cudaStream_t)stream, map_of(map), keep, dev_status));
}

vc_status vc_pages_fork(const vc_page_map *map, int32_t *seq_lens, const int32_t *src, const int32_t *dst, int32_t n,
                        int32_t *dev_status, vc_stream_t stream) {
    if (!map_sizes_ok(map) || n < 0) return VC_ERR_INVALID_ARG;
    if (n == 0 || map->batch == 0) return VC_OK;
    if (!map_ok(map) || !seq_lens || !src || !dst) return VC_ERR_INVALID_ARG;
    return done(launch_pdl(pages_fork_kernel, n, 256, 0, (cudaStream_t)stream, map_of(map), seq_lens, src, dst, n,
                           dev_status));
}

vc_status vc_pages_reserve(const vc_page_map *map, const int32_t *seq_lens, const int32_t *want, int32_t *granted,
                           int32_t *copy_src, int32_t *copy_dst, void *workspace, size_t workspace_bytes,
                           int32_t *dev_status, vc_stream_t stream) {
    if (!map_sizes_ok(map)) return VC_ERR_INVALID_ARG;
    if (map->batch == 0) return VC_OK;
    if (!map_ok(map) || !seq_lens || !want || !granted || !copy_src || !copy_dst || ((uintptr_t)workspace & 3))
        return VC_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < workspace_of(map)) return VC_ERR_WORKSPACE;
    Reserve a;
    a.m = map_of(map);
    a.lens = seq_lens;
    a.want = want;
    a.granted = granted;
    a.copy_src = copy_src;
    a.copy_dst = copy_dst;
    a.count = (int32_t *)workspace;
    a.last = a.count + map->num_pages;
    a.fresh = a.last + map->num_pages;
    a.first = a.fresh + map->num_pages;
    a.anew = a.first + map->batch + 1;
    a.status = dev_status;
    return done(launch_pdl(pages_reserve_kernel, 1, kThreads, 0, (cudaStream_t)stream, a));
}

vc_status vc_pages_compact(const vc_page_map *map, int32_t *move_src, int32_t *move_dst, int32_t max_moves,
                           int32_t *moves, int32_t *remap, void *workspace, size_t workspace_bytes,
                           int32_t *dev_status, vc_stream_t stream) {
    // (no more pages can move than half the pool: each leaves one id for another)
    if (!map_sizes_ok(map) || max_moves < map->num_pages / 2) return VC_ERR_INVALID_ARG;
    if ((max_moves > 0 && (!move_src || !move_dst)) || !moves) return VC_ERR_INVALID_ARG;
    const bool none = map->num_pages == 0;  // (no moves, and that is said)
    if (!none && (!map->refs || (map->batch > 0 && !map_ok(map)) || !remap || ((uintptr_t)workspace & 3)))
        return VC_ERR_INVALID_ARG;
    if (!none && (!workspace || workspace_bytes < workspace_of(map))) return VC_ERR_WORKSPACE;
    Compact a;
    a.m = map_of(map);
    a.src = move_src;
    a.dst = move_dst;
    a.moves = moves;
    a.remap = remap;
    a.cap = max_moves;
    a.live = (int32_t *)workspace;
    a.status = dev_status;
    const cudaStream_t st = (cudaStream_t)stream;
    const int chunks = (int)((map->num_pages + kChunk - 1) / kChunk);
    cudaError_t e;
    if (map->num_pages <= kSmallPool) {
        e = launch_pdl(pages_rank_small_kernel, 1, kThreads, 0, st, a);
    } else {
        e = launch_pdl(pages_count_kernel, chunks, kThreads, 0, st, a);
        if (e == cudaSuccess) e = launch_pdl(pages_rank_kernel, chunks, kThreads, 0, st, a);
        if (e == cudaSuccess) e = launch_pdl(pages_move_kernel, min(ceil_div((int)(map->num_pages / 2) + 1, 256), 304), 256, 0, st, a);
    }
    if (e == cudaSuccess && map->batch > 0 && !none) e = launch_pdl(pages_rename_kernel, map->batch, 256, 0, st, a);
    return done(e);
}

vc_status vc_pages_copy(const vc_page_array *arrays, int32_t n_arrays, int64_t num_pages, const int32_t *src,
                        const int32_t *dst, int32_t n, const int32_t *count, int32_t *dev_status, vc_stream_t stream) {
    if (n_arrays < 0 || num_pages < 0 || n < 0 || (n_arrays > 0 && !arrays)) return VC_ERR_INVALID_ARG;
    for (int i = 0; i < n_arrays; ++i)
        if (!arrays[i].data || arrays[i].page_bytes < 1 || arrays[i].page_bytes % 4 || ((uintptr_t)arrays[i].data & 3))
            return VC_ERR_INVALID_ARG;
    for (int i = 0; i < n_arrays; ++i)
        if (arrays[i].page_bytes > INT32_MAX) return VC_ERR_UNSUPPORTED;
    if (n_arrays == 0 || n == 0) return VC_OK;
    if (!src || !dst || num_pages < 1) return VC_ERR_INVALID_ARG;
    Copy a;
    a.n_pages = num_pages;
    a.src = src;
    a.dst = dst;
    a.count = count;
    a.n = n;
    a.status = dev_status;
    // pages whose bytes allow it in pieces of 16, the others (scales) in pieces of 4
    for (int wide = 1; wide >= 0; --wide) {
        const int size = wide ? 16 : 4;
        for (int i = 0; i < n_arrays;) {
            int k = 0;
            int64_t most = 0;
            for (; i < n_arrays && k < kArrays; ++i) {
                const vc_page_array &x = arrays[i];
                if ((x.page_bytes % 16 == 0 && !((uintptr_t)x.data & 15)) != (wide == 1)) continue;
                a.data[k] = (uint8_t *)x.data;
                a.pieces[k] = (int32_t)(x.page_bytes / size);
                most = most < a.pieces[k] ? a.pieces[k] : most;
                ++k;
            }
            if (k == 0) continue;
            // blocks that fill the GPU eight times over between the arrays, or as many as there are pieces for
            const int64_t blocks = ((int64_t)n * most + 256 * 8 - 1) / (256 * 8), fill = ceil_div(152 * 8, k);
            const dim3 grid((unsigned)(blocks < fill ? blocks : fill), k);
            const cudaError_t e = wide ? launch_pdl(pages_copy_kernel<uint4>, grid, 256, 0, (cudaStream_t)stream, a)
                                       : launch_pdl(pages_copy_kernel<uint32_t>, grid, 256, 0, (cudaStream_t)stream, a);
            if (e != cudaSuccess || cudaGetLastError() != cudaSuccess) return VC_ERR_CUDA;
        }
    }
    return VC_OK;
}

}  // extern "C"
