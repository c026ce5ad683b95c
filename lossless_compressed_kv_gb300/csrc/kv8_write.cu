// vc_kv8_write: pages of KV_full held in 8 bits with a scale for each page and
// kv head.
//
// One pass: a warp holds a block (16 rows of K or of V of one kv head) in
// registers, 16 values a piece, so that the largest magnitude, the scale and
// the codes come of one read.  Read 2 bytes and written 1 byte a value; HBM
// bounds it (64750 tokens of 8 heads of 128, K and V: 63 us, 0.93 of measured
// HBM).  The blocks of all requests, laid end to end, are dealt out in equal
// ranges to the warps of a grid that fills the GPU once: neighbouring warps take
// neighbouring heads, and a call with one new page a request costs little more
// than its pages (8 requests 3.9 us, 64 6.2, 1000 56).  A page that several
// requests hold is made from the longest of them by each (holder_of).
#include "vc_internal.cuh"

namespace vc {
bool kv8_sizes_ok(const vc_paged_kv8 *p);
bool kv8_ok(const vc_paged_kv8 *p);
namespace {

constexpr int kWarps = 8;

struct WriteArgs {
    const uint8_t *kp, *vp;  // full pools
    int64_t f_pages, d_pages;
    const int32_t *f_table, *lens, *first, *d_table;
    int f_maxb, d_maxb, batch, hkv, max_len;
    uint8_t *kc, *vc;
    float *ks, *vs;
    int32_t *status;
};

// Pages of request b that are made anew.
__device__ inline int pages_of(const WriteArgs &a, int b) {
    const int len = a.lens[b], first = a.first ? a.first[b] : 0;
    if (first < 0 || len < 0 || len > a.max_len) return 0;
    return first >= len ? 0 : (len - 1) / kPage + 1 - first / kPage;
}

// The request whose tokens page `dst`, the pg-th of request b, is made of: the
// one with the most tokens in it (the first of those) among all that hold it
// there.  By a warp; `left`: b's tokens in it, then the holder's.  Holders of
// unequal lengths write the same page in one call, in no order, so each of
// them writes what the longest one does.  (Looked for where b's tokens end in
// the page: a full one holds all there are.)
__device__ inline int holder_of(const WriteArgs &a, int b, int pg, int dst, int lane, int &left) {
    int most = left, who = b;
    for (int r = lane; r < a.batch; r += 32) {
        const int len = a.lens[r], n = len <= a.max_len ? min(len - pg * kPage, kPage) : 0;
        if (n > most && a.d_table[(int64_t)r * a.d_maxb + pg] == dst) {
            most = n;
            who = r;
        }
    }
    const int top = __reduce_max_sync(0xffffffffu, most);
    if (top == left) return b;
    left = top;
    return __reduce_min_sync(0xffffffffu, most == top ? who : INT32_MAX);
}

// Two magnitudes (bf16, as whole numbers) that are infinite or NaN.
__device__ inline uint32_t special(uint32_t w) { return ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u; }

template <bool E4M3>
__device__ __forceinline__ uint32_t code4(const float (&x)[4], float r) {
    if constexpr (E4M3) {
        uint32_t d;
        asm("{\n\t.reg .b16 lo, hi;\n\tcvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
            "mov.b32 %0, {lo, hi};\n\t}"
            : "=r"(d)
            : "f"(x[0] * r), "f"(x[1] * r), "f"(x[2] * r), "f"(x[3] * r));
        return d;
    } else {
        // (a sum with 1.5 x 2^23 rounds to nearest even and leaves the whole
        // number in the low bits)
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) u[i] = __float_as_uint(fminf(fmaxf(x[i] * r, -127.0f), 127.0f) + 12582912.0f);
        return __byte_perm(__byte_perm(u[0], u[1], 0x0040), __byte_perm(u[2], u[3], 0x0040), 0x5410);
    }
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(kWarps * 32, 4) kv8_write_kernel(const __grid_constant__ WriteArgs a) {
    pdl_begin();
    constexpr int P = D / 32;           // pieces of 16 values that a lane holds
    constexpr int PR = D / 16;          // pieces of a row
    const int lane = threadIdx.x & 31;
    const int n_warps = gridDim.x * kWarps, me = blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (me == 0) {
        for (int b = lane; b < a.batch; b += 32) {
            const int first = a.first ? a.first[b] : 0, len = a.lens[b];
            if (first < 0 || len < 0 || len > a.max_len) report(a.status, VC_ERR_BAD_INDEX);
        }
    }
    const int per = 2 * a.hkv;  // blocks of a page
    // 32 requests, a lane each, from request b0 on: pages of the request, those up to and with
    // it, and those before all of them
    int b0 = 0, n = lane < a.batch ? pages_of(a, lane) : 0, upto = n, before = 0, total = n;
    for (int i = lane + 32; i < a.batch; i += 32) total += pages_of(a, i);
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    const int64_t items = (int64_t)total * per;
    if (me >= items) return;
    auto sum = [&]() {
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += v;
        }
    };
    sum();
    for (int64_t item = me; item < items; item += n_warps) {
        const int k = (int)(item / per), kind = (int)(item % per), h = kind >> 1;
        unsigned here;  // (k < total: such a request is there)
        while ((here = __ballot_sync(0xffffffffu, k < before + upto)) == 0) {
            before += __shfl_sync(0xffffffffu, upto, 31);
            b0 += 32;
            n = upto = b0 + lane < a.batch ? pages_of(a, b0 + lane) : 0;
            sum();
        }
        const int b = b0 + __ffs(here) - 1, at = before + __shfl_sync(0xffffffffu, upto - n, b - b0);
        const bool is_v = kind & 1;
        const int len = a.lens[b], pg = (a.first ? a.first[b] : 0) / kPage + k - at;
        int left = len - pg * kPage;  // rows of the page that hold tokens
        const int dst = pg < a.d_maxb ? a.d_table[(int64_t)b * a.d_maxb + pg] : -1;
        int src = pg < a.f_maxb ? a.f_table[(int64_t)b * a.f_maxb + pg] : -1;
        if (left < kPage && pg < a.d_maxb) {
            const int from = holder_of(a, b, pg, dst, lane, left);
            if (from != b) src = pg < a.f_maxb ? a.f_table[(int64_t)from * a.f_maxb + pg] : -1;
        }
        if (src < 0 || src >= a.f_pages || dst < 0 || dst >= a.d_pages) {
            if (lane == 0) report(a.status, VC_ERR_BAD_INDEX);
            continue;
        }
        const uint4 *x = reinterpret_cast<const uint4 *>((is_v ? a.vp : a.kp) + ((int64_t)src * a.hkv + h) * kPage * D * 2);
        uint4 u[P][2];
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int e = i * 32 + lane;
            const bool there = e / PR < left;
#pragma unroll
            for (int c = 0; c < 2; ++c) u[i][c] = there ? x[e * 2 + c] : make_uint4(0, 0, 0, 0);
        }
        uint32_t mx = 0, odd = 0;
#pragma unroll
        for (int i = 0; i < P; ++i)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const uint32_t *w = reinterpret_cast<const uint32_t *>(&u[i][c]);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    mx = __vmaxu2(mx, w[j] & 0x7fff7fffu);
                    odd |= special(w[j]);
                }
            }
        if (__any_sync(0xffffffffu, odd != 0)) {  // (rare) without infinities and NaN
            if (odd) report(a.status, VC_ERR_INVALID_ARG);
            mx = 0;
#pragma unroll
            for (int i = 0; i < P; ++i)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t *w = reinterpret_cast<uint32_t *>(&u[i][c]);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int s = 0; s < 32; s += 16) {
                            const uint32_t mag = w[j] >> s & 0x7fffu;
                            if (mag > 0x7f80u) w[j] &= ~(0xffffu << s);
                            else if (mag < 0x7f80u) mx = max(mx, mag);
                        }
                }
        }
        mx = max(mx & 0xffffu, mx >> 16);
        mx = __reduce_max_sync(0xffffffffu, mx);
        constexpr float kInv = E4M3 ? 1.0f / 448.0f : 1.0f / 127.0f;
        const float scale = fmaxf(bf16_bits_to_f32((uint16_t)mx) * kInv, 0x1p-126f), r = __frcp_rn(scale);
        const int64_t block = (int64_t)dst * a.hkv + h;
        uint4 *to = reinterpret_cast<uint4 *>((is_v ? a.vc : a.kc) + block * kPage * D);
#pragma unroll
        for (int i = 0; i < P; ++i) {
            uint32_t d[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const uint32_t *w = reinterpret_cast<const uint32_t *>(&u[i][c >> 1]) + 2 * (c & 1);
                const float v[4] = {__uint_as_float(w[0] << 16), __uint_as_float(w[0] & 0xffff0000u),
                                    __uint_as_float(w[1] << 16), __uint_as_float(w[1] & 0xffff0000u)};
                d[c] = code4<E4M3>(v, r);
            }
            to[i * 32 + lane] = make_uint4(d[0], d[1], d[2], d[3]);
        }
        if (lane == 0) (is_v ? a.vs : a.ks)[block] = scale;
    }
}

template <int D, bool E4M3>
cudaError_t launch(const WriteArgs &a, cudaStream_t st) {
    const int64_t most = ((int64_t)a.batch * (a.max_len / kPage + 1) * a.hkv * 2 + kWarps - 1) / kWarps;
    const int full = 152 * 4;
    return launch_pdl(kv8_write_kernel<D, E4M3>, (int)(most < 1 ? 1 : most < full ? most : full), kWarps * 32, 0, st, a);
}

}  // namespace
}  // namespace vc

using namespace vc;

extern "C" vc_status vc_kv8_write(const vc_paged_kv *full, const int32_t *first, const vc_paged_kv8 *dst,
                                  int32_t max_seq_len, int32_t *dev_status, vc_stream_t stream) {
    if (!paged_fmt_ok(full) || !kv8_sizes_ok(dst) || max_seq_len < 0 || full->batch != dst->batch ||
        full->fmt.num_kv_heads != dst->num_kv_heads || full->fmt.head_dim != dst->head_dim)
        return VC_ERR_INVALID_ARG;
    const int d = dst->head_dim;
    if (full->fmt.bits != 16 || (d != 64 && d != 128) || (dst->code != VC_E4M3 && dst->code != VC_INT8))
        return VC_ERR_UNSUPPORTED;
    // (pages of a call are counted in 32 bits)
    if ((int64_t)full->batch * (max_seq_len / kPage + 1) > INT32_MAX) return VC_ERR_UNSUPPORTED;
    if (full->batch == 0) return VC_OK;
    if (!paged_ok(full) || !kv8_ok(dst) || ((uintptr_t)full->k_pages & 15) || ((uintptr_t)full->v_pages & 15))
        return VC_ERR_INVALID_ARG;
    WriteArgs a;
    a.kp = (const uint8_t *)full->k_pages;
    a.vp = (const uint8_t *)full->v_pages;
    a.f_pages = full->num_pages;
    a.d_pages = dst->num_pages;
    a.f_table = full->block_table;
    a.lens = full->seq_lens;
    a.first = first;
    a.d_table = dst->block_table;
    a.f_maxb = full->max_blocks;
    a.d_maxb = dst->max_blocks;
    a.batch = full->batch;
    a.hkv = dst->num_kv_heads;
    a.max_len = max_seq_len;
    a.kc = (uint8_t *)dst->k_codes;
    a.vc = (uint8_t *)dst->v_codes;
    a.ks = dst->k_scales;
    a.vs = dst->v_scales;
    a.status = dev_status;
    const cudaStream_t st = (cudaStream_t)stream;
    const bool e4m3 = dst->code == VC_E4M3;
    const cudaError_t e = d == 64 ? (e4m3 ? launch<64, true>(a, st) : launch<64, false>(a, st))
                                  : (e4m3 ? launch<128, true>(a, st) : launch<128, false>(a, st));
    return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? VC_OK : VC_ERR_CUDA;
}
