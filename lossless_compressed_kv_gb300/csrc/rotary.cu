// vc_rotary_kv_write: rotary positions in general form, with the rotated K
// and the V of each row written into KV_full.
//
//   (a, b) -> amplitude (a cos t - b sin t, b cos t + a sin t),  t = pos f_i
//
// The angle: f_i / 2pi turns per position is handed over as a binary
// fraction of 64 bits, F_i (computed in double: off by at most 2^-55 turn);
// pos * F_i modulo 2^64 is then the fraction of a turn to within pos * 2^-55
// (2^-35 at a million).  In fp32 the product pos * f_i alone would be off by
// 2^-25 pos radians (0.004 at 131072).
#include <cmath>

#include "vc_internal.cuh"

namespace vc {
namespace {

constexpr int kMaxPairs = VC_MAX_HEAD_DIM / 2;
constexpr int kMaxWidth = 1 << 28;  // channels of a row of qkv

struct RotArgs {
    const void *qkv;
    int64_t stride;  // values per row
    const int32_t *req, *pos, *slot;
    int m, hq, hkv, d, half, inter;
    float amp;
    uint16_t *q;
    uint16_t *kp, *vp;
    int64_t n_pages;
    const int32_t *table;
    int maxb, batch;
    int32_t *status;
    uint64_t turns[kMaxPairs];  // F_i
};

// cos and sin (times the amplitude) of pair i at a position.  The fraction of
// a turn as a signed 32-bit number of 2^-32 turns, so the angle lies in
// [-pi, pi].  Its conversion to fp32 rounds by up to 2^-26 turn (0.94e-7
// radians), the constant and the product by 2^-24 pi and 2^-23 more: 4e-7 in
// all, below 2^-21; the fast sine and cosine are off by at most 2^-21 there.
// The result is rounded to bf16, whose half step is 2^-8 of the value.
__device__ inline float2 cos_sin(uint64_t turns, int pos, float amp) {
    const int32_t frac = (int32_t)((turns * (uint64_t)(uint32_t)pos) >> 32);
    float s, c;
    __sincosf((float)frac * 1.4629180792671596e-9f, &s, &c);  // 2 pi / 2^32
    return make_float2(c * amp, s * amp);
}

// The cache slot a row writes: offset (in values) of kv head 0's row, or -1
// for a row to be skipped (padding, or out of range, which is reported).
__device__ inline int64_t row_base(const RotArgs &a, int r) {
    const int b = a.req[r];
    if (b == -1) return -1;
    const int pos = a.pos[r], slot = a.slot ? a.slot[r] : pos;
    int page = -1;
    if (b >= 0 && b < a.batch && pos >= 0 && slot >= 0 && slot / kPage < a.maxb)
        page = a.table[(int64_t)b * a.maxb + slot / kPage];
    if (page < 0 || page >= a.n_pages) {
        report(a.status, VC_ERR_BAD_INDEX);
        return -1;
    }
    return ((int64_t)page * a.hkv * kPage + slot % kPage) * a.d;
}

__device__ inline float load1(const float *p) { return *p; }
__device__ inline float load1(const uint16_t *p) { return bf16_bits_to_f32(*p); }
__device__ inline uint16_t bf16_bits(float v) { return __bfloat16_as_ushort(__float2bfloat16_rn(v)); }

// Rows, or an output, off 16-byte boundaries: one block per row, one thread per
// channel pair of a head.
template <typename T>
__global__ void __launch_bounds__(256) rotary_pairs_kernel(const __grid_constant__ RotArgs a) {
    pdl_begin();
    __shared__ float2 cs[kMaxPairs];
    __shared__ int64_t base_s;
    const int r = blockIdx.x;
    if (threadIdx.x == 0) base_s = row_base(a, r);
    __syncthreads();
    const int64_t base = base_s;
    if (base < 0) return;
    const int pos = a.pos[r];
    for (int i = threadIdx.x; i < a.half; i += blockDim.x) cs[i] = cos_sin(a.turns[i], pos, a.amp);
    __syncthreads();
    const T *x = reinterpret_cast<const T *>(a.qkv) + (int64_t)r * a.stride;
    const int nh = a.hq + 2 * a.hkv, pairs = a.d / 2;
    for (int e = threadIdx.x; e < nh * pairs; e += blockDim.x) {
        const int h = e / pairs, i = e % pairs;
        // pairs past the rotated ones: neighbouring channels, copied
        const bool turn = i < a.half;
        const int c0 = turn && !a.inter ? i : 2 * i, c1 = turn && !a.inter ? i + a.half : 2 * i + 1;
        const float x0 = load1(x + h * a.d + c0), x1 = load1(x + h * a.d + c1);
        float y0 = x0, y1 = x1;
        if (turn && h < a.hq + a.hkv) {
            y0 = x0 * cs[i].x - x1 * cs[i].y;
            y1 = x1 * cs[i].x + x0 * cs[i].y;
        }
        uint16_t *dst;
        if (h < a.hq)
            dst = a.q + ((int64_t)r * a.hq + h) * a.d;
        else if (h < a.hq + a.hkv)
            dst = a.kp + base + (int64_t)(h - a.hq) * kPage * a.d;
        else
            dst = a.vp + base + (int64_t)(h - a.hq - a.hkv) * kPage * a.d;
        dst[c0] = bf16_bits(y0);
        dst[c1] = bf16_bits(y1);
    }
}

// Rows on 16-byte boundaries: a block takes a few rows; their angles' cosines
// and sines go to shared memory once for all heads, then a thread takes 8
// channels at a time with 16-byte loads and stores.  Bound by memory: each value
// is read once and written once (16384 rows of 32 + 8 + 8 heads of 128, fp32:
// 93 us, 0.95 of a copy's rate).  How the pairs lie:
//   kHalves      the halves are whole pieces: both pieces of 8 pairs at once
//   kNeighbours  a pair is in one piece
//   kOdd         the halves are not whole pieces: the other channel of each pair
//                by itself, from the lines that a neighbour thread loads (50
//                rotated channels of 128: 116 us; pair by pair, as rows off
//                16-byte boundaries are taken, 158)
enum Pairing { kHalves, kNeighbours, kOdd };
constexpr int kThreadsV = 256;

template <typename T>
__device__ inline void load8(const T *p, float (&v)[8]) {
    if constexpr (sizeof(T) == 4) {
        const float4 a = __ldcs(reinterpret_cast<const float4 *>(p)), b = __ldcs(reinterpret_cast<const float4 *>(p) + 1);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
        const uint4 a = __ldcs(reinterpret_cast<const uint4 *>(p));
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
}
__device__ inline void store8(uint16_t *p, const float (&v)[8]) {
    *reinterpret_cast<uint4 *>(p) =
        make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}

constexpr int kMaxRows = 16;
template <typename T, Pairing PAIRING>
__global__ void __launch_bounds__(kThreadsV) rotary_wide_kernel(const __grid_constant__ RotArgs a, int rows) {
    pdl_begin();
    extern __shared__ float2 cs[];  // [rows][half]
    __shared__ int64_t base[kMaxRows];
    const int r0 = blockIdx.x * rows, n = min(rows, a.m - r0);
    if (threadIdx.x < n) base[threadIdx.x] = row_base(a, r0 + threadIdx.x);
    for (int e = threadIdx.x; e < n * a.half; e += kThreadsV) {
        const int k = e / a.half, i = e % a.half;
        cs[e] = cos_sin(a.turns[i], a.pos[r0 + k], a.amp);
    }
    __syncthreads();
    // items of a row: per head, `turned` ones that rotate, then copied ones
    const int turned = PAIRING == kHalves ? a.half / 8 : (a.half + 3) / 4;
    const int per = PAIRING == kHalves ? a.d / 16 : a.d / 8;
    const int items = (a.hq + 2 * a.hkv) * per;
    for (int f = threadIdx.x; f < n * items; f += kThreadsV) {
        const int k = f / items, e = f % items;
        const int64_t kv = base[k];
        if (kv < 0) continue;
        const int h = e / per, i = e % per;
        const T *x = reinterpret_cast<const T *>(a.qkv) + (int64_t)(r0 + k) * a.stride + h * a.d;
        const float2 *c = cs + k * a.half;
        uint16_t *dst = h < a.hq ? a.q + ((int64_t)(r0 + k) * a.hq + h) * a.d
                        : h < a.hq + a.hkv ? a.kp + kv + (int64_t)(h - a.hq) * kPage * a.d
                                           : a.vp + kv + (int64_t)(h - a.hq - a.hkv) * kPage * a.d;
        const bool turn = h < a.hq + a.hkv;
        float u[8];
        if constexpr (PAIRING == kHalves) {
            const int c0 = i < turned ? i * 8 : a.half + i * 8 + (i - turned) * 8, c1 = i < turned ? c0 + a.half : c0 + 8;
            float v[8];
            load8(x + c0, u);
            load8(x + c1, v);
            if (turn && i < turned) {
#pragma unroll
                for (int p = 0; p < 8; ++p) {
                    const float2 w = c[i * 8 + p];
                    const float y0 = u[p] * w.x - v[p] * w.y;
                    v[p] = v[p] * w.x + u[p] * w.y;
                    u[p] = y0;
                }
            }
            store8(dst + c0, u);
            store8(dst + c1, v);
        } else {
            load8(x + i * 8, u);
            if (turn && i < turned) {
                if constexpr (PAIRING == kNeighbours) {
#pragma unroll
                    for (int p = 0; p < 4; ++p) {
                        if (i * 4 + p >= a.half) break;
                        const float2 w = c[i * 4 + p];
                        const float y0 = u[2 * p] * w.x - u[2 * p + 1] * w.y;
                        u[2 * p + 1] = u[2 * p + 1] * w.x + u[2 * p] * w.y;
                        u[2 * p] = y0;
                    }
                } else {
#pragma unroll
                    for (int p = 0; p < 8; ++p) {
                        const int ch = i * 8 + p;
                        if (ch >= 2 * a.half) break;
                        const bool low = ch < a.half;
                        const float2 w = c[low ? ch : ch - a.half];
                        const float o = load1(x + (low ? ch + a.half : ch - a.half));
                        u[p] = u[p] * w.x + (low ? -o : o) * w.y;
                    }
                }
            }
            store8(dst + i * 8, u);
        }
    }
}

template <typename T, Pairing PAIRING>
cudaError_t launch_wide(const RotArgs &a, cudaStream_t st) {
    // a row a block while there are few; else about four items a thread
    const int items = (a.hq + 2 * a.hkv) * a.d / (PAIRING == kHalves ? 16 : 8);
    const int rows = a.m <= 1024 ? 1 : max(1, min(kMaxRows, 4 * kThreadsV / items));
    return launch_pdl(rotary_wide_kernel<T, PAIRING>, ceil_div(a.m, rows), kThreadsV, rows * a.half * 8, st, a, rows);
}
template <typename T>
cudaError_t launch(const RotArgs &a, bool wide, cudaStream_t st) {
    if (!wide) return launch_pdl(rotary_pairs_kernel<T>, a.m, 256, 0, st, a);
    return a.inter           ? launch_wide<T, kNeighbours>(a, st)
           : a.half % 8 == 0 ? launch_wide<T, kHalves>(a, st)
                             : launch_wide<T, kOdd>(a, st);
}

// F_i of every pair, from 64-bit frequencies.
void fill_turns(const vc_rotary &p, uint64_t *turns) {
    constexpr double kTwoPi = 6.283185307179586476925;
    const int half = p.rot_dim / 2;
    const double step = half ? -std::log((double)p.theta) / half : 0.0;
    for (int i = 0; i < half; ++i) {
        double f = std::exp(step * i);
        if (p.factor != 1.0f) {
            double g = 0.0;
            if (p.original_len > 0) {
                g = (p.original_len * f / kTwoPi - p.low_turns) / ((double)p.high_turns - p.low_turns);
                g = g < 0.0 ? 0.0 : g > 1.0 ? 1.0 : g;
            }
            f *= g + (1.0 - g) / p.factor;
        }
        turns[i] = (uint64_t)std::ldexp(f / kTwoPi, 64);  // f <= 1: below half a turn
    }
}

bool rotary_ok(const vc_rotary *p, int d) {
    if (!p || p->rot_dim < 0 || p->rot_dim % 2 || p->rot_dim > d) return false;
    if (!std::isfinite(p->theta) || p->theta < 1.0f || !std::isfinite(p->factor) || p->factor < 1.0f) return false;
    if (p->original_len < 0 || !std::isfinite(p->amplitude)) return false;
    if (p->original_len > 0 && p->factor != 1.0f &&
        !(std::isfinite(p->low_turns) && std::isfinite(p->high_turns) && p->low_turns < p->high_turns))
        return false;
    return true;
}

}  // namespace
}  // namespace vc

using namespace vc;

extern "C" vc_status vc_rotary_kv_write(const void *qkv, int32_t qkv_dtype, int64_t row_stride, int32_t m,
                                        const int32_t *row_req, const int32_t *row_pos, const int32_t *row_slot,
                                        int32_t num_q_heads, const vc_rotary *rotary, void *q_out,
                                        const vc_paged_kv *full, int32_t *dev_status, vc_stream_t stream) {
    if (!paged_fmt_ok(full) || m < 0 || num_q_heads < 1 || !rotary_ok(rotary, full->fmt.head_dim) ||
        row_stride < ((int64_t)num_q_heads + 2 * (int64_t)full->fmt.num_kv_heads) * full->fmt.head_dim)
        return VC_ERR_INVALID_ARG;
    if (full->fmt.bits != 16 || (qkv_dtype != VC_F32 && qkv_dtype != VC_BF16) ||
        ((int64_t)num_q_heads + 2 * (int64_t)full->fmt.num_kv_heads) * full->fmt.head_dim > kMaxWidth)
        return VC_ERR_UNSUPPORTED;
    if (m == 0 || full->batch == 0) return VC_OK;
    if (!qkv || !row_req || !row_pos || !q_out || !full->k_pages || !full->v_pages || !full->block_table ||
        full->max_blocks < 1 || full->num_pages < 1 || (uintptr_t)qkv % dtype_bytes(qkv_dtype) ||
        (((uintptr_t)q_out | (uintptr_t)full->k_pages | (uintptr_t)full->v_pages) & 1))
        return VC_ERR_INVALID_ARG;
    RotArgs a;
    a.qkv = qkv;
    a.stride = row_stride;
    a.req = row_req;
    a.pos = row_pos;
    a.slot = row_slot;
    a.m = m;
    a.hq = num_q_heads;
    a.hkv = full->fmt.num_kv_heads;
    a.d = full->fmt.head_dim;
    a.half = rotary->rot_dim / 2;
    a.inter = rotary->interleaved != 0;
    a.amp = rotary->amplitude;
    a.q = (uint16_t *)q_out;
    a.kp = (uint16_t *)full->k_pages;
    a.vp = (uint16_t *)full->v_pages;
    a.n_pages = full->num_pages;
    a.table = full->block_table;
    a.maxb = full->max_blocks;
    a.batch = full->batch;
    a.status = dev_status;
    fill_turns(*rotary, a.turns);
    const bool f32 = qkv_dtype == VC_F32;
    const bool wide = row_stride % (f32 ? 4 : 8) == 0 &&
                      (((uintptr_t)qkv | (uintptr_t)q_out | (uintptr_t)a.kp | (uintptr_t)a.vp) & 15) == 0;
    const cudaStream_t st = (cudaStream_t)stream;
    const cudaError_t e = f32 ? launch<float>(a, wide, st) : launch<uint16_t>(a, wide, st);
    return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? VC_OK : VC_ERR_CUDA;
}
