// Norms of queries and keys head by head and the rotation to their positions, in one pass over a fused projection's
// rows that also writes the keys and values into the pages of a cache (8-bit or bf16 rows).
//
//   x' = x / sqrt(mean(x^2) + eps) * gamma,   y[d] = x'[d] c_d - x'[d + h] s_d,   y[d + h] = x'[d + h] c_d + x'[d] s_d   (h = D / 2)
//
// Every byte moves once, so HBM bounds it for prompts, and the launch and three dependent loads (length, page and table row,
// the rows) for a step.  A row stands on D / 8 lanes, each with four elements of the lower half and the four that they are rotated with:
// nothing but the sum of squares (and the maximum of an 8-bit row) crosses lanes, and a lane that rotates a token's rows
// keeps its four cosines and sines from head to head.  Everything is fp32 until the result is rounded once.
#include <algorithm>

#include "kv_view.cuh"
#include "qd_device.cuh"
#include "qd_internal.h"

namespace qd {

namespace {

constexpr int kRopeThreads = 256;

struct RopeArgs {
    const uint8_t *in[3];              // q, k, v rows
    uint8_t *out[3];                   // of the results (k, v: may be null)
    int64_t in_token[3], out_token[3]; // bytes
    const float *gamma[2];             // of q, k, or null
    float eps;
    const float *cos, *sin;            // [rope_rows][D / 2], or null
    const int32_t *pos;                // [N] or [3][N], or null: the positions in the cache
    int rope_rows, mrope3;             // frequencies below mrope3 take stream d % 3
    const int32_t *lengths, *offsets, *n_new;
    int B, T, N, qh, kvh, heads;
    KvView pages;                      // k null: none
    const int32_t *table;
    int64_t table_stride;
    int table_pages, n_pages, page_shift;
    int hp, tp, run;                   // heads and tokens of a CTA's groups of lanes; tokens of a CTA
};

// Four elements as floats, and back.
template <typename T> struct Four;
template <> struct Four<float> {
    using V = float4;
    static __device__ __forceinline__ void get(V u, float *x) { x[0] = u.x, x[1] = u.y, x[2] = u.z, x[3] = u.w; }
    static __device__ __forceinline__ V put(const float *x) { return make_float4(x[0], x[1], x[2], x[3]); }
};
template <> struct Four<__nv_bfloat16> {
    using V = uint2;
    static __device__ __forceinline__ void get(V u, float *x) { x[0] = bf16lo(u.x), x[1] = bf16hi(u.x), x[2] = bf16lo(u.y), x[3] = bf16hi(u.y); }
    static __device__ __forceinline__ V put(const float *x) {
        const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
        return make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
    }
};

// A token's stream, its place among the stream's new rows, how many those are; b < 0: the row is not in use.
struct Token {
    int b, t, n;
};
__device__ __forceinline__ Token token_of(const RopeArgs &a, int row) {
    if (!a.offsets) {
        if (!a.lengths) return {0, row, a.N};
        const int b = row / a.T, t = row - b * a.T;
        int n = a.n_new ? a.n_new[b] : a.T;
        n = n < 0 ? 0 : n > a.T ? a.T : n;
        return {t < n ? b : -1, t, n};
    }
    int lo = 0, hi = a.B;                               // the last stream that begins at row or before
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.offsets[mid] <= row)
            lo = mid;
        else
            hi = mid;
    }
    const int first = a.offsets[lo], end = min(a.offsets[lo + 1], a.N);
    return {first >= 0 && first <= row && row < end ? lo : -1, row - first, end - first};
}

// fp32 bits of |x| order like the magnitudes, NaN above infinity.
__device__ __forceinline__ uint32_t mag(float x) { return __float_as_uint(x) & 0x7fffffffu; }

template <typename TI, typename TO, int D, bool Q8, int U>
__global__ void __launch_bounds__(kRopeThreads) qk_norm_rope_kernel(const RopeArgs a) {
    constexpr int LPR = D / 8, HALF = D / 2;
    const int lane = threadIdx.x % LPR, slot = threadIdx.x / LPR, in = slot / a.hp, h0 = slot - in * a.hp;
    const int heads = a.heads;
    const uint32_t mask = LPR == 16 ? 0xffffu << (threadIdx.x & 16) : 0xffu << (threadIdx.x & 24);
    if (in >= a.tp) return;
    const int end = min(a.N, (int)(blockIdx.x + 1) * a.run);
    for (int row = (int)blockIdx.x * a.run + in; row < end; row += a.tp) {
        const Token tk = token_of(a, row);
        if (tk.b < 0) continue;
        // where the token stands
        const int at = a.lengths ? max(a.lengths[tk.b], 0) - tk.n + tk.t : -1;
        int64_t to = -1, to_s = -1;                     // bytes into the pages, of a row of head 0; scales
        if (a.pages.k && at >= 0 && (at >> a.page_shift) < a.table_pages) {
            const int page = a.table[tk.b * a.table_stride + (at >> a.page_shift)], r = at & ((1 << a.page_shift) - 1);
            if ((unsigned)page < (unsigned)a.n_pages) {
                to = page * a.pages.stream + r * a.pages.row;
                to_s = page * a.pages.sstream + r;
            }
        }
        float c[4], s[4];
        if (a.cos) {
            const int most = a.rope_rows;
            if (a.mrope3) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int d = 4 * lane + e, p = a.pos[(int64_t)(d < a.mrope3 ? d % 3 : 0) * a.N + row];
                    const bool there = (unsigned)p < (unsigned)most;
                    c[e] = there ? __ldg(a.cos + (int64_t)p * HALF + d) : __uint_as_float(0x7fc00000u);
                    s[e] = there ? __ldg(a.sin + (int64_t)p * HALF + d) : __uint_as_float(0x7fc00000u);
                }
            } else {
                const int p = a.pos ? a.pos[row] : at;
                if ((unsigned)p < (unsigned)most) {
                    Four<float>::get(__ldg(reinterpret_cast<const float4 *>(a.cos + (int64_t)p * HALF) + lane), c);
                    Four<float>::get(__ldg(reinterpret_cast<const float4 *>(a.sin + (int64_t)p * HALF) + lane), s);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) c[e] = s[e] = __uint_as_float(0x7fc00000u);
                }
            }
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) c[e] = 1.f, s[e] = 0.f;
        }
        for (int h = h0; h < heads; h += U * a.hp) {
            typename Four<TI>::V lo[U], hi[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int hh = h + u * a.hp;
                if (hh >= heads) break;
                const int which = hh < a.qh ? 0 : hh < a.qh + a.kvh ? 1 : 2;
                const int of = which == 0 ? hh : which == 1 ? hh - a.qh : hh - a.qh - a.kvh;
                const TI *src = reinterpret_cast<const TI *>(a.in[which] + row * a.in_token[which]) + of * D + 4 * lane;
                lo[u] = *reinterpret_cast<const typename Four<TI>::V *>(src);
                hi[u] = *reinterpret_cast<const typename Four<TI>::V *>(src + HALF);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int hh = h + u * a.hp;
                if (hh >= heads) break;
                const int which = hh < a.qh ? 0 : hh < a.qh + a.kvh ? 1 : 2;
                const int of = which == 0 ? hh : which == 1 ? hh - a.qh : hh - a.qh - a.kvh;
                float x[8];
                Four<TI>::get(lo[u], x);
                Four<TI>::get(hi[u], x + 4);
                if (which < 2) {
                    const float *gamma = a.gamma[which];
                    if (gamma) {
                        float ss = 0.f;
#pragma unroll
                        for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
                        for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(mask, ss, o);
                        const float inv = 1.f / sqrtf(ss / (float)D + a.eps);
                        float g[8];
                        Four<float>::get(__ldg(reinterpret_cast<const float4 *>(gamma) + lane), g);
                        Four<float>::get(__ldg(reinterpret_cast<const float4 *>(gamma + HALF) + lane), g + 4);
#pragma unroll
                        for (int e = 0; e < 8; ++e) x[e] = x[e] * inv * g[e];
                    }
                    if (a.cos) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float l = x[e], u2 = x[4 + e];
                            x[e] = l * c[e] - u2 * s[e];
                            x[4 + e] = u2 * c[e] + l * s[e];
                        }
                    }
                }
                if (a.out[which]) {
                    TO *dst = reinterpret_cast<TO *>(a.out[which] + row * a.out_token[which]) + of * D + 4 * lane;
                    *reinterpret_cast<typename Four<TO>::V *>(dst) = Four<TO>::put(x);
                    *reinterpret_cast<typename Four<TO>::V *>(dst + HALF) = Four<TO>::put(x + 4);
                }
                if (which && to >= 0) {
                    uint8_t *dst = const_cast<uint8_t *>(which == 1 ? a.pages.k : a.pages.v) + to + of * a.pages.head;
                    if constexpr (Q8) {
                        uint32_t m = 0;
#pragma unroll
                        for (int e = 0; e < 8; ++e) m = max(m, mag(x[e]));
#pragma unroll
                        for (int o = LPR / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(mask, m, o));
                        // even lanes take one quotient, odd ones the other
                        const bool finite = m < 0x7f800000u, zero = m < 0x05800000u;   // below 2^-116
                        const float top = zero || !finite ? 1.f : __uint_as_float(m);
                        float quot = lane & 1 ? __fdiv_rn(top, 127.f) : __fdiv_rn(127.f, top);
                        if (zero) quot = 0.f;
                        const float by = __shfl_sync(mask, quot, 0, LPR), scale = __shfl_sync(mask, quot, 1, LPR);
                        uint32_t w[2];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            uint32_t k[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                k[e] = __float_as_uint(__fadd_rn(__fmul_rn(finite ? x[4 * i + e] : 0.f, by), 12582912.f));
                            w[i] = __byte_perm(__byte_perm(k[0], k[1], 0x0040), __byte_perm(k[2], k[3], 0x0040), 0x5410);
                        }
                        *reinterpret_cast<uint32_t *>(dst + 4 * lane) = w[0];
                        *reinterpret_cast<uint32_t *>(dst + HALF + 4 * lane) = w[1];
                        if (lane == 0)
                            const_cast<float *>(which == 1 ? a.pages.ks : a.pages.vs)[to_s + of * a.pages.shead] =
                                finite ? scale : __uint_as_float(0x7fc00000u);
                    } else {
                        __nv_bfloat16 *row16 = reinterpret_cast<__nv_bfloat16 *>(dst) + 4 * lane;
                        *reinterpret_cast<uint2 *>(row16) = Four<__nv_bfloat16>::put(x);
                        *reinterpret_cast<uint2 *>(row16 + HALF) = Four<__nv_bfloat16>::put(x + 4);
                    }
                }
            }
        }
    }
}

typedef void (*RopeFn)(const RopeArgs);
template <typename TI, typename TO> RopeFn rope_fn(int d, bool q8) {
    constexpr int U = 2;
    if (d == 64) return q8 ? qk_norm_rope_kernel<TI, TO, 64, true, U> : qk_norm_rope_kernel<TI, TO, 64, false, U>;
    return q8 ? qk_norm_rope_kernel<TI, TO, 128, true, U> : qk_norm_rope_kernel<TI, TO, 128, false, U>;
}

}  // namespace

}  // namespace qd

using namespace qd;

extern "C" qd_status qd_qk_norm_rope(const qd_rope_rows *x, void *cuda_stream) {
    if (!x || !x->q || !x->k || !x->q_out || x->n_tokens < 1 || x->n_q_heads < 1 || x->n_kv_heads < 1) return QD_EINVAL;
    if ((x->dtype != QD_F32 && x->dtype != QD_BF16) || (x->out_dtype != QD_F32 && x->out_dtype != QD_BF16)) return QD_EINVAL;
    if (x->head_dim != 64 && x->head_dim != 128) return QD_EUNSUPPORTED;
    const int d = x->head_dim;
    if (x->n_tokens > (1 << 30) || (int64_t)x->n_q_heads + 2 * (int64_t)x->n_kv_heads > 65536) return QD_EUNSUPPORTED;
    if (!(x->eps >= 0.0 && x->eps < 1e30)) return QD_EINVAL;
    if (!x->v && (x->v_out || x->pages)) return QD_EINVAL;
    if ((x->cos == nullptr) != (x->sin == nullptr) || (x->cos && x->rope_rows < 1)) return QD_EINVAL;
    if (x->mrope_h < 0 || 3 * (int64_t)x->mrope_h > d / 2 || (x->mrope_h && (!x->positions || !x->cos))) return QD_EINVAL;
    if (x->cos && !x->positions && !x->lengths) return QD_EINVAL;
    if (x->n_streams < 0 || (!x->lengths && (x->pages || x->offsets || x->n_new)) || (x->offsets && x->n_new)) return QD_EINVAL;
    if (x->lengths && (x->n_streams < 1 || (!x->offsets && x->n_tokens % x->n_streams))) return QD_EINVAL;
    const int64_t unit = x->dtype == QD_F32 ? 4 : 8, ou = x->out_dtype == QD_F32 ? 4 : 8, e = 16 / unit, oe = 16 / ou;
    const void *in[3] = {x->q, x->k, x->v};
    void *out[3] = {x->q_out, x->k_out, x->v_out};
    const int64_t in_stride[3] = {x->q_stride, x->k_stride, x->v_stride}, out_stride[3] = {x->q_out_stride, x->k_out_stride, x->v_out_stride};
    const int64_t N = x->n_tokens;
    for (int i = 0; i < 3; ++i) {
        const int64_t inner = (int64_t)(i ? x->n_kv_heads : x->n_q_heads) * d;
        if (in[i] && (in_stride[i] < 0 || in_stride[i] % unit || in_stride[i] > (int64_t(1) << 40) || !is_aligned(in[i], 16))) return QD_EINVAL;
        if (out[i] && (out_stride[i] % ou || out_stride[i] > (int64_t(1) << 40) || !is_aligned(out[i], 16) || (N > 1 && out_stride[i] < inner)))
            return QD_EINVAL;
    }
    // what is written lies over nothing else: a result may take its own rows' place (same type and stride), or a gap of a fused projection
    for (int i = 0; i < 3; ++i) {
        if (!out[i]) continue;
        const int64_t inner = (int64_t)(i ? x->n_kv_heads : x->n_q_heads) * d;
        for (int j = 0; j < 6; ++j) {
            const void *p = j < 3 ? in[j] : out[j - 3];
            if (!p || j == 3 + i) continue;
            const int64_t pe = j < 3 ? e : oe, ps = j < 3 ? in_stride[j] : out_stride[j - 3];
            const int64_t pi = (int64_t)(j % 3 ? x->n_kv_heads : x->n_q_heads) * d;
            if (j == i && p == out[i] && pe == oe && (N == 1 || ps == out_stride[i])) continue;
            if (!rows_beside(out[i], oe, N, out_stride[i], inner, p, pe, N, ps, pi)) return QD_EINVAL;
        }
    }
    for (const void *p : {(const void *)x->q_gamma, (const void *)x->k_gamma, (const void *)x->cos, (const void *)x->sin})
        if (!is_aligned(p, 16)) return QD_EINVAL;
    for (const void *p : {(const void *)x->positions, (const void *)x->lengths, (const void *)x->offsets, (const void *)x->n_new, (const void *)x->page_table})
        if (!is_aligned(p, 4)) return QD_EINVAL;
    qd_status st;
    int shift = 0;
    const qd_kv_cache *c = x->pages;
    if (c) {
        if ((st = check_pages(c, x->page_table, x->table_stride, x->table_pages, x->n_streams, -1, &shift)) != QD_OK) return st;
        if (c->n_kv_heads != x->n_kv_heads || c->head_dim != d) return QD_EINVAL;
        const int64_t ce = c->format == QD_KV_Q8 ? 1 : 2, H = c->n_kv_heads, P = c->n_streams;
        if (c->k == c->v || !apart(ce, d, {{H, c->head_stride}, {c->smax, c->row_stride}, {P, c->stream_stride}}, bytes_between(c->k, c->v)))
            return QD_EINVAL;
        if (c->format == QD_KV_Q8 && (c->k_scale == c->v_scale || !apart(4, c->smax, {{H, c->scale_head_stride}, {P, c->scale_stream_stride}},
                                                                        bytes_between(c->k_scale, c->v_scale))))
            return QD_EINVAL;
    }
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return QD_ECUDA;
    if (c && (st = check_pages(c, x->page_table, x->table_stride, x->table_pages, x->n_streams, dev, &shift)) != QD_OK) return st;
    for (const void *p : {x->q, x->k, (const void *)x->q_out})
        if (!on_device(p, dev)) return QD_EINVAL;
    for (const void *p : {x->v, (const void *)x->k_out, (const void *)x->v_out, (const void *)x->q_gamma, (const void *)x->k_gamma,
                          (const void *)x->cos, (const void *)x->sin, (const void *)x->positions, (const void *)x->lengths,
                          (const void *)x->offsets, (const void *)x->n_new})
        if (p && !on_device(p, dev)) return QD_EINVAL;

    RopeArgs a = {};
    for (int i = 0; i < 3; ++i) {
        a.in[i] = static_cast<const uint8_t *>(in[i]), a.out[i] = static_cast<uint8_t *>(out[i]);
        a.in_token[i] = in_stride[i] * e, a.out_token[i] = out_stride[i] * oe;
    }
    a.gamma[0] = x->q_gamma, a.gamma[1] = x->k_gamma, a.eps = (float)x->eps;
    a.cos = x->cos, a.sin = x->sin, a.pos = x->positions, a.rope_rows = x->rope_rows, a.mrope3 = 3 * x->mrope_h;
    a.lengths = x->lengths, a.offsets = x->offsets, a.n_new = x->n_new;
    a.B = x->n_streams, a.N = x->n_tokens, a.qh = x->n_q_heads, a.kvh = x->n_kv_heads;
    a.T = x->lengths && !x->offsets ? x->n_tokens / x->n_streams : 1;
    if (c) {
        a.pages = kv_view(c);
        a.table = x->page_table, a.table_stride = x->table_stride, a.table_pages = x->table_pages;
        a.n_pages = c->n_streams, a.page_shift = shift;
    }
    const int groups = kRopeThreads / (d / 8), heads = a.qh + (a.in[2] ? 2 : 1) * a.kvh;
    a.heads = heads, a.hp = std::min(heads, groups), a.tp = groups / a.hp;
    const int sms = sms_of(dev);
    a.run = std::max(a.tp, (a.N + sms * 16 - 1) / (sms * 16));
    const dim3 grid((unsigned)((a.N + a.run - 1) / a.run));
    const bool q8 = c && c->format == QD_KV_Q8;
    const RopeFn fn = x->dtype == QD_F32 ? (x->out_dtype == QD_F32 ? rope_fn<float, float>(d, q8) : rope_fn<float, __nv_bfloat16>(d, q8))
                                         : (x->out_dtype == QD_F32 ? rope_fn<__nv_bfloat16, float>(d, q8)
                                                                   : rope_fn<__nv_bfloat16, __nv_bfloat16>(d, q8));
    fn<<<grid, kRopeThreads, 0, static_cast<cudaStream_t>(cuda_stream)>>>(a);
    return cudaGetLastError() == cudaSuccess ? QD_OK : QD_ECUDA;
}
