// Writing new keys and values into a caller-held cache, and reading them back.
//
// 8-bit rows: scale s = max|x| / 127, code = rint(x * (127 / max|x|)), value = code * s,
// one scale for a row of head_dim.  The scale multiplies whole rows, so that attention
// folds it into the scores (keys) and the probabilities (values) instead of every element.
//
// Both directions move each byte once and are bound by HBM for long prompts, by the launch and two
// dependent loads for a decode step.  A row is spread over the lanes so that each
// lane's 16-byte access is contiguous with its neighbours' (fp32: 4 elements, bf16: 8); the row
// maximum is a butterfly over those lanes, taken on the bits of |x| (integers order like
// the magnitudes, NaN above infinity, so one comparison finds a row that is not finite).  The
// issue rate comes next (20 instructions an element held the first form at half of HBM): the two IEEE quotients of a row are
// taken by one lane each, and rounding to a whole number is an add of 1.5 * 2^23, whose low byte is the code.
#include "kv_view.cuh"
#include "qd_device.cuh"
#include "qd_internal.h"

namespace qd {

namespace {

constexpr int kRowThreads = 256;

struct RowsArgs {
    KvView c;
    const uint8_t *rows[2];            // k, v rows
    int64_t stream, token, head;       // bytes
    const int32_t *lengths, *n_new;
    int n_tokens, kvh, smax;
    int hp, tp, sets;                  // heads and tokens of a CTA's threads; of those sets, a CTA's share at a time
};

// 16 bytes of T as floats
template <typename T> struct Vec16 {
    static constexpr int E = 16 / sizeof(T);
    static __device__ void unpack(uint4 u, float *f) { Elem<T>::unpack(u, f); }
};

// The largest magnitude of 16 bytes as fp32 bits (NaN above infinity above all finite ones).
template <typename T> __device__ __forceinline__ uint32_t top_of(uint4 u) {
    if constexpr (sizeof(T) == 2) {
        // pairs of bf16: 16-bit maxima of the magnitudes
        const uint32_t a = __vmaxu2(u.x & 0x7fff7fffu, u.y & 0x7fff7fffu), b = __vmaxu2(u.z & 0x7fff7fffu, u.w & 0x7fff7fffu);
        const uint32_t m = __vmaxu2(a, b);
        return max(m & 0xffff0000u, m << 16);
    } else {
        return max(max(u.x & 0x7fffffffu, u.y & 0x7fffffffu), max(u.z & 0x7fffffffu, u.w & 0x7fffffffu));
    }
}

__device__ __forceinline__ uint32_t pack2_bf16(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// A CTA's threads stand for hp heads (of one of ceil(kvh / hp) groups) times tp tokens, so that a thread keeps
// its head and walks the tokens with its addresses growing by constants; U tokens at a time, their loads first.
// LPR lanes a row.
template <typename T, int D> struct RowWalk {
    static constexpr int E = Vec16<T>::E, LPR = D / E;
    int h, t, tp, n, first;
    bool idle;
    __device__ __forceinline__ RowWalk(const RowsArgs &a) {
        const NewRows nr = new_rows(a.lengths, a.n_new, (int)blockIdx.y, a.n_tokens);
        n = nr.n, first = nr.first;
        const int slot = threadIdx.x / LPR, in = slot / a.hp;
        tp = a.tp;
        h = (blockIdx.z >> 1) * a.hp + slot - in * a.hp;
        idle = in >= tp || h >= a.kvh;
        if (idle) h = 0;
        t = blockIdx.x * tp * a.sets + in;
    }
    __device__ __forceinline__ bool live(const RowsArgs &a, int tt) const {
        return !idle && tt < n && (unsigned)first + (unsigned)tt < (unsigned)a.smax;   // (past the last token it may wrap)
    }
};

// grid (token blocks, streams, head groups x (K, V))
template <typename T, int D, bool Q8, int U>
__global__ void __launch_bounds__(kRowThreads) kv_append_kernel(const RowsArgs a) {
    using S = RowWalk<T, D>;
    constexpr int E = S::E, LPR = S::LPR;
    const int b = blockIdx.y, which = blockIdx.z & 1, lane = threadIdx.x % LPR;
    S s(a);
    const uint8_t *src = a.rows[which] + b * a.stream + s.h * a.head + s.t * a.token + lane * 16;
    uint8_t *dst = const_cast<uint8_t *>(which ? a.c.v : a.c.k) + b * a.c.stream + s.h * a.c.head +
                   ((int64_t)s.first + s.t) * a.c.row + lane * (Q8 ? E : 2 * E);
    float *scales = nullptr;
    if constexpr (Q8)
        scales = const_cast<float *>(which ? a.c.vs : a.c.ks) + b * a.c.sstream + s.h * a.c.shead + s.first + s.t;
    const int64_t hop_in = s.tp * a.token, hop_out = s.tp * a.c.row;
    // the same number of turns for every thread of the CTA
    for (int t0 = blockIdx.x * s.tp * U; t0 < s.n; t0 += gridDim.x * s.tp * U) {
        uint4 in[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            in[u] = make_uint4(0, 0, 0, 0);
            if (s.live(a, s.t + u * s.tp)) in[u] = __ldcs(reinterpret_cast<const uint4 *>(src + u * hop_in));
        }
        // the rows' largest magnitudes; then each lane of a row's group takes one of the U rows' two quotients
        float by[U], scale[U];
        bool finite[U];
        if constexpr (Q8) {
            static_assert(2 * U <= LPR, "a lane per quotient");
            uint32_t mine = 0;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                uint32_t m = top_of<T>(in[u]);
#pragma unroll
                for (int o = LPR / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
                finite[u] = m < 0x7f800000u;
                if (lane / 2 == u) mine = m;
            }
            const bool zero = mine < 0x05800000u;   // below 2^-116
            const float t = __uint_as_float(mine), one = zero || mine >= 0x7f800000u ? 1.f : t;
            const float quot = zero ? 0.f : lane & 1 ? __fdiv_rn(one, 127.f) : __fdiv_rn(127.f, one);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                by[u] = __shfl_sync(0xffffffffu, quot, 2 * u, LPR);
                scale[u] = __shfl_sync(0xffffffffu, quot, 2 * u + 1, LPR);
                if (!finite[u]) scale[u] = __uint_as_float(0x7fc00000u);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float x[E];
            Vec16<T>::unpack(in[u], x);
            const bool live = s.live(a, s.t + u * s.tp);
            uint8_t *to = dst + u * hop_out;
            if constexpr (Q8) {
                uint32_t w[E / 4];
#pragma unroll
                for (int e = 0; e < E; e += 4) {
                    uint32_t c[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        c[i] = __float_as_uint(__fadd_rn(__fmul_rn(finite[u] ? x[e + i] : 0.f, by[u]), 12582912.f));
                    w[e / 4] = __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
                }
                if (live) {
                    if constexpr (E == 8)
                        *reinterpret_cast<uint2 *>(to) = make_uint2(w[0], w[1]);
                    else
                        *reinterpret_cast<uint32_t *>(to) = w[0];
                    if (lane == 0) scales[u * s.tp] = scale[u];
                }
            } else if (live) {
                if constexpr (E == 8)
                    *reinterpret_cast<uint4 *>(to) = in[u];
                else
                    *reinterpret_cast<uint2 *>(to) = make_uint2(pack2_bf16(x[0], x[1]), pack2_bf16(x[2], x[3]));
            }
        }
        s.t += gridDim.x * s.tp * U;
        src += (int64_t)gridDim.x * U * hop_in, dst += (int64_t)gridDim.x * U * hop_out;
        if constexpr (Q8) scales += gridDim.x * s.tp * U;
    }
}

template <typename T, int D, bool Q8, int U>
__global__ void __launch_bounds__(kRowThreads) kv_read_kernel(const RowsArgs a) {
    using S = RowWalk<T, D>;
    constexpr int E = S::E, LPR = S::LPR, W = Q8 ? E / 4 : E / 2;   // words a lane reads
    const int b = blockIdx.y, which = blockIdx.z & 1, lane = threadIdx.x % LPR;
    S s(a);
    uint8_t *dst = const_cast<uint8_t *>(a.rows[which]) + b * a.stream + s.h * a.head + s.t * a.token + lane * 16;
    const uint8_t *src = (which ? a.c.v : a.c.k) + b * a.c.stream + s.h * a.c.head + ((int64_t)s.first + s.t) * a.c.row + lane * (W * 4);
    const float *scales = nullptr;
    if constexpr (Q8) scales = (which ? a.c.vs : a.c.ks) + b * a.c.sstream + s.h * a.c.shead + s.first + s.t;
    const int64_t hop_in = s.tp * a.c.row, hop_out = s.tp * a.token;
    for (; s.t < s.n; s.t += gridDim.x * s.tp * U) {
        uint32_t w[U][W];
        float scale[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int i = 0; i < W; ++i) w[u][i] = 0;
            scale[u] = 0.f;
            if (!s.live(a, s.t + u * s.tp)) continue;
            const uint8_t *at = src + u * hop_in;
            if constexpr (W == 4) {
                const uint4 v = *reinterpret_cast<const uint4 *>(at);
                w[u][0] = v.x, w[u][1] = v.y, w[u][2] = v.z, w[u][3] = v.w;
            } else if constexpr (W == 2) {
                const uint2 v = *reinterpret_cast<const uint2 *>(at);
                w[u][0] = v.x, w[u][1] = v.y;
            } else {
                w[u][0] = *reinterpret_cast<const uint32_t *>(at);
            }
            if constexpr (Q8) scale[u] = scales[u * s.tp];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (!s.live(a, s.t + u * s.tp)) continue;
            float x[E];
#pragma unroll
            for (int e = 0; e < E; ++e)
                x[e] = Q8 ? __fmul_rn((float)(int8_t)(w[u][(e / 4) % W] >> (8 * (e & 3))), scale[u])
                          : (e & 1 ? bf16hi(w[u][(e / 2) % W]) : bf16lo(w[u][(e / 2) % W]));
            uint4 o;
            if constexpr (E == 8)
                o = make_uint4(pack2_bf16(x[0], x[1]), pack2_bf16(x[2], x[3]), pack2_bf16(x[4], x[5]),
                               pack2_bf16(x[6], x[7]));
            else
                o = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                               __float_as_uint(x[3]));
            __stcs(reinterpret_cast<uint4 *>(dst + u * hop_out), o);
        }
        src += (int64_t)gridDim.x * U * hop_in, dst += (int64_t)gridDim.x * U * hop_out;
        if constexpr (Q8) scales += gridDim.x * s.tp * U;
    }
}

// Rows in flight a thread, where there are that many (64 x 1792 bf16 rows in and out: 2 and 2 241 us, 4 and 4 227, 4
// and 8 226 against 210 for the bytes at HBM's rate).
constexpr int kAppendSets = 4, kReadSets = 8;

typedef void (*RowsFn)(const RowsArgs);
template <typename T, int D, bool Q8> RowsFn rows_fn(bool read, bool many) {
    if (read) return many ? kv_read_kernel<T, D, Q8, kReadSets> : kv_read_kernel<T, D, Q8, 1>;
    return many ? kv_append_kernel<T, D, Q8, kAppendSets> : kv_append_kernel<T, D, Q8, 1>;
}
template <typename T> RowsFn rows_fn(bool read, bool many, int d, bool q8) {
    if (d == 64) return q8 ? rows_fn<T, 64, true>(read, many) : rows_fn<T, 64, false>(read, many);
    return q8 ? rows_fn<T, 128, true>(read, many) : rows_fn<T, 128, false>(read, many);
}

qd_status move_rows(bool read, const qd_kv_cache *cache, const void *k_rows, const void *v_rows, int dtype,
                    int n_tokens, int64_t stream_stride, int64_t token_stride, int64_t head_stride,
                    const int32_t *lengths, const int32_t *n_new, void *cuda_stream) {
    qd_status st = check_cache(cache, -1, false);
    if (st != QD_OK) return st;
    if ((dtype != QD_F32 && dtype != QD_BF16) || n_tokens < 1 || cache->n_streams > 65535) return QD_EINVAL;
    if (n_tokens > INT32_MAX - (1 << 20)) return QD_EUNSUPPORTED;   // a turn past the last token has to fit the kernels' counters
    if (!k_rows || !v_rows || !lengths) return QD_EINVAL;
    const int64_t unit = dtype == QD_F32 ? 4 : 8, e = dtype == QD_F32 ? 4 : 2;
    if (stream_stride < 0 || token_stride < 0 || head_stride < 0 || stream_stride % unit || token_stride % unit ||
        head_stride % unit)
        return QD_EINVAL;
    if (!is_aligned(k_rows, 16) || !is_aligned(v_rows, 16) || !is_aligned(lengths, 4) || !is_aligned(n_new, 4))
        return QD_EINVAL;
    // the side that is written
    const int64_t d64 = cache->head_dim, B = cache->n_streams, H = cache->n_kv_heads, ce = cache->format == QD_KV_Q8 ? 1 : 2;
    if (read ? k_rows == v_rows || !apart(e, d64, {{H, head_stride}, {n_tokens, token_stride}, {B, stream_stride}},
                                          bytes_between(k_rows, v_rows))
             : cache->k == cache->v || !apart(ce, d64, {{H, cache->head_stride}, {cache->smax, cache->row_stride}, {B, cache->stream_stride}},
                                              bytes_between(cache->k, cache->v)))
        return QD_EINVAL;
    if (!read && cache->format == QD_KV_Q8 &&
        (cache->k_scale == cache->v_scale || !apart(4, cache->smax, {{H, cache->scale_head_stride}, {B, cache->scale_stream_stride}},
                                                    bytes_between(cache->k_scale, cache->v_scale))))
        return QD_EINVAL;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return QD_ECUDA;
    if ((st = check_cache(cache, dev, false)) != QD_OK) return st;
    if (!on_device(k_rows, dev) || !on_device(v_rows, dev) || !on_device(lengths, dev) ||
        (n_new && !on_device(n_new, dev)))
        return QD_EINVAL;
    RowsArgs a;
    a.c = kv_view(cache);
    a.rows[0] = static_cast<const uint8_t *>(k_rows);
    a.rows[1] = static_cast<const uint8_t *>(v_rows);
    a.stream = stream_stride * e, a.token = token_stride * e, a.head = head_stride * e;
    a.lengths = lengths, a.n_new = n_new;
    a.n_tokens = n_tokens, a.kvh = cache->n_kv_heads, a.smax = cache->smax;
    const int rpb = kRowThreads / (cache->head_dim / (int)unit), d = cache->head_dim;
    a.hp = std::min(a.kvh, rpb), a.tp = rpb / a.hp;
    const bool many = n_tokens > a.tp, q8 = cache->format == QD_KV_Q8;
    a.sets = many ? (read ? kReadSets : kAppendSets) : 1;
    const int64_t per = (int64_t)a.tp * a.sets, hgroups = (a.kvh + a.hp - 1) / a.hp;
    if (hgroups > 32767) return QD_EUNSUPPORTED;
    // about 16 CTAs' worth of turns per SM: a few waves, whatever the lengths
    const int64_t most = std::max<int64_t>(1, sms_of(dev) * 16 / (cache->n_streams * hgroups));
    const dim3 grid((unsigned)std::min((n_tokens + per - 1) / per, most), (unsigned)cache->n_streams, (unsigned)(2 * hgroups));
    const RowsFn fn = dtype == QD_F32 ? rows_fn<float>(read, many, d, q8) : rows_fn<__nv_bfloat16>(read, many, d, q8);
    fn<<<grid, kRowThreads, 0, static_cast<cudaStream_t>(cuda_stream)>>>(a);
    return cudaGetLastError() == cudaSuccess ? QD_OK : QD_ECUDA;
}

}  // namespace

}  // namespace qd

using namespace qd;

extern "C" {

qd_status qd_kv_append(const qd_kv_cache *cache, const void *k_rows_dev, const void *v_rows_dev, int dtype,
                       int n_tokens, int64_t stream_stride, int64_t token_stride, int64_t head_stride,
                       const int32_t *lengths_dev, const int32_t *n_new_dev, void *cuda_stream) {
    return move_rows(false, cache, k_rows_dev, v_rows_dev, dtype, n_tokens, stream_stride, token_stride, head_stride,
                     lengths_dev, n_new_dev, cuda_stream);
}

qd_status qd_kv_read(const qd_kv_cache *cache, void *k_rows_dev, void *v_rows_dev, int dtype, int n_tokens,
                     int64_t stream_stride, int64_t token_stride, int64_t head_stride, const int32_t *lengths_dev,
                     const int32_t *n_new_dev, void *cuda_stream) {
    return move_rows(true, cache, k_rows_dev, v_rows_dev, dtype, n_tokens, stream_stride, token_stride, head_stride,
                     lengths_dev, n_new_dev, cuda_stream);
}

}  // extern "C"
