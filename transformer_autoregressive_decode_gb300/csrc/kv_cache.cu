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

// Byte i of a word of codes as a float: offset by 128 under the exponent of 2^23, less 2^23 + 128 (a
// permutation and an add at full rate, where a conversion has a quarter of it).
__device__ __forceinline__ float code_of(uint32_t w, int i) {
    return __fsub_rn(__uint_as_float(__byte_perm(w ^ 0x80808080u, 0x4b000000u, 0x7440 + i)), 8388736.f);
}

// A CTA takes U sets of its threads' rows at a time, their loads first.  LPR lanes a row.
template <typename T, int D, int U> struct RowSet {
    static constexpr int E = Vec16<T>::E, LPR = D / E, RPB = kRowThreads / LPR;
    int t[U], h[U], pos[U];
    bool live[U];
    __device__ __forceinline__ void at(const RowsArgs &a, const NewRows &nr, int first) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = first + u * RPB + (int)threadIdx.x / LPR;
            t[u] = (int)((unsigned)r / (unsigned)a.kvh), h[u] = r - t[u] * a.kvh;
            pos[u] = nr.first + t[u];
            live[u] = t[u] < nr.n && pos[u] >= 0 && pos[u] < a.smax;
        }
    }
};

// grid (row blocks, streams, K and V)
template <typename T, int D, bool Q8, int U>
__global__ void __launch_bounds__(kRowThreads) kv_append_kernel(const RowsArgs a) {
    using S = RowSet<T, D, U>;
    constexpr int E = S::E, LPR = S::LPR;
    const int b = blockIdx.y, which = blockIdx.z, lane = threadIdx.x % LPR;
    const NewRows nr = new_rows(a.lengths, a.n_new, b, a.n_tokens);
    const uint8_t *rows = a.rows[which] + b * a.stream + lane * 16;
    uint8_t *cache = const_cast<uint8_t *>(which ? a.c.v : a.c.k) + b * a.c.stream + lane * (Q8 ? E : 2 * E);
    float *scales = Q8 ? const_cast<float *>(which ? a.c.vs : a.c.ks) + b * a.c.sstream : nullptr;
    S s;
    for (int r0 = blockIdx.x * (U * S::RPB); r0 < nr.n * a.kvh; r0 += gridDim.x * (U * S::RPB)) {
        s.at(a, nr, r0);
        uint4 in[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            in[u] = make_uint4(0, 0, 0, 0);
            if (s.live[u]) in[u] = __ldcs(reinterpret_cast<const uint4 *>(rows + s.t[u] * a.token + s.h[u] * a.head));
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
            uint8_t *dst = cache + s.h[u] * a.c.head + s.pos[u] * a.c.row;
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
                if (s.live[u]) {
                    if constexpr (E == 8)
                        *reinterpret_cast<uint2 *>(dst) = make_uint2(w[0], w[1]);
                    else
                        *reinterpret_cast<uint32_t *>(dst) = w[0];
                    if (lane == 0) scales[s.h[u] * a.c.shead + s.pos[u]] = scale[u];
                }
            } else if (s.live[u]) {
                if constexpr (E == 8)
                    *reinterpret_cast<uint4 *>(dst) = in[u];
                else
                    *reinterpret_cast<uint2 *>(dst) = make_uint2(pack2_bf16(x[0], x[1]), pack2_bf16(x[2], x[3]));
            }
        }
    }
}

template <typename T, int D, bool Q8, int U>
__global__ void __launch_bounds__(kRowThreads) kv_read_kernel(const RowsArgs a) {
    using S = RowSet<T, D, U>;
    constexpr int E = S::E, LPR = S::LPR, W = Q8 ? E / 4 : E / 2;   // words a lane reads
    const int b = blockIdx.y, which = blockIdx.z, lane = threadIdx.x % LPR;
    const NewRows nr = new_rows(a.lengths, a.n_new, b, a.n_tokens);
    uint8_t *rows = const_cast<uint8_t *>(a.rows[which]) + b * a.stream + lane * 16;
    const uint8_t *cache = (which ? a.c.v : a.c.k) + b * a.c.stream + lane * (W * 4);
    const float *scales = Q8 ? (which ? a.c.vs : a.c.ks) + b * a.c.sstream : nullptr;
    S s;
    for (int r0 = blockIdx.x * (U * S::RPB); r0 < nr.n * a.kvh; r0 += gridDim.x * (U * S::RPB)) {
        s.at(a, nr, r0);
        uint32_t w[U][W];
        float scale[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int i = 0; i < W; ++i) w[u][i] = 0;
            scale[u] = 0.f;
            if (!s.live[u]) continue;
            const uint8_t *src = cache + s.h[u] * a.c.head + s.pos[u] * a.c.row;
            if constexpr (W == 4) {
                const uint4 v = *reinterpret_cast<const uint4 *>(src);
                w[u][0] = v.x, w[u][1] = v.y, w[u][2] = v.z, w[u][3] = v.w;
            } else if constexpr (W == 2) {
                const uint2 v = *reinterpret_cast<const uint2 *>(src);
                w[u][0] = v.x, w[u][1] = v.y;
            } else {
                w[u][0] = *reinterpret_cast<const uint32_t *>(src);
            }
            if constexpr (Q8) scale[u] = scales[s.h[u] * a.c.shead + s.pos[u]];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (!s.live[u]) continue;
            float x[E];
#pragma unroll
            for (int e = 0; e < E; ++e)
                x[e] = Q8 ? __fmul_rn(code_of(w[u][(e / 4) % W], e & 3), scale[u])
                          : (e & 1 ? bf16hi(w[u][(e / 2) % W]) : bf16lo(w[u][(e / 2) % W]));
            uint4 o;
            if constexpr (E == 8)
                o = make_uint4(pack2_bf16(x[0], x[1]), pack2_bf16(x[2], x[3]), pack2_bf16(x[4], x[5]),
                               pack2_bf16(x[6], x[7]));
            else
                o = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                               __float_as_uint(x[3]));
            __stcs(reinterpret_cast<uint4 *>(rows + s.t[u] * a.token + s.h[u] * a.head), o);
        }
    }
}

constexpr int kRowSets = 4;   // rows in flight a thread, where there are that many

typedef void (*RowsFn)(const RowsArgs);
template <typename T, int U> RowsFn rows_fn(bool read, int d, bool q8) {
    if (d == 64) {
        if (read) return q8 ? kv_read_kernel<T, 64, true, U> : kv_read_kernel<T, 64, false, U>;
        return q8 ? kv_append_kernel<T, 64, true, U> : kv_append_kernel<T, 64, false, U>;
    }
    if (read) return q8 ? kv_read_kernel<T, 128, true, U> : kv_read_kernel<T, 128, false, U>;
    return q8 ? kv_append_kernel<T, 128, true, U> : kv_append_kernel<T, 128, false, U>;
}

qd_status move_rows(bool read, const qd_kv_cache *cache, const void *k_rows, const void *v_rows, int dtype,
                    int n_tokens, int64_t stream_stride, int64_t token_stride, int64_t head_stride,
                    const int32_t *lengths, const int32_t *n_new, void *cuda_stream) {
    qd_status st = check_cache(cache, -1, false);
    if (st != QD_OK) return st;
    if ((dtype != QD_F32 && dtype != QD_BF16) || n_tokens < 1 || cache->n_streams > 65535) return QD_EINVAL;
    if (!k_rows || !v_rows || !lengths) return QD_EINVAL;
    const int64_t unit = dtype == QD_F32 ? 4 : 8, e = dtype == QD_F32 ? 4 : 2;
    if (stream_stride < 0 || token_stride < 0 || head_stride < 0 || stream_stride % unit || token_stride % unit ||
        head_stride % unit)
        return QD_EINVAL;
    if (!is_aligned(k_rows, 16) || !is_aligned(v_rows, 16) || !is_aligned(lengths, 4) || !is_aligned(n_new, 4))
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
    const int rpb = kRowThreads / (cache->head_dim / (int)unit);
    const long long rows = (long long)n_tokens * cache->n_kv_heads;
    if (rows > INT32_MAX / 2) return QD_EUNSUPPORTED;
    const bool many = rows > rpb, q8 = cache->format == QD_KV_Q8;
    const long long per = (long long)rpb * (many ? kRowSets : 1);
    const long long most = std::max(1, sms_of(dev) * 16 / cache->n_streams);
    const dim3 grid((unsigned)std::min((rows + per - 1) / per, most), (unsigned)cache->n_streams, 2);
    const int d = cache->head_dim;
    const RowsFn fn = dtype == QD_F32 ? (many ? rows_fn<float, kRowSets>(read, d, q8) : rows_fn<float, 1>(read, d, q8))
                                      : (many ? rows_fn<__nv_bfloat16, kRowSets>(read, d, q8)
                                              : rows_fn<__nv_bfloat16, 1>(read, d, q8));
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
