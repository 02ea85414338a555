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
// the magnitudes, NaN above infinity, so one comparison finds a row that is not finite).
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

__device__ __forceinline__ uint32_t pack2_bf16(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// grid (row blocks, streams, K and V); LPR lanes a row
template <typename T, int D, bool Q8>
__global__ void __launch_bounds__(kRowThreads) kv_append_kernel(const RowsArgs a) {
    constexpr int E = Vec16<T>::E, LPR = D / E, RPB = kRowThreads / LPR;
    const int b = blockIdx.y, which = blockIdx.z;
    const NewRows nr = new_rows(a.lengths, a.n_new, b, a.n_tokens);
    const int lane = threadIdx.x % LPR;
    const long long n = (long long)nr.n * a.kvh;
    for (long long r = (long long)blockIdx.x * RPB + threadIdx.x / LPR; r - threadIdx.x / LPR < n; r += (long long)gridDim.x * RPB) {
        const int t = (int)(r / a.kvh), h = (int)(r - (long long)t * a.kvh);
        const int pos = nr.first + t;
        const bool live = r < n && pos >= 0 && pos < a.smax;
        float x[E];
        uint4 u = make_uint4(0, 0, 0, 0);
        if (live)
            u = *reinterpret_cast<const uint4 *>(a.rows[which] + b * a.stream + t * a.token + h * a.head + lane * 16);
        Vec16<T>::unpack(u, x);
        uint8_t *dst = const_cast<uint8_t *>(which ? a.c.v : a.c.k) + b * a.c.stream + h * a.c.head + (int64_t)pos * a.c.row;
        if constexpr (Q8) {
            uint32_t m = 0;
#pragma unroll
            for (int e = 0; e < E; ++e) m = max(m, __float_as_uint(x[e]) & 0x7fffffffu);
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
            const bool finite = m < 0x7f800000u, zero = m < 0x05800000u;   // below 2^-116
            const float top = __uint_as_float(m);
            const float by = (zero || !finite) ? 0.f : __fdiv_rn(127.f, top);
            const float scale = !finite ? __uint_as_float(0x7fc00000u) : zero ? 0.f : __fdiv_rn(top, 127.f);
            uint32_t w[E / 4];
#pragma unroll
            for (int e = 0; e < E; e += 4) {
                uint32_t p = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int c = by != 0.f ? __float2int_rn(__fmul_rn(x[e + i], by)) : 0;
                    p |= (uint32_t)(c & 0xff) << (8 * i);
                }
                w[e / 4] = p;
            }
            if (live) {
                if constexpr (E == 8)
                    *reinterpret_cast<uint2 *>(dst + lane * 8) = make_uint2(w[0], w[1]);
                else
                    *reinterpret_cast<uint32_t *>(dst + lane * 4) = w[0];
                if (lane == 0)
                    const_cast<float *>(which ? a.c.vs : a.c.ks)[b * a.c.sstream + h * a.c.shead + pos] = scale;
            }
        } else if (live) {
            if constexpr (E == 8)
                *reinterpret_cast<uint4 *>(dst + lane * 16) = u;
            else
                *reinterpret_cast<uint2 *>(dst + lane * 8) = make_uint2(pack2_bf16(x[0], x[1]), pack2_bf16(x[2], x[3]));
        }
    }
}

template <typename T, int D, bool Q8>
__global__ void __launch_bounds__(kRowThreads) kv_read_kernel(const RowsArgs a) {
    constexpr int E = Vec16<T>::E, LPR = D / E, RPB = kRowThreads / LPR;
    const int b = blockIdx.y, which = blockIdx.z;
    const NewRows nr = new_rows(a.lengths, a.n_new, b, a.n_tokens);
    const int lane = threadIdx.x % LPR;
    const long long n = (long long)nr.n * a.kvh;
    for (long long r = (long long)blockIdx.x * RPB + threadIdx.x / LPR; r < n; r += (long long)gridDim.x * RPB) {
        const int t = (int)(r / a.kvh), h = (int)(r - (long long)t * a.kvh);
        const int pos = nr.first + t;
        if (pos < 0 || pos >= a.smax) continue;
        const uint8_t *src = (which ? a.c.v : a.c.k) + b * a.c.stream + h * a.c.head + (int64_t)pos * a.c.row;
        float x[E];
        if constexpr (Q8) {
            const float s = (which ? a.c.vs : a.c.ks)[b * a.c.sstream + h * a.c.shead + pos];
            uint32_t w[E / 4];
            if constexpr (E == 8) {
                const uint2 u = *reinterpret_cast<const uint2 *>(src + lane * 8);
                w[0] = u.x, w[1] = u.y;
            } else {
                w[0] = *reinterpret_cast<const uint32_t *>(src + lane * 4);
            }
#pragma unroll
            for (int e = 0; e < E; ++e) x[e] = __fmul_rn((float)(int8_t)(w[e / 4] >> (8 * (e & 3))), s);
        } else if constexpr (E == 8) {
            Vec16<T>::unpack(*reinterpret_cast<const uint4 *>(src + lane * 16), x);
        } else {
            const uint2 u = *reinterpret_cast<const uint2 *>(src + lane * 8);
            x[0] = bf16lo(u.x), x[1] = bf16hi(u.x), x[2] = bf16lo(u.y), x[3] = bf16hi(u.y);
        }
        uint4 *dst = reinterpret_cast<uint4 *>(const_cast<uint8_t *>(a.rows[which]) + b * a.stream + t * a.token +
                                               h * a.head + lane * 16);
        if constexpr (E == 8)
            *dst = make_uint4(pack2_bf16(x[0], x[1]), pack2_bf16(x[2], x[3]), pack2_bf16(x[4], x[5]),
                              pack2_bf16(x[6], x[7]));
        else
            *dst = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                              __float_as_uint(x[3]));
    }
}

typedef void (*RowsFn)(const RowsArgs);
template <typename T> RowsFn rows_fn(bool read, int d, bool q8) {
    if (d == 64) {
        if (read) return q8 ? kv_read_kernel<T, 64, true> : kv_read_kernel<T, 64, false>;
        return q8 ? kv_append_kernel<T, 64, true> : kv_append_kernel<T, 64, false>;
    }
    if (read) return q8 ? kv_read_kernel<T, 128, true> : kv_read_kernel<T, 128, false>;
    return q8 ? kv_append_kernel<T, 128, true> : kv_append_kernel<T, 128, false>;
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
    const long long most = std::max(1, sms_of(dev) * 16 / cache->n_streams);
    const dim3 grid((unsigned)std::min((rows + rpb - 1) / rpb, most), (unsigned)cache->n_streams, 2);
    const RowsFn fn = dtype == QD_F32 ? rows_fn<float>(read, cache->head_dim, cache->format == QD_KV_Q8)
                                      : rows_fn<__nv_bfloat16>(read, cache->head_dim, cache->format == QD_KV_Q8);
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
