// What the operators over caller-held caches share: the device form of a qd_kv_cache,
// its host checks, and the positions of a stream's new rows.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>
#include <initializer_list>

#include "qd.h"

namespace qd {

struct KvView {
    const uint8_t *k, *v;              // rows of codes or bf16
    const float *ks, *vs;              // row scales (8-bit format)
    int64_t stream, head, row;         // BYTES between streams, heads, rows
    int64_t sstream, shead;            // floats between the scales' streams, heads
};

// Rows of stream b that a call uses, and the position of the first.
struct NewRows {
    int n, first;
};
__device__ __forceinline__ NewRows new_rows(const int32_t *lengths, const int32_t *n_new, int b, int n_tokens) {
    int n = n_new ? n_new[b] : n_tokens;
    n = n < 0 ? 0 : n > n_tokens ? n_tokens : n;
    return {n, max(lengths[b], 0) - n};   // (below 0 all positions are, with no overflow)
}

// Device (or managed) memory of the current device.
inline bool on_device(const void *p, int dev) {
    if (!p) return false;
    cudaPointerAttributes at;
    if (cudaPointerGetAttributes(&at, p) != cudaSuccess) {
        cudaGetLastError();
        return false;
    }
    return (at.type == cudaMemoryTypeDevice && at.device == dev) || at.type == cudaMemoryTypeManaged;
}

// SMs of the current device (152 on a GB300), looked up once per device.
inline int sms_of(int dev) {
    static std::atomic<int> known[64] = {};
    if (dev < 0 || dev >= 64) return 152;
    int n = known[dev].load(std::memory_order_relaxed);
    if (n) return n;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 152;
    known[dev].store(n, std::memory_order_relaxed);
    return n;
}

inline bool is_aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// The checks of a cache that need no device, then those of its memory (dev >= 0).
inline qd_status check_cache(const qd_kv_cache *c, int dev, bool one_stream) {
    if (!c || !c->k || !c->v || c->n_streams < 1 || c->n_kv_heads < 1 || c->smax < 1) return QD_EINVAL;
    if (c->format != QD_KV_BF16 && c->format != QD_KV_Q8) return QD_EINVAL;
    if (c->head_dim != 64 && c->head_dim != 128) return QD_EUNSUPPORTED;
    const int64_t unit = c->format == QD_KV_Q8 ? 16 : 8;   // elements of 16 bytes
    if (c->row_stride < c->head_dim || c->row_stride % unit || c->head_stride < 0 || c->head_stride % unit)
        return QD_EINVAL;
    if (!one_stream && (c->stream_stride < 0 || c->stream_stride % unit)) return QD_EINVAL;
    if (!is_aligned(c->k, 16) || !is_aligned(c->v, 16)) return QD_EINVAL;
    if (c->format == QD_KV_Q8) {
        if (!c->k_scale || !c->v_scale || !is_aligned(c->k_scale, 4) || !is_aligned(c->v_scale, 4)) return QD_EINVAL;
        if (c->scale_head_stride < 0 || (!one_stream && c->scale_stream_stride < 0)) return QD_EINVAL;
    }
    if (dev >= 0) {
        if (!on_device(c->k, dev) || !on_device(c->v, dev)) return QD_EINVAL;
        if (c->format == QD_KV_Q8 && (!on_device(c->k_scale, dev) || !on_device(c->v_scale, dev))) return QD_EINVAL;
    }
    return QD_OK;
}

// What a call writes must have bytes of its own: pieces of `inner` elements of e bytes at every combination of the
// axes' steps (in elements), in one array or in two `pair` bytes apart.  From the smallest step on, each has to pass over all that the
// smaller ones span; axes that interleave without nesting are refused too.
struct Axis {
    int64_t n, stride;
};
inline bool apart(int64_t e, int64_t inner, std::initializer_list<Axis> axes, int64_t pair = 0) {
    constexpr int64_t kMost = int64_t(1) << 62;   // no address is as far
    Axis a[5];
    int n = 0;
    for (const Axis &x : axes)
        if (x.n > 1) {
            if (x.stride > kMost / e) return false;
            a[n++] = {x.n, x.stride * e};
        }
    if (pair) a[n++] = {2, pair < 0 ? -pair : pair};
    std::sort(a, a + n, [](const Axis &x, const Axis &y) { return x.stride < y.stride; });
    int64_t span = inner * e;
    for (int i = 0; i < n; ++i) {
        if (a[i].stride < span || a[i].n - 1 > (kMost - span) / a[i].stride) return false;
        span += (a[i].n - 1) * a[i].stride;
    }
    return true;
}
inline int64_t bytes_between(const void *a, const void *b) {
    return (int64_t)(reinterpret_cast<uintptr_t>(b) - reinterpret_cast<uintptr_t>(a));
}

inline KvView kv_view(const qd_kv_cache *c) {
    const int64_t e = c->format == QD_KV_Q8 ? 1 : 2;
    return {static_cast<const uint8_t *>(c->k), static_cast<const uint8_t *>(c->v), c->k_scale, c->v_scale,
            c->stream_stride * e, c->head_stride * e, c->row_stride * e, c->scale_stream_stride,
            c->scale_head_stride};
}

}  // namespace qd
