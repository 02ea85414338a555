// Attention of each stream's new tokens over a cache in pages (bf16 or 8-bit rows): the passes of attn_pass.cuh, a
// cluster of CTAs per (stream, key head, rows) for small batches, equal runs of tiles and a join for larger ones.
//
// A page holds a power of two of positions, 16 or more, so a block of 16 positions, the unit of the tensor core's products,
// lies in one page: a tile is one or two blocks, each with a page of its own, and a page that ends inside a tile
// needs nothing further.  The pages of a tile are looked up while the one before it is being copied; that look-up (through L2 at
// the first touch of a line of the table, from L1 then) is all that the pages cost beside the contiguous form.  What bounds the passes: as there,
// HBM for long caches, the chain of loads for short ones.
#include "attn_pass.cuh"

namespace qd {

namespace {

// The checks of sizes that the call and its workspace query share.
qd_status check_paged(const qd_kv_cache *pages, const int32_t *table, int64_t table_stride, int table_pages, int n_streams, int dtype,
                      int n_tokens, int n_q_heads, int max_length, int *shift) {
    const qd_status st = check_pages(pages, table, table_stride, table_pages, n_streams, -1, shift);
    if (st != QD_OK) return st;
    const int kvh = pages->n_kv_heads;
    if ((dtype != QD_F32 && dtype != QD_BF16) || n_tokens < 1 || n_q_heads < kvh || n_q_heads % kvh) return QD_EINVAL;
    if (max_length < 1 || max_length > (int64_t)table_pages * pages->smax) return QD_EINVAL;
    if (n_tokens > kAcMaxTokens) return QD_EUNSUPPORTED;
    const int64_t all = (int64_t)n_tokens * (n_q_heads / kvh) * n_streams;
    if (all > (1 << 24) || all * kvh > (1 << 26)) return QD_EUNSUPPORTED;
    return QD_OK;
}

}  // namespace

}  // namespace qd

using namespace qd;

extern "C" {

qd_status qd_attn_paged_workspace(const qd_kv_cache *pages, int n_streams, int table_pages, int dtype, int n_tokens, int n_q_heads,
                                  int max_length, size_t *bytes) {
    if (!bytes) return QD_EINVAL;
    *bytes = 0;
    int shift = 0;
    static const int32_t some = 0;                   // the table itself is not looked at
    qd_status st = check_paged(pages, &some, 0, table_pages, n_streams, dtype, n_tokens, n_q_heads, max_length, &shift);
    if (st != QD_OK) return st;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return QD_ECUDA;
    Plan p;
    if ((st = make_plan<true>(pages, n_streams, nullptr, 0, dtype == QD_F32, n_tokens, n_q_heads, max_length, dev, &p)) != QD_OK) return st;
    *bytes = p.bytes;
    return QD_OK;
}

qd_status qd_attn_paged(const qd_kv_cache *pages, const int32_t *page_table_dev, int64_t table_stride, int table_pages, int n_streams,
                        const void *q_dev, int64_t q_stream_stride, int64_t q_token_stride, void *out_dev, int64_t out_stream_stride,
                        int64_t out_token_stride, int dtype, int n_tokens, int n_q_heads, float scale, const int32_t *lengths_dev,
                        const int32_t *n_new_dev, int max_length, void *workspace_dev, size_t workspace_bytes, void *cuda_stream) {
    int shift = 0;
    qd_status st = check_paged(pages, page_table_dev, table_stride, table_pages, n_streams, dtype, n_tokens, n_q_heads, max_length, &shift);
    if (st != QD_OK) return st;
    const bool f32 = dtype == QD_F32;
    if (!(scale > -3e38f && scale < 3e38f) || !q_dev || !out_dev || !lengths_dev) return QD_EINVAL;
    const int64_t unit = f32 ? 4 : 8, e = f32 ? 4 : 2;
    for (int64_t v : {q_stream_stride, q_token_stride, out_stream_stride, out_token_stride})
        if (v < 0 || v % unit) return QD_EINVAL;
    if (!is_aligned(q_dev, 16) || !is_aligned(out_dev, 16) || !is_aligned(lengths_dev, 4) || !is_aligned(n_new_dev, 4))
        return QD_EINVAL;
    if (!rows_apart(q_dev, q_stream_stride, q_token_stride, out_dev, out_stream_stride, out_token_stride, e, n_streams, n_tokens,
                    (int64_t)n_q_heads * pages->head_dim))
        return QD_EINVAL;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return QD_ECUDA;
    if ((st = check_pages(pages, page_table_dev, table_stride, table_pages, n_streams, dev, &shift)) != QD_OK) return st;
    if (!on_device(q_dev, dev) || !on_device(out_dev, dev) || !on_device(lengths_dev, dev) ||
        (n_new_dev && !on_device(n_new_dev, dev)))
        return QD_EINVAL;
    Plan p;
    if ((st = make_plan<true>(pages, n_streams, nullptr, 0, f32, n_tokens, n_q_heads, max_length, dev, &p)) != QD_OK) return st;
    if (p.bytes && (!workspace_dev || workspace_bytes < p.bytes || !is_aligned(workspace_dev, 256) || !on_device(workspace_dev, dev)))
        return QD_EINVAL;

    const int kvh = pages->n_kv_heads, d = pages->head_dim, B = n_streams;
    uint8_t *ws = static_cast<uint8_t *>(workspace_dev);
    cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
    CachedArgs a = {};
    a.c = kv_view(pages);
    a.table = page_table_dev, a.table_stride = table_stride, a.page_shift = shift, a.n_pages = pages->n_streams;
    a.q = static_cast<const uint8_t *>(q_dev), a.out = static_cast<uint8_t *>(out_dev);
    a.q_stream = q_stream_stride * e, a.q_token = q_token_stride * e;
    a.o_stream = out_stream_stride * e, a.o_token = out_token_stride * e;
    a.lengths = lengths_dev, a.n_new = n_new_dev;
    a.B = B, a.T = n_tokens, a.G = n_q_heads / kvh, a.kvh = kvh;
    a.scale2 = scale * 1.4426950408889634f;
    a.rows = n_tokens * a.G, a.groups = p.groups, a.max_len = max_length;
    const bool q8 = pages->format == QD_KV_Q8;
    if (p.nsplit) {
        unsigned ctas = (unsigned)((int64_t)B * kvh * p.groups * p.nsplit);
        return dispatch<true>(kPassCluster, q8, f32, d, p.nt, a, &ctas, p.nsplit, dev, s) == cudaSuccess ? QD_OK : QD_ECUDA;
    }
    a.s_ml = reinterpret_cast<float2 *>(ws + p.s_ml), a.s_o = reinterpret_cast<float *>(ws + p.s_o);
    if (dispatch<true>(kPassShare, q8, f32, d, p.nt, a, &p.ctas, 0, dev, s) != cudaSuccess) return QD_ECUDA;
    const unsigned warps = p.ctas * kAcWarps, items = (unsigned)((int64_t)B * kvh * p.groups);
    return launch_join(f32, d, a, p.rw, p.tp, warps, warps / items > 16, sms_of(dev), s) == cudaSuccess ? QD_OK : QD_ECUDA;
}

}  // extern "C"
