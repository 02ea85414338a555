// Attention of each stream's new tokens over its cached keys and values (bf16 or 8-bit
// rows), and over a prefix that all streams share.
//
// Per stream, key head and row r = (new token, query head of the group):
//   s_j = log2(e) scale q_r . k_j,   p_j = 2^(s_j - ref),   out = sum p_j v_j / sum p_j
// in one pass over the positions: ref follows the running maximum and the sums are
// rescaled when it moves.  8-bit rows stand for code * scale, one scale a row: the keys'
// scale multiplies s_j, the values' scale multiplies p_j on its way into the product, so
// the tensor cores work on the codes themselves (exact in fp16).
//
// Decoding has few rows and many positions, so the positions are the long side (M = 16) of
// m16n8k16 and the rows its N = 8 columns.  Where a value must keep more bits than the
// tensor core's type has, it takes C columns, one per part (q and p alike; the parts'
// products are added afterwards): fp32 rows 2 fp16 parts over an 8-bit cache, 3 bf16 parts of 4 columns over
// a bf16 one.  bf16 rows have one part of q and two of p (16 bits of bf16, 22 of fp16), in two columns for up to 8 rows of a
// bf16 cache, else in one column each and two products (hi, then lo) into the same sums.
//
// Neither K nor V is laid out anew in shared memory.  The products' sums run over head_dim
// (scores) and positions (output) in any order, so each lane takes 16 contiguous bytes of a
// row as its share of the A fragment, and q is laid out to match.  For the output, V^T is
// A: a lane holds the same dims of the four positions its fragment pairs, and a byte
// permutation pairs them up, the same that widens the codes.  The probabilities turn from
// the accumulator's layout into the B fragment's with movmatrix.  Each warp has a ring of
// tiles of its own that it fills with cp.async, whole 128-byte lines at a time (a copy by
// fragment made a write into shared memory of every 32-byte sector: 46 us against 37 for 64
// ragged 8-bit streams), the 16-byte pieces of a row placed so that fragments read without
// bank conflicts; no barrier is wider than the warp.
//
// Three ways over a stream's cache, by the sizes alone (make_plan):
//  - small batches: a cluster of CTAs per (stream, key head, rows) item, one wave of them; the
//    warps take the tiles in turn and their partial results (ref, sum, output) meet in
//    distributed shared memory, in a fixed order.  One launch, no scratch; bound by its
//    chain of loads (1 x 600 positions 5.4 us, as many of them the launch).
//  - larger ones: attn_share_kernel's equal runs over all warps and attn_join_kernel.  Bound by HBM:
//    3 streams of up to 65536 8-bit positions, 334 MB, 58 us (0.85 of the measured rate); 64
//    of 257 to 2048, 156 MB, 34 us (0.68: 23 for the bytes, the launches, a pipeline's start and
//    the join the rest).
//  - a prefix: read by every stream's own pass while that is cheap, else by
//    attn_prefix_tc_kernel (bf16 rows) or once for every group of rows (PREFIX here).
#include "attn_pass.cuh"

namespace qd {

namespace {

// The checks of sizes that the call and its workspace query share.
qd_status check_sizes(const qd_kv_cache *cache, const qd_kv_cache *prefix, int prefix_length, int dtype, int n_tokens,
                      int n_q_heads, int max_length) {
    qd_status st = check_cache(cache, -1, false);
    if (st != QD_OK) return st;
    if (prefix_length < 0 || (!prefix && prefix_length)) return QD_EINVAL;
    if (prefix && prefix_length > 0) {
        if ((st = check_cache(prefix, -1, true)) != QD_OK) return st;
        if (prefix->n_kv_heads != cache->n_kv_heads || prefix->head_dim != cache->head_dim ||
            prefix_length > prefix->smax)
            return QD_EINVAL;
    }
    const int kvh = cache->n_kv_heads;
    if ((dtype != QD_F32 && dtype != QD_BF16) || n_tokens < 1 || n_q_heads < kvh || n_q_heads % kvh) return QD_EINVAL;
    if (max_length < 1 || max_length > cache->smax) return QD_EINVAL;
    if (n_tokens > kAcMaxTokens || max_length > kAcMaxPositions || prefix_length > kAcMaxPositions) return QD_EUNSUPPORTED;
    const int64_t all = (int64_t)n_tokens * (n_q_heads / kvh) * cache->n_streams;
    if (all > (1 << 24) || all * kvh > (1 << 26)) return QD_EUNSUPPORTED;
    return QD_OK;
}

}  // namespace

}  // namespace qd

using namespace qd;

extern "C" {

qd_status qd_attn_cached_workspace(const qd_kv_cache *cache, const qd_kv_cache *prefix, int prefix_length, int dtype,
                                   int n_tokens, int n_q_heads, int max_length, size_t *bytes) {
    if (!bytes) return QD_EINVAL;
    *bytes = 0;
    qd_status st = check_sizes(cache, prefix, prefix_length, dtype, n_tokens, n_q_heads, max_length);
    if (st != QD_OK) return st;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return QD_ECUDA;
    Plan p;
    if ((st = make_plan<false>(cache, cache->n_streams, prefix, prefix_length, dtype == QD_F32, n_tokens, n_q_heads, max_length, dev, &p)) != QD_OK)
        return st;
    *bytes = p.bytes;
    return QD_OK;
}

qd_status qd_attn_cached(const qd_kv_cache *cache, const qd_kv_cache *prefix, int prefix_length, const void *q_dev,
                         int64_t q_stream_stride, int64_t q_token_stride, void *out_dev, int64_t out_stream_stride,
                         int64_t out_token_stride, int dtype, int n_tokens, int n_q_heads, float scale,
                         const int32_t *lengths_dev, const int32_t *n_new_dev, int max_length, void *workspace_dev,
                         size_t workspace_bytes, void *cuda_stream) {
    qd_status st = check_sizes(cache, prefix, prefix_length, dtype, n_tokens, n_q_heads, max_length);
    if (st != QD_OK) return st;
    const bool with_prefix = prefix && prefix_length > 0, f32 = dtype == QD_F32;
    if (!(scale > -3e38f && scale < 3e38f) || !q_dev || !out_dev || !lengths_dev) return QD_EINVAL;
    const int64_t unit = f32 ? 4 : 8, e = f32 ? 4 : 2;
    for (int64_t v : {q_stream_stride, q_token_stride, out_stream_stride, out_token_stride})
        if (v < 0 || v % unit) return QD_EINVAL;
    if (!is_aligned(q_dev, 16) || !is_aligned(out_dev, 16) || !is_aligned(lengths_dev, 4) || !is_aligned(n_new_dev, 4))
        return QD_EINVAL;
    if (!rows_apart(q_dev, q_stream_stride, q_token_stride, out_dev, out_stream_stride, out_token_stride, e, cache->n_streams, n_tokens,
                    (int64_t)n_q_heads * cache->head_dim))
        return QD_EINVAL;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return QD_ECUDA;
    if ((st = check_cache(cache, dev, false)) != QD_OK) return st;
    if (with_prefix && (st = check_cache(prefix, dev, true)) != QD_OK) return st;
    if (!on_device(q_dev, dev) || !on_device(out_dev, dev) || !on_device(lengths_dev, dev) ||
        (n_new_dev && !on_device(n_new_dev, dev)))
        return QD_EINVAL;
    Plan p;
    if ((st = make_plan<false>(cache, cache->n_streams, prefix, prefix_length, f32, n_tokens, n_q_heads, max_length, dev, &p)) != QD_OK) return st;
    if (p.bytes && (!workspace_dev || workspace_bytes < p.bytes || !is_aligned(workspace_dev, 256) ||
                    !on_device(workspace_dev, dev)))
        return QD_EINVAL;

    const int kvh = cache->n_kv_heads, d = cache->head_dim, B = cache->n_streams;
    uint8_t *ws = static_cast<uint8_t *>(workspace_dev);
    cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
    CachedArgs a = {};
    a.q = static_cast<const uint8_t *>(q_dev), a.out = static_cast<uint8_t *>(out_dev);
    a.q_stream = q_stream_stride * e, a.q_token = q_token_stride * e;
    a.o_stream = out_stream_stride * e, a.o_token = out_token_stride * e;
    a.lengths = lengths_dev, a.n_new = n_new_dev;
    a.B = B, a.T = n_tokens, a.G = n_q_heads / kvh, a.kvh = kvh;
    a.scale2 = scale * 1.4426950408889634f;
    if (p.inline_prefix) {
        a.pc = kv_view(prefix);
        a.pre_len = prefix_length, a.pre_tiles = (prefix_length + p.tp - 1) / p.tp;
    } else if (with_prefix) {
        a.p_ml = reinterpret_cast<float2 *>(ws + p.p_ml), a.p_o = reinterpret_cast<float *>(ws + p.p_o);
        a.splits = p.splits;
        if (p.wide) a.wide = p.wide, a.wide_chunks = (prefix_length + kWideKeys - 1) / kWideKeys;
        CachedArgs x = a;
        x.c = kv_view(prefix);
        x.rows = (int)p.rows_all, x.groups = p.p_groups, x.max_len = prefix_length;
        unsigned ctas = (unsigned)(p.p_groups * kvh * p.splits);
        if (p.wide) {
            if (launch_attn_prefix_tc(prefix->format == QD_KV_Q8, d, x, p.wide, s) != cudaSuccess) return QD_ECUDA;
        } else if (dispatch<false>(kPassPrefix, prefix->format == QD_KV_Q8, f32, d, p.p_nt, x, &ctas, p.splits, dev, s) != cudaSuccess)
            return QD_ECUDA;
    }
    const bool q8 = cache->format == QD_KV_Q8;
    a.c = kv_view(cache);
    a.rows = n_tokens * a.G, a.groups = p.groups, a.max_len = max_length;
    if (p.nsplit) {
        unsigned ctas = (unsigned)((int64_t)B * kvh * p.groups * p.nsplit);
        return dispatch<false>(kPassCluster, q8, f32, d, p.nt, a, &ctas, p.nsplit, dev, s) == cudaSuccess ? QD_OK : QD_ECUDA;
    }
    a.s_ml = reinterpret_cast<float2 *>(ws + p.s_ml), a.s_o = reinterpret_cast<float *>(ws + p.s_o);
    if (dispatch<false>(kPassShare, q8, f32, d, p.nt, a, &p.ctas, 0, dev, s) != cudaSuccess) return QD_ECUDA;
    // many partials a row (long streams, few of them): several warps per row
    const unsigned warps = p.ctas * kAcWarps, items = (unsigned)((int64_t)B * kvh * p.groups);
    return launch_join(f32, d, a, p.rw, p.tp, warps, warps / items + p.splits > 16, sms_of(dev), s) == cudaSuccess ? QD_OK : QD_ECUDA;
}

}  // extern "C"
