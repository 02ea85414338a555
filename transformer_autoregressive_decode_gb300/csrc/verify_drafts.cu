// Verification of drafted tokens (speculative sampling): draft x_t passes if u_t q_t(x_t) <
// p_t(x_t); the first that fails is replaced by a draw from max(p_t - q_t, 0), and where all
// pass the next token is drawn from p of the position behind them.
//
// Only one row of p and one of q are needed in full: those of the position that is drawn
// from, which T pairs of scalars decide.  A cluster of CTAs per stream shares that row:
// every CTA finds the position by itself, adds up its slice (one sum per warp), reads all
// the cluster's warp sums through distributed shared memory, and the one warp whose slice holds
// the mark walks it.  One launch, no scratch memory; 8 bytes per vocabulary entry are read
// once, which bounds large vocabularies by HBM and small ones by the launch and the
// three dependent loads before the sum.
//
// The weights are whole numbers, floor(w 2^44): their sums are exact in any order, so the
// drawn id does not depend on how the row is split, and 2^19 of them fit 63 bits.
#include "kv_view.cuh"
#include "qd_device.cuh"
#include "qd_internal.h"

namespace qd {

namespace {

constexpr int kVfThreads = 512, kVfWarps = kVfThreads / 32;
constexpr int kVfCluster = 8;
constexpr int kVfMaxTokens = 64, kVfMaxVocab = 524288;

struct VerifyArgs {
    const float *p, *q;
    int64_t p_stream, p_row, q_stream, q_row;   // elements
    const int32_t *ids, *n_draft;
    const float *u;
    int T, V;
    int32_t *out, *accepted;
};

// floor(w 2^44); fmaxf takes a NaN to 0
__device__ __forceinline__ unsigned long long weight(float w) {
    w = fminf(fmaxf(w, 0.f), 1.f);
    return __float2ull_rz(__fmul_rn(w, 17592186044416.f));
}

__device__ __forceinline__ unsigned long long warp_sum_u64(unsigned long long v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// The weights of entries [i, i + 4) of the row drawn from: p, p - q, or p without the drafted id.
struct Row {
    const float *p, *q;
    int hole, V;
    bool vec;
    __device__ __forceinline__ float left(float a, float b) const { return q ? __fsub_rn(a, b) : a; }
    __device__ __forceinline__ void load4(int i, unsigned long long *w) const {
        float a[4] = {0.f, 0.f, 0.f, 0.f}, b[4] = {0.f, 0.f, 0.f, 0.f};
        if (vec && i + 4 <= V) {
            const float4 x = __ldg(reinterpret_cast<const float4 *>(p + i));
            a[0] = x.x, a[1] = x.y, a[2] = x.z, a[3] = x.w;
            if (q) {
                const float4 y = __ldg(reinterpret_cast<const float4 *>(q + i));
                b[0] = y.x, b[1] = y.y, b[2] = y.z, b[3] = y.w;
            }
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (i + e < V) {
                    a[e] = __ldg(p + i + e);
                    if (q) b[e] = __ldg(q + i + e);
                }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = i + e == hole ? 0ull : weight(left(a[e], b[e]));
    }
};

__global__ void __cluster_dims__(kVfCluster, 1, 1) __launch_bounds__(kVfThreads) verify_kernel(const VerifyArgs a) {
    __shared__ unsigned long long sums[kVfWarps];
    __shared__ unsigned long long all[kVfCluster * kVfWarps];
    __shared__ int s_pass;
    const int b = blockIdx.x / kVfCluster, rank = (int)cluster_ctarank();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int n = a.n_draft ? a.n_draft[b] : a.T;
    n = n < 0 ? 0 : n > a.T ? a.T : n;

    // the drafts that pass: each lane of warp 0 decides two of them
    if (warp == 0) {
        int first = n;
        for (int t0 = 0; t0 < n; t0 += 32) {
            const int t = t0 + lane;
            bool ok = true;
            if (t < n) {
                const int x = a.ids[(int64_t)b * a.T + t];
                ok = x >= 0 && x < a.V;
                if (ok) {
                    const float px = a.p[b * a.p_stream + t * a.p_row + x];
                    const float qx = a.q ? a.q[b * a.q_stream + t * a.q_row + x] : 1.f;
                    // 24-bit factors: the product is exact in fp64
                    ok = (double)a.u[(int64_t)b * (a.T + 1) + t] * (double)qx < (double)px;
                }
            }
            const uint32_t bad = ~__ballot_sync(0xffffffffu, ok);
            if (bad) {
                first = t0 + __ffs(bad) - 1;
                break;
            }
        }
        if (lane == 0) s_pass = first;
    }
    __syncthreads();
    const int pass = s_pass;
    if (rank == 0) {
        for (int s = threadIdx.x; s <= a.T; s += kVfThreads)
            if (s != pass) a.out[(int64_t)b * (a.T + 1) + s] = s < pass ? a.ids[(int64_t)b * a.T + s] : -1;
        if (threadIdx.x == 0) a.accepted[b] = pass;
    }

    Row row;
    row.p = a.p + b * a.p_stream + pass * a.p_row;
    row.q = (pass < n && a.q) ? a.q + b * a.q_stream + pass * a.q_row : nullptr;
    row.hole = (pass < n && !a.q) ? a.ids[(int64_t)b * a.T + pass] : -1;
    row.V = a.V;
    row.vec = ((reinterpret_cast<uintptr_t>(row.p) | reinterpret_cast<uintptr_t>(row.q)) & 15) == 0;

    // slices in multiples of 128 entries (one float4 a lane), one per warp of the cluster
    const int parts = kVfCluster * kVfWarps;
    const int per = ((a.V + parts - 1) / parts + 127) / 128 * 128;
    const int me = rank * kVfWarps + warp;
    const int i0 = min(me * per, a.V), i1 = min(i0 + per, a.V);
    unsigned long long total = 0;
    for (int round = 0; round < 2; ++round) {
        unsigned long long s = 0;
        for (int i = i0 + lane * 4; i < i1; i += 128) {
            unsigned long long w[4];
            row.load4(i, w);
            s += (w[0] + w[1]) + (w[2] + w[3]);
        }
        s = warp_sum_u64(s);
        if (lane == 0) sums[warp] = s;
        cluster_sync();
        if (threadIdx.x < parts) {
            const uint32_t at = cluster_map(&sums[threadIdx.x % kVfWarps], threadIdx.x / kVfWarps);
            unsigned long long v;
            asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(at) : "memory");
            all[threadIdx.x] = v;
        }
        cluster_sync();      // every CTA has read the sums: they may be written again, and CTAs may leave
        total = 0;
        for (int i = 0; i < parts; ++i) total += all[i];
        if (total != 0 || (!row.q && row.hole < 0)) break;
        row.q = nullptr;     // nothing left of p - q: the draw is from p
        row.hole = -1;
        row.vec = (reinterpret_cast<uintptr_t>(row.p) & 15) == 0;
    }

    if (total == 0) {
        if (rank == 0 && threadIdx.x == 0) a.out[(int64_t)b * (a.T + 1) + pass] = -1;
        return;
    }
    const double u = (double)a.u[(int64_t)b * (a.T + 1) + a.T];
    unsigned long long mark = (unsigned long long)floor(u * __ull2double_rn(total));
    if (mark >= total) mark = total - 1;   // u in [0, 1) gives less
    unsigned long long before = 0;
    for (int i = 0; i < me; ++i) before += all[i];
    if (mark < before || mark - before >= all[me]) return;

    // this warp's slice holds the mark: 128 entries a step, then the lane, then the entry
    for (int i = i0; i < i1; i += 128) {
        unsigned long long w[4];
        row.load4(i + lane * 4, w);
        if (i + lane * 4 >= i1) w[0] = w[1] = w[2] = w[3] = 0;
        const unsigned long long own = (w[0] + w[1]) + (w[2] + w[3]);
        unsigned long long upto = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned long long v = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += v;
        }
        const uint32_t over = __ballot_sync(0xffffffffu, before + upto > mark);
        if (over) {
            if (lane == __ffs(over) - 1) {
                unsigned long long c = before + upto - own;
                int e = 0;
                while (e < 3 && c + w[e] <= mark) c += w[e++];
                a.out[(int64_t)b * (a.T + 1) + pass] = i + lane * 4 + e;
            }
            return;
        }
        before += __shfl_sync(0xffffffffu, upto, 31);
    }
}

}  // namespace

}  // namespace qd

using namespace qd;

extern "C" qd_status qd_verify_drafts(const float *target_probs_dev, int64_t target_stream_stride,
                                      int64_t target_row_stride, const float *draft_probs_dev,
                                      int64_t draft_stream_stride, int64_t draft_row_stride,
                                      const int32_t *draft_ids_dev, const int32_t *n_draft_dev, const float *u_dev,
                                      int n_streams, int n_tokens, int vocab, int32_t *out_ids_dev,
                                      int32_t *n_accepted_dev, void *cuda_stream) {
    if (n_streams < 1 || n_streams > (1 << 24) || n_tokens < 1 || n_tokens > kVfMaxTokens || vocab < 1 ||
        vocab > kVfMaxVocab)
        return QD_EINVAL;
    if (target_stream_stride < 0 || target_row_stride < 0) return QD_EINVAL;
    if (draft_probs_dev && (draft_stream_stride < 0 || draft_row_stride < 0)) return QD_EINVAL;
    if (!target_probs_dev || !draft_ids_dev || !u_dev || !out_ids_dev || !n_accepted_dev) return QD_EINVAL;
    const void *ptrs[7] = {target_probs_dev, draft_ids_dev, u_dev, out_ids_dev, n_accepted_dev, draft_probs_dev,
                           n_draft_dev};
    for (const void *p : ptrs)
        if (!is_aligned(p, 4)) return QD_EINVAL;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return QD_ECUDA;
    for (int i = 0; i < 7; ++i)
        if ((i < 5 || ptrs[i]) && !on_device(ptrs[i], dev)) return QD_EINVAL;
    VerifyArgs a;
    a.p = target_probs_dev, a.q = draft_probs_dev;
    a.p_stream = target_stream_stride, a.p_row = target_row_stride;
    a.q_stream = draft_stream_stride, a.q_row = draft_row_stride;
    a.ids = draft_ids_dev, a.n_draft = n_draft_dev, a.u = u_dev;
    a.T = n_tokens, a.V = vocab;
    a.out = out_ids_dev, a.accepted = n_accepted_dev;
    verify_kernel<<<n_streams * kVfCluster, kVfThreads, 0, static_cast<cudaStream_t>(cuda_stream)>>>(a);
    return cudaGetLastError() == cudaSuccess ? QD_OK : QD_ECUDA;
}
