// Verification of drafted tokens (speculative sampling): draft x_t passes if u_t q_t(x_t) <
// p_t(x_t); the first that fails is replaced by a draw from max(p_t - q_t, 0), and where all
// pass the next token is drawn from p of the position behind them.
//
// Only one row of p and one of q are needed in full: those of the position that is drawn
// from, which T pairs of scalars decide.  A CTA, or a cluster of them, per stream shares that row:
// every CTA finds the position by itself, adds up its slices (one per warp), reads all
// the cluster's slice sums through distributed shared memory, and the one warp whose slice holds
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

constexpr int kVfThreads = 256, kVfWarps = kVfThreads / 32;
constexpr int kVfMaxCluster = 8;
constexpr int kVfStep = 128, kVfAhead = 4;    // entries of a warp's step (a float4 a lane); steps whose loads go out together
constexpr int kVfRound = kVfStep * kVfAhead;
constexpr int kVfMaxTokens = 64, kVfMaxVocab = 524288;
constexpr int kVfRounds = kVfMaxVocab / (kVfMaxCluster * kVfWarps * kVfRound);   // of a slice, at most
static_assert(kVfRounds <= 32, "a lane per round");
static_assert(kVfRound <= 512, "a round's sums fit 32 bits");

struct VerifyArgs {
    const float *p, *q;
    int64_t p_stream, p_row, q_stream, q_row;   // elements
    const int32_t *ids, *n_draft;
    const float *u;
    int T, V, per;                              // per: entries of a warp's slice
    int32_t *out, *accepted;
};

// floor(w 2^44) of w in [0, 1] as hi 2^23 + lo, lo < 2^23, both as the low bits of a float at 2^23
// (adding 2^23 towards zero leaves the whole part there; every other step is exact).  fp32
// adds, where a conversion to 64 bits runs at a small fraction of their rate.  fmaxf takes a NaN to 0.
constexpr float kVfWhole = 8388608.f;
constexpr uint32_t kVfWholeBits = 0x4b000000u;
struct Weight {
    uint32_t hi, lo;                            // with kVfWholeBits
    __device__ __forceinline__ unsigned long long value() const {
        return ((unsigned long long)(hi - kVfWholeBits) << 23) + (lo - kVfWholeBits);
    }
};
__device__ __forceinline__ Weight weight(float w) {
    const float x = __fmul_rn(fminf(fmaxf(w, 0.f), 1.f), 2097152.f);   // 2^21
    const float h = __fadd_rz(x, kVfWhole);
    const float rest = __fsub_rn(x, __fsub_rn(h, kVfWhole));
    return {__float_as_uint(h), __float_as_uint(__fadd_rz(__fmul_rn(rest, kVfWhole), kVfWhole))};
}

__device__ __forceinline__ unsigned long long warp_scan_u64(unsigned long long v, int lane) {   // inclusive
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long x = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += x;
    }
    return v;
}

// The row drawn from: p, p - q, or p without the drafted id.
struct Row {
    const float *p, *q;
    int hole;
    bool vec;
    __device__ __forceinline__ void set(const float *p_, const float *q_, int hole_) {
        p = p_, q = q_, hole = hole_;
        vec = ((reinterpret_cast<uintptr_t>(p) | reinterpret_cast<uintptr_t>(q)) & 15) == 0;
    }
    // entries [i, i + 4) below `end` of one of the two
    __device__ __forceinline__ float4 load4(const float *x, int i, int end) const {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (vec && i + 4 <= end) return __ldg(reinterpret_cast<const float4 *>(x + i));
        if (i < end) v.x = __ldg(x + i);
        if (i + 1 < end) v.y = __ldg(x + i + 1);
        if (i + 2 < end) v.z = __ldg(x + i + 2);
        if (i + 3 < end) v.w = __ldg(x + i + 3);
        return v;
    }
    // what is left of entries [i, i + 4) of kVfAhead steps, all loads first
    __device__ __forceinline__ void round(int i, int end, float (&v)[kVfAhead][4]) const {
        float4 x[kVfAhead], y[kVfAhead];
#pragma unroll
        for (int k = 0; k < kVfAhead; ++k) x[k] = load4(p, i + k * kVfStep, end);
        if (q) {
#pragma unroll
            for (int k = 0; k < kVfAhead; ++k) y[k] = load4(q, i + k * kVfStep, end);
        }
#pragma unroll
        for (int k = 0; k < kVfAhead; ++k) {
            v[k][0] = x[k].x, v[k][1] = x[k].y, v[k][2] = x[k].z, v[k][3] = x[k].w;
            if (q) {
                v[k][0] = __fsub_rn(v[k][0], y[k].x), v[k][1] = __fsub_rn(v[k][1], y[k].y);
                v[k][2] = __fsub_rn(v[k][2], y[k].z), v[k][3] = __fsub_rn(v[k][3], y[k].w);
            }
            const int at = hole - i - k * kVfStep;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (at == e) v[k][e] = 0.f;
        }
    }
};

// One stream per cluster of CL CTAs.
template <int CL> __global__ void __launch_bounds__(kVfThreads, 4) verify_kernel(const VerifyArgs a) {
    constexpr int kParts = CL * kVfWarps, kPer = (kParts + 31) / 32;   // slices; of them, a lane's
    __shared__ unsigned long long sums[kVfWarps], rounds[kVfWarps][kVfRounds];
    __shared__ unsigned long long all[kPer * 32];
    __shared__ int s_pass;
    const int b = blockIdx.x / CL, rank = blockIdx.x % CL;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int32_t *ids = a.ids + (int64_t)b * a.T;
    const float *u = a.u + (int64_t)b * (a.T + 1);
    int32_t *out = a.out + (int64_t)b * (a.T + 1);
    int n = a.n_draft ? __ldg(a.n_draft + b) : a.T;
    n = n < 0 ? 0 : n > a.T ? a.T : n;

    // the drafts that pass: a lane of warp 0 decides one (of up to 64)
    if (warp == 0) {
        int first = n;
        for (int t0 = 0; t0 < a.T; t0 += 32) {
            const int t = t0 + lane;
            bool ok = true;
            if (t < a.T) {
                const int x = __ldg(ids + t);
                ok = x >= 0 && x < a.V;
                if (ok) {
                    const float px = a.p[b * a.p_stream + t * a.p_row + x];
                    const float qx = a.q ? a.q[b * a.q_stream + t * a.q_row + x] : 1.f;
                    // 24-bit factors: the product is exact in fp64
                    ok = (double)u[t] * (double)qx < (double)px;
                }
            }
            const uint32_t bad = ~__ballot_sync(0xffffffffu, ok);
            if (bad) {
                first = min(n, t0 + __ffs(bad) - 1);
                break;
            }
        }
        if (lane == 0) s_pass = first;
    }
    if (threadIdx.x < kPer * 32) all[threadIdx.x] = 0;
    __syncthreads();
    const int pass = s_pass;
    if (rank == 0) {
        for (int s = threadIdx.x; s <= a.T; s += kVfThreads)
            if (s != pass) out[s] = s < pass ? ids[s] : -1;
        if (threadIdx.x == 0) a.accepted[b] = pass;
    }

    Row row;
    row.set(a.p + b * a.p_stream + pass * a.p_row, pass < n && a.q ? a.q + b * a.q_stream + pass * a.q_row : nullptr,
            pass < n && !a.q ? __ldg(ids + pass) : -1);
    const int me = rank * kVfWarps + warp;
    const int i0 = min(me * a.per, a.V), i1 = min(i0 + a.per, a.V);
    unsigned long long mine[kPer], upto = 0, total = 0;
    for (int turn = 0; turn < 2; ++turn) {
        unsigned long long s = 0;
        for (int i = i0; i < i1; i += kVfRound) {
            float v[kVfAhead][4];
            row.round(i + lane * 4, i1, v);
            // 512 entries: the whole parts stay below 2^30, the rest below 2^32
            uint32_t hi = 0, lo = 0;
#pragma unroll
            for (int k = 0; k < kVfAhead; ++k)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const Weight w = weight(v[k][e]);
                    hi += w.hi, lo += w.lo;
                }
            hi = __reduce_add_sync(0xffffffffu, hi - 4 * kVfAhead * kVfWholeBits);
            lo = __reduce_add_sync(0xffffffffu, lo - 4 * kVfAhead * kVfWholeBits);
            const unsigned long long r = ((unsigned long long)hi << 23) + lo;
            if (lane == 0) rounds[warp][(i - i0) / kVfRound] = r;
            s += r;
        }
        __syncwarp();
        if constexpr (CL == 1) {
            if (lane == 0) all[warp] = s;
            __syncthreads();
        } else {
            if (lane == 0) sums[warp] = s;
            cluster_sync();
            if (threadIdx.x < kParts) {
                const uint32_t at = cluster_map(&sums[threadIdx.x % kVfWarps], threadIdx.x / kVfWarps);
                unsigned long long v;
                asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(at) : "memory");
                all[threadIdx.x] = v;
            }
            cluster_sync();      // every CTA has read the sums: they may be written again, and CTAs may leave
        }
        // every warp scans the slices by itself
        unsigned long long lane_sum = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) lane_sum += mine[i] = all[lane * kPer + i];
        upto = warp_scan_u64(lane_sum, lane);
        total = __shfl_sync(0xffffffffu, upto, 31);
        upto -= lane_sum;
        if (total != 0 || (!row.q && row.hole < 0)) break;
        row.set(row.p, nullptr, -1);   // nothing left of p - q: the draw is from p
        if constexpr (CL == 1) __syncthreads();
    }

    if (total == 0) {
        if (rank == 0 && threadIdx.x == 0) out[pass] = -1;
        return;
    }
    unsigned long long mark = (unsigned long long)floor((double)u[a.T] * __ull2double_rn(total));
    if (mark >= total) mark = total - 1;   // u in [0, 1) gives less
    // the slice that holds the mark, and the sum before it
    int slice = 0;
    unsigned long long before = upto;
    bool here = false;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
        if (!here) {
            if (mark >= before && mark - before < mine[i])
                here = true, slice = lane * kPer + i;
            else
                before += mine[i];
        }
    const int src = __ffs(__ballot_sync(0xffffffffu, here)) - 1;
    if (__shfl_sync(0xffffffffu, slice, src) != me) return;
    before = __shfl_sync(0xffffffffu, before, src);

    // this warp finds the round of its slice, reads it again, and finds the step, the lane, the entry
    const int n_rounds = (i1 - i0 + kVfRound - 1) / kVfRound;
    const unsigned long long in_round = lane < n_rounds ? rounds[warp][lane] : 0;
    const unsigned long long ends = warp_scan_u64(in_round, lane);
    const int r = __ffs(__ballot_sync(0xffffffffu, lane < n_rounds && before + ends > mark)) - 1;
    before += __shfl_sync(0xffffffffu, ends - in_round, r);
    float v[kVfAhead][4];
    row.round(i0 + r * kVfRound + lane * 4, i1, v);
#pragma unroll
    for (int k = 0; k < kVfAhead; ++k) {
        unsigned long long w[4] = {weight(v[k][0]).value(), weight(v[k][1]).value(), weight(v[k][2]).value(),
                                   weight(v[k][3]).value()};
        const unsigned long long own = (w[0] + w[1]) + (w[2] + w[3]), scan = warp_scan_u64(own, lane);
        const uint32_t over = __ballot_sync(0xffffffffu, before + scan > mark);
        if (over) {
            if (lane == __ffs(over) - 1) {
                unsigned long long c = before + scan - own;
                int e = 0;
#pragma unroll
                for (int j = 0; j < 3; ++j)
                    if (e == j && c + w[j] <= mark) c += w[j], ++e;
                out[pass] = i0 + r * kVfRound + k * kVfStep + lane * 4 + e;
            }
            return;
        }
        before += __shfl_sync(0xffffffffu, scan, 31);
    }
}

template <int CL> cudaError_t launch_verify(VerifyArgs &a, int n_streams, cudaStream_t s) {
    constexpr int parts = CL * kVfWarps;
    a.per = ((a.V + parts - 1) / parts + kVfStep - 1) / kVfStep * kVfStep;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(n_streams * CL));
    cfg.blockDim = dim3(kVfThreads);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = CL;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = CL > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, verify_kernel<CL>, (const VerifyArgs)a);
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
    // a stream's CTAs read the ids, counts and numbers while others write the results
    struct Ints {
        const void *at;
        int64_t n;
    };
    const int64_t B = n_streams, T = n_tokens;
    const Ints out = {out_ids_dev, B * (T + 1)}, acc = {n_accepted_dev, B};
    const Ints in[3] = {{draft_ids_dev, B * T}, {u_dev, B * (T + 1)}, {n_draft_dev, n_draft_dev ? B : 0}};
    auto meet = [](const Ints &a, const Ints &b) {
        const int64_t d = bytes_between(a.at, b.at);
        return a.n && b.n && (d < 0 ? -d < 4 * b.n : d < 4 * a.n);
    };
    if (meet(out, acc)) return QD_EINVAL;
    for (const Ints &x : in)
        if (meet(out, x) || meet(acc, x)) return QD_EINVAL;
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
    // CTAs of a stream: a warp's slice at most a round, as far as a cluster goes
    cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
    constexpr int kCta = kVfWarps * kVfRound;
    const cudaError_t e = vocab <= kCta       ? launch_verify<1>(a, n_streams, s)
                          : vocab <= 2 * kCta ? launch_verify<2>(a, n_streams, s)
                          : vocab <= 4 * kCta ? launch_verify<4>(a, n_streams, s)
                                              : launch_verify<kVfMaxCluster>(a, n_streams, s);
    return e == cudaSuccess ? QD_OK : QD_ECUDA;
}
