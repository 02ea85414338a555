// Causal attention over whole prompts of different lengths that stand packed one after the other (bf16), on the tcgen05
// tensor cores.
//
//   out[i] = sum_{j < lim_i} 2^(s_ij - ref) v_j / sum_{j < lim_i} 2^(s_ij - ref),   s_ij = log2(e) scale q_i . k_j,   lim_i = past + i + 1
//
// The rows of a sequence and key head are its (token, query head of the group) pairs, token by token, so a group's heads share
// every key that is read, and short prompts of grouped heads still fill tiles.  A tile has the rows of 128 / G whole tokens (the M
// of an MMA, a few rows unused where G does not divide 128), a CTA works a pair of them against the same chunks of 128 keys, one tile's
// products under the other's softmax:
//   S = Q K^T          128 x 128 fp32 in tensor memory; Q and K from shared memory, by TMA
//   softmax            thread = row; P as bf16 over S's own columns, 64 keys' in the first half of theirs
//   O += P V           P from tensor memory, V from shared memory (keys x dims: the MN-major operand)
// The reference comes from a row's first 32 scores and moves only when the sum of 128 weights passes 2^40 (bf16 weights have
// fp32's range; 2^40 leaves V as much as 2^87), so the scores are read once and O stays where it is.
//
// P is one bf16 part (a weight keeps 8 bits): a second part takes half as many products again, and its rounding, unbiased and
// independent from key to key, adds to that of a bf16 result about as much again (2-norm against 64 bits: 1.8e-3 to 2.3e-3, the result's own
// rounding 1.6e-3).  The sum is that of the weights before their rounding, in fp32.
//
// What a row does not see never reaches it: hidden scores are replaced, not added to, and a V row that is not finite among
// the chunks that some rows see only in part is zeroed in shared memory and added by the rows that see it (0 x infinity is
// NaN).  Two warps look those chunks through while their scores are worked out.
//
// Pairs differ in length, and only the device knows the lengths.  Few pairs (OwnPlan) every CTA ranks for itself, longest first, and takes those of
// its place in each round, there and back; or, where few pairs are long, all CTAs take equal runs of chunks, the pieces of a pair going
// through memory to attn_prompt_join_kernel.  Many are sorted by attn_prompt_plan_kernel, and the CTAs take them from a counter.
//
// Measured: one prompt of 8192 under 32 heads, 550 GFLOP, 346 us (1590 TFLOP/s, 0.83 of the measured peak): a pair of tiles takes about 2650 clocks
// a chunk where its products take 2048, because a tile's softmax (1150: 128 exponentials a thread are 512 at the unit's rate, the rest
// issue slots, the way from and to tensor memory and the vote) and its two products (1024, and 400 until they have begun and been
// noticed) follow one another, and S and O of two tiles fill the tensor memory of head_dim 128.  Not better: two warps a tile's rows, 64 keys each, which
// have to agree on the reference (357 us; short prompts 1 to 2 % faster); the product of the first 64 keys begun while the others are
// weighed (397); for heads of 64, P in columns of its own, so that the next S need not wait for P's product (288 us where this form
// takes 266: both tiles' softmaxes then meet on the same units).  8 x 512 tokens, 16 of 8 heads, 50 MB, 20.8 us: the start (plan 1.2 us, first
// loads 1.2), 4 chunks a CTA, the results' way out (4 us).
//
// Roles (384 threads): warps 0-3 and 4-7 the softmax of the two tiles, warp 8 owns the tensor memory and issues the MMAs, warp 9 takes the
// pairs and loads, warps 10 and 11 look V through.  Registers a thread: 168 at launch, then 208 and 88.  Every wait is bounded; where one
// expires the pair's results become NaN and the roles run to their ends.
#include <cuda.h>

#include <algorithm>
#include <atomic>

#include "attn_cached.cuh"
#include "qd_internal.h"
#include "tc_common.cuh"

namespace qd {

namespace {

constexpr int kPtThreads = 384, kPtSoft = 256;
constexpr int kPtRegsSoft = 208, kPtRegsRest = 88;
static_assert(kPtSoft * kPtRegsSoft + (kPtThreads - kPtSoft) * kPtRegsRest <= kPtThreads * 168, "registers");
constexpr uint32_t kPtBox = 128 * 128;        // 128 rows of 128 bytes, 128-byte swizzle
constexpr uint32_t kPtS = 0, kPtO = 256;      // tensor memory columns: S of the tiles (P of 64 keys over the first half of theirs), O
constexpr int kPtKeys = 128;                  // of a chunk
constexpr int kPtSlots = 4;                   // pairs in flight between the roles
constexpr int kPtUsers = 11;                  // warps that read a slot
constexpr int kPtBuckets = 1024;              // of the plan's sort
constexpr float kPtTop = 1.0995116e12f;       // 2^40

struct PromptArgs {
    const uint8_t *v;
    uint8_t *out;
    int64_t v_token, o_token;                 // bytes
    const int32_t *offsets, *kv_offsets;      // kv_offsets: may be offsets
    int N, M, B, G, kvh;                      // tokens, keys
    int tpt;                                  // tokens of a tile
    bool wide_out;                            // out's rows stand at multiples of 32 bytes
    float scale2;                             // softmax scale times log2(e)
    // the list of pairs, longest first, room for `cap`; [0] their number, [1] those taken beyond the first of each CTA.  null: every CTA
    // finds its own
    int4 *list;
    int *count;
    int cap, cost_shift;
    // room for pieces of pairs, two a CTA; null: pairs stay whole
    struct Join *join;
    float2 *p_ml;                             // [piece][256] reference, sum
    float *p_o;                               // [piece][256][D]
};

// A pair whose chunks several CTAs have worked: pieces 2 first + second of the first CTA's, then 2 w of the `more` that follow.  more 0: none.
struct Join {
    int q0, tokens, hk, lim0;
    int first, second, more, pad;
};

// A pair of tiles, as the roles see it.
struct __align__(16) Pair {
    int q0, tokens;                           // first token row, tokens (of both tiles)
    int k0, lim0;                             // first key row; keys that the first token sees
    int n0, n1;                               // chunks of either tile
    int hk;                                   // key head, and above it (1 + the piece's place) << 20 for a piece; below 0: no more pairs
    uint32_t odd;                             // chunks, counted from first_edge(), in which V was not finite
    __device__ __forceinline__ int head() const { return hk & 0xfffff; }
    __device__ __forceinline__ int piece() const { return (hk >> 20) - 1; }
    __device__ __forceinline__ int n(int h) const { return h ? n1 : n0; }
    __device__ __forceinline__ int most() const { return max(n0, n1); }
    __device__ __forceinline__ int work() const { return max(1, most()); }   // a pair that sees nothing is written all the same
};
// The first chunk that the pair's first token does not see all of.
__device__ __forceinline__ int first_edge(const Pair &p) { return p.lim0 > 0 ? p.lim0 / kPtKeys : 0; }

struct __align__(16) Sequence {
    int q0, n, k0, m;
};
__device__ __forceinline__ Sequence sequence(const PromptArgs &a, int b) {
    Sequence s;
    s.q0 = min(max(a.offsets[b], 0), a.N);
    s.n = min(max(a.offsets[b + 1], s.q0), a.N) - s.q0;
    s.k0 = min(max(a.kv_offsets[b], 0), a.M);
    s.m = min(max(a.kv_offsets[b + 1], s.k0), a.M) - s.k0;
    return s;
}
__device__ __forceinline__ int chunks(int keys) { return keys > 0 ? (keys + kPtKeys - 1) / kPtKeys : 0; }

__device__ __forceinline__ Pair pair_of(const PromptArgs &a, const Sequence &s, int pair, int hk) {
    const int t0 = pair * 2 * a.tpt;
    Pair p;
    p.hk = hk;
    p.q0 = s.q0 + t0, p.tokens = min(s.n - t0, 2 * a.tpt);
    p.k0 = s.k0, p.lim0 = s.m - s.n + t0 + 1;
    const int first = min(p.tokens, a.tpt);
    p.n0 = chunks(p.lim0 + first - 1);
    p.n1 = p.tokens > first ? chunks(p.lim0 + p.tokens - 1) : 0;
    p.odd = 0;
    return p;
}
__device__ __forceinline__ int pairs_of(const PromptArgs &a, const Sequence &s) { return (s.n + 2 * a.tpt - 1) / (2 * a.tpt); }

// ---- the plan: one CTA, a counting sort of the pairs by their chunks, longest first
__global__ void __launch_bounds__(1024) attn_prompt_plan_kernel(const PromptArgs a) {
    __shared__ int hist[kPtBuckets], sums[32];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    hist[tid] = 0;
    pdl_wait();
    pdl_launch_dependents();
    __syncthreads();
    // as many threads a sequence as there are, a warp at least
    int per = 1024;
    while (per > 32 && a.B * per > 1024) per >>= 1;
    auto walk = [&](auto &&take) {
        for (int b = tid / per; b < a.B; b += 1024 / per) {
            const Sequence s = sequence(a, b);
            const int pairs = pairs_of(a, s);
            for (int i = tid % per; i < pairs; i += per) {
                const int last = min(s.n, (i + 1) * 2 * a.tpt);            // tokens up to the pair's end
                take(s, i, min(chunks(s.m - s.n + last) >> a.cost_shift, kPtBuckets - 1));
            }
        }
    };
    walk([&](const Sequence &, int, int cost) { atomicAdd(&hist[kPtBuckets - 1 - cost], 1); });
    __syncthreads();
    // where each bucket begins
    const int mine = hist[tid];
    int upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
    }
    if (lane == 31) sums[warp] = upto;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < 32; ++w) {
        if (w < warp) before += sums[w];
        all += sums[w];
    }
    hist[tid] = before + upto - mine;
    __syncthreads();
    walk([&](const Sequence &s, int i, int cost) {
        const int at = atomicAdd(&hist[kPtBuckets - 1 - cost], 1);
        if (at >= a.cap) return;                                           // (offsets that do not ascend could name more)
        const Pair p = pair_of(a, s, i, 0);
        a.list[2 * at] = make_int4(p.q0, p.tokens, p.k0, p.lim0);
        a.list[2 * at + 1] = make_int4(p.n0, p.n1, 0, 0);
    });
    if (tid == 0) a.count[0] = min(all, a.cap), a.count[1] = 0;
}

// ---- or, for few pairs, every CTA by itself: the pairs of all sequences ranked by their chunks (equal ones in order, the same in every CTA),
// (pair, key head) dealt out there and back.  The CTA's pairs to mine[0 ..], their number to *n.
constexpr int kPtOwnPairs = 256, kPtOwnRounds = 16, kPtMaxCtas = 512;
// Pairs are cut into pieces, equal runs of chunks for all CTAs, where that takes as many chunks off the one that has most (3 x 700 to 1000 queries
// over up to 6000 keys, 12 of 4 heads: 47 chunks in 104 CTAs, 31 in all; the pieces' way through memory and the joining kernel
// take about 8 us, a chunk 1.4).
constexpr int kPtWorthCutting = 8;
constexpr int kPtMinRun = 4;
struct OwnPlan {
    int cost[kPtOwnPairs];                    // read 16 at a time
    int first[kPtOwnPairs + 1];               // of every sequence
    int pad[3];
    Pair mine[kPtOwnRounds];
    int n;
    int most;                                 // chunks of the CTA that has most, were the pairs dealt out whole
    int load[kPtMaxCtas];
    int sums[8];
    // where the pairs are cut: all of them, the chunks of one key head before each, and this CTA's run
    union {
        Pair pairs[kPtOwnPairs];
        Sequence seqs[kPtOwnPairs];           // until then
    };
    int before[kPtOwnPairs + 1];
    int total, x0, x1;
    unsigned run, more;                       // of the Share
    bool cut;
};
__device__ __forceinline__ int rank_of(const PromptArgs &a, const OwnPlan &w, const Pair &p, int total) {
    const int tid = threadIdx.x;
    if (total * a.kvh <= (int)gridDim.x) return tid;
    int rank = 0;
    const int own = p.most();
    const int4 *cost = reinterpret_cast<const int4 *>(w.cost);
#pragma unroll 4
    for (int j = 0; j < total; j += 4) {      // (what stands past `total` is below every cost)
        const int4 c = cost[j / 4];
        rank += (c.x > own || (c.x == own && j < tid)) + (c.y > own || (c.y == own && j + 1 < tid)) +
                (c.z > own || (c.z == own && j + 2 < tid)) + (c.w > own || (c.w == own && j + 3 < tid));
    }
    return rank;
}
// Every thread of the CTA: whether the pairs are cut, and then this CTA's pieces.  p: pair threadIdx.x, with key head 0.
__device__ __noinline__ bool cut_pairs(const PromptArgs &a, OwnPlan &w, const Pair &p, int total) {
    const int tid = threadIdx.x, lane = tid & 31, grid = (int)gridDim.x, own = tid < total ? p.work() : 0;
    if (tid < total) {
        const int rank = rank_of(a, w, p, total);
        int round = rank * a.kvh / grid, at = rank * a.kvh - round * grid;
        for (int hk = 0; hk < a.kvh; ++hk) {
            atomicAdd(&w.load[round & 1 ? grid - 1 - at : at], own);
            if (++at == grid) at = 0, ++round;
        }
    }
    // chunks before this pair, of one key head
    int upto = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
    }
    if (lane == 31 && tid < kPtOwnPairs) w.sums[tid / 32] = upto;
    __syncthreads();
    int before = upto - own, all = 0;
#pragma unroll
    for (int i = 0; i < kPtOwnPairs / 32; ++i) {
        if (i < tid / 32) before += w.sums[i];
        all += w.sums[i];
    }
    int most = 0;
    for (int i = tid; i < grid; i += kPtThreads) most = max(most, w.load[i]);
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 0) atomicMax(&w.most, most);
    __syncthreads();
    const unsigned work = (unsigned)all * (unsigned)a.kvh;
    Share sh;
    const int ctas = (int)min((unsigned)grid, max(1u, work / kPtMinRun));
    sh.use(work, (unsigned)ctas);
    const bool cut = w.most >= (int)sh.run + kPtWorthCutting;
    Join *join = a.join + 2 * blockIdx.x;
    if (tid < 2) join[tid].more = 0;
    if (!cut) return false;
    if (tid < kPtOwnPairs) w.pairs[tid] = p, w.before[tid] = before;
    if (tid == 0) {
        w.before[kPtOwnPairs] = all, w.total = total, w.cut = true, w.run = sh.run, w.more = sh.more;
        w.x0 = (int)blockIdx.x < ctas ? (int)sh.first(blockIdx.x) : 0;
        w.x1 = (int)blockIdx.x < ctas ? (int)sh.first(blockIdx.x + 1) : 0;
    }
    return true;
}
// The piece that begins at chunk x of the list (pair after pair, head after head); x moves on to the next.
__device__ __forceinline__ Pair piece_at(const PromptArgs &a, const OwnPlan &w, int &x) {
    Pair q = {};
    q.hk = -1;
    if (x >= w.x1) return q;
    int lo = 0, hi = kPtOwnPairs;             // before[lo] kvh <= x < before[hi] kvh
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (w.before[mid] * a.kvh <= x)
            lo = mid;
        else
            hi = mid;
    }
    const Pair p = w.pairs[lo];
    const int own = p.work(), y = x - w.before[lo] * a.kvh, hk = y / own, c0 = y - hk * own, c1 = min(own, c0 + w.x1 - x);
    // a piece's place among the two that a CTA can have: its run begins with it, or ends
    const int place = x == w.x0 ? 0 : 1;
    q = p;
    q.hk = hk;
    if (c0 > 0 || c1 < own) q.hk |= (1 + 2 * (int)blockIdx.x + place) << 20;
    q.k0 += c0 * kPtKeys, q.lim0 -= c0 * kPtKeys;
    q.n0 = max(0, min(p.n0, c1) - c0), q.n1 = max(0, min(p.n1, c1) - c0);
    if (c0 == 0 && c1 < own && (threadIdx.x & 31) == 0) {
        Share sh;
        sh.run = w.run, sh.more = w.more;
        a.join[2 * blockIdx.x + place] = {p.q0, p.tokens, hk, p.lim0, (int)blockIdx.x, place,
                                          (int)sh.owner((unsigned)(x + own) - 1u) - (int)blockIdx.x, 0};
    }
    x += c1 - c0;
    return q;
}
// Pair p's key heads, the pair's rank given, to the CTAs there and back: this CTA's to w.mine.
__device__ __forceinline__ void deal(const PromptArgs &a, OwnPlan &w, Pair p, int rank) {
    const int grid = (int)gridDim.x;
    // this CTA's place in the rounds that the pair's key heads fall into
    const int j0 = rank * a.kvh, j1 = j0 + a.kvh;
    for (int round = j0 / grid; round * grid < j1 && round < kPtOwnRounds; ++round) {
        const int j = round * grid + (round & 1 ? grid - 1 - (int)blockIdx.x : (int)blockIdx.x);
        if (j < j0 || j >= j1) continue;
        p.hk = j - j0;
        w.mine[round] = p;
        atomicMax(&w.n, round + 1);           // (no round is left out before the last)
    }
}
__device__ __forceinline__ void plan_own(const PromptArgs &a, OwnPlan &w) {
    const int tid = threadIdx.x, lane = tid & 31;
    if (a.B == 1 && !a.join) {                // one prompt: the later a pair, the longer
        const Sequence s = sequence(a, 0);
        if (tid == 0) w.n = 0, w.cut = false;
        __syncthreads();
        const int total = min(pairs_of(a, s), kPtOwnPairs);
        if (tid < total) deal(a, w, pair_of(a, s, tid, 0), total - 1 - tid);
        return;
    }
    Sequence s;
    if (tid < a.B) {
        s = sequence(a, tid);
        w.first[tid + 1] = pairs_of(a, s);
        w.seqs[tid] = s;
    }
    if (tid == 0) w.n = 0, w.most = 0, w.cut = false;
    if (tid < kPtOwnPairs) w.cost[tid] = -1;
    for (int i = tid; a.join && i < kPtMaxCtas; i += kPtThreads) w.load[i] = 0;
    __syncthreads();
    if (tid < 32) {                           // running sums, 8 sequences a lane
        int v[kPtOwnPairs / 32], sum = 0;
#pragma unroll
        for (int i = 0; i < kPtOwnPairs / 32; ++i) {
            const int b = lane * (kPtOwnPairs / 32) + i;
            v[i] = sum += b < a.B ? w.first[b + 1] : 0;
        }
        int upto = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += x;
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < kPtOwnPairs / 32; ++i) {
            const int b = lane * (kPtOwnPairs / 32) + i;
            if (b < a.B) w.first[b + 1] = upto - sum + v[i];
        }
        if (lane == 0) w.first[0] = 0;
    }
    __syncthreads();
    const int total = min(w.first[a.B], kPtOwnPairs);   // (offsets that do not ascend could name more)
    Pair p = {};
    if (tid < total) {
        int lo = 0, hi = a.B;                 // first[lo] <= tid < first[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (w.first[mid] <= tid)
                lo = mid;
            else
                hi = mid;
        }
        p = pair_of(a, w.seqs[lo], tid - w.first[lo], 0);
        w.cost[tid] = p.most();
    }
    __syncthreads();
    if (a.join && cut_pairs(a, w, p, total)) return;
    if (tid >= total) return;
    deal(a, w, p, rank_of(a, w, p, total));
}

template <int D> struct PtCfg {
    static constexpr int KB = D / 64;                         // 64-wide blocks of head_dim
    static constexpr int kStages = 4 / KB;                    // of K and of V
    static constexpr uint32_t kTile = KB * kPtBox;            // of Q, K or V
    static constexpr uint32_t kQ = 0;                         // Q [tile]
    static constexpr uint32_t kK = kQ + 2 * kTile;            // K [stage]
    static constexpr uint32_t kV = kK + kStages * kTile;    // V [stage]
    static constexpr uint32_t kSlot = kV + kStages * kTile;
    static constexpr uint32_t kOwn = kSlot + kPtSlots * sizeof(Pair);
    static constexpr uint32_t kBar = kOwn + (sizeof(OwnPlan) + 15) / 16 * 16;
    static constexpr uint32_t kBars = 46;
    static constexpr uint32_t kSmem = 1024 + kBar + kBars * 8;
};
static_assert(sizeof(Pair) == 32, "two loads of 16 bytes");

// 32 scores of a row as weights against its reference, packed; their sums join la and lb.  (Single products and packed sums: 64 scores take one
// warp of a scheduler 349 clocks, two of them 566, near the exponentials' 8 a clock; packed products 328 and 556.)
__device__ __forceinline__ void weigh(const uint32_t *x, float cs, float rf, uint32_t *y, uint64_t &la, uint64_t &lb) {
#pragma unroll
    for (int e = 0; e < 32; e += 4) {
        float s[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] = ex2(fmaf(__uint_as_float(x[e + i]), cs, rf));
        la = add2(la, pk(s[0], s[1])), lb = add2(lb, pk(s[2], s[3]));
        y[e / 2] = pack_bf16(s[0], s[1]), y[e / 2 + 1] = pack_bf16(s[2], s[3]);
    }
}
// Scores past the first `left` of 32 become `none`, whose weight is zero whatever stood there.
__device__ __forceinline__ void hide(uint32_t *x, int left, uint32_t none) {
#pragma unroll
    for (int e = 0; e < 32; ++e) x[e] = e < left ? x[e] : none;
}
// The largest of N scores, in log2 units.
template <int N> __device__ __forceinline__ float largest(const uint32_t *x, float cs) {
    float m = -INFINITY;
#pragma unroll
    for (int e = 0; e < N; ++e) m = fmaxf(m, __uint_as_float(x[e]) * cs);
    return m;
}
__device__ __forceinline__ bool not_finite(uint32_t w) { return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u; }
// Two bf16: acc + 0 x w, NaN from the first that is not finite on.
__device__ __forceinline__ uint32_t add_none(uint32_t w, uint32_t acc) {
    uint32_t d;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(w), "r"(0u), "r"(acc));
    return d;
}

// 32 bytes at a multiple of 32.
__device__ __forceinline__ void st32(void *to, const uint32_t *v) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]),
                 "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

template <int D>
__global__ void __launch_bounds__(kPtThreads, 1)
    attn_prompt_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                       const __grid_constant__ CUtensorMap mv, const PromptArgs a) {
    using C = PtCfg<D>;
    constexpr int KB = C::KB;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    Pair *slots = reinterpret_cast<Pair *>(sm + C::kSlot);
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + C::kBar);
    uint64_t *slot_full = bars, *slot_empty = bars + 4;                                              // [slot]
    uint64_t *q_full = bars + 8, *q_empty = bars + 10, *s_full = bars + 12, *p_full = bars + 14;     // [tile]
    uint64_t *o_full = bars + 16, *o_empty = bars + 18;                                              // [tile]
    uint64_t *k_full = bars + 22, *k_empty = bars + 26, *v_full = bars + 30, *v_empty = bars + 34, *v_clean = bars + 38;   // [stage]
    uint64_t *drain = bars + 42;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 43);
    volatile int *bad = reinterpret_cast<volatile int *>(bars + 44);

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kPtSlots; ++i) mbar_init(&slot_full[i], 1), mbar_init(&slot_empty[i], kPtUsers);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&q_full[i], 1), mbar_init(&q_empty[i], 1), mbar_init(&s_full[i], 1), mbar_init(&p_full[i], 4);
            mbar_init(&o_full[i], 1), mbar_init(&o_empty[i], 4);
        }
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(&k_full[i], 1), mbar_init(&k_empty[i], 1);
            mbar_init(&v_full[i], 1), mbar_init(&v_empty[i], 1), mbar_init(&v_clean[i], 2);
        }
        mbar_init(drain, 1);
        *bad = 0;
        fence_barrier_init();
    }
    if (warp == 9 && lane < 3) {
        const CUtensorMap *m = lane == 0 ? &mq : lane == 1 ? &mk : &mv;
        asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
    }
    // the predecessor first, the tensor memory then: held while waiting it could be what a predecessor's CTA on this SM waits for
    pdl_wait();
    if (warp == 8) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    pdl_launch_dependents();                  // the whole grid is resident, so what follows may be placed as SMs fall free
    OwnPlan &own = *reinterpret_cast<OwnPlan *>(sm + C::kOwn);
    if (!a.list) plan_own(a, own);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    auto slot_of = [&](int i) -> Pair & { return slots[i % kPtSlots]; };
    // the i-th pair of this CTA, or none (hk < 0)
    auto pair_at = [&](int i) {
        Pair p;
        p.hk = -1;
        // (a wait may expire for some lanes alone: all of a warp leave together, here and below)
        if (__all_sync(0xffffffffu, wt_wait(&slot_full[i % kPtSlots], (uint32_t)(i / kPtSlots) & 1u, bad))) p = slot_of(i);
        return p;
    };
    auto done_with = [&](int i) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&slot_empty[i % kPtSlots]);
    };

    if (warp == 9) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kPtRegsRest));
        // ---- the pairs, and their loads (the whole warp walks along; one lane issues)
        int kc = 0, nq[2] = {0, 0}, next = (int)blockIdx.x;
        const int total = a.list ? a.count[0] * a.kvh : min(own.n, kPtOwnRounds);
        int x = own.x0;                             // where the pairs are cut: the next chunk
        bool ok = true;
        // pair `i` of the list, or of this CTA's own
        auto pair_no = [&](int i) {
            Pair p = {};
            p.hk = -1;
            if (i >= total && (a.list || !own.cut)) return p;
            if (!a.list) return own.cut ? piece_at(a, own, x) : own.mine[i];
            const int4 u = a.list[2 * (i / a.kvh)], v = a.list[2 * (i / a.kvh) + 1];
            p.q0 = u.x, p.tokens = u.y, p.k0 = u.z, p.lim0 = u.w, p.n0 = v.x, p.n1 = v.y;
            p.hk = i % a.kvh;
            return p;
        };
        Pair p = pair_no(a.list ? next : 0);
        for (int it = 0; ok; ++it) {
            if (it >= kPtSlots) ok = wt_wait(&slot_empty[it % kPtSlots], (uint32_t)(it / kPtSlots + 1) & 1u, bad);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            if (lane == 0) {
                slot_of(it) = p;
                mbar_arrive(&slot_full[it % kPtSlots]);
            }
            __syncwarp();
            if (p.hk < 0) break;
            if (a.list && lane == 0) next = (int)gridDim.x + atomicAdd(&a.count[1], 1);     // in flight under this pair's loads
            const int n = p.most();
            for (int c = 0; ok && c < n; ++c, ++kc) {
                const int st = kc % C::kStages;
                const uint32_t was = (uint32_t)(kc / C::kStages + 1) & 1u;
                const int key = p.k0 + c * kPtKeys;
                auto load = [&](const CUtensorMap *m, uint32_t at, uint64_t *full, uint32_t bytes, int head, int row) {
                    if (elect_one()) {
                        mbar_arrive_expect_tx(full, bytes);
#pragma unroll
                        for (int b = 0; b < KB; ++b) tma_load_3d_plain(sm + at + b * kPtBox, m, 64 * b, head, row, full);
                    }
                    __syncwarp();
                };
                auto load_q = [&](int h) {
                    if (p.n(h) == 0) return;
                    if (nq[h] > 0) ok = ok && wt_wait(&q_empty[h], (uint32_t)(nq[h] + 1) & 1u, bad);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) return;
                    load(&mq, C::kQ + h * C::kTile, &q_full[h], (uint32_t)(KB * a.tpt * a.G * 128), p.head() * a.G, p.q0 + h * a.tpt);
                    ++nq[h];
                };
                if (c == 0) load_q(p.n0 ? 0 : 1);
                if (kc >= C::kStages) ok = ok && wt_wait(&k_empty[st], was, bad);
                ok = __all_sync(0xffffffffu, ok);
                if (ok) load(&mk, C::kK + st * C::kTile, &k_full[st], C::kTile, p.head(), key);
                if (c == 0 && p.n0) load_q(1);
                if (kc >= C::kStages) ok = ok && wt_wait(&v_empty[st], was, bad);
                ok = __all_sync(0xffffffffu, ok);
                if (ok) load(&mv, C::kV + st * C::kTile, &v_full[st], C::kTile, p.head(), key);
            }
            next = __shfl_sync(0xffffffffu, next, 0);
            if (ok) p = pair_no(a.list ? next : it + 1);
        }
        // copies in flight land before the CTA may end (they have, unless a wait expired)
        if (!ok) {
            for (int h = 0; h < 2; ++h)
                if (nq[h] > 0) (void)mbar_wait_bounded(&q_full[h], (uint32_t)(nq[h] + 1) & 1u, 20000000ull);
            for (int i = 0; i < C::kStages; ++i) {
                const int uses = kc / C::kStages + 1;
                (void)mbar_wait_bounded(&k_full[i], (uint32_t)(uses + 1) & 1u, 20000000ull);
                (void)mbar_wait_bounded(&v_full[i], (uint32_t)(uses + 1) & 1u, 20000000ull);
            }
        }
    } else if (warp == 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kPtRegsRest));
        // ---- the MMAs: always a tile's O followed by its next S, which may be the next pair's first
        constexpr uint32_t base = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(128 >> 4) << 24);
        constexpr uint32_t idesc_s = base | ((uint32_t)(kPtKeys >> 3) << 17);
        constexpr uint32_t idesc_o = base | (1u << 16) | ((uint32_t)(D >> 3) << 17);
        const uint64_t dQ = sw128_desc(smem_addr(sm + C::kQ)), dK = sw128_desc(smem_addr(sm + C::kK));
        const uint64_t dV = sw128_desc_mn(smem_addr(sm + C::kV), kPtBox, 1024u);
        constexpr uint32_t kBox16 = kPtBox / 16;
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        int kc = 0;                                 // chunks before this pair's
        uint32_t nq[2] = {0, 0}, np[2] = {0, 0}, no[2] = {0, 0};   // of either tile: pairs, P's, pairs begun in O
        bool ok = true, begun[2] = {false, false};  // the pair's first S is issued
        Pair p = pair_at(0);
        // S of tile h, chunk c of pair x whose first chunk is the kx-th; `other`: the other tile's S of that chunk is issued, or none is wanted
        auto issue_s = [&](int h, int c, const Pair &x, int kx, bool other) {
            const int st = (kx + c) % C::kStages;
            if (c == 0) ok = ok && wt_wait(&q_full[h], nq[h]++ & 1u, bad);
            ok = ok && wt_wait(&k_full[st], (uint32_t)((kx + c) / C::kStages) & 1u, bad);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) return;
            tc_fence_after();
            const uint32_t d = tm + kPtS + 128u * h;
            const uint64_t q = dQ + h * KB * kBox16, k = dK + st * KB * kBox16;
            if (elect_one()) {
#pragma unroll
                for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                    for (int s = 0; s < 4; ++s)
                        tc_mma(d, q + kb * kBox16 + 2 * s, k + kb * kBox16 + 2 * s, idesc_s, (kb | s) ? 1u : 0u);
                tc_commit(&s_full[h]);
                if (other) tc_commit(&k_empty[st]);
                if (c + 1 == x.n(h)) tc_commit(&q_empty[h]);
            }
            __syncwarp();
        };
        auto issue_o = [&](int h, int c) {
            const int st = (kc + c) % C::kStages;
            const uint32_t ph = (uint32_t)((kc + c) / C::kStages) & 1u;
            if (c == 0) {
                if (no[h] > 0) ok = ok && wt_wait(&o_empty[h], (no[h] + 1) & 1u, bad);
                ++no[h];
            }
            const uint32_t d = tm + kPtO + 128u * h, pt = tm + kPtS + 128u * h;
            const uint64_t v = dV + st * KB * kBox16;
            ok = ok && wt_wait(&v_full[st], ph, bad) && wt_wait(&v_clean[st], ph, bad);
            ok = ok && wt_wait(&p_full[h], np[h] & 1u, bad);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) return;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int i = 0; i < kPtKeys / 16; ++i) tc_mma_ts(d, pt + 8u * i + 32u * (i >> 2), v + i * 128, idesc_o, (c | i) ? 1u : 0u);
                if (h == 1 || p.n1 <= c) tc_commit(&v_empty[st]);
                if (c + 1 == p.n(h)) tc_commit(&o_full[h]);
            }
            __syncwarp();
            ++np[h];
        };
        for (int it = 0; ok && p.hk >= 0; ++it) {
            const int n = p.most();
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if (ok && !begun[h] && p.n(h) > 0) {
                    issue_s(h, 0, p, kc, begun[1 - h] || p.n(1 - h) == 0);
                    begun[h] = true;
                }
            begun[0] = begun[1] = false;
            Pair x;
            x.hk = -2;                              // the next pair: not known yet
            for (int c = 0; ok && c < n; ++c)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (!ok || c >= p.n(h)) continue;
                    issue_o(h, c);
                    if (!ok) continue;
                    if (c + 1 < p.n(h)) {
                        issue_s(h, c + 1, p, kc, h == 1 || p.n1 <= c + 1);
                    } else {
                        if (x.hk == -2) x = pair_at(it + 1);
                        if (x.hk >= 0 && x.n(h) > 0) {
                            // (the second tile's may come first: where this pair had no first)
                            issue_s(h, 0, x, kc + n, begun[1 - h] || x.n(1 - h) == 0);
                            begun[h] = true;
                        }
                    }
                }
            if (x.hk == -2) x = pair_at(it + 1);
            done_with(it);
            kc += n;
            p = x;
        }
        // every MMA issued has completed before the tensor memory can be freed
        if (elect_one()) tc_commit(drain);
        (void)mbar_wait_bounded(drain, 0u, 20000000ull);
        __syncwarp();
    } else if (warp >= 10) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kPtRegsRest));
        // ---- V of chunks that some rows see in part: what is not finite becomes zero, and is noted
        int kc = 0;
        bool ok = true;
        for (int it = 0; ok; ++it) {
            Pair p = pair_at(it);
            if (p.hk < 0) break;
            const int n = p.most(), edge = first_edge(p);
            for (int c = 0; ok && c < n; ++c, ++kc) {
                const int st = kc % C::kStages;
                ok = wt_wait(&v_full[st], (uint32_t)(kc / C::kStages) & 1u, bad);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                if (c >= edge) {
                    uint4 *tile = reinterpret_cast<uint4 *>(sm + C::kV + st * C::kTile) + (warp - 10) * 32 + lane;
                    constexpr int kPieces = KB * 128 * 8;
                    uint32_t acc[4] = {0, 0, 0, 0};
#pragma unroll 8
                    for (int i = 0; i < kPieces; i += 64) {
                        const uint4 u = tile[i];
                        acc[0] = add_none(u.x, acc[0]), acc[1] = add_none(u.y, acc[1]);
                        acc[2] = add_none(u.z, acc[2]), acc[3] = add_none(u.w, acc[3]);
                    }
                    if (not_finite(acc[0]) || not_finite(acc[1]) || not_finite(acc[2]) || not_finite(acc[3])) {
                        for (int i = 0; i < kPieces; i += 64) {
                            auto keep = [](uint32_t w) {
                                if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
                                if ((w & 0x7f800000u) == 0x7f800000u) w &= 0xffffu;
                                return w;
                            };
                            const uint4 u = tile[i];
                            tile[i] = make_uint4(keep(u.x), keep(u.y), keep(u.z), keep(u.w));
                        }
                        fence_proxy_async_smem();
                        atomicOr(&slot_of(it).odd, 1u << (c - edge));
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&v_clean[st]);
            }
            done_with(it);
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kPtRegsSoft));
        // ---- softmax: tile h, row r of it
        const int h = warp >> 2, quarter = warp & 3, r = quarter * 32 + lane;
        const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
        const uint32_t tS = tmem + kPtS + 128u * h + lanes, tO = tmem + kPtO + 128u * h + lanes;
        const int token = r / a.G, head = r - token * a.G;
        const bool in_tile = token < a.tpt;
        const uint32_t none = a.scale2 < 0.f ? 0x7f800000u : 0xff800000u;       // -infinity once it is scaled
        uint32_t ns = 0, no = 0;                    // S's, O's so far
        bool ok = true;
        for (int it = 0; ok; ++it) {
            const Pair p = pair_at(it);
            if (p.hk < 0) break;
            const int tt = h * a.tpt + token, n = p.n(h);
            const bool live = in_tile && tt < p.tokens;
            // rows without a token see what the tile's last one does
            const int lim = p.lim0 + (live ? tt : min(p.tokens, (h + 1) * a.tpt) - 1);
            const int lim_all = __reduce_min_sync(0xffffffffu, lim);        // keys that every row of the warp sees
            float ref = -INFINITY, l = 0.f;
            bool ref_wanted = true;
            for (int c = 0; c < n; ++c) {
                ok = ok && wt_wait(&s_full[h], ns & 1u, bad);
                ++ns;
                tc_fence_after();
                const int left = lim - c * kPtKeys;
                const bool edge = lim_all < (c + 1) * kPtKeys;
                uint32_t x[128], y[64];
                float sum;
                bool all_none = false;
                // one pass as a rule; another where a weight has outgrown its room
#pragma unroll 1
                while (true) {
                    tc_ld32_nowait(tS, x);
                    tc_wait_ld_u32<32>(x);
#pragma unroll
                    for (int i = 1; i < 4; ++i) tc_ld32_nowait(tS + 32u * i, x + 32 * i);           // arrive under the work on the first
                    if (edge) hide(x, left, none);
                    // the first chunk: 32 scores set the reference, which is near enough as a rule
                    if (ref_wanted) ref = largest<32>(x, a.scale2), ref_wanted = false;
                    const float rf = ref == -INFINITY ? 0.f : -ref;
                    uint64_t la = pk(0.f, 0.f), lb = la;
                    weigh(x, a.scale2, rf, y, la, lb);
                    tc_wait_ld_u32<96>(x + 32);
                    if (edge) hide(x + 32, left - 32, none), hide(x + 64, left - 64, none), hide(x + 96, left - 96, none);
#pragma unroll
                    for (int i = 1; i < 4; ++i) weigh(x + 32 * i, a.scale2, rf, y + 16 * i, la, lb);
                    float l0, l1;
                    unpk(add2(la, lb), l0, l1);
                    sum = l0 + l1;
                    if (!__any_sync(0xffffffffu, live && (sum > kPtTop || (ref == -INFINITY && left > 0 && !all_none)))) break;
                    // the scores again: they stand until their weights are written
#pragma unroll
                    for (int i = 0; i < 4; ++i) tc_ld32_nowait(tS + 32u * i, x + 32 * i);
                    tc_wait_ld_u32<128>(x);
                    if (edge) hide(x, left, none), hide(x + 32, left - 32, none), hide(x + 64, left - 64, none), hide(x + 96, left - 96, none);
                    const float m = largest<128>(x, a.scale2);
                    all_none = m == -INFINITY;      // (scores of -infinity alone: the reference stays)
                    float f = 1.f;
                    if (m > ref) {
                        f = ref == -INFINITY ? 0.f : ex2(ref - m);
                        ref = m;
                        l *= f;
                    }
                    // O holds the chunks before, whose products are done (this S came behind them)
#pragma unroll 1
                    for (int i = 0; c > 0 && i < D / 16; ++i) {
                        const uint32_t at = tO + (uint32_t)(16 * i);
                        uint32_t u[16];
                        tc_ld16_nowait(at, u);
                        tc_wait_ld_u32<16>(u);
#pragma unroll
                        for (int e = 0; e < 16; ++e) u[e] = __float_as_uint(__uint_as_float(u[e]) * f);
                        tc_st16(at, u);
                    }
                }
                l += sum;
#pragma unroll
                for (int i = 0; i < 4; ++i) tc_st16(tS + 64u * (i >> 1) + 16u * (i & 1), y + 16 * i);
                tc_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[h]);
            }
            // ---- the rows' results
            if (n > 0) {
                ok = ok && wt_wait(&o_full[h], no & 1u, bad);
                ++no;
                tc_fence_after();
            }
            ok = __all_sync(0xffffffffu, ok && !*bad);
            const float fail = ok ? 0.f : __uint_as_float(0x7fc00000u);
            // no key gives zeros; keys whose scores are all -infinity NaN, as the formula does
            const float by = (lim <= 0 ? 0.f : l == 0.f ? __uint_as_float(0x7fc00000u) : 1.f / l) + fail;
            const uint32_t odd = n > 0 ? *reinterpret_cast<volatile uint32_t *>(&slot_of(it).odd) : 0u;
            uint8_t *dst = a.out + (int64_t)(p.q0 + tt) * a.o_token + (int64_t)(p.head() * a.G + head) * (2 * D);
            uint32_t u[D];
            if (n > 0) {
#pragma unroll
                for (int i = 0; i < D / 32; ++i) tc_ld32_nowait(tO + 32u * i, u + 32 * i);
                tc_wait_ld_u32<D>(u);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&o_empty[h]);        // the next pair's products may begin
            } else {
#pragma unroll
                for (int e = 0; e < D; ++e) u[e] = 0;
            }
            if (odd) {
                // the values that were taken out, by the rows that see them
#pragma unroll 1
                for (int k = 0; k < 32; ++k) {
                    if (!((odd >> k) & 1u)) continue;
                    const int j0 = (first_edge(p) + k) * kPtKeys, j1 = min(lim, j0 + kPtKeys);
                    for (int j = j0; live && j < j1; ++j) {
                        const uint16_t *v = reinterpret_cast<const uint16_t *>(a.v + (int64_t)(p.k0 + j) * a.v_token) + p.head() * D;
#pragma unroll
                        for (int e = 0; e < D; ++e) {
                            const uint32_t w = (uint32_t)v[e] << 16;
                            if ((w & 0x7f800000u) == 0x7f800000u) u[e] = __float_as_uint(__uint_as_float(u[e]) + __uint_as_float(w));
                        }
                    }
                }
            }
            if (p.piece() >= 0) {
                // a piece: the products as they are, with the reference and the sum
                const int64_t at = (int64_t)p.piece() * 256 + h * 128 + r;
                if (live) {
                    float *to = a.p_o + at * D;
#pragma unroll
                    for (int e = 0; e < D; e += 8) st32(to + e, u + e);
                    a.p_ml[at] = make_float2(ref, l + fail);
                }
            } else if (live) {
#pragma unroll
                for (int i = 0; i < D / 32; ++i) {
                    uint32_t o[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) o[e] = pack_bf16(__uint_as_float(u[32 * i + 2 * e]) * by, __uint_as_float(u[32 * i + 2 * e + 1]) * by);
                    if (a.wide_out) {               // whole sectors
                        st32(dst + 64 * i, o);
                        st32(dst + 64 * i + 32, o + 8);
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            *reinterpret_cast<uint4 *>(dst + 64 * i + 16 * e) = make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                    }
                }
            }
            done_with(it);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 8) tmem_dealloc(tmem, 512);
}

// The pieces of a pair that several CTAs worked, weighted to their largest reference: blockIdx.x the pair's first piece, blockIdx.y 16 of
// its 256 rows; D / 8 threads a row.
constexpr int kPtJoinRows = 16;
template <int D> __global__ void __launch_bounds__(kPtJoinRows * D / 8) attn_prompt_join_kernel(const PromptArgs a) {
    pdl_wait();
    const Join j = a.join[blockIdx.x];
    if (j.more == 0) return;
    const int row = blockIdx.y * kPtJoinRows + threadIdx.x / (D / 8), d = threadIdx.x % (D / 8) * 8;
    const int h = row >> 7, r = row & 127, token = r / a.G, head = r - token * a.G, tt = h * a.tpt + token;
    if (token >= a.tpt || tt >= j.tokens) return;
    auto piece = [&](int i) { return (int64_t)(i == 0 ? 2 * j.first + j.second : 2 * (j.first + i)) * 256 + row; };
    float M = -INFINITY;
    for (int i = 0; i <= j.more; ++i) M = fmaxf(M, a.p_ml[piece(i)].x);
    float sum = 0.f, acc[8] = {};
    for (int i = 0; i <= j.more; ++i) {
        const float2 e = a.p_ml[piece(i)];
        if (e.y == 0.f) continue;                   // nothing seen there
        const float f = ex2(e.x - M);
        sum = fmaf(f, e.y, sum);
        const float4 *o = reinterpret_cast<const float4 *>(a.p_o + piece(i) * D + d);
        const float4 x = o[0], y = o[1];
        acc[0] = fmaf(f, x.x, acc[0]), acc[1] = fmaf(f, x.y, acc[1]), acc[2] = fmaf(f, x.z, acc[2]), acc[3] = fmaf(f, x.w, acc[3]);
        acc[4] = fmaf(f, y.x, acc[4]), acc[5] = fmaf(f, y.y, acc[5]), acc[6] = fmaf(f, y.z, acc[6]), acc[7] = fmaf(f, y.w, acc[7]);
    }
    const float by = j.lim0 + tt <= 0 ? 0.f : sum == 0.f ? __uint_as_float(0x7fc00000u) : 1.f / sum;
    *reinterpret_cast<uint4 *>(a.out + (int64_t)(j.q0 + tt) * a.o_token + ((int64_t)(j.hk * a.G + head) * D + d) * 2) =
        make_uint4(pack_bf16(acc[0] * by, acc[1] * by), pack_bf16(acc[2] * by, acc[3] * by), pack_bf16(acc[4] * by, acc[5] * by),
                   pack_bf16(acc[6] * by, acc[7] * by));
}

template <typename F, typename... A>
cudaError_t launch_after(F fn, dim3 ctas, int threads, size_t smem, cudaStream_t s, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = ctas;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fn, args...);
}

template <int D> cudaError_t launch(const CUtensorMap &q, const CUtensorMap &k, const CUtensorMap &v, const PromptArgs &a, unsigned ctas, int dev,
                                    cudaStream_t s) {
    static std::atomic<bool> ready[64] = {};
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    auto fn = attn_prompt_kernel<D>;
    if (!ready[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void *>(fn), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   (int)PtCfg<D>::kSmem);
        if (e != cudaSuccess) return e;
        ready[dev] = true;
    }
    if (a.list) {
        const cudaError_t e = launch_after(attn_prompt_plan_kernel, 1, 1024, 0, s, a);
        if (e != cudaSuccess) return e;
    }
    const cudaError_t e = launch_after(fn, ctas, kPtThreads, PtCfg<D>::kSmem, s, q, k, v, a);
    if (e != cudaSuccess || !a.join) return e;
    return launch_after(attn_prompt_join_kernel<D>, dim3(2 * ctas, 256 / kPtJoinRows), kPtJoinRows * D / 8, 0, s, a);
}

// How a call runs: the most pairs that the sequences can have, and the CTAs.
struct PromptPlan {
    int tpt, cap;
    bool list, join;
    unsigned ctas;
    size_t p_ml, p_o, bytes;
};
// Keys a sequence, in the mean, from which few pairs may be cut into pieces: below, none is long enough to gain by it (kPtWorthCutting), and the
// joining kernel's launch, which the lengths decide about too late, costs 2 us.
constexpr int64_t kPtCutKeys = 16 * kPtKeys;

qd_status plan_prompt(int n_tokens, int n_kv_tokens, int n_seqs, int n_q_heads, int n_kv_heads, int head_dim, int dev, PromptPlan *p) {
    if (n_tokens < 1 || n_kv_tokens < 1 || n_seqs < 1 || n_kv_heads < 1 || n_q_heads < n_kv_heads || n_q_heads % n_kv_heads) return QD_EINVAL;
    if (head_dim != 64 && head_dim != 128) return QD_EUNSUPPORTED;
    const int G = n_q_heads / n_kv_heads;
    if (G > 128 || n_q_heads > 65536 || n_tokens > (1 << 30) || n_kv_tokens > (1 << 30) || n_seqs > (1 << 24)) return QD_EUNSUPPORTED;
    p->tpt = 128 / G;
    const int64_t pairs = (int64_t)n_tokens / (2 * p->tpt) + std::min(n_seqs, n_tokens);
    if (pairs * n_kv_heads > (1 << 30)) return QD_EUNSUPPORTED;
    const int sms = sms_of(dev);
    p->cap = (int)pairs;
    p->list = pairs > kPtOwnPairs || n_seqs > kPtOwnPairs || pairs * n_kv_heads > (int64_t)kPtOwnRounds * sms;
    p->ctas = (unsigned)std::min<int64_t>(pairs * n_kv_heads, sms);
    // few pairs of long sequences: every SM has a CTA, and room for two pieces
    p->join = !p->list && pairs * n_kv_heads <= sms + sms / 4 && n_kv_tokens >= kPtCutKeys * n_seqs && sms <= kPtMaxCtas &&
              pairs * n_kv_heads * (n_kv_tokens / kPtKeys + 1) < (int64_t(1) << 30);   // (the chunks are counted in an int)
    p->bytes = p->list ? 256 + (size_t)pairs * 32 : 0;
    if (p->join) {
        p->ctas = (unsigned)sms;
        const size_t pieces = 2 * (size_t)sms;
        p->p_ml = (pieces * sizeof(Join) + 255) / 256 * 256;
        p->p_o = p->p_ml + pieces * 256 * sizeof(float2);
        p->bytes = p->p_o + pieces * 256 * head_dim * sizeof(float);
    }
    return QD_OK;
}

}  // namespace

}  // namespace qd

using namespace qd;

extern "C" {

qd_status qd_attn_prompt_workspace(int n_tokens, int n_kv_tokens, int n_seqs, int n_q_heads, int n_kv_heads, int head_dim, size_t *bytes) {
    if (!bytes) return QD_EINVAL;
    *bytes = 0;
    int dev = 0;
    PromptPlan p;
    qd_status st = plan_prompt(n_tokens, n_kv_tokens, n_seqs, n_q_heads, n_kv_heads, head_dim, -1, &p);
    if (st != QD_OK) return st;
    if (cudaGetDevice(&dev) != cudaSuccess) return QD_ECUDA;
    st = plan_prompt(n_tokens, n_kv_tokens, n_seqs, n_q_heads, n_kv_heads, head_dim, dev, &p);
    *bytes = p.bytes;
    return st;
}

qd_status qd_attn_prompt(const void *q_dev, int64_t q_stride, const void *k_dev, int64_t k_stride, const void *v_dev, int64_t v_stride,
                         void *out_dev, int64_t out_stride, int n_tokens, int n_kv_tokens, int n_q_heads, int n_kv_heads, int head_dim,
                         float scale, const int32_t *offsets_dev, const int32_t *kv_offsets_dev, int n_seqs, void *workspace_dev,
                         size_t workspace_bytes, void *cuda_stream) {
    PromptPlan p;
    qd_status st = plan_prompt(n_tokens, n_kv_tokens, n_seqs, n_q_heads, n_kv_heads, head_dim, -1, &p);
    if (st != QD_OK) return st;
    if (!q_dev || !k_dev || !v_dev || !out_dev || !offsets_dev || !(scale > -3e38f && scale < 3e38f)) return QD_EINVAL;
    if (!kv_offsets_dev && n_tokens != n_kv_tokens) return QD_EINVAL;
    for (const void *x : {q_dev, k_dev, v_dev, (const void *)out_dev})
        if (!is_aligned(x, 16)) return QD_EINVAL;
    if (!is_aligned(offsets_dev, 4) || !is_aligned(kv_offsets_dev, 4)) return QD_EINVAL;
    const int64_t q_row = (int64_t)n_q_heads * head_dim, k_row = (int64_t)n_kv_heads * head_dim;
    for (int64_t x : {q_stride, k_stride, v_stride, out_stride})
        if (x % 8 || x > (int64_t(1) << 37)) return QD_EINVAL;       // (a tensor map's strides end at 2^40 bytes)
    if ((n_tokens > 1 && (q_stride < q_row || out_stride < q_row)) || (n_kv_tokens > 1 && (k_stride < k_row || v_stride < k_row))) return QD_EINVAL;
    // out lies over none of the inputs, but may stand between their rows
    if (!rows_beside(out_dev, 2, n_tokens, out_stride, q_row, q_dev, 2, n_tokens, q_stride, q_row) ||
        !rows_beside(out_dev, 2, n_tokens, out_stride, q_row, k_dev, 2, n_kv_tokens, k_stride, k_row) ||
        !rows_beside(out_dev, 2, n_tokens, out_stride, q_row, v_dev, 2, n_kv_tokens, v_stride, k_row))
        return QD_EINVAL;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return QD_ECUDA;
    for (const void *x : {q_dev, k_dev, v_dev, (const void *)out_dev, (const void *)offsets_dev})
        if (!on_device(x, dev)) return QD_EINVAL;
    if (kv_offsets_dev && !on_device(kv_offsets_dev, dev)) return QD_EINVAL;
    if ((st = plan_prompt(n_tokens, n_kv_tokens, n_seqs, n_q_heads, n_kv_heads, head_dim, dev, &p)) != QD_OK) return st;
    if (p.bytes && (!workspace_dev || workspace_bytes < p.bytes || !is_aligned(workspace_dev, 256) || !on_device(workspace_dev, dev)))
        return QD_EINVAL;

    PromptArgs a = {};
    a.v = static_cast<const uint8_t *>(v_dev), a.out = static_cast<uint8_t *>(out_dev);
    a.v_token = v_stride * 2, a.o_token = out_stride * 2;
    a.offsets = offsets_dev, a.kv_offsets = kv_offsets_dev ? kv_offsets_dev : offsets_dev;
    a.N = n_tokens, a.M = n_kv_tokens, a.B = n_seqs, a.G = n_q_heads / n_kv_heads, a.kvh = n_kv_heads;
    a.wide_out = is_aligned(out_dev, 32) && (n_tokens == 1 || out_stride % 16 == 0);
    a.tpt = p.tpt;
    a.scale2 = scale == 0.f ? 1e-30f : scale * 1.4426950408889634f;   // (hidden scores are infinite: 0 times them would be NaN)
    if (p.list) {
        a.count = static_cast<int *>(workspace_dev);
        a.list = reinterpret_cast<int4 *>(static_cast<uint8_t *>(workspace_dev) + 256);
        a.cap = p.cap;
        while ((n_kv_tokens / kPtKeys + 1) >> a.cost_shift >= kPtBuckets) ++a.cost_shift;
    }
    if (p.join) {
        uint8_t *ws = static_cast<uint8_t *>(workspace_dev);
        a.join = reinterpret_cast<Join *>(ws);
        a.p_ml = reinterpret_cast<float2 *>(ws + p.p_ml), a.p_o = reinterpret_cast<float *>(ws + p.p_o);
    }
    CUtensorMap mq, mk, mv;
    if (!make_heads_map(&mq, q_dev, head_dim, n_q_heads, n_tokens, n_tokens > 1 ? q_stride : q_row, a.G, a.tpt) ||
        !make_heads_map(&mk, k_dev, head_dim, n_kv_heads, n_kv_tokens, n_kv_tokens > 1 ? k_stride : k_row, 1, kPtKeys) ||
        !make_heads_map(&mv, v_dev, head_dim, n_kv_heads, n_kv_tokens, n_kv_tokens > 1 ? v_stride : k_row, 1, kPtKeys))
        return QD_ECUDA;
    cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
    const cudaError_t e = head_dim == 128 ? launch<128>(mq, mk, mv, a, p.ctas, dev, s) : launch<64>(mq, mk, mv, a, p.ctas, dev, s);
    return e == cudaSuccess ? QD_OK : QD_ECUDA;
}

}  // extern "C"
