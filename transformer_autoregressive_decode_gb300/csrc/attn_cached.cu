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
#include <atomic>

#include "attn_cached.cuh"
#include "qd_internal.h"

namespace qd {

namespace {

constexpr int kAcWarps = 4, kAcThreads = kAcWarps * 32;
constexpr int kAcMaxCluster = 8;
constexpr int kAcMaxTokens = 64;
constexpr int kAcMaxPositions = INT32_MAX - 1024;    // rounded up to tiles or chunks they fit an int

__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool live) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void *src, bool live) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(live ? 4 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void mma16816_f16(float *d, const uint32_t *a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t movmatrix(uint32_t a) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}
// NTX: tiles of 8 columns, plus kOneColumn for bf16 rows over a bf16 cache with a column a row: from 9 rows on, where it
// halves the passes over the cache.  Where a row has one column (over 8-bit rows, too) each step makes two products for the
// output, one per part of p: 16 streams of 64 rows over 4000 bf16 positions 71 us, 67 with the first part alone, which
// keeps 8 bits (11 of fp16); of 16 rows over 8-bit positions 34.6 and 33.6; 64 ragged 8-bit streams 34.6 and 33.9.
constexpr int kOneColumn = 8;
template <bool Q8, bool F32, int D, int NTX> struct AcCfg {
    static constexpr int NT = NTX & 7;
    static constexpr int C = Q8 ? (F32 ? 2 : 1) : F32 ? 4 : NTX & kOneColumn ? 1 : 2;   // columns per row
    static constexpr int PP = C == 1 ? 2 : 1;                      // products of the output, one per part of p
    static constexpr int RW = 8 * NT / C;                          // rows per CTA
    static constexpr int ES = Q8 ? 1 : 2;
    static constexpr int KP = D * ES / 64;                         // 16-byte pieces of a K row per lane
    static constexpr int KW = Q8 ? 4 : 2;                          // k-steps per piece
    static constexpr int KS = D / 16, MT = D / 16;
    static constexpr int LB = D * ES;                              // bytes of a row
    static constexpr int CP = LB / 32;                             // 16-byte copies per lane and block, of K or V
    static constexpr int CR = 512 / LB;                            // rows that one copy instruction covers
    static constexpr int kTurn = 8 / CR;                           // copies after which the places repeat, 8 rows on
    // A step's tile: two blocks of 16 positions where they take 8 KB at most (half the address arithmetic,
    // votes and waits per position, and two independent chains), one of bf16 rows of 128.
    static constexpr int SUB = D * ES <= 128 ? 2 : 1;
    static constexpr int TP = 16 * SUB;                            // positions of a tile
    static constexpr int kV = 16 * LB;                             // byte offset of V in a block
    static constexpr int kBlock = 2 * kV;
    static constexpr int kS = SUB * kBlock;                        // of the scales in a tile: [K, V][TP]
    static constexpr int kTileBytes = kS + (Q8 ? TP * 8 : 0);
    
    static constexpr int kStages = kTileBytes > 8192 ? 2 : 3;
    static constexpr int kRing = kStages * kTileBytes;             // per warp
    // after the pass the rings' space holds the warps' partials
    static constexpr int kMl = kAcWarps * RW * D * 4;
    static constexpr int kEnd = kMl + kAcWarps * RW * 8;
    static constexpr int kSmem = kAcWarps * kRing > kEnd ? kAcWarps * kRing : kEnd;
    // behind them what a cluster's CTAs send each other: [source][slice], [source][rows]
    static constexpr int kRecv = (kSmem + 15) / 16 * 16;
    static constexpr int kRecvMl = kRecv + RW * D * 4 + kAcMaxCluster * 16;
    static constexpr int kSmemCluster = kRecvMl + kAcMaxCluster * RW * 8;
    // CTAs an SM: as many as shared memory holds, but two for two row tiles of 128 (three left 240 bytes a thread in
    // memory: 96 streams of 16 rows 133 us against 128)
    static constexpr int kMinCtas = kSmem > 72 * 1024 || (NT == 2 && D == 128) || NT == 4 ? 2 : NT == 1 && kSmem <= 54 * 1024 ? 4 : 3;
};

__device__ __forceinline__ void st_cluster_f2(uint32_t addr, float2 v) {
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(v.x), "f"(v.y) : "memory");
}
__device__ __forceinline__ void st_cluster_f4(uint32_t addr, float4 v) {
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
                 : "memory");
}
// The cluster barrier in two halves, the first without an order: the CTAs have started.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.aligned;" ::: "memory"); }

// One warp's pass over some of an item's tiles: the item's rows as B fragments, the ring of
// tiles, and the running reference, sums and output.
template <bool Q8, bool F32, int D, int NTX, bool PREFIX> struct WarpPass {
    using K = AcCfg<Q8, F32, D, NTX>;
    static constexpr int NT = K::NT;
    static constexpr int C = K::C, HC = C == 1 ? 2 : 1;
    // bf16 rows over codes: K's codes enter as 1152 + code, and the scores start at -1152 sum q (fp32 sums of
    // 8 steps: within 2^-20 of 1152 sum |q|, 2^-17 of max|k| sum |q|).  fp32 rows and V subtract it from each code.
    static constexpr bool kFold = Q8 && !F32;
    int lane, g, t;
    uint32_t qf[NT][K::KS][2];
    float cs[NT][2], s0[NT][2];                     // of this lane's columns: factor, the scores' start
    int lim[NT][HC];
    int lim_lo, lim_hi;                             // the limits of the item's rows
    float o[K::MT][NT][4], ref[NT][HC], l[NT][HC];
    const uint8_t *kb, *vb, *kp, *vp;               // this lane's column of the item; of the next tile
    const float *ksb, *vsb;
    int64_t row, hop;
    int n_pos, next, end, step;
    uint8_t *ring;
    uint32_t ring_s;
    int put[K::kTurn], kget[2], vget[2];            // this lane's places: copies, K's pieces, V's positions

    __device__ __forceinline__ void init(int lane_) {
        lane = lane_, g = lane_ >> 2, t = lane_ & 3;
        const int at = lane / (32 / K::CR), c = lane % (32 / K::CR);
#pragma unroll
        for (int j = 0; j < K::kTurn; ++j) put[j] = place(K::CR * j + at, c);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            kget[i] = K::LB == 64 ? place(g, t) : place(g, 4 * i + t);
            vget[i] = K::LB == 64 ? place(2 * t + i, g >> 1) + 8 * (g & 1) : place(2 * t + i, g);
        }
    }

    // Where 16-byte piece c of position p stands in a block of K or V: rows in order, the pieces of
    // a 128-byte line permuted by the position, such that the fragments' reads (8 lanes: two rows, four pieces of K;
    // four rows two apart, two pieces of V) meet every bank once.
    static __device__ __forceinline__ int place(int p, int c) {
        const int f = ((p & 1) << 2) ^ (p & 6);
        if constexpr (K::LB == 64) return (p >> 1) * 128 + (((((p & 1) << 2) + c) ^ (p & 6)) << 4);
        return p * K::LB + ((c >> 3) << 7) + (((c & 7) ^ f) << 4);
    }

    // copy the next tile into a stage; positions past n_pos become zeros
    template <bool FULL> __device__ __forceinline__ void fetch_as(int stage) {
        const uint32_t dst = ring_s + stage * K::kTileBytes;
        const int left = n_pos - next * K::TP, at = lane / (32 / K::CR);   // positions of the tile; this lane's first
#pragma unroll
        for (int u = 0; u < K::SUB; ++u)
#pragma unroll
            for (int j = 0; j < K::CP; ++j) {
                const int p = K::CR * j;
                const uint32_t d = dst + u * K::kBlock + put[j % K::kTurn] + (j / K::kTurn) * 8 * K::LB;
                const bool live = FULL || 16 * u + p + at < left;
                cp16(d, live ? kp + (16 * u + p) * row : kb, live);
                cp16(d + K::kV, live ? vp + (16 * u + p) * row : vb, live);
            }
        if constexpr (Q8) {
            static_assert(K::TP == 32, "a lane per position's scales");
            const int p = next * K::TP + lane;
            const bool live = FULL || lane < left;
            cp4(dst + K::kS + lane * 4, ksb + (live ? p : 0), live);
            cp4(dst + K::kS + 128 + lane * 4, vsb + (live ? p : 0), live);
        }
    }
    __device__ __forceinline__ void fetch(int stage) {
        if ((next + 1) * K::TP <= n_pos)
            fetch_as<true>(stage);
        else
            fetch_as<false>(stage);
        kp += hop, vp += hop;
    }

    // tiles first, first + step, ... below end of `len` positions of one stream and head: the first copies start here
    __device__ __forceinline__ void start(const KvView &v, int b, int hk, int len, uint8_t *ring_, int first, int end_,
                                          int step_) {
        const int at = lane / (32 / K::CR), c = lane % (32 / K::CR);
        kb = v.k + b * v.stream + hk * v.head + c * 16;
        vb = v.v + b * v.stream + hk * v.head + c * 16;
        ksb = Q8 ? v.ks + b * v.sstream + hk * v.shead : nullptr;
        vsb = Q8 ? v.vs + b * v.sstream + hk * v.shead : nullptr;
        row = v.row;
        n_pos = len;
        ring = ring_;
        ring_s = smem_addr(ring_);
        next = first, end = end_, step = step_;
        kp = kb + ((int64_t)first * K::TP + at) * row;
        vp = vb + ((int64_t)first * K::TP + at) * row;
        hop = (int64_t)step * K::TP * row;
#pragma unroll 1
        for (int s = 0; s < K::kStages - 1; ++s) {
            if (next < end) fetch(s);
            cp_commit();
            next += step;
        }
    }

    // rows r0 .. of the item as B fragments: column 8 nt + g holds part (column % C) of row r0 +
    // column / C; q scaled by a power of two per row for fp16
    __device__ __forceinline__ void load_rows(const CachedArgs &a, int b, int hk, int r0, int len, int nn) {
        float cs_g[NT], s0_g[NT];
        int lim_g[NT];
        lim_lo = INT32_MAX, lim_hi = 0;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int col = 8 * nt + g, r = r0 + col / C, part = col % C;
            int bb = b, rr = r;
            if constexpr (PREFIX) {
                bb = r / (a.T * a.G);
                rr = r - bb * (a.T * a.G);
            }
            const int tt = rr / a.G, gg = rr - tt * a.G;
            const bool live = r < a.rows && tt < (PREFIX ? clamp_new(a, bb) : nn);   // the others are not read
            const uint8_t *src = a.q + bb * a.q_stream + tt * a.q_token + (int64_t)(hk * a.G + gg) * D * (F32 ? 4 : 2);
            constexpr int E = 16 / K::ES;           // dims of a piece
            float x[K::KP * E];
#pragma unroll
            for (int i = 0; i < K::KP; ++i)
#pragma unroll
                for (int e = 0; e < E; e += F32 ? 4 : 8) {
                    const int d = i * 4 * E + t * E + e;
                    uint4 u = make_uint4(0, 0, 0, 0);
                    if (live) u = *reinterpret_cast<const uint4 *>(src + d * (F32 ? 4 : 2));
                    if constexpr (F32)
                        Elem<float>::unpack(u, x + i * E + e);
                    else
                        Elem<__nv_bfloat16>::unpack(u, x + i * E + e);
                }
            float c = a.scale2, sum = 0.f;
            if constexpr (Q8) {
                uint32_t m = 0;
#pragma unroll
                for (int e = 0; e < K::KP * E; ++e) m = max(m, __float_as_uint(x[e]) & 0x7fffffffu);
                m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
                m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
                // the row's largest value to [2^14, 2^15)
                int up = 268 - (int)(m >> 23);
                up = up > 253 ? 253 : up;
                const float f = __uint_as_float((uint32_t)up << 23);
                c *= __uint_as_float((uint32_t)(254 - up) << 23);
#pragma unroll
                for (int e = 0; e < K::KP * E; ++e) x[e] *= f;
            }
#pragma unroll
            for (int e = 0; e < K::KP * E; ++e) {
                if constexpr (Q8) {
                    if (part == 1) x[e] = x[e] - f16_of(x[e]);
                } else {
                    if (part >= 1) x[e] = x[e] - bf16_of(x[e]);
                    if (part >= 2) x[e] = x[e] - bf16_of(x[e]);
                    if (part >= 3) x[e] = 0.f;
                }
            }
#pragma unroll
            for (int ks = 0; ks < K::KS; ++ks)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float lo = x[ks * 4 + 2 * k], hi = x[ks * 4 + 2 * k + 1];
                    qf[nt][ks][k] = Q8 ? pack_f16(lo, hi) : pack_bf16(lo, hi);
                    if constexpr (kFold) {
                        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&qf[nt][ks][k]));
                        sum += f.x + f.y;
                    }
                }
            if constexpr (kFold) {
                sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                sum += __shfl_xor_sync(0xffffffffu, sum, 2);
            }
            s0_g[nt] = -1152.f * sum;
            cs_g[nt] = c;
            lim_g[nt] = !live ? 0 : PREFIX ? len : max(0, len - (nn - 1 - tt));
            lim_lo = min(lim_lo, __reduce_min_sync(0xffffffffu, live ? lim_g[nt] : INT32_MAX));
            lim_hi = max(lim_hi, __reduce_max_sync(0xffffffffu, lim_g[nt]));
        }
        // the columns of this lane's accumulators
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                cs[nt][k] = __shfl_sync(0xffffffffu, cs_g[nt], (2 * t + k) * 4);
                s0[nt][k] = __shfl_sync(0xffffffffu, s0_g[nt], (2 * t + k) * 4);
            }
#pragma unroll
            for (int k = 0; k < HC; ++k) lim[nt][k] = __shfl_sync(0xffffffffu, lim_g[nt], (2 * t + k) * 4);
        }
#pragma unroll
        for (int mt = 0; mt < K::MT; ++mt)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[mt][nt][e] = 0.f;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < HC; ++k) ref[nt][k] = -INFINITY, l[nt][k] = 0.f;
    }

    // every row sees all `len` positions of the run that follows
    __device__ __forceinline__ void see_all(int len) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < HC; ++k) lim[nt][k] = len;
        lim_lo = lim_hi = len;
    }

    __device__ __forceinline__ void run() {
        int stage = 0;
        for (int tile = next - (K::kStages - 1) * step; tile < end; tile += step) {
            if (next < end) fetch(stage == 0 ? K::kStages - 1 : stage - 1);
            cp_commit();
            next += step;
            cp_wait<K::kStages - 1>();
            __syncwarp();                           // other lanes' copies
            one_tile(ring + stage * K::kTileBytes, tile * K::TP);
            stage = stage == K::kStages - 1 ? 0 : stage + 1;
            __syncwarp();                           // before the stage is written again
        }
        cp_wait<0>();
    }

    // Scores of one block of 16 positions: rows (positions) g and g + 8, columns 2t and 2t + 1
    __device__ __forceinline__ void scores(const uint8_t *st, float (&s)[NT][4]) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[nt][e] = kFold ? s0[nt][e & 1] : 0.f;
#pragma unroll
        for (int i = 0; i < K::KP; ++i) {
            const uint8_t *at = st + kget[i & 1] + (i >> 1) * 128;
            const uint4 ua = *reinterpret_cast<const uint4 *>(at);
            const uint4 ub = *reinterpret_cast<const uint4 *>(at + 8 * K::LB);
            const uint32_t wa[4] = {ua.x, ua.y, ua.z, ua.w}, wb[4] = {ub.x, ub.y, ub.z, ub.w};
#pragma unroll
            for (int w = 0; w < K::KW; ++w) {
                uint32_t f[4];
                if constexpr (Q8) {
                    const uint32_t xa = wa[w] ^ 0x80808080u, xb = wb[w] ^ 0x80808080u;
                    f[0] = codes_f16<kFold>(xa, 0x4140), f[1] = codes_f16<kFold>(xb, 0x4140);
                    f[2] = codes_f16<kFold>(xa, 0x4342), f[3] = codes_f16<kFold>(xb, 0x4342);
                } else {
                    f[0] = wa[2 * w], f[1] = wb[2 * w], f[2] = wa[2 * w + 1], f[3] = wb[2 * w + 1];
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const uint32_t *q = qf[nt][K::KW * i + w];
                    if constexpr (Q8)
                        mma16816_f16(s[nt], f, q[0], q[1]);
                    else
                        mma16816(s[nt], f, q[0], q[1]);
                }
            }
        }
    }

    // Output: rows (dims) of V^T of one block against its probabilities (their parts)
    __device__ __forceinline__ void output(const uint8_t *sv, const uint32_t (&pb)[K::PP][NT][2], int p0) {
        if constexpr (Q8) {
            constexpr int VW = D / 32;
            uint32_t v[4][VW];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint8_t *at = sv + vget[i & 1] + (i >> 1) * 8 * K::LB;
                if constexpr (VW == 4) {
                    const uint4 u = *reinterpret_cast<const uint4 *>(at);
                    v[i][0] = u.x, v[i][1] = u.y, v[i][2] = u.z, v[i][3] = u.w;
                } else {
                    const uint2 u = *reinterpret_cast<const uint2 *>(at);
                    v[i][0] = u.x, v[i][1] = u.y;
                }
            }
#pragma unroll
            for (int w = 0; w < VW; ++w) {
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i][w] ^= 0x80808080u;
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    const uint32_t y = __byte_perm(v[0][w], v[1][w], hh ? 0x7362 : 0x5140);
                    const uint32_t z = __byte_perm(v[2][w], v[3][w], hh ? 0x7362 : 0x5140);
                    const uint32_t f[4] = {codes_f16<false>(y, 0x4140), codes_f16<false>(y, 0x4342),
                                           codes_f16<false>(z, 0x4140), codes_f16<false>(z, 0x4342)};
#pragma unroll
                    for (int pp = 0; pp < K::PP; ++pp)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) mma16816_f16(o[2 * w + hh][nt], f, pb[pp][nt][0], pb[pp][nt][1]);
                }
            }
        } else {
            uint32_t v[4][4 * (K::LB / 128)];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < (K::LB / 128); ++j) {
                    const uint4 u = *reinterpret_cast<const uint4 *>(sv + vget[i & 1] + (i >> 1) * 8 * K::LB + 128 * j);
                    v[i][4 * j] = u.x, v[i][4 * j + 1] = u.y, v[i][4 * j + 2] = u.z, v[i][4 * j + 3] = u.w;
                }
            // A new token's V that is not finite must not reach the rows that do not see it (0 x
            // infinity is NaN): only tiles that some rows see further into than others can hold one.
            bool odd = false;
            if (!PREFIX && p0 + 16 > lim_lo) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int w = 0; w < 4 * (K::LB / 128); ++w)
                        odd |= (v[i][w] & 0x7f80u) == 0x7f80u || (v[i][w] & 0x7f800000u) == 0x7f800000u;
                odd = __any_sync(0xffffffffu, odd);
            }
#pragma unroll
            for (int w = 0; w < 4 * (K::LB / 128); ++w) {
                const uint32_t f[4] = {__byte_perm(v[0][w], v[1][w], 0x5410), __byte_perm(v[0][w], v[1][w], 0x7632),
                                       __byte_perm(v[2][w], v[3][w], 0x5410), __byte_perm(v[2][w], v[3][w], 0x7632)};
                if (!PREFIX && odd) {
                    // one limit after the other: V beyond it zeroed, the result kept by the columns it is theirs
                    for (int cut = lim_lo; cut <= lim_hi; ++cut) {
                        const int at = p0 + 2 * t;
                        const uint32_t m0 = (at < cut ? 0xffffu : 0u) | (at + 1 < cut ? 0xffff0000u : 0u);
                        const uint32_t m1 = (at + 8 < cut ? 0xffffu : 0u) | (at + 9 < cut ? 0xffff0000u : 0u);
                        const uint32_t fm[4] = {f[0] & m0, f[1] & m0, f[2] & m1, f[3] & m1};
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            float acc[4] = {o[w][nt][0], o[w][nt][1], o[w][nt][2], o[w][nt][3]};
#pragma unroll
                            for (int pp = 0; pp < K::PP; ++pp) mma16816(acc, fm, pb[pp][nt][0], pb[pp][nt][1]);
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (lim[nt][HC == 2 ? e & 1 : 0] == cut) o[w][nt][e] = acc[e];
                        }
                    }
                } else {
#pragma unroll
                    for (int pp = 0; pp < K::PP; ++pp)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) mma16816(o[w][nt], f, pb[pp][nt][0], pb[pp][nt][1]);
                }
            }
        }
    }

    // one tile from position p0 on, in its stage
    __device__ __forceinline__ void one_tile(const uint8_t *st, int p0) {
        constexpr int H = 2 * K::SUB;               // this lane's positions: p0 + g + 8 h
        const bool edge = p0 + K::TP > lim_lo;      // some row does not see all of it
        float x[NT][H][HC], vd[H], vl[H];
#pragma unroll
        for (int u = 0; u < K::SUB; ++u) {
            float s[NT][4];
            scores(st + u * K::kBlock, s);
            // in log2 units
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                const int h = 2 * u + hh;
                float kd = 1.f;
                if constexpr (Q8) kd = reinterpret_cast<const float *>(st + K::kS)[g + 8 * h];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int k = 0; k < HC; ++k) {
                        float v = s[nt][2 * hh + k];
                        if constexpr (F32) v += s[nt][2 * hh + 1];   // bf16 q has one part
                        if constexpr (C == 4) v += __shfl_xor_sync(0xffffffffu, v, 1);
                        v *= cs[nt][k];
                        if constexpr (Q8) v *= kd;
                        x[nt][h][k] = v;
                    }
            }
        }
        // z = s + log2|values' scale| bounds the weight that enters the product; a row of zeros
        // does not move the reference
#pragma unroll
        for (int h = 0; h < H; ++h) {
            vd[h] = 1.f, vl[h] = 0.f;
            if constexpr (Q8) {
                vd[h] = reinterpret_cast<const float *>(st + K::kS)[K::TP + g + 8 * h];
                vl[h] = fmaxf(lg2(fabsf(vd[h])), -60.f);
            }
        }
        if (edge) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int h = 0; h < H; ++h)
#pragma unroll
                    for (int k = 0; k < HC; ++k)
                        if (p0 + g + 8 * h >= lim[nt][k]) x[nt][h][k] = -INFINITY;
        }
        bool over = false;
        float m[NT][HC];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < HC; ++k) {
                m[nt][k] = x[nt][0][k] + vl[0];
#pragma unroll
                for (int h = 1; h < H; ++h) m[nt][k] = fmaxf(m[nt][k], x[nt][h][k] + vl[h]);
                over |= m[nt][k] > ref[nt][k] + kAcRoom;
            }
        if (__any_sync(0xffffffffu, over)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float f[HC];
#pragma unroll
                for (int k = 0; k < HC; ++k) {
                    float top = m[nt][k];
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
                    f[k] = 1.f;
                    if (top > ref[nt][k] + kAcRoom) {
                        const float now = top - kAcUp;
                        f[k] = ref[nt][k] == -INFINITY ? 0.f : ex2(ref[nt][k] - now);
                        ref[nt][k] = now;
                        l[nt][k] = l[nt][k] * f[k];
                    }
                }
#pragma unroll
                for (int mt = 0; mt < K::MT; ++mt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[mt][nt][e] *= f[HC == 2 ? (e & 1) : 0];
            }
        }
        // probabilities, their sums, and their parts as the B fragments of the output
        float rf[NT][HC];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < HC; ++k) rf[nt][k] = ref[nt][k] == -INFINITY ? 0.f : ref[nt][k];
#pragma unroll
        for (int u = 0; u < K::SUB; ++u) {
            uint32_t pb[K::PP][NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    const int h = 2 * u + hh;
                    float w[HC];
#pragma unroll
                    for (int k = 0; k < HC; ++k) {
                        w[k] = ex2(x[nt][h][k] - rf[nt][k]);
                        l[nt][k] += w[k];
                        if constexpr (Q8) {
                            w[k] *= vd[h];
                            if (edge && p0 + g + 8 * h >= lim[nt][k]) w[k] = 0.f;   // its scale may be NaN
                        }
                    }
                    uint32_t y;
                    if constexpr (C == 1) {
                        y = Q8 ? pack_f16(w[0], w[1]) : pack_bf16(w[0], w[1]);
                        const float2 hi = Q8 ? __half22float2(*reinterpret_cast<const __half2 *>(&y))
                                             : make_float2(bf16lo(y), bf16hi(y));
                        pb[K::PP - 1][nt][hh] = movmatrix(Q8 ? pack_f16(w[0] - hi.x, w[1] - hi.y) : pack_bf16(w[0] - hi.x, w[1] - hi.y));
                    } else if constexpr (Q8) {
                        const float hi = f16_of(w[0]);
                        y = pack_f16(hi, w[0] - hi);
                    } else if constexpr (C == 2) {
                        const float hi = bf16_of(w[0]);
                        y = pack_bf16(hi, w[0] - hi);
                    } else {
                        const float hi = bf16_of(w[0]), mid = bf16_of(w[0] - hi);
                        y = t & 1 ? pack_bf16(w[0] - hi - mid, 0.f) : pack_bf16(hi, mid);
                    }
                    pb[0][nt][hh] = movmatrix(y);
                }
            output(st + u * K::kBlock + K::kV, pb, p0 + 16 * u);
        }
    }

    // Row r of this lane's columns (k) and eight-column tile nt, its sum over the warp's positions.
    __device__ __forceinline__ int row_of(int nt, int k) const { return (8 * nt + 2 * t + k) / C; }
    __device__ __forceinline__ bool writes() const { return C != 4 || !(t & 1); }
    __device__ __forceinline__ float sum_of(int nt, int k) const {
        float v = l[nt][k];
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
        return v;
    }
    // Four consecutive dims of that row: quad j of this lane's D / 32, at dim_of(j); the parts' columns added.
    static constexpr int kQuads = D / 32;
    __device__ __forceinline__ int dim_of(int j) const {
        return Q8 ? (D / 8) * g + 4 * j : 64 * (j / 2) + 8 * g + 4 * (j % 2);
    }
    __device__ __forceinline__ float4 quad(int nt, int k, int j) const {
        float w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int mt = 2 * j + (e >> 1), h = e & 1;
            w[e] = o[mt][nt][2 * h + k];
            if constexpr (C >= 2) w[e] += o[mt][nt][2 * h + 1];
            if constexpr (C == 4) w[e] += __shfl_xor_sync(0xffffffffu, w[e], 1);
        }
        return make_float4(w[0], w[1], w[2], w[3]);
    }
};

// A stream's tiles of tp positions (a power of two), its own and then those of a short prefix: none where it has no new token.
__device__ __forceinline__ int tiles_of(const CachedArgs &a, int b, int tp) {
    const int len = clamp_len(a.lengths[b], a.max_len);
    return clamp_new(a, b) > 0 ? (int)((unsigned)(len + tp - 1) / (unsigned)tp) + a.pre_tiles : 0;
}

template <bool F32> __device__ __forceinline__ void store4(uint8_t *dst, float4 v, float by) {
    if constexpr (F32)
        *reinterpret_cast<float4 *>(dst) = make_float4(v.x * by, v.y * by, v.z * by, v.w * by);
    else
        *reinterpret_cast<uint2 *>(dst) = make_uint2(pack_bf16(v.x * by, v.y * by), pack_bf16(v.z * by, v.w * by));
}
__device__ __forceinline__ void add4(float4 &acc, float f, float4 v) {
    acc.x = fmaf(f, v.x, acc.x), acc.y = fmaf(f, v.y, acc.y);
    acc.z = fmaf(f, v.z, acc.z), acc.w = fmaf(f, v.w, acc.w);
}

// Small batches: an item per cluster, its warps taking the tiles in turn; the partials meet in
// shared memory and the output is written here.  PREFIX: the rows of every stream over
// the shared prefix, an item per `nsplit` CTAs, partials to global memory.
// blockIdx.x = item * nsplit + split.
template <bool Q8, bool F32, int D, int NTX, bool PREFIX>
__global__ void __launch_bounds__(kAcThreads, AcCfg<Q8, F32, D, NTX>::kMinCtas)
    attn_cached_kernel(const CachedArgs a, int nsplit) {
    using K = AcCfg<Q8, F32, D, NTX>;
    constexpr int NT = K::NT;
    extern __shared__ __align__(16) uint8_t sm[];
    if (!PREFIX && nsplit > 1) cluster_arrive();
    pdl_wait();
    pdl_launch_dependents();                         // after the wait: see attn_join_kernel
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int split = blockIdx.x % nsplit, item = blockIdx.x / nsplit;
    const int grp = item % a.groups, hk = (item / a.groups) % a.kvh, b = PREFIX ? 0 : item / a.groups / a.kvh;
    const int len = PREFIX ? a.max_len : clamp_len(a.lengths[b], a.max_len);
    const int nn = PREFIX ? a.T : clamp_new(a, b);
    const int r0 = grp * K::RW;
    if (PREFIX && a.n_new) {                         // a group without a row in use leaves no partials: nothing asks for them
        const int r = r0 + lane, of = a.T * a.G, bb = r / of;
        if (!__any_sync(0xffffffffu, lane < K::RW && r < a.rows && (r - bb * of) / a.G < clamp_new(a, bb))) return;
    }

    WarpPass<Q8, F32, D, NTX, PREFIX> w;
    w.init(lane);
    {
        const int own = (len + K::TP - 1) / K::TP, step = nsplit * kAcWarps, total = PREFIX ? own : r0 < nn * a.G ? own + a.pre_tiles : 0;
        const int tile = split * kAcWarps + warp;
        bool pre = !PREFIX && tile >= own && tile < total;   // the stream's own tiles, then a short prefix's
        if (pre)
            w.start(a.pc, 0, hk, a.pre_len, sm + warp * K::kRing, tile - own, a.pre_tiles, step);
        else
            w.start(a.c, b, hk, len, sm + warp * K::kRing, tile, min(own, total), step);
        w.load_rows(a, b, hk, r0, len, nn);
        if (pre) w.see_all(a.pre_len);
        w.run();
        if constexpr (!PREFIX) {
            const int then = tile + (own - tile + step - 1) / step * step;   // this warp's first tile past its own
            if (!pre && tile < own && then < total) {
                w.start(a.pc, 0, hk, a.pre_len, sm + warp * K::kRing, then - own, a.pre_tiles, step);
                w.see_all(a.pre_len);
                w.run();
            }
        }
    }
    __syncthreads();

    // ---- the warps' partials
    float *part = reinterpret_cast<float *>(sm);
    float2 *ml = reinterpret_cast<float2 *>(sm + K::kMl);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < w.HC; ++k) {
            const float sum = w.sum_of(nt, k);
            const int row = w.row_of(nt, k);
            if (w.g == 0 && w.writes()) ml[warp * K::RW + row] = make_float2(w.ref[nt][k], sum);
#pragma unroll
            for (int j = 0; j < w.kQuads; ++j) {
                const float4 v = w.quad(nt, k, j);
                if (w.writes()) *reinterpret_cast<float4 *>(part + (warp * K::RW + row) * D + w.dim_of(j)) = v;
            }
        }
    __syncthreads();
    // row `row`, dims 4 (i % (D / 4)) ..: the prefix's partials join, the output is written
    auto finish = [&](int row, int i, float M, float4 acc, float sum) {
        const int r = r0 + row, tt = r / a.G;
        if (tt >= nn) return;
        const int64_t at = (((int64_t)hk * a.B + b) * a.rows + r) * a.splits;
        for (int s = 0; s < a.splits; ++s) {
            const float2 e = a.p_ml[at + s];
            if (e.y == 0.f) continue;
            const float now = fmaxf(M, e.x), keep = part_weight(make_float2(M, sum), now), f = part_weight(e, now);
            acc.x *= keep, acc.y *= keep, acc.z *= keep, acc.w *= keep;
            add4(acc, f, *reinterpret_cast<const float4 *>(a.p_o + (at + s) * D + (i % (D / 4)) * 4));
            sum = fmaf(f, e.y, sum * keep);
            M = now;
        }
        store4<F32>(a.out + b * a.o_stream + tt * a.o_token +
                        ((int64_t)(hk * a.G + (r - tt * a.G)) * D + (i % (D / 4)) * 4) * (F32 ? 4 : 2),
                    acc, sum == 0.f ? 0.f : 1.f / sum);
    };
    // the CTA's (ref, sum) of a row
    auto row_ml = [&](int row) {
        float M = -INFINITY, sum = 0.f;
#pragma unroll
        for (int u = 0; u < kAcWarps; ++u) M = fmaxf(M, ml[u * K::RW + row].x);
#pragma unroll
        for (int u = 0; u < kAcWarps; ++u) {
            const float2 e = ml[u * K::RW + row];
            if (e.y != 0.f) sum = fmaf(part_weight(e, M), e.y, sum);
        }
        return make_float2(M, sum);
    };
    // A cluster's CTAs send their partials to the one that owns the slice (a read of the others' memory instead took a round
    // trip for every CTA, twice): buffers of their own, which no warp's ring uses.
    constexpr int kAll = K::RW * D / 4;
    const int per = (kAll + nsplit - 1) / nsplit;
    float4 *recv = reinterpret_cast<float4 *>(sm + K::kRecv);           // [source][per]
    float2 *recv_ml = reinterpret_cast<float2 *>(sm + K::kRecvMl);      // [source][rows]
    if (!PREFIX && nsplit > 1) cluster_wait();       // every CTA of the cluster has started
    for (int i = threadIdx.x; i < kAll; i += kAcThreads) {
        const int row = i / (D / 4);
        if (r0 + row >= a.rows) continue;
        const float2 own = row_ml(row);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int u = 0; u < kAcWarps; ++u) {
            const float2 e = ml[u * K::RW + row];
            if (e.y != 0.f) add4(acc, part_weight(e, own.x), *reinterpret_cast<const float4 *>(part + u * K::RW * D + i * 4));
        }
        if constexpr (PREFIX) {
            const int64_t at = ((int64_t)hk * a.rows + r0 + row) * nsplit + split;
            *reinterpret_cast<float4 *>(a.p_o + at * D + (i % (D / 4)) * 4) = acc;
            if (i % (D / 4) == 0) a.p_ml[at] = own;
        } else if (nsplit == 1) {
            finish(row, i, own.x, acc, own.y);
        } else {
            const int to = i / per;
            st_cluster_f4(cluster_map(recv + split * per + (i - to * per), (uint32_t)to), acc);
        }
    }
    if constexpr (!PREFIX) {
        if (nsplit == 1) return;
        for (int j = threadIdx.x; j < K::RW * nsplit; j += kAcThreads) {
            const int row = j % K::RW;
            st_cluster_f2(cluster_map(recv_ml + split * K::RW + row, (uint32_t)(j / K::RW)), row_ml(row));
        }
        cluster_sync();
        for (int i = threadIdx.x; i < per && split * per + i < kAll; i += kAcThreads) {
            const int row = (split * per + i) / (D / 4);
            if (r0 + row >= a.rows) continue;
            float M = -INFINITY, sum = 0.f;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int s = 0; s < kAcMaxCluster; ++s)
                if (s < nsplit) M = fmaxf(M, recv_ml[s * K::RW + row].x);
#pragma unroll
            for (int s = 0; s < kAcMaxCluster; ++s) {
                if (s >= nsplit) break;
                const float2 e = recv_ml[s * K::RW + row];
                if (e.y == 0.f) continue;
                const float f = part_weight(e, M);
                add4(acc, f, recv[s * per + i]);
                sum = fmaf(f, e.y, sum);
            }
            finish(row, split * per + i, M, acc, sum);
        }
    }
}

// Large batches: the streams' lengths differ and only the device knows them, so the tiles of all items
// stand in one list (stream, key head, row group, tile) that the grid's warps share out in equal runs,
// whatever the lengths.  A warp's run covers the end of one item, whole items, the beginning of another;
// it leaves a partial for each in slot (warp + item), which no other pair has: along the
// list both only grow.  attn_join_kernel finds them by the same arithmetic.
// A stream's row groups with a row in use (its first rows, token by token): those of tokens that n_new leaves out read
// nothing (fp32, 77 streams of 1 to 3 tokens of 8 rows in groups of 4: 112 us, 149 with every group).
__device__ __forceinline__ int groups_of(const CachedArgs &a, int b, int rw) {
    return (int)((unsigned)(clamp_new(a, b) * a.G + rw - 1) / (unsigned)rw);
}

// The tiles of all items of the streams before b (`upto`), and of all streams.
__device__ __forceinline__ unsigned tiles_before(const CachedArgs &a, int upto, int tp, int rw, unsigned *total) {
    const int lane = threadIdx.x & 31;
    unsigned before = 0, all = 0;
#pragma unroll 4
    for (int b = lane; b < a.B; b += 32) {
        const unsigned n = (unsigned)tiles_of(a, b, tp) * (unsigned)groups_of(a, b, rw);
        all += n;
        if (b < upto) before += n;
    }
    *total = __reduce_add_sync(0xffffffffu, all) * (unsigned)a.kvh;
    return __reduce_add_sync(0xffffffffu, before) * (unsigned)a.kvh;
}

template <bool Q8, bool F32, int D, int NTX>
__global__ void __launch_bounds__(kAcThreads, AcCfg<Q8, F32, D, NTX>::kMinCtas)
    attn_share_kernel(const CachedArgs a) {
    using K = AcCfg<Q8, F32, D, NTX>;
    constexpr int NT = K::NT;
    extern __shared__ __align__(16) uint8_t sm[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const unsigned wid = blockIdx.x * kAcWarps + warp;
    // A prefix's pass before this one let it start when every CTA of that pass had waited for whatever wrote the inputs: those
    // grids are complete, their results in L2, and the fence keeps what is read from anything older (plain loads and
    // cp.async; none of it is read by non-coherent loads, which a fence does not order).  It needs none of that pass's
    // results, so it runs beside it (its idle SMs, its end) and waits at its own end instead, because attn_join_kernel waits
    // for this kernel alone.  (16384 under 96 x 4 x 32 rows 153 us one after the other, 141 so; 4096 under 64 x 16 35.8 and 33.2.)
    const bool beside = a.splits != 0 || a.wide != 0;
    if (beside)
        __threadfence();
    else
        pdl_wait();
    pdl_launch_dependents();                         // after the wait: see attn_join_kernel
    unsigned total;
    tiles_before(a, 0, K::TP, K::RW, &total);
    Share sh;
    sh.use(total, gridDim.x * kAcWarps);
    unsigned x = sh.first(wid);
    const unsigned x1 = sh.first(wid + 1);
    if (x >= x1) {                                   // more warps than tiles: those behind have none
        if (beside) pdl_wait();
        return;
    }

    // the stream that holds tile x: 32 streams a step, the running sum across the lanes
    int b = 0;
    unsigned s_b = 0;
    for (int b0 = 0; b0 < a.B; b0 += 32) {
        const unsigned n = b0 + lane < a.B ? (unsigned)tiles_of(a, b0 + lane, K::TP) * (unsigned)(groups_of(a, b0 + lane, K::RW) * a.kvh) : 0u;
        unsigned upto = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned v = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += v;
        }
        const uint32_t over = __ballot_sync(0xffffffffu, s_b + upto > x);
        if (over) {
            const int at = __ffs(over) - 1;
            b = b0 + at;
            s_b += __shfl_sync(0xffffffffu, upto - n, at);
            break;
        }
        s_b += __shfl_sync(0xffffffffu, upto, 31);
    }

    WarpPass<Q8, F32, D, NTX, false> w;
    w.init(lane);
    while (x < x1) {
        const unsigned tiles = (unsigned)tiles_of(a, b, K::TP);
        const int groups = groups_of(a, b, K::RW);
        const unsigned of_b = tiles * (unsigned)(groups * a.kvh);
        if (x >= s_b + of_b) {                       // (a stream without tiles, too)
            s_b += of_b;
            ++b;
            continue;
        }
        const int in = (int)((x - s_b) / tiles), tile0 = (int)(x - s_b - in * tiles);
        const int n = (int)min(tiles - tile0, x1 - x);
        const int hk = in / groups, grp = in - hk * groups;
        const int len = clamp_len(a.lengths[b], a.max_len);
        // its own tiles, then a short prefix's (two copies of the pass: a loop around one held 250 bytes a thread in memory)
        const int own = (int)tiles - a.pre_tiles, cut = min(max(own, tile0), tile0 + n);
        if (tile0 < own)
            w.start(a.c, b, hk, len, sm + warp * K::kRing, tile0, cut, 1);
        else
            w.start(a.pc, 0, hk, a.pre_len, sm + warp * K::kRing, tile0 - own, tile0 + n - own, 1);
        w.load_rows(a, b, hk, grp * K::RW, len, clamp_new(a, b));
        if (tile0 >= own) w.see_all(a.pre_len);
        w.run();
        if (tile0 < own && cut < tile0 + n) {
            w.start(a.pc, 0, hk, a.pre_len, sm + warp * K::kRing, cut - own, tile0 + n - own, 1);
            w.see_all(a.pre_len);
            w.run();
        }
        __syncwarp();
        const int64_t slot = (int64_t)b * a.kvh * a.groups + in + wid;   // x only grows: so does the pair
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < w.HC; ++k) {
                const float sum = w.sum_of(nt, k);
                const int r = w.row_of(nt, k);
                const bool mine = w.writes() && grp * K::RW + r < a.rows;
                if (w.g == 0 && mine) a.s_ml[slot * K::RW + r] = make_float2(w.ref[nt][k], sum);
#pragma unroll
                for (int j = 0; j < w.kQuads; ++j) {
                    const float4 v = w.quad(nt, k, j);
                    if (mine) *reinterpret_cast<float4 *>(a.s_o + (slot * K::RW + r) * D + w.dim_of(j)) = v;
                }
            }
        x += n;
    }
    if (beside) pdl_wait();
}

// One output row (stream, token, query head) per WPR warps: its partials from attn_share_kernel
// and from the prefix, weighted to a common reference, added in the order of the list.  blockIdx.x: the stream, whose
// place in the lists a warp works out once; blockIdx.y: its share of the stream's rows in use.
constexpr int kJoinWarps = 8;
constexpr int join_warps(int wpr) { return wpr == 1 ? 4 : kJoinWarps; }   // small CTAs find room while attn_share_kernel ends
// WPR 8: few rows of many partials.  WPR 1: a warp a row, BATCH partials in flight: 8 where the rows are few and the time is a
// chain of loads, 4 (half the registers) where they are many.  (64 x 16 rows: 34.2 us a call against 36; 96 x 4 x 32: 143
// against 137.)
template <bool F32, int D, int WPR, int BATCH>
__global__ void __launch_bounds__(join_warps(WPR) * 32, WPR > 1 ? 2 : BATCH == 8 ? 4 : 8) attn_join_kernel(const CachedArgs a, int rw, int tp, unsigned warps) {
    constexpr int JW = join_warps(WPR);
    __shared__ float4 s_acc[JW][32];
    __shared__ float2 s_ml[JW];
    constexpr int LPR = D / 4;                      // lanes of a row's float4s
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, part = warp % WPR;
    // lengths and n_new may be read before the wait: attn_share_kernel lets this kernel start only after
    // its own wait for whatever wrote them, or that of the prefix's pass
    const int b = blockIdx.x, nn = clamp_new(a, b), tiles = tiles_of(a, b, tp);
    unsigned total;
    const unsigned s_b = tiles_before(a, b, tp, rw, &total);
    const int groups = groups_of(a, b, rw);
    Share sh, ws;
    sh.use(total, warps);
    int rows_all = 0, cr0 = 0;
    if (a.wide) cr0 = wide_rows(a, b, &rows_all);
    const WideItems items(rows_all);
    if (a.wide) items.share(a, &ws);
    const int used = nn * a.G, n_rows = a.kvh * used;    // of the stream, key head by key head
    constexpr int kRows = JW / WPR;                 // rows of a CTA's turn
    struct Place {
        int row, hk, r, own, all, subs, sub, cr, in_grp;
        int64_t slot0, p_at, rec0;
    };
    auto place = [&](int i0) {
        Place p;
        p.row = i0 + warp / WPR;
        const int at = min(p.row, n_rows - 1);
        p.hk = at / used, p.r = at - p.hk * used;
        const int grp = p.r / rw, in = p.hk * groups + grp;
        p.in_grp = p.r - grp * rw;
        const unsigned x = s_b + in * tiles;
        const unsigned w0 = tiles ? sh.owner(x) : 0u;
        p.own = tiles ? (int)(sh.owner(x + tiles - 1) + 1 - w0) : 0;
        p.slot0 = (int64_t)b * a.kvh * a.groups + in + w0;
        p.p_at = (((int64_t)p.hk * a.B + b) * a.rows + p.r) * a.splits;
        // the prefix's partials: `splits` of them, or the records of attn_prefix_tc_kernel
        int n_pre = a.splits;
        p.subs = 1, p.sub = 0, p.rec0 = 0, p.cr = cr0 + p.r;
        if (a.wide) {
            const int tile = p.cr / kWideRows, item = items.pairs ? p.hk * items.pairs + tile / 2 : p.hk;
            const unsigned c0 = (unsigned)(item * a.wide_chunks), o0 = ws.owner(c0);
            if (items.pairs)
                p.sub = tile & 1;
            else
                p.subs = 2;
            n_pre = (int)(ws.owner(c0 + a.wide_chunks - 1) + 1 - o0) * p.subs;
            p.rec0 = 2 * ((int64_t)o0 + item);
        }
        p.all = p.own + n_pre;
        return p;
    };
    Place p = {};
    if ((int)blockIdx.y * kRows < n_rows) p = place(blockIdx.y * kRows);
    pdl_wait();                                     // the partials are written

    for (int i0 = blockIdx.y * kRows; i0 < n_rows;) {
        // 32 / LPR partials at a time (one for head_dim 128), LPR lanes each; kBatch of those are loaded
        // together, (ref, sum) with their rows, then weighted to the running reference
        constexpr int kBatch = BATCH, kStep = WPR * (32 / LPR);
        const int d = (lane % LPR) * 4;
        float M = -INFINITY, sum = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int j0 = part * (32 / LPR) + lane / LPR; j0 - lane / LPR < p.all; j0 += kBatch * kStep) {
            float2 e[kBatch];
            float4 v[kBatch];
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                const int i = j0 + j * kStep;
                e[j] = make_float2(-INFINITY, 0.f);
                v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (i < p.own) {
                    const int64_t at = (p.slot0 + i) * rw + p.in_grp;
                    e[j] = a.s_ml[at];
                    v[j] = *reinterpret_cast<const float4 *>(a.s_o + at * D + d);
                } else if (i < p.all) {
                    const int k = i - p.own;
                    const int64_t at = !a.wide ? p.p_at + k
                                               : (p.rec0 + (p.subs == 2 ? k : 2 * k + p.sub)) * kWideRows + p.cr % kWideRows;
                    e[j] = a.p_ml[at];
                    v[j] = *reinterpret_cast<const float4 *>(a.p_o + at * D + d);
                }
            }
            float now = M;
#pragma unroll
            for (int j = 0; j < kBatch; ++j) now = fmaxf(now, e[j].x);
            const float keep = part_weight(make_float2(M, sum), now);
            acc.x *= keep, acc.y *= keep, acc.z *= keep, acc.w *= keep;
            sum *= keep;
            M = now;
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                if (e[j].y == 0.f) continue;
                const float f = part_weight(e[j], M);
                add4(acc, f, v[j]);
                sum = fmaf(f, e[j].y, sum);
            }
        }
        // the lanes' and the warps' own references meet
        if constexpr (LPR == 16) {
            const float now = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, 16));
            const float f = part_weight(make_float2(M, sum), now);
            acc.x *= f, acc.y *= f, acc.z *= f, acc.w *= f;
            sum *= f;
            M = now;
        }
        if constexpr (LPR == 16) {
            acc.x += __shfl_xor_sync(0xffffffffu, acc.x, 16), acc.y += __shfl_xor_sync(0xffffffffu, acc.y, 16);
            acc.z += __shfl_xor_sync(0xffffffffu, acc.z, 16), acc.w += __shfl_xor_sync(0xffffffffu, acc.w, 16);
            sum += __shfl_xor_sync(0xffffffffu, sum, 16);
        }
        if constexpr (WPR > 1) {
            s_acc[warp][lane] = acc;
            if (lane == 0) s_ml[warp] = make_float2(M, sum);
            __syncthreads();
            const int w1 = warp - part;                 // this row's first warp
#pragma unroll
            for (int i = 0; i < WPR; ++i) M = fmaxf(M, s_ml[w1 + i].x);
            acc = make_float4(0.f, 0.f, 0.f, 0.f), sum = 0.f;
#pragma unroll
            for (int i = 0; i < WPR; ++i) {
                const float2 e = s_ml[w1 + i];
                if (e.y == 0.f) continue;
                const float f = part_weight(e, M);
                add4(acc, f, s_acc[w1 + i][lane]);
                sum = fmaf(f, e.y, sum);
            }
            __syncthreads();                            // before the next turn's
        }
        if (p.row < n_rows && part == 0 && lane < LPR) {
            const int tt = p.r / a.G;
            store4<F32>(a.out + b * a.o_stream + tt * a.o_token + ((int64_t)(p.hk * a.G + (p.r - tt * a.G)) * D + d) * (F32 ? 4 : 2),
                        acc, sum == 0.f ? 0.f : 1.f / sum);
        }
        i0 += gridDim.y * kRows;
        if (i0 < n_rows) p = place(i0);
    }
}

// ------------------------------------------------------------------------- launches

// CTAs that share the prefix's positions, per key head and row group.
int prefix_splits(int rows, int kvh, int prefix_len, int rw, int tp, int sms) {
    const int groups = (rows + rw - 1) / rw;
    const int tiles = (prefix_len + tp - 1) / tp;
    const int most = std::max(1, tiles / (2 * kAcWarps));
    const int want = std::max(1, 4 * sms / std::max(1, groups * kvh));
    return std::max(1, std::min(std::min(most, want), 32));
}

enum : int { kPassCluster = 0, kPassPrefix = 1, kPassShare = 2 };

// Shared-memory limit set and resident CTAs per SM (0: not yet) of a variant, looked up once per device.  Host threads
// whose first calls meet look it up twice; none sees the one without the other.
using Ready = std::atomic<int>;
template <typename F> cudaError_t make_ready(Ready *r, F fn, int smem) {
    if (r->load(std::memory_order_acquire)) return cudaSuccess;
    int per_sm = 0;
    cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void *>(fn), cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, fn, kAcThreads, smem);
    if (e != cudaSuccess) return e;
    if (per_sm < 1) return cudaErrorInvalidConfiguration;
    r->store(per_sm, std::memory_order_release);
    return cudaSuccess;
}

template <typename F, typename... A>
cudaError_t launch_ex(F fn, dim3 grid, int threads, int smem, unsigned cluster, cudaStream_t s, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    int n = 0;
    if (cluster > 1) {
        at[n].id = cudaLaunchAttributeClusterDimension;
        at[n].val.clusterDim.x = cluster;
        at[n].val.clusterDim.y = at[n].val.clusterDim.z = 1;
        ++n;
    }
    // every kernel here waits for its predecessor (griddepcontrol.wait) before it reads or writes memory,
    // so its CTAs may be placed while that one ends
    at[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
    cfg.attrs = at;
    cfg.numAttrs = (unsigned)n;
    return cudaLaunchKernelEx(&cfg, fn, args...);
}

// kind Cluster or Prefix: `ctas` of clusters of nsplit; kind Share: every CTA the SMs hold, *ctas says how many.  `plan`: only *ctas,
// for Cluster the CTAs that an SM holds, three at most.
template <bool Q8, bool F32, int D, int NTX>
cudaError_t launch(int kind, const CachedArgs &a, unsigned *ctas, int nsplit, int dev, cudaStream_t s, bool plan) {
    using K = AcCfg<Q8, F32, D, NTX>;
    static Ready ready[3][64] = {};
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    cudaError_t e;
    if (kind == kPassShare) {
        auto fn = attn_share_kernel<Q8, F32, D, NTX>;
        if ((e = make_ready(&ready[kind][dev], fn, K::kSmem)) != cudaSuccess) return e;
        *ctas = (unsigned)(ready[kind][dev].load(std::memory_order_acquire) * sms_of(dev));
        return plan ? cudaSuccess : launch_ex(fn, *ctas, kAcThreads, K::kSmem, 1, s, a);
    }
    if (kind == kPassPrefix) {
        auto fn = attn_cached_kernel<Q8, F32, D, NTX, true>;
        if ((e = make_ready(&ready[kind][dev], fn, K::kSmem)) != cudaSuccess) return e;
        return launch_ex(fn, *ctas, kAcThreads, K::kSmem, 1, s, a, nsplit);
    }
    if (plan) {
        *ctas = (unsigned)std::min(3, K::kMinCtas);
        return cudaSuccess;
    }
    auto fn = attn_cached_kernel<Q8, F32, D, NTX, false>;
    const int smem = nsplit > 1 ? K::kSmemCluster : K::kSmem;
    if ((e = make_ready(&ready[kind][dev], fn, K::kSmemCluster)) != cudaSuccess) return e;
    return launch_ex(fn, *ctas, kAcThreads, smem, (unsigned)nsplit, s, a, nsplit);
}

// Up to here (tiles that the streams would read between them) a prefix is read by every stream's own pass: a launch and
// a pipeline's start less, where its positions cost little (64 streams, one token each, 8-bit: 1024 positions, 16384 tiles, 28 us
// against 30 on the tcgen05 cores; 1536, 24576 tiles, 34 against 30; bf16: 512, 16384 tiles, 25 against 30; 1024, 32768 tiles, 36
// against 32).
constexpr int64_t kInlineTiles = 20000;

// Rows from which the prefix goes to the tcgen05 cores (16000 8-bit positions under 32, 48 and 96 rows of 8 key heads: 37.3, 37.3 and
// 39.1 us there, 37.3, 39.0 and 53.1 a few rows at a time; 8000 bf16 positions under 16, 48 and 96 rows: 21.6, 26.1 and 29.6
// there, 28.2, 31.2 and 43.1).  Not before, although bf16 prefixes would gain: fewer rows keep the finer spacing of faint weights over 8-bit
// rows (2^-35 of the largest, 2^-27 there), and the limit is one for both formats.
constexpr int kWideFrom = 48;

constexpr int tile_positions(bool q8, int d) { return q8 || d == 64 ? 32 : 16; }   // AcCfg::TP
// Column tiles (AcCfg's NTX) for `rows` rows of an item, and the rows that they hold.
int column_tiles(bool q8, bool f32, int d, int64_t rows, int *rw) {
    const int per = 8 / (q8 ? (f32 ? 2 : 1) : (f32 ? 4 : 2));   // rows of a tile
    int nt = rows > per ? 2 : 1;
    *rw = per * nt;
    // more tiles, where their sums fit the registers (head_dim 64), or one column where two were; four tiles of 128 kept 230
    // bytes a thread in memory (fp32 rows, bf16 cache, 66 streams of 12 rows: 92 us against 74 on two, which read it three times)
    if (d == 64 && rows > *rw && (f32 || !q8) && rows > (f32 ? *rw : 16))
        nt = f32 ? 4 : kOneColumn + 4, *rw = f32 ? per * 4 : 32;
    else if (!f32 && !q8 && rows > *rw)
        nt = kOneColumn + 2, *rw = 16;
    return nt;
}

cudaError_t dispatch(int kind, bool q8, bool f32, int d, int nt, const CachedArgs &a, unsigned *ctas, int nsplit, int dev,
                     cudaStream_t s, bool plan = false) {
#define QD_AC(Q, F, DD, N) \
    if (q8 == Q && f32 == F && d == DD && nt == (N)) return launch<Q, F, DD, (N)>(kind, a, ctas, nsplit, dev, s, plan);
#define QD_AC2(Q, F) QD_AC(Q, F, 64, 1) QD_AC(Q, F, 64, 2) QD_AC(Q, F, 128, 1) QD_AC(Q, F, 128, 2)
    QD_AC2(false, false) QD_AC2(false, true) QD_AC2(true, false) QD_AC2(true, true)
    QD_AC(false, false, 64, kOneColumn + 2) QD_AC(false, false, 128, kOneColumn + 2)
    QD_AC(false, false, 64, kOneColumn + 4) QD_AC(false, true, 64, 4) QD_AC(true, true, 64, 4)
#undef QD_AC2
#undef QD_AC
    return cudaErrorInvalidValue;
}

cudaError_t launch_join(bool f32, int d, const CachedArgs &a, int rw, int tp, unsigned warps, bool many, int sms, cudaStream_t s) {
    // about eight CTAs per SM, two waves: the stream's place is worked out once for a few turns
    const int wpr = many ? kJoinWarps : 1, jw = join_warps(wpr), turns = (a.kvh * a.rows * wpr + jw - 1) / jw;
    const dim3 grid((unsigned)a.B, (unsigned)std::min({turns, std::max(1, 64 / jw * sms / a.B), 65535}));
    const int batch = many || (int64_t)a.B * a.kvh * a.rows <= 4096 ? 8 : 4;
#define QD_JOIN(F, DD, W, N) \
    if (f32 == F && d == DD && wpr == W && batch == N) \
        return launch_ex(attn_join_kernel<F, DD, W, N>, grid, jw * 32, 0, 1, s, a, rw, tp, warps);
#define QD_JOIN2(F, DD) QD_JOIN(F, DD, 1, 4) QD_JOIN(F, DD, 1, 8) QD_JOIN(F, DD, kJoinWarps, 8)
    QD_JOIN2(false, 64) QD_JOIN2(false, 128) QD_JOIN2(true, 64) QD_JOIN2(true, 128)
#undef QD_JOIN2
#undef QD_JOIN
    return cudaErrorInvalidValue;
}

// How a call runs, from its sizes alone.
struct Plan {
    int nt, rw, groups, tp;             // own caches: row tiles, rows per CTA, row groups, positions of a tile
    int nsplit;                         // CTAs of a cluster (one cluster per item); 0: shared out
    unsigned ctas;                      // of the shared-out pass
    int64_t rows_all;
    bool inline_prefix;                 // a short prefix: every stream's own pass reads it
    int p_nt, p_rw, p_groups, splits;   // else a few rows of the batch at a time
    int wide;                           // or its CTAs on the tcgen05 cores
    size_t p_ml, p_o, s_ml, s_o, bytes; // workspace offsets
};

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

qd_status make_plan(const qd_kv_cache *cache, const qd_kv_cache *prefix, int prefix_length, bool f32, int T, int QH,
                    int max_length, int dev, Plan *p) {
    *p = {};
    const int kvh = cache->n_kv_heads, d = cache->head_dim, B = cache->n_streams, G = QH / kvh;
    const int sms = sms_of(dev);
    const bool q8 = cache->format == QD_KV_Q8;
    const int rows = T * G;
    p->rows_all = (int64_t)rows * B;
    p->nt = column_tiles(q8, f32, d, rows, &p->rw), p->groups = (rows + p->rw - 1) / p->rw;
    const int64_t items = (int64_t)B * kvh * p->groups;
    p->tp = tile_positions(q8, d);
    int tiles = (max_length + p->tp - 1) / p->tp;
    if (prefix && prefix_length > 0 && prefix->format == cache->format) {
        const int64_t pre = (prefix_length + p->tp - 1) / p->tp;
        const int64_t own = items * pre;
        if (f32 || p->rows_all < kWideFrom)
            p->inline_prefix = own <= (p->rows_all + p->rw - 1) / p->rw * kvh * pre + kInlineTiles;
        else
            p->inline_prefix = own <= kInlineTiles;
        if (p->inline_prefix) tiles += (int)pre;
    }
    if (items * tiles > (1ll << 30)) return QD_EUNSUPPORTED;
    // A cluster per item while the grid is one wave, or little more, and a warp's share short; longer or larger batches are
    // shared out.  (72 items, a short prefix: 576 CTAs 13.8 us, 288 10.2; 592 items of one CTA 14.6 us, shared out 18.)
    // The wave is what the SMs hold of this variant (two CTAs of bf16 rows of 64, whose ring is as large as that of 128: 160 items
    // of up to 700 positions in clusters of two, as if there were room for three, 8.4 us, one CTA each 7.6); the little more goes by the work
    // of an item (560 items of up to 200 or 700 of those positions, nearly two waves, 8.5 and 13.9 us, shared out 9.6 and 14.2).
    const CachedArgs none = {};
    unsigned per_sm = 0;
    if (dispatch(kPassCluster, q8, f32, d, p->nt, none, &per_sm, 0, dev, nullptr, true) != cudaSuccess) return QD_ECUDA;
    const int wave = (int)per_sm * sms;
    const int most = (d == 128 && (!q8 || p->nt == 2)) || (p->nt & 7) == 4 ? wave + wave / 3 : 4 * sms;
    p->nsplit = 1;
    while (p->nsplit < kAcMaxCluster && items * p->nsplit * 2 <= wave && tiles > p->nsplit * kAcWarps) p->nsplit *= 2;
    if (items * p->nsplit > most || tiles > 8 * p->nsplit * kAcWarps) p->nsplit = 0;
    size_t at = 0;
    if (prefix && prefix_length > 0 && !p->inline_prefix) {
        const bool pq8 = prefix->format == QD_KV_Q8;
        if (!f32 && p->rows_all >= kWideFrom) {
            p->wide = sms, p->nsplit = 0;
            const int64_t tiles = (p->rows_all + kWideRows - 1) / kWideRows, items = kvh * ((tiles + 1) / 2);
            const int64_t chunks = (prefix_length + kWideKeys - 1) / kWideKeys;
            if (items * chunks > (1ll << 30)) return QD_EUNSUPPORTED;
            const size_t recs = 2 * (size_t)(p->wide + items);
            p->p_ml = at, at = up256(at + recs * kWideRows * 8);
            p->p_o = at, at = up256(at + recs * kWideRows * d * 4);
        } else {
            p->p_nt = column_tiles(pq8, f32, d, p->rows_all, &p->p_rw);
            p->p_groups = (int)((p->rows_all + p->p_rw - 1) / p->p_rw);
            p->splits = prefix_splits((int)p->rows_all, kvh, prefix_length, p->p_rw, tile_positions(pq8, d), sms);
            p->p_ml = at, at = up256(at + (size_t)kvh * p->rows_all * p->splits * 8);
            p->p_o = at, at = up256(at + (size_t)kvh * p->rows_all * p->splits * d * 4);
        }
    }
    if (!p->nsplit) {
        if (dispatch(kPassShare, q8, f32, d, p->nt, none, &p->ctas, 0, dev, nullptr, true) != cudaSuccess) return QD_ECUDA;
        const size_t slots = (size_t)items + (size_t)p->ctas * kAcWarps;
        p->s_ml = at, at = up256(at + slots * p->rw * 8);
        p->s_o = at, at = up256(at + slots * p->rw * d * 4);
    }
    p->bytes = at;
    return QD_OK;
}

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
    if ((st = make_plan(cache, prefix, prefix_length, dtype == QD_F32, n_tokens, n_q_heads, max_length, dev, &p)) != QD_OK)
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
    // out's rows must lie neither over each other nor over q's
    const int64_t row = (int64_t)n_q_heads * cache->head_dim, B64 = cache->n_streams;
    const bool alike = (n_tokens == 1 || q_token_stride == out_token_stride) && (B64 == 1 || q_stream_stride == out_stream_stride);
    if (q_dev == out_dev || !apart(e, row, {{n_tokens, out_token_stride}, {B64, out_stream_stride}}, alike ? bytes_between(q_dev, out_dev) : 0))
        return QD_EINVAL;
    if (!alike) {                                    // rows of two layouts: not in the same stretch of memory
        const uintptr_t q0 = reinterpret_cast<uintptr_t>(q_dev), o0 = reinterpret_cast<uintptr_t>(out_dev);
        const uintptr_t q1 = ((uintptr_t)(n_tokens - 1) * q_token_stride + (uintptr_t)(B64 - 1) * q_stream_stride + row) * e;
        const uintptr_t o1 = ((uintptr_t)(n_tokens - 1) * out_token_stride + (uintptr_t)(B64 - 1) * out_stream_stride + row) * e;
        if (q0 < o0 ? o0 - q0 < q1 : q0 - o0 < o1) return QD_EINVAL;
    }
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return QD_ECUDA;
    if ((st = check_cache(cache, dev, false)) != QD_OK) return st;
    if (with_prefix && (st = check_cache(prefix, dev, true)) != QD_OK) return st;
    if (!on_device(q_dev, dev) || !on_device(out_dev, dev) || !on_device(lengths_dev, dev) ||
        (n_new_dev && !on_device(n_new_dev, dev)))
        return QD_EINVAL;
    Plan p;
    if ((st = make_plan(cache, prefix, prefix_length, f32, n_tokens, n_q_heads, max_length, dev, &p)) != QD_OK) return st;
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
        } else if (dispatch(kPassPrefix, prefix->format == QD_KV_Q8, f32, d, p.p_nt, x, &ctas, p.splits, dev, s) != cudaSuccess)
            return QD_ECUDA;
    }
    const bool q8 = cache->format == QD_KV_Q8;
    a.c = kv_view(cache);
    a.rows = n_tokens * a.G, a.groups = p.groups, a.max_len = max_length;
    if (p.nsplit) {
        unsigned ctas = (unsigned)((int64_t)B * kvh * p.groups * p.nsplit);
        return dispatch(kPassCluster, q8, f32, d, p.nt, a, &ctas, p.nsplit, dev, s) == cudaSuccess ? QD_OK : QD_ECUDA;
    }
    a.s_ml = reinterpret_cast<float2 *>(ws + p.s_ml), a.s_o = reinterpret_cast<float *>(ws + p.s_o);
    if (dispatch(kPassShare, q8, f32, d, p.nt, a, &p.ctas, 0, dev, s) != cudaSuccess) return QD_ECUDA;
    // many partials a row (long streams, few of them): several warps per row
    const unsigned warps = p.ctas * kAcWarps, items = (unsigned)((int64_t)B * kvh * p.groups);
    return launch_join(f32, d, a, p.rw, p.tp, warps, warps / items + p.splits > 16, sms_of(dev), s) == cudaSuccess ? QD_OK : QD_ECUDA;
}

}  // extern "C"
