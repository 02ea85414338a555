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
// Decoding has few rows and many positions, so the positions are the long side (M = 16) of m16n8k16
// and the rows its N = 8 columns.  Where a value must keep more bits than the tensor
// core's type has, it takes C columns, one per part (q and p alike; the parts' products
// are added afterwards): 8-bit cache, fp16: bf16 rows 1 part, fp32 rows 2; bf16 cache: 2
// parts (hi, lo of p), fp32 rows 3 of 4 columns.
//
// Neither K nor V passes through a layout in shared memory.  The products' sums run over
// head_dim (scores) and positions (output) in any order, so each lane takes 16 contiguous bytes of a row as its
// share of the A fragment, and q is laid out to match.  For the output, V^T is A:
// a lane holds the same dims of the four positions its fragment pairs, and a byte
// permutation pairs them up, the same that widens the codes.  The probabilities turn
// from the accumulator's layout into the B fragment's with movmatrix.  Each lane reads only what it
// copied itself (cp.async, 16 bytes), so the ring of tiles needs no barrier: it serves as
// registers that the loads in flight do not occupy.
//
// A cluster of CTAs shares one (stream, key head, rows) item; its warps take the 16-position
// tiles in turn and their partial results (ref, sum, output) meet in distributed shared
// memory, in a fixed order.  Nothing is kept in global memory but the prefix's partials.
#include <cuda_fp16.h>

#include "kv_view.cuh"
#include "mma_sync.cuh"
#include "qd_device.cuh"
#include "qd_internal.h"

namespace qd {

namespace {

constexpr int kAcWarps = 4, kAcThreads = kAcWarps * 32;
constexpr int kAcStages = 3;
constexpr int kAcTile = 16;                 // positions per warp and step
constexpr int kAcMaxCluster = 8;
constexpr int kAcMaxTokens = 64;
// Probabilities stand 2^10 above 1 at the running maximum and may grow to 2^15 before the
// sums are rescaled: fp16 then keeps 11 (two parts: 22) bits of every weight down to 2^-24
// (2^-10) of the largest, and small moves of the maximum cost nothing.
constexpr float kAcUp = 10.f, kAcRoom = 15.f;

struct CachedArgs {
    KvView c;
    const uint8_t *q;
    uint8_t *out;
    int64_t q_stream, q_token, o_stream, o_token;   // bytes
    const int32_t *lengths, *n_new;
    int T, G, kvh, groups, max_len;
    int rows;                                       // rows of an item: T G, of the prefix B T G
    float scale2;                                   // softmax scale times log2(e)
    // partials over the prefix: [kvh][B T G][splits]
    float2 *p_ml;
    float *p_o;
    int splits;
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float lg2(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool live) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp8(uint32_t dst, const void *src, bool live) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(live ? 8 : 0) : "memory");
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
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ float f16_of(float x) { return __half2float(__float2half_rn(x)); }
__device__ __forceinline__ float bf16_of(float x) { return __bfloat162float(__float2bfloat16_rn(x)); }

// Two code bytes (offset by 128) under the exponent of 1024: 1024 + u, less 1152 = code, exactly.
__device__ __forceinline__ uint32_t codes_f16(uint32_t y, uint32_t sel) {
    const uint32_t h = __byte_perm(y, 0x64646464u, sel);
    const __half2 v = __hsub2(*reinterpret_cast<const __half2 *>(&h), __half2half2(__ushort_as_half(0x6480)));
    return *reinterpret_cast<const uint32_t *>(&v);
}

template <bool Q8, bool F32, int D, int NT> struct AcCfg {
    static constexpr int C = Q8 ? (F32 ? 2 : 1) : (F32 ? 4 : 2);   // columns per row
    static constexpr int RW = 8 * NT / C;                          // rows per CTA
    static constexpr int ES = Q8 ? 1 : 2;
    static constexpr int KP = D * ES / 64;                         // 16-byte pieces of a K row per lane
    static constexpr int KW = Q8 ? 4 : 2;                          // k-steps per piece
    static constexpr int KS = D / 16, MT = D / 16;
    static constexpr int VB = D * ES / 8 < 16 ? D * ES / 8 : 16;   // bytes of a V access (8 or 16)
    static constexpr int VP = D * ES / 8 / VB;                     // V accesses per position and lane
    static constexpr int kV = 2 * KP * 512;                        // byte offset of V in a tile
    static constexpr int kS = kV + 4 * VP * VB * 32;               // of the scales
    static constexpr int kTileBytes = kS + (Q8 ? 128 : 0);
    static constexpr int kRing = kAcStages * kTileBytes;           // per warp
    // after the pass the rings' space holds the warps' partials, then the CTA's
    static constexpr int kPart = kAcWarps * RW * D * 4;
    static constexpr int kMl = kPart + RW * D * 4;
    static constexpr int kEnd = kMl + (kAcWarps + 1) * RW * 8;
    static constexpr int kSmem = kAcWarps * kRing > kEnd ? kAcWarps * kRing : kEnd;
};

// (ref, sum) of one partial: its weight against the reference M
__device__ __forceinline__ float part_weight(float2 ml, float M) { return ml.y == 0.f ? 0.f : ex2(ml.x - M); }

__device__ __forceinline__ float2 ld_cluster_f2(uint32_t addr) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

// PREFIX: the rows of every stream over the shared prefix, partials to global memory.
// Otherwise: a stream's rows over its own cache; joins the prefix's partials and writes
// the output.  blockIdx.x = item * splits + split.
template <bool Q8, bool F32, int D, int NT, bool PREFIX>
__global__ void __launch_bounds__(kAcThreads, NT == 1 ? 4 : 3) attn_cached_kernel(const CachedArgs a, int nsplit) {
    using K = AcCfg<Q8, F32, D, NT>;
    constexpr int C = K::C, HC = C == 1 ? 2 : 1;
    extern __shared__ __align__(16) uint8_t sm[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int split = blockIdx.x % nsplit, item = blockIdx.x / nsplit;
    const int grp = item % a.groups, hk = (item / a.groups) % a.kvh, b = PREFIX ? 0 : item / a.groups / a.kvh;

    int len = a.max_len, nn = a.T;
    if constexpr (!PREFIX) {
        len = a.lengths[b];
        len = len < 0 ? 0 : len > a.max_len ? a.max_len : len;
        nn = a.n_new ? a.n_new[b] : a.T;
        nn = nn < 0 ? 0 : nn > a.T ? a.T : nn;
    }
    const int r0 = grp * K::RW;

    // ---- this item's rows as the B fragments of the scores: column 8 nt + g holds part
    // (column % C) of row r0 + column / C; q scaled by a power of two per row for fp16
    uint32_t qf[NT][K::KS][2];
    float cs_g[NT];
    int lim_g[NT];
    int lim_lo = INT32_MAX, lim_hi = 0;             // over this item's rows
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int col = 8 * nt + g, r = r0 + col / C, part = col % C;
        int bb = b, rr = r;
        if constexpr (PREFIX) {
            bb = r / (a.T * a.G);
            rr = r - bb * (a.T * a.G);
        }
        const int tt = rr / a.G, gg = rr - tt * a.G;
        const bool live = r < a.rows && (PREFIX || tt < nn);
        const uint8_t *src = a.q + bb * a.q_stream + tt * a.q_token + (int64_t)(hk * a.G + gg) * D * (F32 ? 4 : 2);
        constexpr int E = 16 / K::ES;               // dims of a piece
        float x[K::KP * E];
#pragma unroll
        for (int i = 0; i < K::KP; ++i)
#pragma unroll
            for (int e = 0; e < E; e += F32 ? 4 : 8) {
                const int d = i * 4 * E + t * E + e;
                uint4 u = make_uint4(0, 0, 0, 0);
                if (live) u = __ldg(reinterpret_cast<const uint4 *>(src + d * (F32 ? 4 : 2)));
                if constexpr (F32)
                    Elem<float>::unpack(u, x + i * E + e);
                else
                    Elem<__nv_bfloat16>::unpack(u, x + i * E + e);
            }
        float cs = a.scale2;
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
            cs *= __uint_as_float((uint32_t)(254 - up) << 23);
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
            }
        cs_g[nt] = cs;
        lim_g[nt] = !live ? 0 : PREFIX ? len : max(0, len - (nn - 1 - tt));
        lim_lo = min(lim_lo, __reduce_min_sync(0xffffffffu, live ? lim_g[nt] : INT32_MAX));
        lim_hi = max(lim_hi, __reduce_max_sync(0xffffffffu, lim_g[nt]));
    }
    // the columns of this lane's accumulators
    float cs[NT][2];
    int lim[NT][HC];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int k = 0; k < 2; ++k) cs[nt][k] = __shfl_sync(0xffffffffu, cs_g[nt], (2 * t + k) * 4);
#pragma unroll
        for (int k = 0; k < HC; ++k) lim[nt][k] = __shfl_sync(0xffffffffu, lim_g[nt], (2 * t + k) * 4);
    }
    const int n_pos = lim_hi;                       // positions that any row sees
    const int n_tiles = (n_pos + kAcTile - 1) / kAcTile;

    const uint8_t *kb = a.c.k + (PREFIX ? 0 : b * a.c.stream) + hk * a.c.head;
    const uint8_t *vb = a.c.v + (PREFIX ? 0 : b * a.c.stream) + hk * a.c.head;
    const float *ksb = Q8 ? a.c.ks + (PREFIX ? 0 : b * a.c.sstream) + hk * a.c.shead : nullptr;
    const float *vsb = Q8 ? a.c.vs + (PREFIX ? 0 : b * a.c.sstream) + hk * a.c.shead : nullptr;
    uint8_t *ring = sm + warp * K::kRing;
    const uint32_t ring_s = smem_addr(ring);

    // copy this lane's share of the tile into its stage; positions past n_pos become zeros
    auto fetch = [&](int tile, int stage) {
        const int p0 = tile * kAcTile;
        const uint32_t dst = ring_s + stage * K::kTileBytes;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int p = p0 + g + 8 * h;
            const bool live = p < n_pos;
            const uint8_t *src = kb + (int64_t)(live ? p : 0) * a.c.row + t * 16;
#pragma unroll
            for (int i = 0; i < K::KP; ++i) cp16(dst + (h * K::KP + i) * 512 + lane * 16, src + 64 * i, live);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int p = p0 + 2 * t + (i & 1) + 8 * (i >> 1);
            const bool live = p < n_pos;
            const uint8_t *src = vb + (int64_t)(live ? p : 0) * a.c.row + g * K::VB;
#pragma unroll
            for (int j = 0; j < K::VP; ++j) {
                const uint32_t d = dst + K::kV + (i * K::VP + j) * (32 * K::VB) + lane * K::VB;
                if constexpr (K::VB == 16)
                    cp16(d, src + 128 * j, live);
                else
                    cp8(d, src, live);
            }
        }
        if constexpr (Q8) {
            const int p = p0 + (lane & 15);
            const bool live = p < n_pos;
            cp4(dst + K::kS + lane * 4, (lane < 16 ? ksb : vsb) + (live ? p : 0), live);
        }
    };

    float o[K::MT][NT][4];
#pragma unroll
    for (int mt = 0; mt < K::MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[mt][nt][e] = 0.f;
    float ref[NT][HC], l[NT][HC];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < HC; ++k) ref[nt][k] = -INFINITY, l[nt][k] = 0.f;

    const int step = nsplit * kAcWarps;
    int next = split * kAcWarps + warp;             // tile to fetch
#pragma unroll
    for (int s = 0; s < kAcStages - 1; ++s) {
        if (next < n_tiles) fetch(next, s);
        cp_commit();
        next += step;
    }
    int stage = 0;
    for (int tile = split * kAcWarps + warp; tile < n_tiles; tile += step) {
        {
            const int into = stage == 0 ? kAcStages - 1 : stage - 1;
            if (next < n_tiles) fetch(next, into);
            cp_commit();
            next += step;
        }
        cp_wait<kAcStages - 1>();
        __syncwarp();                               // the scales come from other lanes
        const uint8_t *st = ring + stage * K::kTileBytes;
        const int p0 = tile * kAcTile;

        // ---- scores: rows (positions) g and g + 8, columns 2t and 2t + 1
        float s[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
#pragma unroll
        for (int i = 0; i < K::KP; ++i) {
            const uint4 ua = *reinterpret_cast<const uint4 *>(st + i * 512 + lane * 16);
            const uint4 ub = *reinterpret_cast<const uint4 *>(st + (K::KP + i) * 512 + lane * 16);
            const uint32_t wa[4] = {ua.x, ua.y, ua.z, ua.w}, wb[4] = {ub.x, ub.y, ub.z, ub.w};
#pragma unroll
            for (int w = 0; w < K::KW; ++w) {
                uint32_t f[4];
                if constexpr (Q8) {
                    const uint32_t xa = wa[w] ^ 0x80808080u, xb = wb[w] ^ 0x80808080u;
                    f[0] = codes_f16(xa, 0x4140), f[1] = codes_f16(xb, 0x4140);
                    f[2] = codes_f16(xa, 0x4342), f[3] = codes_f16(xb, 0x4342);
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

        // ---- scores in log2 units, the mask, and z = s + log2(values' scale), which bounds
        // the weight that enters the product
        float kd[2] = {1.f, 1.f}, vd[2] = {1.f, 1.f}, vl[2] = {0.f, 0.f};
        if constexpr (Q8) {
            const float *sc = reinterpret_cast<const float *>(st + K::kS);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                kd[h] = sc[g + 8 * h], vd[h] = sc[16 + g + 8 * h];
                vl[h] = fmaxf(lg2(vd[h]), -60.f);   // a row of zeros does not move the reference
            }
        }
        float x[NT][2][HC];
        bool over = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int p = p0 + g + 8 * h;
#pragma unroll
                for (int k = 0; k < HC; ++k) {
                    float v = s[nt][2 * h + k];
                    if constexpr (F32) v += s[nt][2 * h + 1];   // bf16 q has one part
                    if constexpr (C == 4) v += __shfl_xor_sync(0xffffffffu, v, 1);
                    v *= cs[nt][k];
                    if constexpr (Q8) v *= kd[h];
                    v = p < lim[nt][k] ? v : -INFINITY;
                    x[nt][h][k] = v;
                    over |= v + vl[h] > ref[nt][k] + kAcRoom;
                }
            }
        if (__any_sync(0xffffffffu, over)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float f[HC];
#pragma unroll
                for (int k = 0; k < HC; ++k) {
                    float m = fmaxf(x[nt][0][k] + vl[0], x[nt][1][k] + vl[1]);
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
                    f[k] = 1.f;
                    if (m > ref[nt][k] + kAcRoom) {
                        const float now = m - kAcUp;
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

        // ---- probabilities, their sums, and their parts as the B fragments of the output
        uint32_t pb[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float w[HC];
#pragma unroll
                for (int k = 0; k < HC; ++k) {
                    const float rf = ref[nt][k] == -INFINITY ? 0.f : ref[nt][k];
                    w[k] = ex2(x[nt][h][k] - rf);
                    l[nt][k] += w[k];
                    if constexpr (Q8) w[k] = p0 + g + 8 * h < lim[nt][k] ? w[k] * vd[h] : 0.f;
                }
                uint32_t u;
                if constexpr (C == 1) {
                    u = pack_f16(w[0], w[1]);
                } else if constexpr (Q8) {
                    const float hi = f16_of(w[0]);
                    u = pack_f16(hi, w[0] - hi);
                } else if constexpr (C == 2) {
                    const float hi = bf16_of(w[0]);
                    u = pack_bf16(hi, w[0] - hi);
                } else {
                    const float hi = bf16_of(w[0]), mid = bf16_of(w[0] - hi);
                    u = t & 1 ? pack_bf16(w[0] - hi - mid, 0.f) : pack_bf16(hi, mid);
                }
                pb[nt][h] = movmatrix(u);
            }

        // ---- output: rows (dims) of V^T against the probabilities
        const uint8_t *sv = st + K::kV;
        if constexpr (Q8) {
            constexpr int VW = K::VB / 4;
            uint32_t v[4][VW];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (VW == 4) {
                    const uint4 u = *reinterpret_cast<const uint4 *>(sv + i * 512 + lane * 16);
                    v[i][0] = u.x, v[i][1] = u.y, v[i][2] = u.z, v[i][3] = u.w;
                } else {
                    const uint2 u = *reinterpret_cast<const uint2 *>(sv + i * 256 + lane * 8);
                    v[i][0] = u.x, v[i][1] = u.y;
                }
#pragma unroll
                for (int w = 0; w < VW; ++w) v[i][w] ^= 0x80808080u;
            }
#pragma unroll
            for (int w = 0; w < VW; ++w)
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    const uint32_t y = __byte_perm(v[0][w], v[1][w], hh ? 0x7362 : 0x5140);
                    const uint32_t z = __byte_perm(v[2][w], v[3][w], hh ? 0x7362 : 0x5140);
                    const uint32_t f[4] = {codes_f16(y, 0x4140), codes_f16(y, 0x4342), codes_f16(z, 0x4140),
                                           codes_f16(z, 0x4342)};
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma16816_f16(o[2 * w + hh][nt], f, pb[nt][0], pb[nt][1]);
                }
        } else {
            uint32_t v[4][4 * K::VP];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < K::VP; ++j) {
                    const uint4 u = *reinterpret_cast<const uint4 *>(sv + (i * K::VP + j) * 512 + lane * 16);
                    v[i][4 * j] = u.x, v[i][4 * j + 1] = u.y, v[i][4 * j + 2] = u.z, v[i][4 * j + 3] = u.w;
                }
            // A new token's V that is not finite must not reach the rows that do not see it (0 x
            // infinity is NaN): only tiles that some rows see further into than others can hold one.
            bool odd = false;
            if (!PREFIX && p0 + kAcTile > lim_lo) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int w = 0; w < 4 * K::VP; ++w)
                        odd |= (v[i][w] & 0x7f80u) == 0x7f80u || (v[i][w] & 0x7f800000u) == 0x7f800000u;
                odd = __any_sync(0xffffffffu, odd);
            }
#pragma unroll
            for (int w = 0; w < 4 * K::VP; ++w) {
                const uint32_t f[4] = {__byte_perm(v[0][w], v[1][w], 0x5410), __byte_perm(v[0][w], v[1][w], 0x7632),
                                       __byte_perm(v[2][w], v[3][w], 0x5410), __byte_perm(v[2][w], v[3][w], 0x7632)};
                if (!PREFIX && odd) {
                    // one limit after the other: V beyond it zeroed, the result kept by the columns it is theirs
                    for (int cut = max(lim_lo, 0); cut <= lim_hi; ++cut) {
                        const int at = p0 + 2 * t;
                        const uint32_t m0 = (at < cut ? 0xffffu : 0u) | (at + 1 < cut ? 0xffff0000u : 0u);
                        const uint32_t m1 = (at + 8 < cut ? 0xffffu : 0u) | (at + 9 < cut ? 0xffff0000u : 0u);
                        const uint32_t fm[4] = {f[0] & m0, f[1] & m0, f[2] & m1, f[3] & m1};
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            float acc[4] = {o[w][nt][0], o[w][nt][1], o[w][nt][2], o[w][nt][3]};
                            mma16816(acc, fm, pb[nt][0], pb[nt][1]);
                            if (lim[nt][0] == cut) {
#pragma unroll
                                for (int e = 0; e < 4; ++e) o[w][nt][e] = acc[e];
                            }
                        }
                    }
                } else {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma16816(o[w][nt], f, pb[nt][0], pb[nt][1]);
                }
            }
        }
        stage = stage == kAcStages - 1 ? 0 : stage + 1;
        __syncwarp();                               // before a lane's scales are written again
    }
    cp_wait<0>();
    __syncthreads();

    // ---- the warps' partials
    float *part = reinterpret_cast<float *>(sm);
    float *mine = part + kAcWarps * K::RW * D;      // the CTA's
    float2 *ml = reinterpret_cast<float2 *>(sm + K::kMl);
    float2 *ml_mine = ml + kAcWarps * K::RW;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < HC; ++k) {
            float v = l[nt][k];
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
            const int row = (8 * nt + 2 * t + k) / C;
            if (g == 0 && (C != 4 || !(t & 1))) ml[warp * K::RW + row] = make_float2(ref[nt][k], v);
#pragma unroll
            for (int mt = 0; mt < K::MT; ++mt)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float w = o[mt][nt][2 * h + k];
                    if constexpr (C >= 2) w += o[mt][nt][2 * h + 1];
                    if constexpr (C == 4) w += __shfl_xor_sync(0xffffffffu, w, 1);
                    const int d = Q8 ? (D / 8) * g + 2 * mt + h : 64 * (mt / 4) + 8 * g + 2 * (mt % 4) + h;
                    if (C != 4 || !(t & 1)) part[(warp * K::RW + row) * D + d] = w;
                }
        }
    __syncthreads();
    for (int i = threadIdx.x; i < K::RW * D / 4; i += kAcThreads) {
        const int row = i / (D / 4);
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kAcWarps; ++w) M = fmaxf(M, ml[w * K::RW + row].x);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < kAcWarps; ++w) {
            const float2 e = ml[w * K::RW + row];
            if (e.y == 0.f) continue;
            const float f = part_weight(e, M);
            const float4 v = *reinterpret_cast<const float4 *>(part + w * K::RW * D + i * 4);
            acc.x = fmaf(f, v.x, acc.x), acc.y = fmaf(f, v.y, acc.y);
            acc.z = fmaf(f, v.z, acc.z), acc.w = fmaf(f, v.w, acc.w);
            sum = fmaf(f, e.y, sum);
        }
        if constexpr (PREFIX) {
            const int r = r0 + row;
            if (r < a.rows) {
                const int64_t at = ((int64_t)hk * a.rows + r) * nsplit + split;
                *reinterpret_cast<float4 *>(a.p_o + at * D + (i % (D / 4)) * 4) = acc;
                if (i % (D / 4) == 0) a.p_ml[at] = make_float2(M, sum);
            }
        } else {
            *reinterpret_cast<float4 *>(mine + i * 4) = acc;
            if (i % (D / 4) == 0) ml_mine[row] = make_float2(M, sum);
        }
    }
    if constexpr (!PREFIX) {
        if (nsplit > 1)
            cluster_sync();
        else
            __syncthreads();
        // ---- the cluster's partials and the prefix's, each CTA a share of the output
        for (int i = split * kAcThreads + threadIdx.x; i < K::RW * D / 4; i += nsplit * kAcThreads) {
            const int row = i / (D / 4), r = r0 + row, tt = r / a.G;
            if (r >= a.rows || tt >= nn) continue;
            float M = -INFINITY;
            for (int s = 0; s < nsplit; ++s)
                M = fmaxf(M, nsplit > 1 ? ld_cluster_f2(cluster_map(ml_mine + row, s)).x : ml_mine[row].x);
            const int64_t at = ((int64_t)hk * (gridDim.x / (nsplit * a.groups * a.kvh)) * a.rows + (int64_t)b * a.rows + r) * a.splits;
            for (int s = 0; s < a.splits; ++s) M = fmaxf(M, a.p_ml[at + s].x);
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            float sum = 0.f;
            for (int s = 0; s < nsplit + a.splits; ++s) {
                float2 e;
                float4 v;
                if (s >= nsplit) {
                    e = a.p_ml[at + s - nsplit];
                    v = *reinterpret_cast<const float4 *>(a.p_o + (at + s - nsplit) * D + (i % (D / 4)) * 4);
                } else if (nsplit > 1) {
                    e = ld_cluster_f2(cluster_map(ml_mine + row, s));
                    v = ld_cluster_f4(cluster_map(mine + i * 4, s));
                } else {
                    e = ml_mine[row];
                    v = *reinterpret_cast<const float4 *>(mine + i * 4);
                }
                if (e.y == 0.f) continue;
                const float f = part_weight(e, M);
                acc.x = fmaf(f, v.x, acc.x), acc.y = fmaf(f, v.y, acc.y);
                acc.z = fmaf(f, v.z, acc.z), acc.w = fmaf(f, v.w, acc.w);
                sum = fmaf(f, e.y, sum);
            }
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            uint8_t *dst = a.out + b * a.o_stream + tt * a.o_token +
                           ((int64_t)(hk * a.G + (r - tt * a.G)) * D + (i % (D / 4)) * 4) * (F32 ? 4 : 2);
            if constexpr (F32)
                *reinterpret_cast<float4 *>(dst) = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
            else
                *reinterpret_cast<uint2 *>(dst) =
                    make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
        }
        if (nsplit > 1) cluster_sync();              // the others have read this CTA's part
    }
}

// ------------------------------------------------------------------------- launches

// CTAs that share the prefix's positions, per key head and row group.
int prefix_splits(int rows, int kvh, int prefix_len, int rw, int sms) {
    const int groups = (rows + rw - 1) / rw;
    const int tiles = (prefix_len + kAcTile - 1) / kAcTile;
    const int most = std::max(1, tiles / (2 * kAcWarps));
    const int want = std::max(1, 4 * sms / std::max(1, groups * kvh));
    return std::max(1, std::min(std::min(most, want), 32));
}

template <bool Q8, bool F32, int D, int NT, bool PREFIX>
cudaError_t launch(const CachedArgs &a, int items, int nsplit, int dev, cudaStream_t s) {
    using K = AcCfg<Q8, F32, D, NT>;
    auto fn = attn_cached_kernel<Q8, F32, D, NT, PREFIX>;
    static bool ready[64] = {};                     // per device; setting it twice is harmless
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!ready[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void *>(fn),
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, K::kSmem);
        if (e != cudaSuccess) return e;
        ready[dev] = true;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(items * nsplit));
    cfg.blockDim = dim3(kAcThreads);
    cfg.dynamicSmemBytes = K::kSmem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = PREFIX ? 1 : (unsigned)nsplit;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fn, a, nsplit);
}

constexpr int rows_per_tile(bool q8, bool f32) { return 8 / (q8 ? (f32 ? 2 : 1) : (f32 ? 4 : 2)); }

template <bool PREFIX>
cudaError_t dispatch(bool q8, bool f32, int d, int nt, const CachedArgs &a, int items, int nsplit, int dev,
                     cudaStream_t s) {
#define QD_AC(Q, F, DD, N) \
    if (q8 == Q && f32 == F && d == DD && nt == N) return launch<Q, F, DD, N, PREFIX>(a, items, nsplit, dev, s);
#define QD_AC2(Q, F) QD_AC(Q, F, 64, 1) QD_AC(Q, F, 64, 2) QD_AC(Q, F, 128, 1) QD_AC(Q, F, 128, 2)
    QD_AC2(false, false) QD_AC2(false, true) QD_AC2(true, false) QD_AC2(true, true)
#undef QD_AC2
#undef QD_AC
    return cudaErrorInvalidValue;
}

// workspace: (ref, sum) of every partial, then its output row
size_t ml_bytes(int kvh, int64_t rows, int splits) { return ((size_t)kvh * rows * splits * 8 + 255) / 256 * 256; }

}  // namespace

}  // namespace qd

using namespace qd;

extern "C" {

qd_status qd_attn_cached_workspace(int n_streams, int n_tokens, int n_q_heads, int n_kv_heads, int head_dim,
                                   int prefix_length, size_t *bytes) {
    if (!bytes) return QD_EINVAL;
    *bytes = 0;
    if (n_streams < 1 || n_tokens < 1 || n_kv_heads < 1 || n_q_heads < n_kv_heads || n_q_heads % n_kv_heads ||
        prefix_length < 0)
        return QD_EINVAL;
    if ((head_dim != 64 && head_dim != 128) || n_tokens > kAcMaxTokens) return QD_EUNSUPPORTED;
    if (!prefix_length) return QD_OK;
    int dev = 0;
    const int sms = cudaGetDevice(&dev) == cudaSuccess ? sms_of(dev) : 152;
    const int64_t rows = (int64_t)n_streams * n_tokens * (n_q_heads / n_kv_heads);
    if (rows > (1 << 24)) return QD_EUNSUPPORTED;
    // the most splits of any type's tiling
    int most = 1;
    for (int rw = 2; rw <= 16; rw <<= 1) most = std::max(most, prefix_splits((int)rows, n_kv_heads, prefix_length, rw, sms));
    *bytes = ml_bytes(n_kv_heads, rows, most) + (size_t)n_kv_heads * rows * most * head_dim * 4;
    return QD_OK;
}

qd_status qd_attn_cached(const qd_kv_cache *cache, const qd_kv_cache *prefix, int prefix_length, const void *q_dev,
                         int64_t q_stream_stride, int64_t q_token_stride, void *out_dev, int64_t out_stream_stride,
                         int64_t out_token_stride, int dtype, int n_tokens, int n_q_heads, float scale,
                         const int32_t *lengths_dev, const int32_t *n_new_dev, int max_length, void *workspace_dev,
                         size_t workspace_bytes, void *cuda_stream) {
    qd_status st = check_cache(cache, -1, false);
    if (st != QD_OK) return st;
    const bool with_prefix = prefix && prefix_length > 0;
    if (prefix_length < 0 || (!prefix && prefix_length)) return QD_EINVAL;
    if (with_prefix) {
        if ((st = check_cache(prefix, -1, true)) != QD_OK) return st;
        if (prefix->n_kv_heads != cache->n_kv_heads || prefix->head_dim != cache->head_dim ||
            prefix_length > prefix->smax)
            return QD_EINVAL;
    }
    const int kvh = cache->n_kv_heads, d = cache->head_dim, B = cache->n_streams;
    if ((dtype != QD_F32 && dtype != QD_BF16) || n_tokens < 1 || n_q_heads < kvh || n_q_heads % kvh) return QD_EINVAL;
    if (max_length < 1 || max_length > cache->smax || !(scale > -3e38f && scale < 3e38f)) return QD_EINVAL;
    if (n_tokens > kAcMaxTokens) return QD_EUNSUPPORTED;
    if (!q_dev || !out_dev || !lengths_dev) return QD_EINVAL;
    const int64_t unit = dtype == QD_F32 ? 4 : 8, e = dtype == QD_F32 ? 4 : 2;
    for (int64_t v : {q_stream_stride, q_token_stride, out_stream_stride, out_token_stride})
        if (v < 0 || v % unit) return QD_EINVAL;
    if (!is_aligned(q_dev, 16) || !is_aligned(out_dev, 16) || !is_aligned(lengths_dev, 4) || !is_aligned(n_new_dev, 4))
        return QD_EINVAL;
    const int G = n_q_heads / kvh;
    const int64_t rows = (int64_t)n_tokens * G, all = rows * B;
    if (all > (1 << 24) || all * kvh > (1 << 26)) return QD_EUNSUPPORTED;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return QD_ECUDA;
    const int sms = sms_of(dev);
    if ((st = check_cache(cache, dev, false)) != QD_OK) return st;
    if (with_prefix && (st = check_cache(prefix, dev, true)) != QD_OK) return st;
    if (!on_device(q_dev, dev) || !on_device(out_dev, dev) || !on_device(lengths_dev, dev) ||
        (n_new_dev && !on_device(n_new_dev, dev)))
        return QD_EINVAL;

    const bool f32 = dtype == QD_F32;
    cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
    CachedArgs a = {};
    a.q = static_cast<const uint8_t *>(q_dev), a.out = static_cast<uint8_t *>(out_dev);
    a.q_stream = q_stream_stride * e, a.q_token = q_token_stride * e;
    a.o_stream = out_stream_stride * e, a.o_token = out_token_stride * e;
    a.lengths = lengths_dev, a.n_new = n_new_dev;
    a.T = n_tokens, a.G = G, a.kvh = kvh;
    a.scale2 = scale * 1.4426950408889634f;

    if (with_prefix) {
        size_t need = 0;
        if ((st = qd_attn_cached_workspace(B, n_tokens, n_q_heads, kvh, d, prefix_length, &need)) != QD_OK) return st;
        if (!workspace_dev || workspace_bytes < need || !is_aligned(workspace_dev, 256) || !on_device(workspace_dev, dev))
            return QD_EINVAL;
        const bool q8 = prefix->format == QD_KV_Q8;
        const int per = rows_per_tile(q8, f32), nt = all > per ? 2 : 1, rw = per * nt;
        CachedArgs p = a;
        p.c = kv_view(prefix);
        p.rows = (int)all, p.groups = (int)((all + rw - 1) / rw), p.max_len = prefix_length;
        const int splits = prefix_splits((int)all, kvh, prefix_length, rw, sms);
        p.p_ml = static_cast<float2 *>(workspace_dev);
        p.p_o = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace_dev) + ml_bytes(kvh, all, splits));
        p.splits = splits;
        if (dispatch<true>(q8, f32, d, nt, p, p.groups * kvh, splits, dev, s) != cudaSuccess) return QD_ECUDA;
        a.p_ml = p.p_ml, a.p_o = p.p_o, a.splits = splits;
    }

    const bool q8 = cache->format == QD_KV_Q8;
    const int per = rows_per_tile(q8, f32), nt = rows > per ? 2 : 1, rw = per * nt;
    a.c = kv_view(cache);
    a.rows = (int)rows, a.groups = (int)((rows + rw - 1) / rw), a.max_len = max_length;
    const int64_t items = (int64_t)B * kvh * a.groups;
    // split a stream until the CTAs fill the SMs, but leave every warp a tile
    int nsplit = 1;
    while (nsplit < kAcMaxCluster && items * nsplit < 3 * sms && max_length > nsplit * kAcWarps * kAcTile) nsplit *= 2;
    return dispatch<false>(q8, f32, d, nt, a, (int)items, nsplit, dev, s) == cudaSuccess ? QD_OK : QD_ECUDA;
}

}  // extern "C"
