// Attention of many bf16 rows (all streams' new tokens and query heads) over the shared
// prefix on the tcgen05 tensor cores: the prefix is read once per 128 or 256 rows.
//
// Per key head the batch's rows in use stand one after the other in tiles of 128 (the M of an MMA); the keys
// come in chunks of 128.  A CTA has two halves, each with a tile of its own in flight (S, P and O in tensor
// memory), so that the tensor core works for one half while the other takes its softmax:
//   S = Q K^T          128 x 128 fp32 in tensor memory; Q and K from shared memory
//   softmax            thread = row: P = 2^(s - ref) as two 16-bit parts over S's own columns, 64 keys at a time
//   O += P V           P's parts from tensor memory, V from shared memory (keys x dims: the MN-major operand)
// With more than 128 rows the halves take two tiles of rows over the same chunks (K and V are shared);
// otherwise both take the one tile, every other chunk each.  The list (key head, tile pair, chunk) is cut into equal
// runs, one per CTA; each leaves (ref, sum, O) of its rows for attn_join_kernel.
//
// bf16 prefix: P is two bf16 parts (16 bits).  8-bit prefix: the codes are widened to fp16, exactly, on their way into shared
// memory; the keys' scales multiply S's columns, the values' scales P's, and P is two fp16 parts (22 bits).  32 keys'
// scores stand in 32 columns, and so do their parts: 16 columns of the first, 16 of the second.
//
// 64 keys' probabilities are formed with the reference as it stands and written over their scores when none has outgrown
// its room (32 keys at a time, a vote each, took 150 us where this takes 140); otherwise the reference moves first, with O in
// tensor memory (the half's previous O product has finished when its next S has) and what the chunk has written so
// far.  So the scores are usually read once.
//
// Measured: 16384 8-bit positions under 768 of 1536 rows and 8 key heads, 52.7 GFLOP (79 with P's second part), 85 us, the
// tensor pipe 44 % of its cycles; 71 us with one part, which keeps 11 bits (8 of bf16).  A chunk needs 1536 clocks of products in each
// half, and 1024 of the exponentials' units (16 a clock and SM), and a pair takes about twice the products' time: a half's softmax
// and its two products follow one another, and S and O of two halves fill the tensor memory of head_dim 128.  Not tried: O's products begun on the
// first keys while the others' weights are formed, and a share of the exponentials on the FMA units.
//
// Roles (512 threads): warps 0-3 and 4-7 the softmax of the two halves (a row each, also Q and the results),
// warps 8-11 load K and V, warp 12 owns the tensor memory and issues the MMAs, warps 13-15 only complete its
// warpgroup.  Registers a thread: 128 at launch, then 176, 176, 104 and 56 (all of the 65,536).  Every wait
// is bounded; where one expires the CTA's partials become NaN and the roles run to their ends.
#include <cuda.h>

#include <atomic>

#include "attn_cached.cuh"
#include "qd_internal.h"
#include "tc_common.cuh"

namespace qd {

namespace {

constexpr int kWtThreads = 512;
constexpr int kWtSoft = 256, kWtLoad = 128;   // softmax threads, loading threads
constexpr int kWtRegsSoft = 176, kWtRegsLoad = 104, kWtRegsMma = 56;
static_assert(128 * (2 * kWtRegsSoft + kWtRegsLoad + kWtRegsMma) <= kWtThreads * 128, "registers");
constexpr uint32_t kWtBox = 128 * 128;        // 128 rows of 128 bytes, 128-byte swizzle
constexpr uint32_t kWtS = 0, kWtO = 256;      // tensor memory columns: S (and P) of the halves, O

template <int D> struct WtCfg {
    static constexpr int KB = D / 64;                         // 64-wide blocks of head_dim
    static constexpr uint32_t kQ = 0;                         // Q [half][KB]
    static constexpr uint32_t kK = kQ + 2 * KB * kWtBox;      // K [stage][KB]
    static constexpr uint32_t kV = kK + 2 * KB * kWtBox;      // V [stage][KB]
    static constexpr uint32_t kSc = kV + 2 * KB * kWtBox;     // scales [stage][keys', values', log2 of |values'|][128]
    static constexpr uint32_t kOff = kSc + 2 * 3 * 128 * 4;   // first row of each stream
    static constexpr uint32_t kBar = kOff + (kWideMaxStreams + 1) * 4 + 4;
    static constexpr uint32_t kSmem = 1024 + kBar + 32 * 8;
};

// 32 consecutive fp32 columns of this thread's lane
__device__ __forceinline__ void ld32(uint32_t taddr, float *v) {
    uint32_t r[32];
    tc_ld16_nowait(taddr, r);
    tc_ld16_nowait(taddr + 16, r + 16);
    tc_wait_ld_u32<32>(r);
#pragma unroll
    for (int e = 0; e < 32; ++e) v[e] = __uint_as_float(r[e]);
}
// Byte of 16-byte piece c (of 8) of row r in a swizzled box.
__device__ __forceinline__ uint32_t swz(int r, int c) { return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4)); }

// The reference of a half's rows stands 2^kWtUp<> below 2^0.. of the largest weight when it is set, and moves when a
// weight has passed kWtTop<>.  fp16 weights (8-bit prefix): from 2^2 to 2^15, the type's range less a factor of two; below
// 2^-14 they lose bits, 2^-25 at most, 2^-27 of the largest.  bf16 weights have fp32's range: practically once.
template <bool Q8> constexpr float kWtUp = Q8 ? 2.f : 0.f;
template <bool Q8> constexpr float kWtTop = Q8 ? 32768.f : 1.e18f;

// The largest weight, in log2 units, that 32 keys (`left` of them there) have in a row.
template <bool Q8> __device__ __forceinline__ float largest(const uint32_t (&x)[32], const float *sc, float cs, int left) {
    float m = -INFINITY;
#pragma unroll
    for (int e = 0; e < 32; ++e) {
        float s = __uint_as_float(x[e]);
        s = Q8 ? fmaf(s * sc[e], cs, sc[256 + e]) : s * cs;
        m = fmaxf(m, e < left ? s : -INFINITY);
    }
    return m;
}

// 32 keys of a row against its reference: the weights of the product, the largest of them, and the sum of the
// probabilities.  A weight past kWtTop means that the reference has to move.
template <bool Q8, bool EDGE>
__device__ __forceinline__ void weigh(const uint32_t (&x)[32], const float *sc, float cs, float ref, int left, float (&w)[32],
                                      float &top, float &sum) {
    const float rf = ref == -INFINITY ? 0.f : ref;
    const uint64_t cs2 = pk(cs, cs), rf2 = pk(-rf, -rf);
    uint64_t l2 = pk(0.f, 0.f);
    float t0 = 0.f, t1 = 0.f;
#pragma unroll
    for (int e = 0; e < 32; e += 4) {
        uint64_t x0 = pk(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), x1 = pk(__uint_as_float(x[e + 2]), __uint_as_float(x[e + 3]));
        if constexpr (Q8) {
            const ulonglong2 k = *reinterpret_cast<const ulonglong2 *>(sc + e);
            x0 = mul2(x0, k.x), x1 = mul2(x1, k.y);
        }
        float s0, s1, s2, s3;
        unpk(fma2(x0, cs2, rf2), s0, s1);
        unpk(fma2(x1, cs2, rf2), s2, s3);
        s0 = ex2(s0), s1 = ex2(s1), s2 = ex2(s2), s3 = ex2(s3);
        if constexpr (EDGE) {
            s0 = e < left ? s0 : 0.f, s1 = e + 1 < left ? s1 : 0.f;
            s2 = e + 2 < left ? s2 : 0.f, s3 = e + 3 < left ? s3 : 0.f;
        }
        x0 = pk(s0, s1), x1 = pk(s2, s3);
        l2 = add2(l2, add2(x0, x1));
        if constexpr (Q8) {
            const ulonglong2 v = *reinterpret_cast<const ulonglong2 *>(sc + 128 + e);
            unpk(mul2(x0, v.x), s0, s1);
            unpk(mul2(x1, v.y), s2, s3);
        }
        t0 = fmaxf(t0, fmaxf(fabsf(s0), fabsf(s1))), t1 = fmaxf(t1, fmaxf(fabsf(s2), fabsf(s3)));   // (a scale may be negative)
        w[e] = s0, w[e + 1] = s1, w[e + 2] = s2, w[e + 3] = s3;
    }
    float l0, l1;
    unpk(l2, l0, l1);
    sum = l0 + l1, top = fmaxf(t0, t1);
}

// A pair of weights as two 16-bit parts each, and back.
template <bool Q8> __device__ __forceinline__ float2 pair_of(uint32_t y) {
    return Q8 ? __half22float2(*reinterpret_cast<const __half2 *>(&y)) : make_float2(bf16lo(y), bf16hi(y));
}
template <bool Q8> __device__ __forceinline__ void parts(float a, float b, uint32_t &hi, uint32_t &lo) {
    hi = Q8 ? pack_f16(a, b) : pack_bf16(a, b);
    const float2 h = pair_of<Q8>(hi);
    lo = Q8 ? pack_f16(a - h.x, b - h.y) : pack_bf16(a - h.x, b - h.y);
}
// 32 weights over the columns of their scores
template <bool Q8> __device__ __forceinline__ void put_weights(uint32_t taddr, const float (&w)[32]) {
    uint32_t y[32];
#pragma unroll
    for (int e = 0; e < 16; ++e) parts<Q8>(w[2 * e], w[2 * e + 1], y[e], y[16 + e]);
    tc_st16(taddr, y);
    tc_st16(taddr + 16u, y + 16);
}

__device__ __forceinline__ void soft_sync() { named_sync(1, kWtSoft); }

// A CTA's run, segment by segment (an item's chunks c0 .. c0 + n); the same walk in every role.
struct Walk {
    Share sh;
    int chunks;
    unsigned x, x1;
    int item, c0, n;
    __device__ __forceinline__ bool next() {
        if (x >= x1) return false;
        item = (int)(x / (unsigned)chunks), c0 = (int)(x - (unsigned)item * chunks);
        n = (int)min((unsigned)(chunks - c0), x1 - x);
        x += n;
        return true;
    }
};

template <bool Q8, int D>
__global__ void __launch_bounds__(kWtThreads, 1) attn_prefix_tc_kernel(const CachedArgs a) {
    using C = WtCfg<D>;
    constexpr int KB = C::KB;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + ((C::kBar + 7u) & ~7u));
    uint64_t *s_full = bars, *p_full = bars + 2, *q_full = bars + 4, *o_done = bars + 6;          // [half]
    uint64_t *k_full = bars + 8, *k_empty = bars + 10, *v_full = bars + 12, *v_empty = bars + 14;   // [stage]
    uint64_t *drain = bars + 16;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 17);
    volatile int *bad = reinterpret_cast<volatile int *>(bars + 18);
    int *off = reinterpret_cast<int *>(sm + C::kOff);

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1), mbar_init(&p_full[i], 4), mbar_init(&q_full[i], 4), mbar_init(&o_done[i], 1);
            mbar_init(&k_full[i], kWtLoad), mbar_init(&k_empty[i], 1);
            mbar_init(&v_full[i], kWtLoad), mbar_init(&v_empty[i], 1);
        }
        mbar_init(drain, 1);
        *bad = 0;
        fence_barrier_init();
    }
    // The predecessor first, the tensor memory then: held while waiting it could be what a predecessor's CTA on this SM
    // waits for.
    pdl_wait();
    if (warp == 12) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    pdl_launch_dependents();
    // where each stream's rows in use begin, and how many there are
    const bool gaps = a.n_new && a.B <= kWideMaxStreams;
    if (gaps && warp == 0) {
        int sum = 0;
        for (int b0 = 0; b0 < a.B; b0 += 32) {
            const int n = b0 + lane < a.B ? clamp_new(a, b0 + lane) * a.G : 0;
            int upto = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += v;
            }
            if (b0 + lane < a.B) off[b0 + lane] = sum + upto - n;
            sum += __shfl_sync(0xffffffffu, upto, 31);
        }
        if (lane == 0) off[a.B] = sum;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int rows = gaps ? off[a.B] : a.B * a.T * a.G;

    const WideItems items(rows);
    const bool pairs = items.pairs > 0;
    Walk w;
    const bool works = blockIdx.x < items.share(a, &w.sh) && rows > 0;
    w.chunks = a.wide_chunks;
    w.x = works ? w.sh.first(blockIdx.x) : 0u;
    w.x1 = works ? w.sh.first(blockIdx.x + 1) : 0u;
    const int P = a.max_len;

    if (warp >= 8 && warp < 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kWtRegsLoad));
        // ---- K and V chunks into the operands' layout, 16 bytes of the cache a thread and turn
        const int tid = threadIdx.x - kWtSoft;
        int kc = 0;                                 // chunks so far
        bool ok = true;
        while (w.next()) {
            const int hk = w.item / items.per_head();
            const uint8_t *kb = a.c.k + hk * a.c.head, *vb = a.c.v + hk * a.c.head;
            if constexpr (Q8) {
                // this thread: piece j (16 codes) of rows r0, r0 + 32, .. of each 64-wide block
                constexpr int N = 4 * KB;
                const float *ks = a.c.ks + hk * a.c.shead, *vs = a.c.vs + hk * a.c.shead;
                const int j = tid & 3, r0 = tid >> 2;
                const int64_t hop = 32 * a.c.row;
                kb += r0 * a.c.row + j * 16, vb += r0 * a.c.row + j * 16;
                uint4 uk[N], uv[N];                 // the next chunk's codes
                float sk, sv;                       // and scales, of key tid
                auto load = [&](const uint8_t *base, int c, uint4 *to) {
                    const uint8_t *at = base + (int64_t)c * kWideKeys * a.c.row;
                    const int left = P - c * kWideKeys;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int k = 0; k < KB; ++k) {
                            to[KB * i + k] = make_uint4(0, 0, 0, 0);
                            if (r0 + 32 * i < left) to[KB * i + k] = __ldg(reinterpret_cast<const uint4 *>(at + i * hop + 64 * k));
                        }
                };
                auto load_scales = [&](int c) {
                    const int key = c * kWideKeys + tid;
                    sk = key < P ? __ldg(ks + key) : 0.f, sv = key < P ? __ldg(vs + key) : 0.f;
                };
                const uint32_t put0 = swz(r0, 2 * j), put1 = swz(r0, 2 * j + 1);   // rows 32 apart swizzle alike
                auto store = [&](uint8_t *tile, const uint4 *from) {
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        const uint32_t x[4] = {from[i].x ^ 0x80808080u, from[i].y ^ 0x80808080u, from[i].z ^ 0x80808080u,
                                               from[i].w ^ 0x80808080u};
                        // eight lanes: two rows, whose swizzles differ in the last bit, and four even (odd) pieces
                        uint8_t *box = tile + (i % KB) * kWtBox + (i / KB) * 32 * 128;
                        *reinterpret_cast<uint4 *>(box + put0) =
                            make_uint4(codes_f16<false>(x[0], 0x4140), codes_f16<false>(x[0], 0x4342),
                                       codes_f16<false>(x[1], 0x4140), codes_f16<false>(x[1], 0x4342));
                        *reinterpret_cast<uint4 *>(box + put1) =
                            make_uint4(codes_f16<false>(x[2], 0x4140), codes_f16<false>(x[2], 0x4342),
                                       codes_f16<false>(x[3], 0x4140), codes_f16<false>(x[3], 0x4342));
                    }
                };
                load(kb, w.c0, uk);
                load(vb, w.c0, uv);
                load_scales(w.c0);
                for (int i = 0; i < w.n; ++i, ++kc) {
                    const int st = kc & 1;
                    const uint32_t was = ((uint32_t)(kc >> 1) & 1u) ^ 1u;
                    if (kc >= 2) ok = ok && wt_wait(&k_empty[st], was, bad);
                    store(sm + C::kK + (uint32_t)(st * KB) * kWtBox, uk);
                    fence_proxy_async_smem();
                    mbar_arrive(&k_full[st]);
                    if (i + 1 < w.n) load(kb, w.c0 + i + 1, uk);
                    if (kc >= 2) ok = ok && wt_wait(&v_empty[st], was, bad);
                    store(sm + C::kV + (uint32_t)(st * KB) * kWtBox, uv);
                    // the scales come with V, which is not given up before its softmax is done (K's tile is)
                    float *sc = reinterpret_cast<float *>(sm + C::kSc) + st * 384;
                    sc[tid] = sk, sc[128 + tid] = sv, sc[256 + tid] = fminf(fmaxf(lg2(fabsf(sv)), -60.f), kScaleMost);
                    fence_proxy_async_smem();
                    mbar_arrive(&v_full[st]);
                    if (i + 1 < w.n) {
                        load(vb, w.c0 + i + 1, uv);
                        load_scales(w.c0 + i + 1);
                    }
                }
            } else {
                // this thread: piece j (8 dims) of rows r0, r0 + RPI, ..
                constexpr int PPR = 8 * KB, RPI = kWtLoad / PPR, N = 128 / RPI;
                const int j = tid % PPR, r0 = tid / PPR;
                const int64_t hop = RPI * a.c.row;
                kb += r0 * a.c.row + j * 16, vb += r0 * a.c.row + j * 16;
                auto copy = [&](const uint8_t *base, int c, uint8_t *tile) {
                    const uint8_t *at = base + (int64_t)c * kWideKeys * a.c.row;
                    const int left = P - c * kWideKeys;
                    const uint32_t to = smem_addr(tile) + (uint32_t)(j >> 3) * kWtBox;
#pragma unroll
                    for (int n = 0; n < N; ++n) {
                        const int r = r0 + n * RPI;
                        const bool live = r < left;
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + swz(r, j & 7)),
                                     "l"(live ? at + n * hop : a.c.k), "r"(live ? 16 : 0)
                                     : "memory");
                    }
                    asm volatile("cp.async.commit_group;" ::: "memory");
                };
                for (int i = 0; i < w.n; ++i, ++kc) {
                    const int st = kc & 1;
                    const uint32_t was = ((uint32_t)(kc >> 1) & 1u) ^ 1u;
                    if (kc >= 2) ok = ok && wt_wait(&k_empty[st], was, bad);
                    copy(kb, w.c0 + i, sm + C::kK + (uint32_t)(st * KB) * kWtBox);
                    if (kc >= 2) ok = ok && wt_wait(&v_empty[st], was, bad);
                    copy(vb, w.c0 + i, sm + C::kV + (uint32_t)(st * KB) * kWtBox);
                    asm volatile("cp.async.wait_group 1;" ::: "memory");
                    fence_proxy_async_smem();
                    mbar_arrive(&k_full[st]);
                    asm volatile("cp.async.wait_group 0;" ::: "memory");
                    fence_proxy_async_smem();
                    mbar_arrive(&v_full[st]);
                }
            }
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
    } else if (warp >= 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kWtRegsMma));
        if (warp == 12) {
        // ---- the MMAs: S of both halves, then always a half's O followed by its next S.  The whole warp walks
        // along, and one lane of its choosing issues (elect.sync always names the same): the operands then live in uniform
        // registers.  A branch on lane 0 instead took 140 to 190 clocks for each MMA of 64.
        constexpr uint32_t bf = Q8 ? 0u : (1u << 7) | (1u << 10);
        constexpr uint32_t base = (1u << 4) | bf | ((uint32_t)(kWideRows >> 4) << 24);
        constexpr uint32_t idesc_s = base | ((uint32_t)(kWideKeys >> 3) << 17);
        constexpr uint32_t idesc_o = base | (1u << 16) | ((uint32_t)(D >> 3) << 17);
        // descriptors of the first bytes; an offset of n bytes adds n / 16
        const uint64_t dQ = sw128_desc(smem_addr(sm + C::kQ)), dK = sw128_desc(smem_addr(sm + C::kK));
        const uint64_t dV = sw128_desc_mn(smem_addr(sm + C::kV), kWtBox, 1024u);
        constexpr uint32_t kBox16 = kWtBox / 16;
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        int kc = 0, seg = 0;
        uint32_t np[2] = {0, 0};                   // P's so far
        bool ok = true;
        for (; ok && w.next(); ++seg) {
            const int N = pairs ? 2 * w.n : w.n;
            ok = wt_wait(&q_full[0], (uint32_t)seg & 1u, bad) && (!pairs || wt_wait(&q_full[1], (uint32_t)seg & 1u, bad));
            ok = __all_sync(0xffffffffu, ok);       // a wait may expire for some lanes alone: all leave together
            auto issue_s = [&](int i) {
                const int h = i & 1, c = kc + (pairs ? i >> 1 : i), st = c & 1;
                if (!pairs || !h) ok = ok && wt_wait(&k_full[st], (uint32_t)(c >> 1) & 1u, bad);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) return;
                tc_fence_after();
                const uint32_t d = tm + kWtS + 128u * h;
                const uint64_t q = dQ + (pairs ? h * KB : 0) * kBox16, k = dK + st * KB * kBox16;
                if (elect_one()) {
#pragma unroll
                    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                        for (int s = 0; s < 4; ++s)
                            tc_mma(d, q + kb * kBox16 + 2 * s, k + kb * kBox16 + 2 * s, idesc_s, (kb | s) ? 1u : 0u);
                    tc_commit(&s_full[h]);
                    if (!pairs || h) tc_commit(&k_empty[st]);
                }
                __syncwarp();
            };
            auto issue_o = [&](int i) {
                const int h = i & 1, c = kc + (pairs ? i >> 1 : i), st = c & 1;
                ok = ok && wt_wait(&p_full[h], np[h] & 1u, bad);
                if (!pairs || !h) ok = ok && wt_wait(&v_full[st], (uint32_t)(c >> 1) & 1u, bad);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) return;
                ++np[h];
                tc_fence_after();
                const uint32_t d = tm + kWtO + 128u * h, p = tm + kWtS + 128u * h;
                const uint64_t v = dV + st * KB * kBox16;
                if (elect_one()) {
#pragma unroll
                    for (int ks = 0; ks < kWideKeys / 16; ++ks)
#pragma unroll
                        for (int part = 0; part < 2; ++part)
                            tc_mma_ts(d, p + 32u * (ks >> 1) + 8u * (ks & 1) + 16u * part, v + ks * 128, idesc_o,
                                      (ks | part) ? 1u : (i >= 2 ? 1u : 0u));
                    if (!pairs || h) tc_commit(&v_empty[st]);
                    if (i + 2 >= N) tc_commit(&o_done[h]);
                }
                __syncwarp();
            };
            for (int i = 0; ok && i < 2 && i < N; ++i) issue_s(i);
            for (int i = 0; ok && i < N; ++i) {
                issue_o(i);
                if (ok && i + 2 < N) issue_s(i + 2);
            }
            kc += w.n;
        }
        // every MMA issued has completed before the tensor memory can be freed
        if (elect_one()) tc_commit(drain);
        (void)mbar_wait_bounded(drain, 0u, 20000000ull);
        __syncwarp();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kWtRegsSoft));
        // ---- softmax: half h, row r of its tile
        const int h = warp >> 2, quarter = warp & 3, r = quarter * 32 + lane;
        const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
        const uint32_t tS = tmem + kWtS + 128u * h + lanes, tO = tmem + kWtO + 128u * h + lanes;
        int kc = 0, seg = 0;
        uint32_t ns = 0, no = 0;                   // S's, O's so far
        bool ok = true;
        for (; w.next(); ++seg) {
            const int per = items.per_head(), hk = w.item / per, tile = pairs ? 2 * (w.item - hk * per) + h : 0;
            const int row = tile * kWideRows + r;
            // the row's query: compact row -> stream, token, head
            const uint8_t *src = nullptr;
            if (row < rows) {
                int b, in;
                if (gaps) {
                    int lo = 0, hi = a.B;           // off[lo] <= row < off[hi]
                    while (hi - lo > 1) {
                        const int mid = (lo + hi) >> 1;
                        if (off[mid] <= row)
                            lo = mid;
                        else
                            hi = mid;
                    }
                    b = lo, in = row - off[lo];
                } else {
                    b = row / (a.T * a.G), in = row - b * (a.T * a.G);
                }
                const int tt = in / a.G, g = in - tt * a.G;
                if (tt < clamp_new(a, b)) src = a.q + b * a.q_stream + tt * a.q_token + (int64_t)(hk * a.G + g) * D * 2;
            }
            // the warp's 32 rows, D / 8 lanes a row: whole lines, where a row a thread took a line for every 16 bytes
            float cs = a.scale2;
            {
                constexpr int LPR = D / 8, RPI = 32 / LPR, N = LPR;   // lanes a row, rows a turn, turns
                const int j = lane % LPR, in = lane / LPR;
                uint4 u[N];
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const uint64_t at = __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(src), RPI * i + in);
                    u[i] = make_uint4(0, 0, 0, 0);
                    if (at) u[i] = __ldg(reinterpret_cast<const uint4 *>(at) + j);
                }
                uint8_t *q = sm + C::kQ + (uint32_t)((pairs ? h : 0) * KB + (j >> 3)) * kWtBox;
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const int rr = RPI * i + in;
                    if constexpr (Q8) {
                        // fp16, scaled by a power of two: the row's largest value to [2^14, 2^15)
                        uint32_t m = __vmaxu2(__vmaxu2(u[i].x & 0x7fff7fffu, u[i].y & 0x7fff7fffu),
                                              __vmaxu2(u[i].z & 0x7fff7fffu, u[i].w & 0x7fff7fffu));
                        m = max(m >> 16, m & 0xffffu);
#pragma unroll
                        for (int o = LPR / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
                        const int up = min(268 - (int)(m >> 7), 253);   // from the exponent
                        const float f = __uint_as_float((uint32_t)up << 23);
                        // the row's own thread takes the inverse into its factor
                        const int mine = __shfl_sync(0xffffffffu, up, (lane % RPI) * LPR);
                        if (lane / RPI == i) cs = a.scale2 * __uint_as_float((uint32_t)(254 - mine) << 23);
                        u[i].x = pack_f16(bf16lo(u[i].x) * f, bf16hi(u[i].x) * f);
                        u[i].y = pack_f16(bf16lo(u[i].y) * f, bf16hi(u[i].y) * f);
                        u[i].z = pack_f16(bf16lo(u[i].z) * f, bf16hi(u[i].z) * f);
                        u[i].w = pack_f16(bf16lo(u[i].w) * f, bf16hi(u[i].w) * f);
                    }
                    if (pairs || h == 0) *reinterpret_cast<uint4 *>(q + swz(quarter * 32 + rr, j & 7)) = u[i];
                }
                if (pairs || h == 0) {
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&q_full[h]);
                }
            }
            float ref = -INFINITY, l = 0.f;
            const int N = pairs ? 2 * w.n : w.n;
            for (int i = h; i < N; i += 2) {
                const int c = pairs ? i >> 1 : i, st = (kc + c) & 1;
                const int left = P - (w.c0 + c) * kWideKeys;        // keys of the chunk
                const float *sc = reinterpret_cast<const float *>(sm + C::kSc) + st * 384;
                ok = ok && wt_wait(&s_full[h], ns & 1u, bad);
                ++ns;
                if constexpr (Q8) ok = ok && wt_wait(&v_full[st], (uint32_t)((kc + c) >> 1) & 1u, bad);
                tc_fence_after();
                // 64 keys at a time; the next ones' scores arrive while these are packed
                uint32_t x[2][2][32];
                ld32_start(tS, x[0][0]);
                ld32_start(tS + 32u, x[0][1]);
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const uint32_t tq = tS + 64u * q;
                    const int here = left - 64 * q; // keys there
                    const float *scq = sc + 64 * q;
                    float w[2][32], top, sum;
                    auto weigh_all = [&](const uint32_t (&y)[2][32]) {
                        float t1, s1;
                        if (here < 64) {
                            weigh<Q8, true>(y[0], scq, cs, ref, here, w[0], top, sum);
                            weigh<Q8, true>(y[1], scq + 32, cs, ref, here - 32, w[1], t1, s1);
                        } else {
                            weigh<Q8, false>(y[0], scq, cs, ref, here, w[0], top, sum);
                            weigh<Q8, false>(y[1], scq + 32, cs, ref, here, w[1], t1, s1);
                        }
                        top = fmaxf(top, t1), sum += s1;
                    };
                    tc_wait_ld_u32<32>(x[q][0]);
                    tc_wait_ld_u32<32>(x[q][1]);
                    // a half's first keys set the reference, which is near enough as a rule
                    const bool first = q == 0 && i < 2;
                    if (first) {
                        const float m = fmaxf(largest<Q8>(x[q][0], scq, cs, here), largest<Q8>(x[q][1], scq + 32, cs, here - 32));
                        if (m - kWtUp<Q8> > ref) ref = m - kWtUp<Q8>;
                    }
                    weigh_all(x[q]);
                    if (!first && __any_sync(0xffffffffu, top > kWtTop<Q8> || ref == -INFINITY)) {
                        uint32_t y[2][32];          // the scores again: they stand until their weights are written
                        ld32_start(tq, y[0]);
                        ld32_start(tq + 32u, y[1]);
                        tc_wait_ld_u32<32>(y[0]);
                        tc_wait_ld_u32<32>(y[1]);
                        const float m = fmaxf(largest<Q8>(y[0], scq, cs, here), largest<Q8>(y[1], scq + 32, cs, here - 32));
                        // this half's earlier O products are done: its next S, which came behind them, is
                        float f = 1.f;
                        if (m - kWtUp<Q8> > ref) {
                            f = ref == -INFINITY ? 0.f : ex2(ref - (m - kWtUp<Q8>));
                            ref = m - kWtUp<Q8>;
                            l *= f;
                        }
                        if (i >= 2) {
#pragma unroll 1
                            for (int c = 0; c < D / 32; ++c) {
                                float v[32];
                                uint32_t u[32];
                                ld32(tO + 32u * c, v);
#pragma unroll
                                for (int e = 0; e < 32; ++e) u[e] = __float_as_uint(v[e] * f);
                                tc_st16(tO + 32u * c, u);
                                tc_st16(tO + 32u * c + 16u, u + 16);
                            }
                        }
                        // and the chunk's weights so far
                        if (q > 0) tc_wait_st();
#pragma unroll 1
                        for (int c = 0; c < 2 * q; ++c) {
                            float v[32];
                            uint32_t u[32];
                            ld32(tS + 32u * c, v);
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                const float2 a0 = pair_of<Q8>(__float_as_uint(v[e])), a1 = pair_of<Q8>(__float_as_uint(v[16 + e]));
                                parts<Q8>((a0.x + a1.x) * f, (a0.y + a1.y) * f, u[e], u[16 + e]);
                            }
                            tc_st16(tS + 32u * c, u);
                            tc_st16(tS + 32u * c + 16u, u + 16);
                        }
                        weigh_all(y);
                    }
                    l += sum;
                    put_weights<Q8>(tq, w[0]);
                    if (q == 0) ld32_start(tS + 64u, x[1][0]);
                    put_weights<Q8>(tq + 32u, w[1]);
                    if (q == 0) ld32_start(tS + 96u, x[1][1]);
                }
                tc_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[h]);
            }
            // ---- this half's partial of its rows
            const int64_t rec = 2 * ((int64_t)blockIdx.x + w.item) + h;
            const int steps = (N - h + 1) / 2;
            if (steps > 0) {
                ok = ok && wt_wait(&o_done[h], no & 1u, bad);
                ++no;
            }
            tc_fence_after();
            const float fail = ok && !*bad ? 0.f : __uint_as_float(0x7fc00000u);
            if (row < rows) a.p_ml[rec * kWideRows + r] = make_float2(ref, l + fail);
            // O by way of shared memory, so that the stores are whole lines: D / 4 columns of the warp's rows at a time, over Q
            // (this half's own, all of whose products are done; with one tile for both halves, the unused second)
            if (steps > 0) {
                constexpr int CW = D / 4, PC = CW / 4;   // columns a turn, 16-byte pieces of them
                uint8_t *stage = sm + C::kQ + (pairs ? (uint32_t)(h * KB) * kWtBox : (uint32_t)KB * kWtBox + h * (32u * D * 4)) +
                                 quarter * (8u * D * 4);
                float *dst = a.p_o + (rec * kWideRows + quarter * 32) * D;
                auto place = [&](int row32, int c) {
                    return PC == 8 ? row32 * 128 + ((c ^ (row32 & 7)) << 4) : row32 * 64 + ((c ^ ((row32 >> 1) & 3)) << 4);
                };
#pragma unroll 1
                for (int q = 0; q < 4; ++q) {
                    uint32_t v[CW];
#pragma unroll
                    for (int e = 0; e < CW; e += 16) tc_ld16_nowait(tO + (uint32_t)(CW * q + e), v + e);
                    tc_wait_ld_u32<CW>(v);
#pragma unroll
                    for (int c = 0; c < PC; ++c)
                        *reinterpret_cast<uint4 *>(stage + place(lane, c)) = make_uint4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < PC; ++i) {
                        const int row32 = i * (32 / PC) + lane / PC, c = lane % PC;
                        const uint4 x = *reinterpret_cast<const uint4 *>(stage + place(row32, c));
                        if (tile * kWideRows + quarter * 32 + row32 < rows)
                            *reinterpret_cast<uint4 *>(dst + row32 * D + CW * q + 4 * c) = x;
                    }
                    __syncwarp();
                }
            }
            tc_fence_before();
            kc += w.n;
            soft_sync();                            // the next segment's Q may replace this one's
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 12) tmem_dealloc(tmem, 512);
}

template <bool Q8, int D> cudaError_t launch(const CachedArgs &a, int ctas, int dev, cudaStream_t s) {
    static std::atomic<bool> ready[64] = {};
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    auto fn = attn_prefix_tc_kernel<Q8, D>;
    if (!ready[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void *>(fn),
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, (int)WtCfg<D>::kSmem);
        if (e != cudaSuccess) return e;
        ready[dev] = true;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(kWtThreads);
    cfg.dynamicSmemBytes = WtCfg<D>::kSmem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fn, a);
}

}  // namespace

cudaError_t launch_attn_prefix_tc(bool q8, int d, const CachedArgs &a, int ctas, cudaStream_t s) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (d == 128) return q8 ? launch<true, 128>(a, ctas, dev, s) : launch<false, 128>(a, ctas, dev, s);
    return q8 ? launch<true, 64>(a, ctas, dev, s) : launch<false, 64>(a, ctas, dev, s);
}

}  // namespace qd
