// Attention of many bf16 rows (all streams' new tokens and query heads) over the shared
// prefix on the tcgen05 tensor cores: the prefix is read once per 128 or 256 rows.
//
// Per key head the batch's rows in use stand one after the other in tiles of 128 (the M of an MMA); the keys
// come in chunks of 128.  A CTA has two halves, each with a tile of its own in flight (S, P and O in tensor
// memory), so that the tensor core works for one half while the other takes its softmax:
//   S = Q K^T          128 x 128 fp32 in tensor memory; Q and K from shared memory
//   softmax            thread = row: maximum, then P = 2^(s - ref) packed to 16 bits over S's own columns
//   O += P V           P from tensor memory, V from shared memory (keys x dims: the MN-major operand)
// With more than 128 rows the halves take two tiles of rows over the same chunks (K and V are shared);
// otherwise both take the one tile, every other chunk each.  The list (key head, tile pair, chunk) is cut into equal
// runs, one per CTA; each leaves (ref, sum, O) of its rows for attn_join_kernel.
//
// ref follows the running maximum at a distance (kAcUp, kAcRoom), so O is rescaled in tensor memory only
// when the maximum has moved far; the half's previous O product has finished when its next S has.
//
// bf16 prefix: P is one bf16 part (half a step 2^-8 of each probability, at random; a second part would add half the MMA
// time again).  8-bit prefix: the codes are widened to fp16, exactly, on their way into shared
// memory; the keys' scales multiply S's columns, the values' scales P's, and P is fp16 (2^-11).
//
// Roles (416 threads): warps 0-3 and 4-7 the softmax of the two halves (a row each, also Q and the results),
// warps 8 and 9 load K, 10 and 11 V, warp 12 owns the tensor memory and its lane 0 issues the MMAs.  Every wait
// is bounded; where one expires the CTA's partials become NaN and the roles run to their ends.
#include <cuda.h>

#include "attn_cached.cuh"
#include "qd_internal.h"
#include "tc_common.cuh"

namespace qd {

namespace {

constexpr int kWtThreads = 416;
constexpr int kWtSoft = 256, kWtLoad = 64;   // softmax threads, loading threads of K and of V
constexpr uint32_t kWtBox = 128 * 128;        // 128 rows of 128 bytes, 128-byte swizzle
constexpr uint32_t kWtS = 0, kWtO = 256;      // tensor memory columns: S (and P) of the halves, O

template <int D> struct WtCfg {
    static constexpr int KB = D / 64;                         // 64-wide blocks of head_dim
    static constexpr uint32_t kQ = 0;                         // Q [half][KB]
    static constexpr uint32_t kK = kQ + 2 * KB * kWtBox;      // K [stage][KB]
    static constexpr uint32_t kV = kK + 2 * KB * kWtBox;      // V [stage][KB]
    static constexpr uint32_t kSc = kV + 2 * KB * kWtBox;     // scales [stage][keys', values', log2 of values'][128]
    static constexpr uint32_t kOff = kSc + 2 * 3 * 128 * 4;   // first row of each stream
    static constexpr uint32_t kBar = kOff + (kWideMaxStreams + 1) * 4 + 4;
    static constexpr uint32_t kSmem = 1024 + kBar + 32 * 8;
};

// D (tensor memory) (+)= A (tensor memory, 16-bit pairs along K) * B^T (shared memory descriptor).
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(bdesc), "r"(idesc), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void tc_st16(uint32_t taddr, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// 32 consecutive fp32 columns of this thread's lane
__device__ __forceinline__ void ld32(uint32_t taddr, float *v) {
    uint32_t r[32];
    tc_ld16_nowait(taddr, r);
    tc_ld16_nowait(taddr + 16, r + 16);
    tc_wait_ld_u32<32>(r);
#pragma unroll
    for (int e = 0; e < 32; ++e) v[e] = __uint_as_float(r[e]);
}
// pairs of fp32 in one instruction
__device__ __forceinline__ uint64_t pk(float x, float y) {
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(x), "f"(y));
    return v;
}
__device__ __forceinline__ void unpk(uint64_t v, float &x, float &y) { asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v)); }
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
// 32 columns without waiting; ld_done makes them usable
__device__ __forceinline__ void ld32_start(uint32_t taddr, uint32_t *r) {
    tc_ld16_nowait(taddr, r);
    tc_ld16_nowait(taddr + 16, r + 16);
}

__device__ __forceinline__ uint64_t desc_mn(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)((lbo >> 4) & 0x3FFFu) << 16) |
           ((uint64_t)((sbo >> 4) & 0x3FFFu) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// Byte of 16-byte piece c (of 8) of row r in a swizzled box.
__device__ __forceinline__ uint32_t swz(int r, int c) { return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4)); }

__device__ __forceinline__ void soft_sync() { named_sync(1, kWtSoft); }

// Bounded wait; the flag ends all later ones at once.
__device__ __forceinline__ bool wt_wait(uint64_t *bar, uint32_t parity, volatile int *bad) {
    if (mbar_try_wait(bar, parity)) return true;
    const unsigned long long t0 = cycles_now();
    while (!mbar_try_wait(bar, parity)) {
        if (*bad) return false;
        if (cycles_now() - t0 > wait_cycles(kWaitLimitNs)) {
            *bad = 1;
            return false;
        }
    }
    return true;
}

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

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
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
    if (warp == 12) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    pdl_wait();
    pdl_launch_dependents();
    // rows in use, and where each stream's begin
    int rows;
    (void)wide_rows(a, 0, &rows);
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

    const WideItems items(rows);
    const bool pairs = items.pairs > 0;
    Walk w;
    const bool works = blockIdx.x < items.share(a, &w.sh) && rows > 0;
    w.chunks = a.wide_chunks;
    w.x = works ? w.sh.first(blockIdx.x) : 0u;
    w.x1 = works ? w.sh.first(blockIdx.x + 1) : 0u;
    const int P = a.max_len;

    if (warp >= 8 && warp < 12) {
        // ---- K or V chunks into the operands' layout
        const bool is_v = warp >= 10;
        const int tid = (threadIdx.x - kWtSoft) & (kWtLoad - 1);
        uint64_t *full = is_v ? v_full : k_full, *empty = is_v ? v_empty : k_empty;
        uint8_t *tiles = sm + (is_v ? C::kV : C::kK);
        int kc = 0;                                 // chunks so far
        bool ok = true;
        while (w.next()) {
            const int hk = w.item / items.per_head();
            const uint8_t *base = (is_v ? a.c.v : a.c.k) + hk * a.c.head;
            if constexpr (Q8) {
                constexpr int RPI = kWtLoad / 4, N = 128 / RPI * KB;   // four lanes a row of one 64-wide block
                const float *ks = a.c.ks + hk * a.c.shead, *vs = a.c.vs + hk * a.c.shead;
                const int j = tid & 3, r0 = tid >> 2;
                uint4 u[N];                         // the next chunk's codes
                float s[2][2];                      // V's warps: K's and V's scales of keys tid and tid + 64
                auto load = [&](int c) {
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        const int key = c * kWideKeys + r0 + (i / KB) * RPI;
                        u[i] = make_uint4(0, 0, 0, 0);
                        if (key < P) u[i] = __ldg(reinterpret_cast<const uint4 *>(base + (int64_t)key * a.c.row + (i % KB) * 64 + j * 16));
                    }
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int key = c * kWideKeys + tid + i * kWtLoad;
                        const bool live = is_v && key < P;
                        s[i][0] = live ? __ldg(ks + key) : 0.f, s[i][1] = live ? __ldg(vs + key) : 0.f;
                    }
                };
                load(w.c0);
                for (int i = 0; i < w.n; ++i, ++kc) {
                    const int st = kc & 1;
                    if (kc >= 2) ok = ok && wt_wait(&empty[st], ((uint32_t)(kc >> 1) & 1u) ^ 1u, bad);
                    uint8_t *tile = tiles + (uint32_t)(st * KB) * kWtBox;
#pragma unroll
                    for (int n = 0; n < N; ++n) {
                        const int r = r0 + (n / KB) * RPI;
                        const uint32_t x[4] = {u[n].x ^ 0x80808080u, u[n].y ^ 0x80808080u, u[n].z ^ 0x80808080u,
                                               u[n].w ^ 0x80808080u};
                        // eight lanes: two rows, whose swizzles differ in the last bit, and four even (odd) pieces
                        uint8_t *box = tile + (n % KB) * kWtBox;
                        *reinterpret_cast<uint4 *>(box + swz(r, 2 * j)) =
                            make_uint4(codes_f16<false>(x[0], 0x4140), codes_f16<false>(x[0], 0x4342),
                                       codes_f16<false>(x[1], 0x4140), codes_f16<false>(x[1], 0x4342));
                        *reinterpret_cast<uint4 *>(box + swz(r, 2 * j + 1)) =
                            make_uint4(codes_f16<false>(x[2], 0x4140), codes_f16<false>(x[2], 0x4342),
                                       codes_f16<false>(x[3], 0x4140), codes_f16<false>(x[3], 0x4342));
                    }
                    // the scales come with V, which is not given up before its softmax is done (K's tile is)
                    if (is_v) {
                        float *sc = reinterpret_cast<float *>(sm + C::kSc) + st * 384;
#pragma unroll
                        for (int n = 0; n < 2; ++n) {
                            const int key = tid + n * kWtLoad;
                            sc[key] = s[n][0], sc[128 + key] = s[n][1], sc[256 + key] = fmaxf(lg2(s[n][1]), -60.f);
                        }
                    }
                    fence_proxy_async_smem();
                    mbar_arrive(&full[st]);
                    if (i + 1 < w.n) load(w.c0 + i + 1);
                }
            } else {
                constexpr int PPR = D / 8, RPI = kWtLoad / PPR, N = 128 / RPI;
                const int j = tid % PPR, r0 = tid / PPR;
                for (int i = 0; i < w.n; ++i, ++kc) {
                    const int st = kc & 1;
                    if (kc >= 2) ok = ok && wt_wait(&empty[st], ((uint32_t)(kc >> 1) & 1u) ^ 1u, bad);
                    const uint32_t box = smem_addr(tiles + (uint32_t)(st * KB) * kWtBox) + (uint32_t)(j >> 3) * kWtBox;
#pragma unroll
                    for (int n = 0; n < N; ++n) {
                        const int r = r0 + n * RPI, key = (w.c0 + i) * kWideKeys + r;
                        const bool live = key < P;
                        const uint8_t *src = base + (int64_t)(live ? key : 0) * a.c.row + j * 16;
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(box + swz(r, j & 7)), "l"(src),
                                     "r"(live ? 16 : 0)
                                     : "memory");
                    }
                    asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;" ::: "memory");
                    fence_proxy_async_smem();
                    mbar_arrive(&full[st]);
                }
            }
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
    } else if (warp == 12) {
        // ---- the MMAs: S of both halves, then always a half's O followed by its next S
        if (lane == 0) {
            constexpr uint32_t bf = Q8 ? 0u : (1u << 7) | (1u << 10);
            constexpr uint32_t base = (1u << 4) | bf | ((uint32_t)(kWideRows >> 4) << 24);
            constexpr uint32_t idesc_s = base | ((uint32_t)(kWideKeys >> 3) << 17);
            constexpr uint32_t idesc_o = base | (1u << 16) | ((uint32_t)(D >> 3) << 17);
            const uint32_t sQ = smem_addr(sm + C::kQ), sK = smem_addr(sm + C::kK), sV = smem_addr(sm + C::kV);
            int kc = 0, seg = 0;
            uint32_t np[2] = {0, 0};               // P's so far
            bool ok = true;
            for (; ok && w.next(); ++seg) {
                const int N = pairs ? 2 * w.n : w.n;
                ok = wt_wait(&q_full[0], (uint32_t)seg & 1u, bad) && (!pairs || wt_wait(&q_full[1], (uint32_t)seg & 1u, bad));
                auto issue_s = [&](int i) {
                    const int h = i & 1, c = kc + (pairs ? i >> 1 : i), st = c & 1;
                    if (!pairs || !h) ok = ok && wt_wait(&k_full[st], (uint32_t)(c >> 1) & 1u, bad);
                    if (!ok) return;
                    tc_fence_after();
                    const uint32_t d = tmem + kWtS + 128u * h, q = sQ + (uint32_t)(pairs ? h * KB : 0) * kWtBox;
                    const uint32_t k = sK + (uint32_t)(st * KB) * kWtBox;
#pragma unroll
                    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                        for (int s = 0; s < 4; ++s)
                            tc_mma(d, sw128_desc(q + (uint32_t)kb * kWtBox + 32u * s),
                                   sw128_desc(k + (uint32_t)kb * kWtBox + 32u * s), idesc_s, (kb | s) ? 1u : 0u);
                    tc_commit(&s_full[h]);
                    if (!pairs || h) tc_commit(&k_empty[st]);
                };
                auto issue_o = [&](int i) {
                    const int h = i & 1, c = kc + (pairs ? i >> 1 : i), st = c & 1;
                    ok = ok && wt_wait(&p_full[h], np[h] & 1u, bad);
                    if (!pairs || !h) ok = ok && wt_wait(&v_full[st], (uint32_t)(c >> 1) & 1u, bad);
                    if (!ok) return;
                    ++np[h];
                    tc_fence_after();
                    const uint32_t d = tmem + kWtO + 128u * h, p = tmem + kWtS + 128u * h;
                    const uint32_t v = sV + (uint32_t)(st * KB) * kWtBox;
#pragma unroll
                    for (int ks = 0; ks < kWideKeys / 16; ++ks)
                        tc_mma_ts(d, p + 8u * ks, desc_mn(v + (uint32_t)ks * 2048u, kWtBox, 1024u), idesc_o,
                                  (i >= 2 || ks) ? 1u : 0u);
                    if (!pairs || h) tc_commit(&v_empty[st]);
                    if (i + 2 >= N) tc_commit(&o_done[h]);
                };
                for (int i = 0; ok && i < 2 && i < N; ++i) issue_s(i);
                for (int i = 0; ok && i < N; ++i) {
                    issue_o(i);
                    if (i + 2 < N) issue_s(i + 2);
                }
                kc += w.n;
            }
            // every MMA issued has completed before the tensor memory can be freed
            tc_commit(drain);
            (void)mbar_wait_bounded(drain, 0u, 20000000ull);
        }
        __syncwarp();
    } else {
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
            float cs = a.scale2;
            {
                uint4 u[D / 8];
#pragma unroll
                for (int i = 0; i < D / 8; ++i) u[i] = make_uint4(0, 0, 0, 0);
                if (row < rows) {
                    int b, in;
                    if (gaps) {
                        int lo = 0, hi = a.B;       // off[lo] <= row < off[hi]
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
                    const uint4 *src = reinterpret_cast<const uint4 *>(a.q + b * a.q_stream + tt * a.q_token +
                                                                       (int64_t)(hk * a.G + g) * D * 2);
#pragma unroll
                    for (int i = 0; i < D / 8; ++i) u[i] = __ldg(src + i);
                }
                if constexpr (Q8) {
                    // fp16, scaled by a power of two: the row's largest value to [2^14, 2^15)
                    uint32_t m = 0;
#pragma unroll
                    for (int i = 0; i < D / 8; ++i) {
                        const uint32_t x = __vmaxu2(__vmaxu2(u[i].x & 0x7fff7fffu, u[i].y & 0x7fff7fffu),
                                                    __vmaxu2(u[i].z & 0x7fff7fffu, u[i].w & 0x7fff7fffu));
                        m = __vmaxu2(m, x);
                    }
                    m = max(m >> 16, m & 0xffffu) >> 7;             // the exponent
                    const int up = min(268 - (int)m, 253);
                    const float f = __uint_as_float((uint32_t)up << 23);
                    cs *= __uint_as_float((uint32_t)(254 - up) << 23);
#pragma unroll
                    for (int i = 0; i < D / 8; ++i) {
                        u[i].x = pack_f16(bf16lo(u[i].x) * f, bf16hi(u[i].x) * f);
                        u[i].y = pack_f16(bf16lo(u[i].y) * f, bf16hi(u[i].y) * f);
                        u[i].z = pack_f16(bf16lo(u[i].z) * f, bf16hi(u[i].z) * f);
                        u[i].w = pack_f16(bf16lo(u[i].w) * f, bf16hi(u[i].w) * f);
                    }
                }
                if (pairs || h == 0) {
                    uint8_t *q = sm + C::kQ + (uint32_t)(h * KB) * kWtBox;
#pragma unroll
                    for (int i = 0; i < D / 8; ++i) *reinterpret_cast<uint4 *>(q + (uint32_t)(i >> 3) * kWtBox + swz(r, i & 7)) = u[i];
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&q_full[h]);
                }
            }
            float ref = -INFINITY, l = 0.f;
            const uint64_t cs2 = pk(cs, cs);
            const int N = pairs ? 2 * w.n : w.n;
            for (int i = h; i < N; i += 2) {
                const int c = pairs ? i >> 1 : i, st = (kc + c) & 1;
                const int left = P - (w.c0 + c) * kWideKeys;        // keys of the chunk
                const float *sc = reinterpret_cast<const float *>(sm + C::kSc) + st * 384;
                ok = ok && wt_wait(&s_full[h], ns & 1u, bad);
                ++ns;
                if constexpr (Q8) ok = ok && wt_wait(&v_full[st], (uint32_t)((kc + c) >> 1) & 1u, bad);
                tc_fence_after();
                // the chunk's largest score (with the values' scales: the largest weight), 64 keys at a time
                float m = -INFINITY;
#pragma unroll 1
                for (int q = 0; q < 2; ++q) {
                    uint32_t u[64];
                    ld32_start(tS + 64u * q, u);
                    ld32_start(tS + 64u * q + 32u, u + 32);
                    tc_wait_ld_u32<64>(u);
                    float m2 = -INFINITY;
#pragma unroll
                    for (int e = 0; e < 64; e += 4) {
                        float s0 = __uint_as_float(u[e]), s1 = __uint_as_float(u[e + 1]), s2 = __uint_as_float(u[e + 2]),
                              s3 = __uint_as_float(u[e + 3]);
                        if constexpr (Q8) {
                            const ulonglong2 k = *reinterpret_cast<const ulonglong2 *>(sc + 64 * q + e);
                            const ulonglong2 v = *reinterpret_cast<const ulonglong2 *>(sc + 256 + 64 * q + e);
                            unpk(fma2(mul2(pk(s0, s1), k.x), cs2, v.x), s0, s1);
                            unpk(fma2(mul2(pk(s2, s3), k.y), cs2, v.y), s2, s3);
                        } else {
                            unpk(mul2(pk(s0, s1), cs2), s0, s1);
                            unpk(mul2(pk(s2, s3), cs2), s2, s3);
                        }
                        if (left < kWideKeys) {
                            const int key = 64 * q + e;
                            s0 = key < left ? s0 : -INFINITY, s1 = key + 1 < left ? s1 : -INFINITY;
                            s2 = key + 2 < left ? s2 : -INFINITY, s3 = key + 3 < left ? s3 : -INFINITY;
                        }
                        m = fmaxf(m, fmaxf(s0, s1)), m2 = fmaxf(m2, fmaxf(s2, s3));
                    }
                    m = fmaxf(m, m2);
                }
                if (__any_sync(0xffffffffu, m > ref + kAcRoom)) {
                    // this half's earlier O products are done: its next S, which came behind them, is
                    float f = 1.f;
                    if (m > ref + kAcRoom) {
                        const float now = m - kAcUp;
                        f = ref == -INFINITY ? 0.f : ex2(ref - now);
                        ref = now;
                        l *= f;
                    }
                    if (i >= 2) {
#pragma unroll 1
                        for (int q = 0; q < D / 32; ++q) {
                            float v[32];
                            uint32_t u[32];
                            ld32(tO + 32u * q, v);
#pragma unroll
                            for (int e = 0; e < 32; ++e) u[e] = __float_as_uint(v[e] * f);
                            tc_st16(tO + 32u * q, u);
                            tc_st16(tO + 32u * q + 16u, u + 16);
                        }
                    }
                }
                const float rf = ref == -INFINITY ? 0.f : ref;
                const uint64_t rf2 = pk(-rf, -rf);
                uint64_t l2 = pk(l, 0.f);
                uint32_t u[2][32];                  // the next 32 keys' scores arrive while these are worked
                ld32_start(tS, u[0]);
                tc_wait_ld_u32<32>(u[0]);
#pragma unroll 1
                for (int q = 0; q < 4; q += 2) {
#pragma unroll
                    for (int z = 0; z < 2; ++z) {
                        const int key0 = 32 * (q + z);
                        if (z == 0 || q == 0) ld32_start(tS + key0 + 32u, u[z ^ 1]);
                        uint32_t o[16];
#pragma unroll
                        for (int e = 0; e < 32; e += 4) {
                            uint64_t x0 = pk(__uint_as_float(u[z][e]), __uint_as_float(u[z][e + 1]));
                            uint64_t x1 = pk(__uint_as_float(u[z][e + 2]), __uint_as_float(u[z][e + 3]));
                            if constexpr (Q8) {
                                const ulonglong2 k = *reinterpret_cast<const ulonglong2 *>(sc + key0 + e);
                                x0 = mul2(x0, k.x), x1 = mul2(x1, k.y);
                            }
                            float s0, s1, s2, s3;
                            unpk(fma2(x0, cs2, rf2), s0, s1);
                            unpk(fma2(x1, cs2, rf2), s2, s3);
                            s0 = ex2(s0), s1 = ex2(s1), s2 = ex2(s2), s3 = ex2(s3);
                            if (left < kWideKeys) {
                                const int key = key0 + e;
                                s0 = key < left ? s0 : 0.f, s1 = key + 1 < left ? s1 : 0.f;
                                s2 = key + 2 < left ? s2 : 0.f, s3 = key + 3 < left ? s3 : 0.f;
                            }
                            x0 = pk(s0, s1), x1 = pk(s2, s3);
                            l2 = add2(l2, add2(x0, x1));
                            if constexpr (Q8) {
                                const ulonglong2 v = *reinterpret_cast<const ulonglong2 *>(sc + 128 + key0 + e);
                                unpk(mul2(x0, v.x), s0, s1);
                                unpk(mul2(x1, v.y), s2, s3);
                            }
                            o[e / 2] = Q8 ? pack_f16(s0, s1) : pack_bf16(s0, s1);
                            o[e / 2 + 1] = Q8 ? pack_f16(s2, s3) : pack_bf16(s2, s3);
                        }
                        // these keys' columns lie in the first half of S's that have been read
                        if (z == 0 || q == 0) tc_wait_ld_u32<32>(u[z ^ 1]);
                        tc_st16(tS + key0 / 2, o);
                    }
                }
                {
                    float l0, l1;
                    unpk(l2, l0, l1);
                    l = l0 + l1;
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
            float *dst = a.p_o + (rec * kWideRows + r) * D;
            if (steps > 0) {
#pragma unroll 1
                for (int q = 0; q < D / 32; ++q) {
                    float v[32];
                    ld32(tO + 32u * q, v);
                    if (row < rows) {
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            *reinterpret_cast<float4 *>(dst + 32 * q + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
                    }
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
    static bool ready[64] = {};
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
