// Norms of queries and keys head by head and the rotation to their positions, in one pass over a fused projection's
// rows that also writes the keys and values into the pages of a cache (8-bit or bf16 rows).
//
//   x' = x / sqrt(mean(x^2) + eps) * gamma,   y[d] = x'[d] c_d - x'[d + h] s_d,   y[d + h] = x'[d + h] c_d + x'[d] s_d   (h = D / 2)
//
// Every byte moves once, so HBM bounds it for prompts (28000 tokens of 32 + 16 heads, 688 MB, 121 us, 0.84 of the measured rate;
// 3248 fp32 tokens of 16 + 16 heads into 8-bit pages, 73 MB, 16 us, 0.68: the start's loads and the end take the rest), and the launch
// and three dependent loads (length, page and table row) for a step (64 tokens 3.2 us).  A row stands on D / 16 lanes, each with eight
// elements of the lower half and the eight that they are rotated with: nothing but the sum of squares (and the maximum of an
// 8-bit row) crosses lanes, and a lane keeps its eight cosines and sines of a token from head to head.  Everything is fp32 until the
// result is rounded once.
#include <algorithm>

#include "kv_view.cuh"
#include "mma_sync.cuh"
#include "qd_device.cuh"
#include "qd_internal.h"
#include "tc_common.cuh"

namespace qd {

namespace {

// CTAs an SM and rows ahead of a thread, the one at hand among them (16 x 2500 bf16 tokens of 32 + 16 heads, 8 x 512 fp32 tokens of 16 + 16:
// 4 CTAs 124 and 16.6 us, 5 121 and 15.9, 6 127 and 17.6; a row less 121 and 16.0, one more 122 and 16.9).
constexpr int kRopeThreads = 128, kRopeCtas = 5;
template <typename T> constexpr int kRopeAhead = sizeof(T) == 2 ? 4 : 3;

struct RopeArgs {
    const uint8_t *in[3];              // q, k, v rows
    uint8_t *out[3];                   // of the results (k, v: may be null)
    int64_t in_token[3], out_token[3]; // bytes
    const float *gamma[2];             // of q, k, or null
    float eps;
    const float *cos, *sin;            // [rope_rows][D / 2], or null
    const int32_t *pos;                // [N] or [3][N], or null: the positions in the cache
    int rope_rows, mrope3;             // frequencies below mrope3 take stream d % 3
    const int32_t *lengths, *offsets, *n_new;
    int B, T, N, qh, kvh;
    KvView pages;                      // k null: none
    const int32_t *table;
    int64_t table_stride;
    int table_pages, n_pages, page_shift;
    int units, run;                    // of heads of a token (a warp's rows each); of those of a warp
};

// A lane's 16 elements of a row of D: eight of the lower half (in chunks of 16 bytes, which are contiguous across the lanes: 32 bytes a lane in two loads
// took every 32-byte sector twice, 8 x 512 fp32 tokens 24 us) and the eight that they are rotated with.
template <typename T, int D> struct Sixteen {
    static constexpr int P = (int)sizeof(T), E = 16 / P;             // chunks, elements of one
    // chunk i's first element
    static __device__ __forceinline__ int at(int i, int lane) { return i * (D / P) + E * lane; }
    static __device__ __forceinline__ void get(const uint4 *u, float *f) {
#pragma unroll
        for (int i = 0; i < P; ++i) Elem<T>::unpack(u[i], f + i * E);
    }
};
// N elements as T, to memory.
template <typename T, int N> __device__ __forceinline__ void put(uint8_t *to, const float *f) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < N; i += 4) *reinterpret_cast<float4 *>(to + 4 * i) = make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]);
    } else if constexpr (N == 8) {
        *reinterpret_cast<uint4 *>(to) = make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
    } else {
        *reinterpret_cast<uint2 *>(to) = make_uint2(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]));
    }
}

// The stream of the token rows that a warp walks.
struct Stream {
    int b, first, end, base;                            // rows [first, end) are the stream's; row r stands at position base + r - first
    // The last stream that begins at row or before: 32 offsets at a time, coarse to fine.
    __device__ __forceinline__ void find(const RopeArgs &a, int row) {
        b = 0, first = 0, end = a.N, base = 0;
        if (!a.lengths) return;
        if (!a.offsets) {
            b = row / a.T;
            load(a);
            return;
        }
        const int lane = threadIdx.x & 31;
        int n = a.B;
        while (n > 1) {
            const int step = (n + 31) / 32, at = lane * step;
            const bool before = at < n && a.offsets[b + at] <= row;
            const int k = max(__popc(__ballot_sync(0xffffffffu, before)), 1) - 1;
            b += k * step, n = min(step, n - k * step);
        }
        load(a);
    }
    __device__ __forceinline__ void load(const RopeArgs &a) {
        if (a.offsets) {
            first = a.offsets[b], end = min(a.offsets[b + 1], a.N);
        } else {
            const int n = a.n_new ? a.n_new[b] : a.T;
            first = b * a.T, end = first + (n < 0 ? 0 : n > a.T ? a.T : n);
        }
        base = max(a.lengths[b], 0) - (end - first);
    }
    // On to the stream of a later row.
    __device__ __forceinline__ void go(const RopeArgs &a, int row) {
        if (row < end || !a.lengths) return;
        int then = b;
        if (a.offsets)
            while (then + 1 < a.B && a.offsets[then + 1] <= row) ++then;
        else
            then = row / a.T;
        if (then != b) {
            b = then;
            load(a);
        }
    }
};

// Where a token goes in the pages, and which rows of the tables it is rotated by.
struct Place {
    int page, r;                                        // page -1: not written, -2: the row is not in use
    int p[3];                                           // its position in every stream of positions
};
__device__ __forceinline__ Place place_of(const RopeArgs &a, Stream &s, int row, bool there) {
    Place x;
    x.page = -2, x.r = 0, x.p[0] = x.p[1] = x.p[2] = -1;
    if (!there) return x;
    s.go(a, row);
    if (row < s.first || row >= s.end || s.first < 0) return x;
    x.page = -1;
    const int at = a.lengths ? s.base + row - s.first : -1;
    if (a.table && at >= 0 && (at >> a.page_shift) < a.table_pages) {
        const int page = a.table[s.b * a.table_stride + (at >> a.page_shift)];
        x.r = at & ((1 << a.page_shift) - 1);
        if ((unsigned)page < (unsigned)a.n_pages) x.page = page;
    }
    if (a.pos) {
        x.p[0] = a.pos[row];
        if (a.mrope3) x.p[1] = a.pos[(int64_t)a.N + row], x.p[2] = a.pos[2 * (int64_t)a.N + row];
    } else {
        x.p[0] = at;
    }
    return x;
}

__device__ __forceinline__ void cp16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// A warp takes a few heads of one kind (q, k, v) of one token at a time (a row on D / 16 lanes) and walks a run of those, token by token, the same number
// for every warp, so that whatever goes by the kind or the token is the same for its lanes.  The rows ahead are on their way
// into shared memory, S of them, each thread's own 16 elements into a place of its own: nothing waits for another thread, and
// 64 KB an SM are in flight, where as many registers would leave no room (two rows ahead in registers: 16 x 2500 tokens 205 to
// 310 us).  A token's place is looked up two tokens ahead, its cosines and sines are loaded one ahead.
template <typename TI, typename TO, int D, bool Q8>
__global__ void __launch_bounds__(kRopeThreads, kRopeCtas) qk_norm_rope_kernel(const RopeArgs a) {
    using X = Sixteen<TI, D>;
    constexpr int LPR = D / 16, RPW = 32 / LPR, HALF = D / 2, P = X::P, E = X::E, S = kRopeAhead<TI>;
    __shared__ uint4 ring[S][P][kRopeThreads];
    const int lane = threadIdx.x % LPR, in = (threadIdx.x & 31) / LPR;    // this lane's share of a row; the row's place among the warp's
    pdl_wait();                                         // whatever wrote the rows
    pdl_launch_dependents();                            // (they wait for the whole grid before they read)
    const int warp = __shfl_sync(0xffffffffu, (int)(blockIdx.x * (kRopeThreads / 32) + threadIdx.x / 32), 0);
    const int64_t x0 = (int64_t)warp * a.run, left = (int64_t)a.N * a.units - x0;
    if (left <= 0) return;
    const int n = left < a.run ? (int)left : a.run;
    int row = (int)(x0 / a.units), unit = (int)(x0 - (int64_t)row * a.units);
    const int uq = (a.qh + RPW - 1) / RPW, uk = (a.kvh + RPW - 1) / RPW;   // units of q, of k
    const int last = row + (n + unit - 1) / a.units;    // the run's last token

    // the copies: of rows that no stream uses, too, which are there all the same
    int ci = 0, cu = unit, crow = row;                  // units so far; unit and token of the next
    const uint32_t mine = smem_addr(&ring[0][0][threadIdx.x]);
    auto copy = [&](int stage) {
        if (ci < n) {
            const int kind = cu < uq ? 0 : cu < uq + uk ? 1 : 2, of = (cu - (kind == 0 ? 0 : kind == 1 ? uq : uq + uk)) * RPW + in;
            const uint8_t *src = a.in[kind] + crow * a.in_token[kind] + (of * D + E * lane) * (int)sizeof(TI);
            if (of < (kind ? a.kvh : a.qh)) {
#pragma unroll
                for (int i = 0; i < P; ++i)
                    cp16(mine + (uint32_t)((stage * P + i) * kRopeThreads * 16), src + i * (D / P) * (int)sizeof(TI));
            }
            ++ci;
            if (++cu == a.units) cu = 0, ++crow;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    // of a vector in this lane's order: elements 4 i .. of its 16
    auto four = [&](const float *v, int i) {
        return __ldg(reinterpret_cast<const ulonglong2 *>(v + X::at(4 * i / E, lane) + 4 * i % E));
    };
    struct Angles {
        uint64_t c[4], s[4];
    };
    auto angles = [&](const Place &p) {
        Angles x;
        const float nan = __uint_as_float(0x7fc00000u);
#pragma unroll
        for (int i = 0; i < 4; ++i) x.c[i] = x.s[i] = pk(nan, nan);
        if (!a.cos || p.page == -2) return x;
        if (a.mrope3) {
            float c[8], s[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int d = X::at(e / E, lane) + e % E, k = d < a.mrope3 ? d % 3 : 0, q = k == 0 ? p.p[0] : k == 1 ? p.p[1] : p.p[2];
                const bool there = (unsigned)q < (unsigned)a.rope_rows;
                c[e] = there ? __ldg(a.cos + (int64_t)q * HALF + d) : nan;
                s[e] = there ? __ldg(a.sin + (int64_t)q * HALF + d) : nan;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) x.c[i] = pk(c[2 * i], c[2 * i + 1]), x.s[i] = pk(s[2 * i], s[2 * i + 1]);
        } else if ((unsigned)p.p[0] < (unsigned)a.rope_rows) {
            const float *c = a.cos + (int64_t)p.p[0] * HALF, *s = a.sin + (int64_t)p.p[0] * HALF;
            const ulonglong2 c0 = four(c, 0), c1 = four(c, 1), s0 = four(s, 0), s1 = four(s, 1);
            x.c[0] = c0.x, x.c[1] = c0.y, x.c[2] = c1.x, x.c[3] = c1.y;
            x.s[0] = s0.x, x.s[1] = s0.y, x.s[2] = s1.x, x.s[3] = s1.y;
        }
        return x;
    };
    const uint64_t minus = pk(-1.f, -1.f);
    // one unit of a token; every lane comes here (the sums cross lanes), `live` ones write
    auto finish = [&](const uint4 *in16, const Place &p, int row, int kind, int of, bool live, const Angles &w) {
        float f[16];
        X::get(in16, f);
        if (kind < 2) {
            uint64_t y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = pk(f[2 * e], f[2 * e + 1]);
            // the row's mean square crosses lanes while the elements are weighted and rotated; its root multiplies them last
            float inv = 1.f;
            const float *g = a.gamma[kind];
            if (g) {
                uint64_t sq = mul2(y[0], y[0]), sr = mul2(y[1], y[1]);
#pragma unroll
                for (int e = 2; e < 8; e += 2) sq = fma2(y[e], y[e], sq), sr = fma2(y[e + 1], y[e + 1], sr);
                float s0, s1;
                unpk(add2(sq, sr), s0, s1);
                float ss = s0 + s1;
#pragma unroll
                for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                inv = rsqrtf(fmaf(ss, 1.f / (float)D, a.eps));
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const ulonglong2 v = four(g, i);
                    y[2 * i] = mul2(y[2 * i], v.x), y[2 * i + 1] = mul2(y[2 * i + 1], v.y);
                }
            }
            if (a.cos) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint64_t l = y[e], u = y[4 + e];
                    y[e] = fma2(mul2(u, w.s[e]), minus, mul2(l, w.c[e]));
                    y[4 + e] = fma2(u, w.c[e], mul2(l, w.s[e]));
                }
            }
            const uint64_t inv2 = pk(inv, inv);
#pragma unroll
            for (int e = 0; e < 8; ++e) unpk(mul2(y[e], inv2), f[2 * e], f[2 * e + 1]);
        }
        if (live && a.out[kind]) {
            uint8_t *dst = a.out[kind] + row * a.out_token[kind] + (of * D + E * lane) * (int)sizeof(TO);
#pragma unroll
            for (int i = 0; i < P; ++i) put<TO, E>(dst + i * (D / P) * (int)sizeof(TO), f + i * E);
        }
        if (kind == 0 || p.page < 0) return;
        const int64_t to = p.page * a.pages.stream + p.r * a.pages.row + of * a.pages.head;
        uint8_t *dst = const_cast<uint8_t *>(kind == 1 ? a.pages.k : a.pages.v) + to;
        if constexpr (Q8) {
            uint64_t z = pk(0.f, 0.f);
            const uint64_t none = z;
            float most = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                z = fma2(pk(f[2 * e], f[2 * e + 1]), none, z);   // 0, or NaN where an element is not finite
                most = fmaxf(most, fmaxf(fabsf(f[2 * e]), fabsf(f[2 * e + 1])));
            }
            float z0, z1;
            unpk(z, z0, z1);
            uint32_t m = z0 + z1 == 0.f ? __float_as_uint(most) : 0x7fc00000u;
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
            // even lanes take one quotient, odd ones the other
            const bool finite = m < 0x7f800000u, zero = m < 0x05800000u;   // below 2^-116
            const float top = zero || !finite ? 1.f : __uint_as_float(m);
            float quot = __fdiv_rn(lane & 1 ? top : 127.f, lane & 1 ? 127.f : top);
            if (zero) quot = 0.f;
            const float by = __shfl_sync(0xffffffffu, quot, 0, LPR), scale = __shfl_sync(0xffffffffu, quot, 1, LPR);
            const uint64_t magic = pk(12582912.f, 12582912.f);
            uint32_t q[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                // the low byte is the code (the products singly: a packed product and sum became one fused operation, which rounds once)
                const uint64_t c0 = add2(pk(__fmul_rn(f[4 * i], by), __fmul_rn(f[4 * i + 1], by)), magic);
                const uint64_t c1 = add2(pk(__fmul_rn(f[4 * i + 2], by), __fmul_rn(f[4 * i + 3], by)), magic);
                q[i] = __byte_perm(__byte_perm((uint32_t)c0, (uint32_t)(c0 >> 32), 0x0040), __byte_perm((uint32_t)c1, (uint32_t)(c1 >> 32), 0x0040),
                                   0x5410);
                if (!finite) q[i] = 0;
            }
            if (live) {
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    if constexpr (E == 8)
                        *reinterpret_cast<uint2 *>(dst + X::at(i, lane)) = make_uint2(q[2 * i], q[2 * i + 1]);
                    else
                        *reinterpret_cast<uint32_t *>(dst + X::at(i, lane)) = q[i];
                }
                if (lane == 0)
                    const_cast<float *>(kind == 1 ? a.pages.ks : a.pages.vs)[p.page * a.pages.sstream + of * a.pages.shead + p.r] =
                        finite ? scale : __uint_as_float(0x7fc00000u);
            }
        } else if (live) {
#pragma unroll
            for (int i = 0; i < P; ++i) put<__nv_bfloat16, E>(dst + 2 * X::at(i, lane), f + i * E);
        }
    };

#pragma unroll
    for (int i = 0; i < S - 1; ++i) copy(i);
    Stream s;
    s.find(a, row);
    Place p0 = place_of(a, s, row, true), p1 = place_of(a, s, row + 1, row < last);
    Angles w0 = angles(p0), w1 = angles(p1);
    Place p2 = place_of(a, s, row + 2, row + 1 < last);
    int stage = 0;
    for (int i = 0; i < n; ++i) {
        copy(stage == 0 ? S - 1 : stage - 1);
        asm volatile("cp.async.wait_group %0;" ::"n"(S - 1) : "memory");
        uint4 u[P];
#pragma unroll
        for (int j = 0; j < P; ++j) u[j] = ring[stage][j][threadIdx.x];
        const int kind = unit < uq ? 0 : unit < uq + uk ? 1 : 2, of = (unit - (kind == 0 ? 0 : kind == 1 ? uq : uq + uk)) * RPW + in;
        if (p0.page != -2) finish(u, p0, row, kind, of, of < (kind ? a.kvh : a.qh), w0);
        stage = stage == S - 1 ? 0 : stage + 1;
        if (++unit == a.units) {
            unit = 0, ++row;
            p0 = p1, w0 = w1, p1 = p2;
            w1 = angles(p1);
            p2 = place_of(a, s, row + 2, row + 1 < last);
        }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

typedef void (*RopeFn)(const RopeArgs);
template <typename TI, typename TO> RopeFn rope_fn(int d, bool q8) {
    if (d == 64) return q8 ? qk_norm_rope_kernel<TI, TO, 64, true> : qk_norm_rope_kernel<TI, TO, 64, false>;
    return q8 ? qk_norm_rope_kernel<TI, TO, 128, true> : qk_norm_rope_kernel<TI, TO, 128, false>;
}

}  // namespace

}  // namespace qd

using namespace qd;

extern "C" qd_status qd_qk_norm_rope(const qd_rope_rows *x, void *cuda_stream) {
    if (!x || !x->q || !x->k || !x->q_out || x->n_tokens < 1 || x->n_q_heads < 1 || x->n_kv_heads < 1) return QD_EINVAL;
    if ((x->dtype != QD_F32 && x->dtype != QD_BF16) || (x->out_dtype != QD_F32 && x->out_dtype != QD_BF16)) return QD_EINVAL;
    if (x->head_dim != 64 && x->head_dim != 128) return QD_EUNSUPPORTED;
    const int d = x->head_dim;
    if (x->n_tokens > (1 << 30) || (int64_t)x->n_q_heads + 2 * (int64_t)x->n_kv_heads > 65536) return QD_EUNSUPPORTED;
    if (!(x->eps >= 0.0 && x->eps < 1e30)) return QD_EINVAL;
    if (!x->v && (x->v_out || x->pages)) return QD_EINVAL;
    if ((x->cos == nullptr) != (x->sin == nullptr) || (x->cos && x->rope_rows < 1)) return QD_EINVAL;
    if (x->mrope_h < 0 || 3 * (int64_t)x->mrope_h > d / 2 || (x->mrope_h && (!x->positions || !x->cos))) return QD_EINVAL;
    if (x->cos && !x->positions && !x->lengths) return QD_EINVAL;
    if (x->n_streams < 0 || (!x->lengths && (x->pages || x->offsets || x->n_new)) || (x->offsets && x->n_new)) return QD_EINVAL;
    if (x->lengths && (x->n_streams < 1 || (!x->offsets && x->n_tokens % x->n_streams))) return QD_EINVAL;
    const int64_t unit = x->dtype == QD_F32 ? 4 : 8, ou = x->out_dtype == QD_F32 ? 4 : 8, e = 16 / unit, oe = 16 / ou;
    const void *in[3] = {x->q, x->k, x->v};
    void *out[3] = {x->q_out, x->k_out, x->v_out};
    const int64_t in_stride[3] = {x->q_stride, x->k_stride, x->v_stride}, out_stride[3] = {x->q_out_stride, x->k_out_stride, x->v_out_stride};
    const int64_t N = x->n_tokens;
    for (int i = 0; i < 3; ++i) {
        const int64_t inner = (int64_t)(i ? x->n_kv_heads : x->n_q_heads) * d;
        if (in[i] && (in_stride[i] < 0 || in_stride[i] % unit || in_stride[i] > (int64_t(1) << 40) || !is_aligned(in[i], 16))) return QD_EINVAL;
        if (out[i] && (out_stride[i] % ou || out_stride[i] > (int64_t(1) << 40) || !is_aligned(out[i], 16) || (N > 1 && out_stride[i] < inner)))
            return QD_EINVAL;
    }
    // what is written lies over nothing else: a result may take its own rows' place (same type and stride), or a gap of a fused projection
    for (int i = 0; i < 3; ++i) {
        if (!out[i]) continue;
        const int64_t inner = (int64_t)(i ? x->n_kv_heads : x->n_q_heads) * d;
        for (int j = 0; j < 6; ++j) {
            const void *p = j < 3 ? in[j] : out[j - 3];
            if (!p || j == 3 + i) continue;
            const int64_t pe = j < 3 ? e : oe, ps = j < 3 ? in_stride[j] : out_stride[j - 3];
            const int64_t pi = (int64_t)(j % 3 ? x->n_kv_heads : x->n_q_heads) * d;
            if (j == i && p == out[i] && pe == oe && (N == 1 || ps == out_stride[i])) continue;
            if (!rows_beside(out[i], oe, N, out_stride[i], inner, p, pe, N, ps, pi)) return QD_EINVAL;
        }
    }
    for (const void *p : {(const void *)x->q_gamma, (const void *)x->k_gamma, (const void *)x->cos, (const void *)x->sin})
        if (!is_aligned(p, 16)) return QD_EINVAL;
    for (const void *p : {(const void *)x->positions, (const void *)x->lengths, (const void *)x->offsets, (const void *)x->n_new, (const void *)x->page_table})
        if (!is_aligned(p, 4)) return QD_EINVAL;
    qd_status st;
    int shift = 0;
    const qd_kv_cache *c = x->pages;
    if (c) {
        if ((st = check_pages(c, x->page_table, x->table_stride, x->table_pages, x->n_streams, -1, &shift)) != QD_OK) return st;
        if (c->n_kv_heads != x->n_kv_heads || c->head_dim != d) return QD_EINVAL;
        const int64_t ce = c->format == QD_KV_Q8 ? 1 : 2, H = c->n_kv_heads, P = c->n_streams;
        if (c->k == c->v || !apart(ce, d, {{H, c->head_stride}, {c->smax, c->row_stride}, {P, c->stream_stride}}, bytes_between(c->k, c->v)))
            return QD_EINVAL;
        if (c->format == QD_KV_Q8 && (c->k_scale == c->v_scale || !apart(4, c->smax, {{H, c->scale_head_stride}, {P, c->scale_stream_stride}},
                                                                        bytes_between(c->k_scale, c->v_scale))))
            return QD_EINVAL;
    }
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return QD_ECUDA;
    if (c && (st = check_pages(c, x->page_table, x->table_stride, x->table_pages, x->n_streams, dev, &shift)) != QD_OK) return st;
    for (const void *p : {x->q, x->k, (const void *)x->q_out})
        if (!on_device(p, dev)) return QD_EINVAL;
    for (const void *p : {x->v, (const void *)x->k_out, (const void *)x->v_out, (const void *)x->q_gamma, (const void *)x->k_gamma,
                          (const void *)x->cos, (const void *)x->sin, (const void *)x->positions, (const void *)x->lengths,
                          (const void *)x->offsets, (const void *)x->n_new})
        if (p && !on_device(p, dev)) return QD_EINVAL;

    RopeArgs a = {};
    for (int i = 0; i < 3; ++i) {
        a.in[i] = static_cast<const uint8_t *>(in[i]), a.out[i] = static_cast<uint8_t *>(out[i]);
        a.in_token[i] = in_stride[i] * e, a.out_token[i] = out_stride[i] * oe;
    }
    a.gamma[0] = x->q_gamma, a.gamma[1] = x->k_gamma, a.eps = (float)x->eps;
    a.cos = x->cos, a.sin = x->sin, a.pos = x->positions, a.rope_rows = x->rope_rows, a.mrope3 = 3 * x->mrope_h;
    a.lengths = x->lengths, a.offsets = x->offsets, a.n_new = x->n_new;
    a.B = x->n_streams, a.N = x->n_tokens, a.qh = x->n_q_heads, a.kvh = x->n_kv_heads;
    a.T = x->lengths && !x->offsets ? x->n_tokens / x->n_streams : 1;
    if (c) {
        a.pages = kv_view(c);
        a.table = x->page_table, a.table_stride = x->table_stride, a.table_pages = x->table_pages;
        a.n_pages = c->n_streams, a.page_shift = shift;
    }
    // a run for every warp that the SMs hold at once
    const int rpw = 512 / d, sms = sms_of(dev);
    a.units = (a.qh + rpw - 1) / rpw + (a.in[2] ? 2 : 1) * ((a.kvh + rpw - 1) / rpw);
    const int64_t units = (int64_t)a.N * a.units, warps = (int64_t)sms * kRopeCtas * (kRopeThreads / 32);
    a.run = (int)((units + warps - 1) / warps);
    const int64_t per = (int64_t)a.run * (kRopeThreads / 32);
    const dim3 grid((unsigned)((units + per - 1) / per));
    const bool q8 = c && c->format == QD_KV_Q8;
    const RopeFn fn = x->dtype == QD_F32 ? (x->out_dtype == QD_F32 ? rope_fn<float, float>(d, q8) : rope_fn<float, __nv_bfloat16>(d, q8))
                                         : (x->out_dtype == QD_F32 ? rope_fn<__nv_bfloat16, float>(d, q8)
                                                                   : rope_fn<__nv_bfloat16, __nv_bfloat16>(d, q8));
    // placed while a predecessor that allows it ends
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kRopeThreads);
    cfg.stream = static_cast<cudaStream_t>(cuda_stream);
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fn, a) == cudaSuccess ? QD_OK : QD_ECUDA;
}
