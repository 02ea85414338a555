// What the attention over caller-held caches shares between its passes: the arguments, the
// exact widening of codes, partial results, and the equal runs of a list of tiles.
#pragma once
#include <cuda_fp16.h>

#include "kv_view.cuh"
#include "mma_sync.cuh"
#include "qd_device.cuh"

namespace qd {

struct CachedArgs {
    KvView c;
    const uint8_t *q;
    uint8_t *out;
    int64_t q_stream, q_token, o_stream, o_token;   // bytes
    const int32_t *lengths, *n_new;
    int B, T, G, kvh, groups, max_len;
    int rows;                                       // rows of an item: T G, of the prefix B T G
    float scale2;                                   // softmax scale times log2(e)
    // a short prefix is read by every stream's own pass, behind its cache: its view, positions and tiles
    KvView pc;
    int pre_len, pre_tiles;
    // partials over the prefix: [kvh][B T G][splits]
    float2 *p_ml;
    float *p_o;
    int splits;
    // or, by attn_prefix_tc_kernel, of 128 rows each: records 2 (CTA + item) + {0, 1}, `wide` CTAs at most
    int wide, wide_chunks;
    // partials of attn_share_kernel: [slot][rows of a CTA]
    float2 *s_ml;
    float *s_o;
};

// Probabilities stand 2^10 above 1 at the running maximum and may grow to 2^15 before the
// sums are rescaled: fp16 then keeps 11 (two parts: 22) bits of every weight down to 2^-24
// (2^-10) of the largest, and small moves of the maximum cost nothing.
constexpr float kAcUp = 10.f, kAcRoom = 15.f;

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
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ float f16_of(float x) { return __half2float(__float2half_rn(x)); }
__device__ __forceinline__ float bf16_of(float x) { return __bfloat162float(__float2bfloat16_rn(x)); }

// Two code bytes (offset by 128) under the exponent of 1024: 1024 + u, less 1152 = code, exactly.
// RAW: 1152 + code, for a sum that starts at the offset's share.
template <bool RAW> __device__ __forceinline__ uint32_t codes_f16(uint32_t y, uint32_t sel) {
    const uint32_t h = __byte_perm(y, 0x64646464u, sel);
    if constexpr (RAW) return h;
    const __half2 v = __hsub2(*reinterpret_cast<const __half2 *>(&h), __half2half2(__ushort_as_half(0x6480)));
    return *reinterpret_cast<const uint32_t *>(&v);
}

// (ref, sum) of one partial: its weight against the reference M
__device__ __forceinline__ float part_weight(float2 ml, float M) { return ml.y == 0.f ? 0.f : ex2(ml.x - M); }

__device__ __forceinline__ int clamp_len(int len, int most) { return len < 0 ? 0 : len > most ? most : len; }
// Lengths, counts and queries are read by plain loads, which the fence or wait at a kernel's start orders (attn_share_kernel), not
// by non-coherent ones, which nothing does.
__device__ __forceinline__ int clamp_new(const CachedArgs &a, int b) {
    const int n = a.n_new ? a.n_new[b] : a.T;
    return n < 0 ? 0 : n > a.T ? a.T : n;
}
// A list of `total` tiles in equal runs, one per worker (warp or CTA).
struct Share {
    unsigned total, run, more;                       // tiles; a warp's run; the first `more` warps take one tile more
    __device__ __forceinline__ void use(unsigned all, unsigned warps) {
        total = all;
        run = all / warps, more = all - run * warps;
    }
    __device__ __forceinline__ unsigned first(unsigned w) const { return w * run + min(w, more); }
    __device__ __forceinline__ unsigned owner(unsigned x) const {   // x < total
        const unsigned big = more * (run + 1);
        return x < big ? x / (run + 1) : more + (x - big) / run;
    }
};

// ---- the prefix on the tcgen05 tensor cores (attn_prefix_tc.cu): bf16 rows, many of them
constexpr int kWideRows = 128;   // rows of a tile
constexpr int kWideKeys = 128;   // keys of a chunk
// The shortest run of chunks.  A longer one saves starts and partials; a shorter one takes more SMs, of which the own caches' pass
// beside it gets the rest.  Both move the time in steps, so no run is best everywhere; 2, 4, 6 and 8 chunks, call in us, 8 key heads: 2048
// bf16 positions under 64 x 16 rows 30.8, 33.5, 38.6, 39.0; 4096 37.1, 34.2, 39.1, 40.4, next to no own caches 23.2, 21.2,
// 28.0, 25.9; 8000 47.0, 42.7, 42.9, 45.8; 3000 under 32 x 2 x 16 26.6, 27.6, 30.0, 32.3; 8000 8-bit under 48 x 16
// 39.1, 38.4, 40.5, 42.4; 2000 under 96 x 4 x 32 90.3, 90.3, 92.2, 97.4.
constexpr unsigned kWideMinRun = 4;
constexpr int kWideMaxStreams = 2048;   // up to here the unused rows of a batch are left out

// Rows of the streams before `upto` (unused ones left out where n_new says so), and of all.
__device__ __forceinline__ int wide_rows(const CachedArgs &a, int upto, int *all) {
    const int per = a.T * a.G;
    if (!a.n_new || a.B > kWideMaxStreams) {
        *all = a.B * per;
        return upto * per;
    }
    const int lane = threadIdx.x & 31;
    int before = 0, sum = 0;
    for (int b = lane; b < a.B; b += 32) {
        const int n = clamp_new(a, b) * a.G;
        sum += n;
        if (b < upto) before += n;
    }
    *all = __reduce_add_sync(0xffffffffu, sum);
    return __reduce_add_sync(0xffffffffu, before);
}

// How the tiles of `rows` rows are worked: alone (both halves of a CTA take every other chunk of one tile) or in pairs.
struct WideItems {
    int pairs;                                      // items of a key head; 0: one tile alone
    __device__ __forceinline__ explicit WideItems(int rows) { pairs = rows > kWideRows ? (rows + 2 * kWideRows - 1) / (2 * kWideRows) : 0; }
    __device__ __forceinline__ int per_head() const { return pairs ? pairs : 1; }
    __device__ __forceinline__ unsigned share(const CachedArgs &a, Share *s) const {   // the CTAs that have a run
        const unsigned total = (unsigned)(a.kvh * per_head() * a.wide_chunks);
        const unsigned ctas = min((unsigned)a.wide, max(1u, total / kWideMinRun));
        s->use(total, ctas);
        return ctas;
    }
};

cudaError_t launch_attn_prefix_tc(bool q8, int d, const CachedArgs &a, int ctas, cudaStream_t s);

}  // namespace qd
