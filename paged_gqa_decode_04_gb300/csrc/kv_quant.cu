// The write side of a serving step over ragged batches: K and V rows into the
// pages, quantised as they are written (paged_kv_write), and the same with the
// per-head norm of queries and keys and the rotation by position in one pass
// (paged_qk_norm_rope_write).  See include/paged_kv_manager.h for the contract.
//
// Mathematics of a head vector x of D elements at position p:
//     r = rsqrt(mean(x^2) + eps)                                (norm, optional)
//     y_e = r (x_e w_e cos - x_f w_f sin)   or   r (x_e w_e cos + x_f w_f sin)
// for the first or second of a rotated pair (e, f), cos and sin from the caller's table at
// p, and y_e = r x_e w_e outside the rotated part: with w_e cos and -+ w_f sin made once
// for a token, two products, a sum and r for all its heads.
//     8-bit pages: code = rn(y / scale), saturated.
// All of it in float32 and in registers, with one rounding at the end: to the output
// type, or to the code.
//
// What bounds it: bytes, once the instructions are few.  Every row is read once and written
// once.  16-byte accesses, a lane holds 8 consecutive elements of a head (16 lanes a vector
// at D = 128), sums of squares and rotation partners by shuffles, and a warp issues the
// loads of 16 head vectors before it uses the first.
//
// Work of a warp.  One token's 16 query heads, or 8 KV heads with K and V, whose angles and
// weights are loaded once.  Where a scale belongs to a block, K and V go by blocks instead,
// since the largest magnitude of a block's new rows has to be known before its first code.
// A plain write takes one (block, KV head, K or V) a warp; its rows stay in registers in
// between (but for blocks of 256 tokens, whose first half is loaded again), and blocks of more
// than 16 tokens are shared by up to 8 warps of a CTA, which exchange their maxima through
// shared memory.  With norm and rotation a CTA takes a block of 8 KV heads, and its rows are
// loaded, normed and rotated twice, for the maxima and for the codes.  Its warps join their
// maxima with an atomic maximum in shared memory, which has no order; no two warps write one
// scale: the pages do not depend on timing.
//
// Measured, 8 KV heads of 128 (share of the time a plain copy of the bytes takes): 67k tokens
// into e4m3 pages with a scale per block 71.6 us (86%); norm, rotation and write of 67k tokens
// with 32 query heads into bfloat16 pages 287 us (88%), of 17k tokens with 64 query heads into
// e4m3 pages with a scale per block 142 us (69%: instructions, issued in 65% of the cycles, of
// the keys' norm and rotation done twice, and of spills: 368 bytes of stores and 356 of loads at
// the 80 registers of three CTAs).  2737 tokens of 40 heads into int8 pages with a scale per head
// 22.0 us; a copy of the same 84 MB takes 20.7.
#include <cuda_fp8.h>

#include "page_ops.h"
#include "paged_kv_manager.h"
#include "ragged.cuh"

namespace pgd {
namespace {

constexpr int kWarps = 8;         // warps of a CTA
constexpr int kChunk = 16;        // head vectors a warp loads before it uses them
constexpr float kTiny = 1.17549435e-38f;  // smallest normal number

struct Prep {
    const void* q_weight;  // [D], null: no norm of the queries
    const void* k_weight;
    int weight_f32;        // weights in float32, else bfloat16
    float eps;
    const float* rope;     // [rows][2][rope_dim / 2], null: no rotation
    int rope_dim;
    int interleaved;       // pairs (2j, 2j + 1), else (j, j + rope_dim / 2)
};

struct WriteArgs {
    Ragged r;
    Prep prep;
    const void* q;
    void* q_out;
    int64_t q_stride, q_out_stride;
    int hq;
    const void* k;
    const void* v;
    int64_t k_stride, v_stride;
    int hkv;
    void* k_pool;
    void* v_pool;
    float* k_scale;
    float* v_scale;
    int chunk_shift;      // scale per block: log2 of the block's tokens,
    int warps_per_unit;   // warps sharing one (block, head, K or V),
    uint32_t block_ctas;  // and the CTAs of these units; token units follow
    uint32_t q_groups;    // units of a token: 16 query heads each,
    uint32_t kv_groups;   // then 8 KV heads each
};

// ---------------------------------------------------------- 8 elements of a lane
template <typename Act>
struct Raw;
template <>
struct Raw<__nv_bfloat16> {
    uint4 a;
    __device__ void load(const __nv_bfloat16* p) { a = *reinterpret_cast<const uint4*>(p); }
    __device__ void zero() { a = make_uint4(0, 0, 0, 0); }
    __device__ Raw from(int lane) const {  // the same 8 places of another lane
        Raw r;
        r.a = make_uint4(__shfl_sync(0xffffffffu, a.x, lane), __shfl_sync(0xffffffffu, a.y, lane),
                         __shfl_sync(0xffffffffu, a.z, lane), __shfl_sync(0xffffffffu, a.w, lane));
        return r;
    }
    __device__ void get(float (&x)[8]) const {
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
};
template <>
struct Raw<float> {
    float4 a, b;
    __device__ void load(const float* p) {
        a = reinterpret_cast<const float4*>(p)[0];
        b = reinterpret_cast<const float4*>(p)[1];
    }
    __device__ void zero() { a = b = make_float4(0, 0, 0, 0); }
    __device__ Raw from(int lane) const {
        Raw r;
        r.a = make_float4(__shfl_sync(0xffffffffu, a.x, lane), __shfl_sync(0xffffffffu, a.y, lane),
                          __shfl_sync(0xffffffffu, a.z, lane), __shfl_sync(0xffffffffu, a.w, lane));
        r.b = make_float4(__shfl_sync(0xffffffffu, b.x, lane), __shfl_sync(0xffffffffu, b.y, lane),
                          __shfl_sync(0xffffffffu, b.z, lane), __shfl_sync(0xffffffffu, b.w, lane));
        return r;
    }
    __device__ void get(float (&x)[8]) const {
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
        x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    }
};

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&x)[8]) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]),
                                              pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}

// ------------------------------------------------------------------------ codes
template <int PAGE>
__device__ __forceinline__ constexpr float code_max() {
    return PAGE == PGD_INT8 ? 127.f : 448.f;
}

// 0 for scales below the smallest normal number, whose reciprocal may be infinite (zeros would
// become NaN).
__device__ __forceinline__ float inverse(float scale) {
    return scale >= kTiny ? 1.f / scale : 0.f;
}

// 8 codes of values already divided by their scale: nearest, ties to even, saturated.
// NaN gives the NaN code of e4m3 and 0 in int8, which has none.
template <int PAGE>
__device__ __forceinline__ uint2 codes8(const float (&x)[8]) {
    uint32_t w[2];
    if (PAGE == PGD_INT8) {
        // 1.5 * 2^23 more, a float32 has its integer, rounded to even, in its low bits
        uint32_t c[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float v = x[i] == x[i] ? fminf(fmaxf(x[i], -127.f), 127.f) : 0.f;
            c[i] = __float_as_uint(v + 12582912.f);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
            w[i] = __byte_perm(__byte_perm(c[4 * i], c[4 * i + 1], 0x0040),
                               __byte_perm(c[4 * i + 2], c[4 * i + 3], 0x0040), 0x5410);
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * i], x[4 * i + 1]),
                                                         __NV_SATFINITE, __NV_E4M3);
            const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * i + 2], x[4 * i + 3]),
                                                         __NV_SATFINITE, __NV_E4M3);
            w[i] = lo | hi << 16;
        }
    }
    return make_uint2(w[0], w[1]);
}

template <int PAGE>
__device__ __forceinline__ void values8(uint2 c, float (&x)[8]) {
    const uint32_t w[2] = {c.x, c.y};
    if (PAGE == PGD_INT8) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = float(int8_t(w[i / 4] >> (8 * (i % 4))));
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
                __nv_fp8x2_storage_t(w[i / 2] >> (16 * (i % 2))), __NV_E4M3);
            const float2 f = __half22float2(__half2(h));
            x[2 * i] = f.x, x[2 * i + 1] = f.y;
        }
    }
}

// ------------------------------------------------------------- norm and rotation
// The lane's 8 weights at d0 (ones without a norm).
__device__ __forceinline__ void load_weights(const void* w, int f32, int d0, float (&out)[8]) {
    if (!w) {
#pragma unroll
        for (int i = 0; i < 8; ++i) out[i] = 1.f;
    } else if ((reinterpret_cast<uintptr_t>(w) & 15) != 0) {  // a weight inside a larger tensor
#pragma unroll
        for (int i = 0; i < 8; ++i)
            out[i] = f32 ? __ldg(static_cast<const float*>(w) + d0 + i)
                         : __bfloat162float(static_cast<const __nv_bfloat16*>(w)[d0 + i]);
    } else if (f32) {
        Raw<float> r;
        r.load(static_cast<const float*>(w) + d0);
        r.get(out);
    } else {
        Raw<__nv_bfloat16> r;
        r.load(static_cast<const __nv_bfloat16*>(w) + d0);
        r.get(out);
    }
}

__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p));
    const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}

// Place of the lane's 8 elements in the rotation, and their weights and partners' weights.
struct Place {
    int d0;
    bool in, low;  // inside the rotated part; first of a pair (two halves)
    int src;       // lane that has the partners (two halves), else this one
    bool norm;
    float w[8], wp[8];

    __device__ __forceinline__ Place(const Prep& pr, const void* weight, int d) {
        const int half = pr.rope_dim / 2, lane = threadIdx.x & 31;
        d0 = d;
        in = d < pr.rope_dim;
        low = d < half;
        src = !in || pr.interleaved ? lane : low ? lane + half / 8 : lane - half / 8;
        norm = weight != nullptr;
        load_weights(weight, pr.weight_f32, d, w);
        if (in && !pr.interleaved)
            load_weights(weight, pr.weight_f32, low ? d + half : d - half, wp);
    }
};

// What the lane's 8 elements of a token's heads are multiplied with: themselves and their
// partners.
struct Turn {
    float own[8], other[8];

    __device__ __forceinline__ Turn(const Prep& pr, const Place& at, int p) {
        const int half = pr.rope_dim / 2;
        const float* const t = pr.rope + (int64_t)p * pr.rope_dim;
#pragma unroll
        for (int i = 0; i < 8; ++i) own[i] = at.w[i], other[i] = 0.f;
        if (!at.in) return;  // also without a rotation
        if (pr.interleaved) {
            const float4 c4 = __ldg(reinterpret_cast<const float4*>(t + at.d0 / 2));
            const float4 s4 = __ldg(reinterpret_cast<const float4*>(t + half + at.d0 / 2));
            const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                other[2 * i] = -own[2 * i + 1] * s[i];
                other[2 * i + 1] = own[2 * i] * s[i];
                own[2 * i] *= c[i];
                own[2 * i + 1] *= c[i];
            }
        } else {
            float c[8], s[8];
            load8(t + (at.low ? at.d0 : at.d0 - half), c);
            load8(t + half + (at.low ? at.d0 : at.d0 - half), s);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                own[i] *= c[i];
                other[i] = at.low ? -at.wp[i] * s[i] : at.wp[i] * s[i];
            }
        }
    }

    // The lane's 8 elements of a vector, normed and rotated; a whole warp calls it together.
    template <typename Act, int D>
    __device__ __forceinline__ void apply(const Prep& pr, const Place& at, const Raw<Act>& raw,
                                          float (&y)[8]) const {
        float x[8], z[8];
        raw.get(x);
        float r = 1.f;
        if (at.norm) {
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
            for (int k = 1; k < D / 8; k *= 2) ss += __shfl_xor_sync(0xffffffffu, ss, k);
            r = rsqrtf(ss * (1.f / D) + pr.eps);
        }
        if (pr.interleaved) {
#pragma unroll
            for (int i = 0; i < 8; ++i) z[i] = x[i ^ 1];
        } else {
            raw.from(at.src).get(z);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            y[i] = x[i] * own[i];
            if (at.in) y[i] = fmaf(z[i], other[i], y[i]);
            y[i] *= r;
        }
    }
};

template <int PAGE>
struct PageType {
    using type = uint8_t;
};
template <>
struct PageType<PGD_F32> {
    using type = float;
};
template <>
struct PageType<PGD_BF16> {
    using type = __nv_bfloat16;
};

// ------------------------------------------------- K, V with a scale for each block
// Largest finite magnitude of 8 elements, joined with `top`.
__device__ __forceinline__ float finite_max(const float (&x)[8], float top) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float m = fabsf(x[i]);
        top = fmaxf(top, m < INFINITY ? m : 0.f);
    }
    return top;
}

// Block number `piece` of the call: its sequence, its first token, its rows [lo, hi) to
// write and its place in the pool (-1: none, or out of range).
struct Block {
    Seq s;
    int at, lo, hi;
    int64_t id;

    __device__ __forceinline__ Block(const WriteArgs& a, uint32_t piece) {
        s.ok = false;
        at = lo = hi = 0;
        id = -1;
        const int b = find_seq(a.r, piece, 1, a.chunk_shift, 2);
        if (b >= a.r.B) return;
        s = load_seq(a.r, b);
        if (!s.ok || s.n > s.len) return;
        const int start = s.len - s.n;
        const int i = (start >> a.chunk_shift) +
                      int(piece - first_piece(a.r, b, 1, a.chunk_shift, 2));
        const int64_t first = (int64_t)i << a.chunk_shift;
        lo = int(max(first, (int64_t)start) - first);
        hi = first < s.len ? int(min((int64_t)s.len - first, (int64_t)1 << a.chunk_shift)) : 0;
        if (hi <= lo) return;
        at = int(first);
        id = block_of(a.r, b, i);
    }
    // packed row of the block's row 0
    __device__ __forceinline__ int64_t row() const { return s.row0 + at - (s.len - s.n); }
};

// The scale a block takes from the largest magnitude of its new rows and the scale before.
template <int PAGE>
__device__ __forceinline__ float new_scale(float top, float was) {
    const float now = top * (1.f / code_max<PAGE>());
    return fmaxf(now >= kTiny ? now : 0.f, was);
}

// 8 codes at a larger scale: rows cached in a block before this call.
template <int PAGE>
__device__ __forceinline__ void requantise(uint8_t* p, float ratio) {
    float x[8];
    values8<PAGE>(*reinterpret_cast<uint2*>(p), x);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] *= ratio;
    *reinterpret_cast<uint2*>(p) = codes8<PAGE>(x);
}

// Largest finite magnitude of some vectors of a lane.  bfloat16 magnitudes are ordered like
// their bits, two of them at once.
template <int N>
__device__ __forceinline__ float largest(const Raw<__nv_bfloat16> (&raw)[N]) {
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        most = __vmaxu2(most, raw[i].a.x & 0x7fff7fffu);
        most = __vmaxu2(most, raw[i].a.y & 0x7fff7fffu);
        most = __vmaxu2(most, raw[i].a.z & 0x7fff7fffu);
        most = __vmaxu2(most, raw[i].a.w & 0x7fff7fffu);
    }
    most = max(most & 0xffffu, most >> 16);
    if (most < 0x7f80u) return __uint_as_float(most << 16);
    float top = 0.f;  // an infinity or NaN, which take no part
#pragma unroll
    for (int i = 0; i < N; ++i) {
        float x[8];
        raw[i].get(x);
        top = finite_max(x, top);
    }
    return top;
}

template <int PAGE, int D>
__device__ __forceinline__ void write_blocks(const WriteArgs& a, float* smax) {
    using Act = __nv_bfloat16;
    constexpr int kLanes = D / 8;              // lanes of a head vector
    constexpr int kRows = 32 / kLanes;         // vectors of a warp at once
    constexpr int kIters = kChunk / kRows;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int sub = lane / kLanes, d0 = lane % kLanes * 8;
    const int W = a.warps_per_unit, part = warp % W;
    const uint32_t unit = blockIdx.x * (kWarps / W) + warp / W, per = 2 * a.hkv;
    const int side = int(unit % per) / a.hkv, h = int(unit % per) % a.hkv;
    const Block blk(a, unit / per);
    const int lo = blk.lo, hi = blk.hi;
    const int64_t stride = side ? a.v_stride : a.k_stride;
    // this lane's elements of packed row j of the block, and of pool row j
    const Act* const src =
        static_cast<const Act*>(side ? a.v : a.k) + blk.row() * stride + h * D + d0;
    const int row = a.hkv * D;
    const int64_t id = max(blk.id, (int64_t)0);
    uint8_t* const dst = static_cast<uint8_t*>(side ? a.v_pool : a.k_pool) +
                         (id << a.chunk_shift) * row + h * D + d0;
    float* const scale = (side ? a.v_scale : a.k_scale) + id * a.hkv + h;
    const int rows = 1 << a.chunk_shift;
    const int passes = (rows + W * kChunk - 1) / (W * kChunk);

    Raw<Act> raw[kIters];
    auto load = [&](int j0) {
#pragma unroll
        for (int i = 0; i < kIters; ++i) {
            const int j = j0 + i * kRows + sub;
            raw[i].zero();
            if (j >= lo && j < hi) raw[i].load(src + j * stride);
        }
    };
    // the old scale first: its latency passes under the rows' loads
    const float was = blk.id >= 0 && lo > 0 ? *scale : 0.f;
    float top = 0.f;
    for (int p = 0; p < passes && blk.id >= 0; ++p) {
        load((p * W + part) * kChunk);
        top = fmaxf(top, largest(raw));
    }
#pragma unroll
    for (int m = 1; m < 32; m *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
    if (W > 1) {
        if (lane == 0) smax[warp] = top;
        __syncthreads();
        for (int i = 0; i < W; ++i) top = fmaxf(top, smax[warp / W * W + i]);
    }
    if (blk.id < 0) return;
    const float now = new_scale<PAGE>(top, was), inv = inverse(now);
    if (part == 0 && lane == 0) *scale = now;
    if (now > was)
        for (int j = part * kRows + sub; j < lo; j += W * kRows)
            requantise<PAGE>(dst + j * row, was * inv);
    for (int p = passes - 1; p >= 0; --p) {
        const int j0 = (p * W + part) * kChunk;
        if (p != passes - 1) load(j0);
#pragma unroll
        for (int i = 0; i < kIters; ++i) {
            const int j = j0 + i * kRows + sub;
            float x[8];
            raw[i].get(x);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] *= inv;
            if (j >= lo && j < hi) *reinterpret_cast<uint2*>(dst + j * row) = codes8<PAGE>(x);
        }
    }
}

// The same with keys normed and rotated first: a CTA takes a block of 8 KV heads, K and V,
// and a warp one token after the other, so that a token's angles serve all its heads.  Rows
// are read twice (the second time from L1) instead of held: 8 heads of float32 values would
// leave room for few warps.  `smax`: the largest magnitudes of [K, V][8 heads].
template <int PAGE, int D>
__device__ __forceinline__ void norm_blocks(const WriteArgs& a, float* smax) {
    using Act = __nv_bfloat16;
    constexpr int kLanes = D / 8, kRows = 32 / kLanes, kHeads = kChunk / 2;
    constexpr int kIters = kHeads / kRows;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int sub = lane / kLanes, d0 = lane % kLanes * 8;
    const uint32_t groups = (a.hkv + kHeads - 1) / kHeads;
    const int h0 = int(blockIdx.x % groups) * kHeads + sub;  // head of vector i: h0 + i kRows
    const Block blk(a, blockIdx.x / groups);
    if (blk.id < 0) return;  // the whole CTA
    const int lo = blk.lo, hi = blk.hi, row = a.hkv * D;
    const Act* const k = static_cast<const Act*>(a.k) + blk.row() * a.k_stride + h0 * D + d0;
    const Act* const v = static_cast<const Act*>(a.v) + blk.row() * a.v_stride + h0 * D + d0;
    const int64_t pool_at = (blk.id << a.chunk_shift) * row + h0 * D + d0;
    const Place place(a.prep, a.prep.k_weight, d0);

    Raw<Act> rk[kIters], rv[kIters];
    auto load = [&](int j) {
#pragma unroll
        for (int i = 0; i < kIters; ++i) {
            rk[i].zero();
            rv[i].zero();
            if (h0 + i * kRows < a.hkv) {
                rk[i].load(k + j * a.k_stride + i * kRows * D);
                rv[i].load(v + j * a.v_stride + i * kRows * D);
            }
        }
    };
    float top[2][kIters] = {}, was[2][kIters] = {};
    if (threadIdx.x < 2 * kHeads) smax[threadIdx.x] = 0.f;
    for (int j = lo + warp; j < hi; j += kWarps) {
        load(j);
        const Turn turn(a.prep, place, blk.at + j);
#pragma unroll
        for (int i = 0; i < kIters; ++i) {
            float y[8];
            turn.template apply<Act, D>(a.prep, place, rk[i], y);
            top[0][i] = finite_max(y, top[0][i]);
            const Raw<Act> one[1] = {rv[i]};
            top[1][i] = fmaxf(top[1][i], largest(one));
        }
    }
    __syncthreads();  // smax is zero
#pragma unroll
    for (int side = 0; side < 2; ++side)
#pragma unroll
        for (int i = 0; i < kIters; ++i) {
            const int h = h0 + i * kRows;
            float t = top[side][i];
#pragma unroll
            for (int m = 1; m < kLanes; m *= 2) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, m));
            // magnitudes are ordered like their bits; a maximum has no order of arrival
            if (lane % kLanes == 0)
                atomicMax(reinterpret_cast<int*>(smax) + side * kHeads + i * kRows + sub,
                          __float_as_int(t));
            if (lo > 0 && h < a.hkv)
                was[side][i] = (side ? a.v_scale : a.k_scale)[blk.id * a.hkv + h];
        }
    __syncthreads();
    float inv[2][kIters];
#pragma unroll
    for (int side = 0; side < 2; ++side)
#pragma unroll
        for (int i = 0; i < kIters; ++i) {
            const int h = h0 + i * kRows;
            uint8_t* const dst =
                static_cast<uint8_t*>(side ? a.v_pool : a.k_pool) + pool_at + i * kRows * D;
            const float now =
                new_scale<PAGE>(smax[side * kHeads + i * kRows + sub], was[side][i]);
            inv[side][i] = inverse(now);
            if (h >= a.hkv) continue;
            if (warp == 0 && lane % kLanes == 0)
                (side ? a.v_scale : a.k_scale)[blk.id * a.hkv + h] = now;
            if (now > was[side][i])
                for (int j = warp; j < lo; j += kWarps)
                    requantise<PAGE>(dst + j * row, was[side][i] * inv[side][i]);
        }
    for (int j = lo + warp; j < hi; j += kWarps) {
        load(j);
        const Turn turn(a.prep, place, blk.at + j);
#pragma unroll
        for (int i = 0; i < kIters; ++i) {
            float y[8], x[8];
            turn.template apply<Act, D>(a.prep, place, rk[i], y);
            rv[i].get(x);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                y[e] *= inv[0][i];
                x[e] *= inv[1][i];
            }
            if (h0 + i * kRows >= a.hkv) continue;
            const int64_t to = pool_at + j * row + i * kRows * D;
            *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.k_pool) + to) = codes8<PAGE>(y);
            *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.v_pool) + to) = codes8<PAGE>(x);
        }
    }
}

// ------------------------------------------------------------------ heads of a token
template <typename Act, int PAGE, int D, bool PREP>
__device__ __forceinline__ void write_tokens(const WriteArgs& a) {
    constexpr int kLanes = D / 8, kRows = 32 / kLanes, kIters = kChunk / kRows;
    constexpr bool q8 = PAGE == PGD_FP8_E4M3 || PAGE == PGD_INT8;
    using Page = typename PageType<PAGE>::type;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int sub = lane / kLanes, d0 = lane % kLanes * 8;
    const uint32_t groups = a.q_groups + a.kv_groups;
    const uint32_t unit = (blockIdx.x - a.block_ctas) * kWarps + warp;
    const int t = unit / groups, group = unit % groups;
    if (t >= a.r.total) return;
    const bool kv = group >= (int)a.q_groups;
    const int h0 = kv ? (group - a.q_groups) * (kChunk / 2) : group * kChunk;
    // vector i of the unit: query head h0 + i, or K of KV head h0 + i, i < 8, then V
    Raw<Act> raw[kIters];
    const Act* const q = static_cast<const Act*>(a.q) + t * a.q_stride + d0;
    const Act* const k = static_cast<const Act*>(a.k) + t * a.k_stride + d0;
    const Act* const v = static_cast<const Act*>(a.v) + t * a.v_stride + d0;
#pragma unroll
    for (int i = 0; i < kIters; ++i) {  // the rows do not wait for the sequence's tables
        const int h = h0 + i % (kv ? kIters / 2 : kIters) * kRows + sub;
        raw[i].zero();
        if (h < (kv ? a.hkv : a.hq)) raw[i].load((kv ? i < kIters / 2 ? k : v : q) + h * D);
    }
    const int b = find_seq(a.r, t, 1, 0, 0);
    if (b >= a.r.B) return;  // a row behind the last sequence
    Seq s = load_seq(a.r, b);
    if (s.n > s.len) s.ok = false;
    if (t < s.row0 || (s.ok && t >= s.row0 + s.n)) return;
    const int pos = s.ok ? s.len - s.n + (t - s.row0) : 0;
    const Place place(a.prep, !PREP ? nullptr : kv ? a.prep.k_weight : a.prep.q_weight, d0);
    const Turn turn(a.prep, place, pos);
    if (!kv) {
        if constexpr (PREP) {
            Act* const out = static_cast<Act*>(a.q_out) + t * a.q_out_stride + d0;
#pragma unroll
            for (int i = 0; i < kIters; ++i) {
                const int h = h0 + i * kRows + sub;
                float y[8];
                turn.template apply<Act, D>(a.prep, place, raw[i], y);
                if (!s.ok) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[e] = NAN;
                }
                if (h < a.hq) store8(out + h * D, y);
            }
        }
        return;
    }
    if (!s.ok) return;
    const int64_t blk = block_of(a.r, b, pos / a.r.block_size);
    if (blk < 0) return;
    const int64_t to = ((blk * a.r.block_size + pos % a.r.block_size) * a.hkv) * D + d0;
#pragma unroll
    for (int i = 0; i < kIters; ++i) {
        const bool val = i >= kIters / 2;
        const int h = h0 + i % (kIters / 2) * kRows + sub;
        float y[8];
        if (PREP && !val)
            turn.template apply<Act, D>(a.prep, place, raw[i], y);
        else
            raw[i].get(y);
        if (h >= a.hkv) continue;
        Page* const dst = static_cast<Page*>(val ? a.v_pool : a.k_pool) + to + h * D;
        if constexpr (q8) {
            const float inv = inverse(__ldg((val ? a.v_scale : a.k_scale) + h));
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] *= inv;
            *reinterpret_cast<uint2*>(dst) = codes8<PAGE>(y);
        } else {
            store8(dst, y);
        }
    }
}

// CTAs an SM is to hold, which bounds a thread's registers: 3 (80 registers) where a token's
// heads are normed and rotated (67k tokens: 285 us, 353 with 2 CTAs, 363 with 4 and spills),
// 4 for plain writes; one fewer with float32 rows.
template <typename Act, bool PREP>
constexpr int ctas_per_sm() {
    return (PREP ? 3 : 4) - (sizeof(Act) == 4);
}

template <typename Act, int PAGE, int D, bool PB, bool PREP>
__global__ void __launch_bounds__(kWarps * 32, ctas_per_sm<Act, PREP>())
    write_kernel(const WriteArgs a) {
    __shared__ float smax[2 * kWarps];
    if (blockIdx.x == 0) check_all(a.r, true);
    if (PB && blockIdx.x < a.block_ctas) {
        if constexpr (PB && PREP)
            norm_blocks<PAGE, D>(a, smax);
        else if constexpr (PB)
            write_blocks<PAGE, D>(a, smax);
    } else {
        write_tokens<Act, PAGE, D, PREP>(a);
    }
}

template <typename Act, int PAGE, int D>
cudaError_t launch(const WriteArgs& a, bool pb, bool prep, int64_t ctas, cudaStream_t s) {
    constexpr bool q8 = PAGE == PGD_FP8_E4M3 || PAGE == PGD_INT8;
    const dim3 grid((unsigned)ctas);
    if (pb) {
        if (prep)
            write_kernel<Act, PAGE, D, q8, true><<<grid, kWarps * 32, 0, s>>>(a);
        else
            write_kernel<Act, PAGE, D, q8, false><<<grid, kWarps * 32, 0, s>>>(a);
    } else {
        if (prep)
            write_kernel<Act, PAGE, D, false, true><<<grid, kWarps * 32, 0, s>>>(a);
        else
            write_kernel<Act, PAGE, D, false, false><<<grid, kWarps * 32, 0, s>>>(a);
    }
    return cudaGetLastError();
}

int run_write(const Pool& p, WriteArgs& a, bool prep, void* stream) {
    const bool pb = is_q8(p.dtype) && p.scale_per_block;
    int64_t block_ctas = 0;
    if (pb) {  // block_size is a power of two in 8 .. 256
        a.chunk_shift = 3;
        a.warps_per_unit = 1;
        while ((1 << a.chunk_shift) < p.block_size) ++a.chunk_shift;
        while (a.warps_per_unit < kWarps && a.warps_per_unit * kChunk < p.block_size)
            a.warps_per_unit *= 2;
        const int64_t blocks = max_pieces(a.r.total, a.r.B, 1, a.chunk_shift, 2);
        const int64_t units = blocks * 2 * p.hkv, per_cta = kWarps / a.warps_per_unit;
        if (units > INT32_MAX) return PGD_ERR_SHAPE;
        block_ctas = prep ? blocks * ((p.hkv + kChunk / 2 - 1) / (kChunk / 2))
                          : (units + per_cta - 1) / per_cta;
    }
    a.block_ctas = uint32_t(block_ctas);
    a.q_groups = prep ? (a.hq + kChunk - 1) / kChunk : 0;
    a.kv_groups = pb ? 0 : (a.hkv + kChunk / 2 - 1) / (kChunk / 2);
    const int64_t units = (int64_t)a.r.total * (a.q_groups + a.kv_groups);
    const int64_t ctas = block_ctas + (units + kWarps - 1) / kWarps;
    if (units > INT32_MAX || ctas > INT32_MAX) return PGD_ERR_SHAPE;
    OnDevice dev(p.device);
    if (!dev.ok) return PGD_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (p.dtype == PGD_F32)
        e = p.d == 64 ? launch<float, PGD_F32, 64>(a, false, prep, ctas, s)
                      : launch<float, PGD_F32, 128>(a, false, prep, ctas, s);
    else if (p.dtype == PGD_BF16)
        e = p.d == 64 ? launch<__nv_bfloat16, PGD_BF16, 64>(a, false, prep, ctas, s)
                      : launch<__nv_bfloat16, PGD_BF16, 128>(a, false, prep, ctas, s);
    else if (p.dtype == PGD_FP8_E4M3)
        e = launch<__nv_bfloat16, PGD_FP8_E4M3, 128>(a, pb, prep, ctas, s);
    else
        e = launch<__nv_bfloat16, PGD_INT8, 128>(a, pb, prep, ctas, s);
    return e == cudaSuccess ? PGD_OK : PGD_ERR_CUDA;
}

// The K/V half of a call's arguments: checks, then the fields they fill.
int check_kv(const Pool& p, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
             int total, const int32_t* cu, int B, const int32_t* table, int max_blocks,
             const int32_t* lens, int max_len, WriteArgs* a) {
    int rc = check_ragged(p, total, cu, B, table, max_blocks, lens);
    if (rc != PGD_OK || B == 0 || total == 0) return rc;
    const int64_t width = (int64_t)p.hkv * p.d;
    rc = check_rows(k, k_stride, width, act_bytes(p));
    if (rc == PGD_OK) rc = check_rows(v, v_stride, width, act_bytes(p));
    if (rc != PGD_OK) return rc;
    const int cap = max_blocks * p.block_size;
    a->r = {cu, table, lens, B, total, max_blocks, p.block_size, p.num_blocks,
            max_len < cap ? max_len : cap, p.err};
    a->k = k;
    a->v = v;
    a->k_stride = k_stride;
    a->v_stride = v_stride;
    a->hkv = p.hkv;
    a->k_pool = const_cast<void*>(p.k);
    a->v_pool = const_cast<void*>(p.v);
    a->k_scale = const_cast<float*>(p.k_scale);
    a->v_scale = const_cast<float*>(p.v_scale);
    return PGD_OK;
}

// Rows of `width` bytes, `stride` apart, from `p` on.
struct Span {
    const char* p;
    int64_t stride, width;
};

// Whether no row of one meets a row of the other: apart altogether, or columns of the
// rows of one packed tensor.
bool apart(const Span& x, const Span& y, int64_t total) {
    if (x.p + (total - 1) * x.stride + x.width <= y.p ||
        y.p + (total - 1) * y.stride + y.width <= x.p)
        return true;
    if (x.stride != y.stride) return false;
    int64_t off = (y.p - x.p) % x.stride;
    if (off < 0) off += x.stride;
    return off >= x.width && off + y.width <= x.stride;
}

}  // namespace
}  // namespace pgd

using namespace pgd;

extern "C" int paged_kv_write(pgd_pool_t pool, const void* k, int64_t k_stride, const void* v,
                              int64_t v_stride, int total, const int32_t* cu_seqlens, int B,
                              const int32_t* block_table, int max_blocks,
                              const int32_t* seq_lens, void* stream) {
    if (!pool) return PGD_ERR_ARG;
    const Pool& p = pool_desc(pool);
    WriteArgs a = {};
    const int rc = check_kv(p, k, k_stride, v, v_stride, total, cu_seqlens, B, block_table,
                            max_blocks, seq_lens, INT32_MAX, &a);
    if (rc != PGD_OK || B == 0 || total == 0) return rc;
    return run_write(p, a, false, stream);
}

extern "C" int paged_qk_norm_rope_write(
    pgd_pool_t pool, const void* q, int64_t q_stride, void* q_out, int64_t q_out_stride, int Hq,
    const void* k, int64_t k_stride, const void* v, int64_t v_stride, int total,
    const void* q_weight, const void* k_weight, int weight_dtype, float eps, const float* rope,
    int rope_len, int rope_dim, int interleaved, const int32_t* cu_seqlens, int B,
    const int32_t* block_table, int max_blocks, const int32_t* seq_lens, void* stream) {
    if (!pool || Hq < 1 || !(eps >= 0.f) || !isfinite(eps)) return PGD_ERR_ARG;
    const Pool& p = pool_desc(pool);
    if (Hq % p.hkv != 0) return PGD_ERR_SHAPE;
    if ((q_weight || k_weight) && weight_dtype != PGD_F32 && weight_dtype != PGD_BF16)
        return PGD_ERR_DTYPE;
    if (interleaved != 0 && interleaved != 1) return PGD_ERR_ARG;
    if (rope) {
        if (rope_len < 1) return PGD_ERR_ARG;
        if (rope_dim < 16 || rope_dim > p.d || rope_dim % 16 != 0) return PGD_ERR_SHAPE;
        if (!is_aligned(rope, 16)) return PGD_ERR_ALIGN;
    }
    WriteArgs a = {};
    int rc = check_kv(p, k, k_stride, v, v_stride, total, cu_seqlens, B, block_table, max_blocks,
                      seq_lens, rope ? rope_len : INT32_MAX, &a);
    if (rc != PGD_OK || B == 0 || total == 0) return rc;
    const int64_t width = (int64_t)Hq * p.d;
    const int elt = act_bytes(p);
    rc = check_rows(q, q_stride, width, elt);
    if (rc == PGD_OK) rc = check_rows(q_out, q_out_stride, width, elt);
    if (rc != PGD_OK) return rc;
    const Span in = {static_cast<const char*>(q), q_stride * elt, width * elt};
    const Span out = {static_cast<const char*>(q_out), q_out_stride * elt, width * elt};
    const Span ks = {static_cast<const char*>(k), k_stride * elt, (int64_t)p.hkv * p.d * elt};
    const Span vs = {static_cast<const char*>(v), v_stride * elt, ks.width};
    const bool in_place = in.p == out.p && (in.stride == out.stride || total == 1);
    if ((!in_place && !apart(in, out, total)) || !apart(ks, out, total) || !apart(vs, out, total))
        return PGD_ERR_ARG;
    const int w_align = weight_dtype == PGD_F32 ? 4 : 2;
    if (!is_aligned(q_weight, w_align) || !is_aligned(k_weight, w_align)) return PGD_ERR_ALIGN;
    a.prep = {q_weight, k_weight, weight_dtype == PGD_F32, eps, rope, rope ? rope_dim : 0,
              interleaved};
    a.q = q;
    a.q_out = q_out;
    a.q_stride = q_stride;
    a.q_out_stride = q_out_stride;
    a.hq = Hq;
    return run_write(p, a, true, stream);
}
