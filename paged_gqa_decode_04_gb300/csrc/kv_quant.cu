// The write side of a serving step over ragged batches: K and V rows into the
// pages, quantised as they are written (paged_kv_write), and the same with the
// per-head norm of queries and keys and the rotation by position in one pass
// (paged_qk_norm_rope_write).  See include/paged_kv_manager.h for the contract.
//
// Mathematics of a head vector x of D elements at position p:
//     y = x * rsqrt(mean(x^2) + eps) * w                        (norm, optional)
//     (a, b) -> (a cos - b sin, b cos + a sin) for the pairs j < R / 2 of the first R
//     elements, cos and sin from the caller's table at p        (rotation, optional)
//     8-bit pages: code = rn(y / scale), saturated.
// All of it in float32 and in registers, with one rounding at the end: to the output
// type, or to the code.
//
// What bounds it: bytes.  Every row is read once and written once, about ten operations
// an element.  So: 16-byte accesses, a lane holds 8 consecutive elements of a head (16
// lanes a vector at D = 128), the sum of squares and the rotation partner by shuffles,
// and a warp issues the loads of 16 head vectors before it uses the first.
//
// Work of a warp.  K and V: one (chunk of tokens, KV head, K or V).  Where the scale
// belongs to a block, the chunk is the block: the largest magnitude of its new rows has
// to be known before the first code, and the rows stay in registers in between; blocks
// of more than 16 tokens are shared by up to 8 warps of a CTA, which exchange their
// maxima through shared memory.  Otherwise chunks are 16 tokens.  No two warps write one
// scale and there are no atomics, so the pages do not depend on timing.  Queries: one
// (token, 16 heads), whose cosines, sines and weights are loaded once.
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
    int chunk_shift;      // log2 of the tokens of a K/V chunk
    int warps_per_unit;   // warps sharing one (chunk, head, K or V)
    int64_t kv_ctas;      // CTAs of the K/V part; the query part follows
};

// ---------------------------------------------------------- 8 elements of a lane
template <typename Act>
struct Raw;
template <>
struct Raw<__nv_bfloat16> {
    uint4 a;
    __device__ void load(const __nv_bfloat16* p) { a = *reinterpret_cast<const uint4*>(p); }
    __device__ void zero() { a = make_uint4(0, 0, 0, 0); }
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

__device__ __forceinline__ float inverse(float scale) { return scale > 0.f ? 1.f / scale : 0.f; }

// 8 codes of values already divided by their scale: nearest, ties to even, saturated.
// NaN gives the NaN code of e4m3 and 0 in int8, which has none.
template <int PAGE>
__device__ __forceinline__ uint2 codes8(const float (&x)[8]) {
    uint32_t w[2];
    if (PAGE == PGD_INT8) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            w[i] = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float v = x[4 * i + j];
                const int c = v == v ? __float2int_rn(fminf(fmaxf(v, -127.f), 127.f)) : 0;
                w[i] |= uint32_t(c & 0xff) << (8 * j);
            }
        }
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
// The lane's 8 weights (ones without a norm).
__device__ __forceinline__ void load_weights(const void* w, int f32, int d0, float (&out)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
        out[i] = !w ? 1.f
                 : f32 ? __ldg(static_cast<const float*>(w) + d0 + i)
                       : __bfloat162float(static_cast<const __nv_bfloat16*>(w)[d0 + i]);
}

// The lane's 8 cosines and sines at position p (interleaved: 4 of each).
__device__ __forceinline__ void load_angles(const Prep& pr, int p, int d0, float (&cs)[8],
                                            float (&sn)[8]) {
    const int half = pr.rope_dim / 2;
    const float* t = pr.rope + (int64_t)p * pr.rope_dim;
    if (d0 >= pr.rope_dim) {
#pragma unroll
        for (int i = 0; i < 8; ++i) cs[i] = 1.f, sn[i] = 0.f;
    } else if (pr.interleaved) {
        const float4 c = __ldg(reinterpret_cast<const float4*>(t + d0 / 2));
        const float4 s = __ldg(reinterpret_cast<const float4*>(t + half + d0 / 2));
        cs[0] = c.x, cs[1] = c.y, cs[2] = c.z, cs[3] = c.w;
        sn[0] = s.x, sn[1] = s.y, sn[2] = s.z, sn[3] = s.w;
    } else {
        const int j = d0 < half ? d0 : d0 - half;
        const float4* c = reinterpret_cast<const float4*>(t + j);
        const float4* s = reinterpret_cast<const float4*>(t + half + j);
        const float4 c0 = __ldg(c), c1 = __ldg(c + 1), s0 = __ldg(s), s1 = __ldg(s + 1);
        cs[0] = c0.x, cs[1] = c0.y, cs[2] = c0.z, cs[3] = c0.w;
        cs[4] = c1.x, cs[5] = c1.y, cs[6] = c1.z, cs[7] = c1.w;
        sn[0] = s0.x, sn[1] = s0.y, sn[2] = s0.z, sn[3] = s0.w;
        sn[4] = s1.x, sn[5] = s1.y, sn[6] = s1.z, sn[7] = s1.w;
    }
}

// Norm and rotate the lane's 8 elements of a head vector; the D / 8 lanes of a vector
// (and the whole warp) call this together.
template <int D>
__device__ __forceinline__ void norm_rotate(const Prep& pr, bool norm, const float (&w)[8],
                                            const float (&cs)[8], const float (&sn)[8], int d0,
                                            float (&x)[8]) {
    if (norm) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
        for (int m = 1; m < D / 8; m *= 2) ss += __shfl_xor_sync(0xffffffffu, ss, m);
        const float r = rsqrtf(ss * (1.f / D) + pr.eps);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = x[i] * r * w[i];
    }
    if (!pr.rope) return;
    if (pr.interleaved) {
        if (d0 < pr.rope_dim) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float a = x[2 * i], b = x[2 * i + 1];
                x[2 * i] = a * cs[i] - b * sn[i];
                x[2 * i + 1] = b * cs[i] + a * sn[i];
            }
        }
        return;
    }
    // the partner of element j is j +- rope_dim / 2: the same place in another lane
    const int half = pr.rope_dim / 2, lane = threadIdx.x & 31;
    const bool low = d0 < half, in = d0 < pr.rope_dim;
    const int src = !in ? lane : low ? lane + half / 8 : lane - half / 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float o = __shfl_sync(0xffffffffu, x[i], src);
        if (in) x[i] = low ? x[i] * cs[i] - o * sn[i] : x[i] * cs[i] + o * sn[i];
    }
}

// -------------------------------------------------------------------------- K, V
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

template <typename Act, int PAGE, int D, bool PB, bool PREP>
__device__ __forceinline__ void write_kv(const WriteArgs& a, float* smax) {
    constexpr int kLanes = D / 8;              // lanes of a head vector
    constexpr int kRows = 32 / kLanes;         // vectors of a warp at once
    constexpr int kIters = kChunk / kRows;
    using Page = typename PageType<PAGE>::type;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int sub = lane / kLanes, d0 = lane % kLanes * 8;
    const int W = PB ? a.warps_per_unit : 1;
    const int64_t unit = (int64_t)blockIdx.x * (kWarps / W) + warp / W;
    const int part = warp % W;
    const int per = 2 * a.hkv;
    const int64_t piece = unit / per;
    const int side = int(unit % per) / a.hkv, h = int(unit % per) % a.hkv;

    Seq s;
    s.ok = false;
    int chunk = 0, lo = 0, hi = 0;  // the chunk's number in the sequence; rows of it to write
    const int b = find_seq(a.r, piece, 1, a.chunk_shift, 2);
    if (b < a.r.B) {
        s = load_seq(a.r, b);
        if (s.n > s.len) s.ok = false;
        if (s.ok) {
            const int start = s.len - s.n;
            chunk = (start >> a.chunk_shift) +
                    int(piece - first_piece(a.r, b, 1, a.chunk_shift, 2));
            const int64_t at = (int64_t)chunk << a.chunk_shift;
            lo = int(max(at, (int64_t)start) - at);
            hi = at < s.len ? int(min((int64_t)s.len - at, (int64_t)1 << a.chunk_shift)) : 0;
            if (hi <= lo) s.ok = false;
        }
    }
    const Act* src = static_cast<const Act*>(side ? a.v : a.k);
    const int64_t stride = side ? a.v_stride : a.k_stride;
    Page* pool = static_cast<Page*>(side ? a.v_pool : a.k_pool);
    float* scales = side ? a.v_scale : a.k_scale;
    const int64_t at = (int64_t)chunk << a.chunk_shift;
    // packed row of the chunk's row j: row0 + (at + j) - (len - n)
    const int64_t row_of = s.ok ? s.row0 + at - (s.len - s.n) : 0;
    const bool prep = PREP && side == 0;
    float w[8];
    if (prep) load_weights(a.prep.k_weight, a.prep.weight_f32, d0, w);

    Raw<Act> raw[kIters];
    auto load = [&](int j0) {
#pragma unroll
        for (int i = 0; i < kIters; ++i) {
            const int j = j0 + i * kRows + sub;
            raw[i].zero();
            if (j >= lo && j < hi) raw[i].load(src + (row_of + j) * stride + h * D + d0);
        }
    };
    // values of row j (all lanes of the warp call this for the same i)
    auto value = [&](int i, int j, float (&x)[8]) {
        raw[i].get(x);
        if (prep) {
            float cs[8], sn[8];
            if (a.prep.rope)
                load_angles(a.prep, j >= lo && j < hi ? int(at) + j : 0, d0, cs, sn);
            norm_rotate<D>(a.prep, a.prep.k_weight != nullptr, w, cs, sn, d0, x);
        }
    };
    auto slot_of = [&](int64_t blk, int64_t pos) {
        return ((blk * a.r.block_size + pos % a.r.block_size) * a.hkv + h) * D + d0;
    };

    if (!PB) {
        if (!s.ok) return;
        float inv = 1.f;
        if (PAGE == PGD_FP8_E4M3 || PAGE == PGD_INT8) inv = inverse(__ldg(scales + h));
        load(0);
#pragma unroll
        for (int i = 0; i < kIters; ++i) {
            const int j = i * kRows + sub;
            float x[8];
            value(i, j, x);
            if (j < lo || j >= hi) continue;
            const int64_t pos = at + j;
            const int64_t blk = block_of(a.r, s.b, int(pos / a.r.block_size));
            if (blk < 0) continue;
            if constexpr (PAGE == PGD_FP8_E4M3 || PAGE == PGD_INT8) {
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] *= inv;
                *reinterpret_cast<uint2*>(pool + slot_of(blk, pos)) = codes8<PAGE>(x);
            } else {
                store8(pool + slot_of(blk, pos), x);
            }
        }
    } else if constexpr (PAGE == PGD_FP8_E4M3 || PAGE == PGD_INT8) {
        const int64_t blk = s.ok ? block_of(a.r, s.b, chunk) : -1;
        const int rows = 1 << a.chunk_shift;
        const int passes = (rows + W * kChunk - 1) / (W * kChunk);
        // the old scale first: its latency passes under the rows' loads
        const float was = blk >= 0 && lo > 0 ? scales[blk * a.hkv + h] : 0.f;
        float top = 0.f;
        for (int p = 0; p < passes; ++p) {
            if (blk < 0) break;
            const int j0 = (p * W + part) * kChunk;
            load(j0);
#pragma unroll
            for (int i = 0; i < kIters; ++i) {
                float x[8];
                value(i, j0 + i * kRows + sub, x);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float m = fabsf(x[e]);
                    top = fmaxf(top, m < INFINITY ? m : 0.f);  // NaN and infinities left out
                }
            }
        }
#pragma unroll
        for (int m = 1; m < 32; m *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
        if (W > 1) {
            if (lane == 0) smax[warp] = top;
            __syncthreads();
            for (int i = 0; i < W; ++i) top = fmaxf(top, smax[warp / W * W + i]);
        }
        if (blk < 0) return;
        float now = top * (1.f / code_max<PAGE>());
        if (!(now >= kTiny)) now = 0.f;
        now = fmaxf(now, was);
        const float inv = inverse(now);
        if (part == 0 && lane == 0) scales[blk * a.hkv + h] = now;
        // rows cached in the block before this call take the larger scale
        if (now > was && lo > 0) {
            const float ratio = was * inv;
            for (int j = part * kRows + sub; j < lo; j += W * kRows) {
                uint2* c = reinterpret_cast<uint2*>(pool + slot_of(blk, j));
                float x[8];
                values8<PAGE>(*c, x);
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] *= ratio;
                *c = codes8<PAGE>(x);
            }
        }
        for (int p = passes - 1; p >= 0; --p) {
            const int j0 = (p * W + part) * kChunk;
            if (p != passes - 1) load(j0);
#pragma unroll
            for (int i = 0; i < kIters; ++i) {
                const int j = j0 + i * kRows + sub;
                float x[8];
                value(i, j, x);
                if (j < lo || j >= hi) continue;
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] *= inv;
                *reinterpret_cast<uint2*>(pool + slot_of(blk, j)) = codes8<PAGE>(x);
            }
        }
    }
}

// ----------------------------------------------------------------------- queries
template <typename Act, int D>
__device__ __forceinline__ void prep_q(const WriteArgs& a) {
    constexpr int kLanes = D / 8, kRows = 32 / kLanes, kIters = kChunk / kRows;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int sub = lane / kLanes, d0 = lane % kLanes * 8;
    const int groups = (a.hq + kChunk - 1) / kChunk;
    const int64_t unit = ((int64_t)blockIdx.x - a.kv_ctas) * kWarps + warp;
    const int64_t t = unit / groups;
    const int h0 = int(unit % groups) * kChunk;
    if (t >= a.r.total) return;
    const Act* q = static_cast<const Act*>(a.q) + t * a.q_stride + d0;
    Raw<Act> raw[kIters];
#pragma unroll
    for (int i = 0; i < kIters; ++i) {  // the rows do not wait for the sequence's tables
        const int h = h0 + i * kRows + sub;
        raw[i].zero();
        if (h < a.hq) raw[i].load(q + h * D);
    }
    float w[8], cs[8], sn[8];
    load_weights(a.prep.q_weight, a.prep.weight_f32, d0, w);
    const int b = find_seq(a.r, t, 1, 0, 0);
    if (b >= a.r.B) return;  // a row behind the last sequence
    Seq s = load_seq(a.r, b);
    if (s.n > s.len) s.ok = false;
    if (t < s.row0 || (s.ok && t >= s.row0 + s.n)) return;
    if (s.ok && a.prep.rope) load_angles(a.prep, s.len - s.n + int(t - s.row0), d0, cs, sn);
    Act* out = static_cast<Act*>(a.q_out) + t * a.q_out_stride + d0;
#pragma unroll
    for (int i = 0; i < kIters; ++i) {
        const int h = h0 + i * kRows + sub;
        float x[8];
        raw[i].get(x);
        norm_rotate<D>(a.prep, a.prep.q_weight != nullptr, w, cs, sn, d0, x);
        if (!s.ok) {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = NAN;
        }
        if (h < a.hq) store8(out + h * D, x);
    }
}

template <typename Act, int PAGE, int D, bool PB, bool PREP>
__global__ void __launch_bounds__(kWarps * 32) write_kernel(const WriteArgs a) {
    __shared__ float smax[kWarps];
    if (blockIdx.x == 0) check_all(a.r, true);
    if (blockIdx.x < a.kv_ctas)
        write_kv<Act, PAGE, D, PB, PREP>(a, smax);
    else if (PREP)
        prep_q<Act, D>(a);
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
    a.chunk_shift = 4;
    a.warps_per_unit = 1;
    if (pb) {  // block_size is a power of two in 8 .. 256
        a.chunk_shift = 3;
        while ((1 << a.chunk_shift) < p.block_size) ++a.chunk_shift;
        while (a.warps_per_unit < kWarps && a.warps_per_unit * kChunk < p.block_size)
            a.warps_per_unit *= 2;
    }
    const int64_t units = max_pieces(a.r.total, a.r.B, 1, a.chunk_shift, 2) * 2 * p.hkv;
    const int per_cta = kWarps / a.warps_per_unit;
    a.kv_ctas = (units + per_cta - 1) / per_cta;
    const int64_t q_units = prep ? (int64_t)a.r.total * ((a.hq + kChunk - 1) / kChunk) : 0;
    const int64_t ctas = a.kv_ctas + (q_units + kWarps - 1) / kWarps;
    if (ctas > INT32_MAX) return PGD_ERR_SHAPE;
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

// Whether q_out may be written while q is read: the same rows, or rows that never meet.
bool q_out_fits(const char* q, int64_t q_stride, const char* o, int64_t o_stride, int64_t width,
                int64_t total) {
    if (q == o) return q_stride == o_stride || total == 1;
    const char* q_end = q + (total - 1) * q_stride + width;
    const char* o_end = o + (total - 1) * o_stride + width;
    if (q_end <= o || o_end <= q) return true;
    if (q_stride != o_stride) return false;
    int64_t off = (o - q) % q_stride;  // columns of one packed row
    if (off < 0) off += q_stride;
    return off >= width && off + width <= q_stride;
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
    if (!q_out_fits(static_cast<const char*>(q), q_stride * elt, static_cast<char*>(q_out),
                    q_out_stride * elt, width * elt, total))
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
