// The attention of many query tokens on the asynchronous tensor cores.
//
//     S = q K^T,  m = running maximum of a row's scores,  P = exp2(c S - m),
//     O += P V,   l += sum of P,   out = O / l
//
// with S and O in float32 in TMEM, m and l in float32 in registers and P rounded to 16
// bits, the type the product takes (at most half a step of each weight, 2^-8 in bfloat16 and
// 2^-11 in f16 over 8-bit pages); l is the sum of the weights before they are rounded.
//
// Rows.  The G query heads of a KV head see the same keys, so a CTA takes 256 consecutive
// rows (token, head of the group) of one sequence and KV head: a key tile is fetched once
// for all of them, and a few tokens still fill rows.  They are two blocks of 128 rows,
// the height of the tensor cores' accumulator, each with one thread a row for its softmax
// (no shuffles): while one block's weights are computed, the tensor cores run the other's
// products.
//
// Keys.  Tiles of 128 tokens.  Producer warps walk the block table and fetch each page of
// the tile with one TMA copy for every 64 elements of the head, so that pages land as
// one tile in the swizzled layout both products read: K with its head dimension contiguous,
// V with its tokens as rows (the transposed operand).  A warp issues its lanes' copies one
// after the other, 54 cycles each (measured), and a tile of 16-token pages takes 16 for K
// and 16 for V: one warp needs 2830 cycles for what the products take 2048 for, four need
// 1650.  (Copies of 16 bytes by the threads of four warps, cp.async: 4850.)  Pages no query
// of the CTA sees are not fetched, and V rows outside the visible range are zeroed, so that
// nothing in an unused slot is multiplied.  A page whose block id is out of range has V
// zeroed as well (8-bit pages: fetched from a coordinate outside the tensor, which reads zeros),
// so that rows that do not see it stay right; those that do are marked (mark_lost) and become
// NaN at the end.
//
// Warps: 0-3 and 4-7 the softmax of the two blocks, 8-11 the producers, 12 and 13 issue the
// products of one block each; 14 and 15 only round the group up to four warps, the unit
// registers are handed over in.  Weights take the place of the scores they came from in
// TMEM, in halves, so that the first half's product starts early.  A block's products go P V(j),
// q K(j+1), P V(j+1), .., in turns with the other's: its softmax runs during the other's
// turn.  The issuing warp of the next turn has waited for its tiles and weights before the
// turn is handed over; one warp that issued both blocks' products left the tensor cores
// idle a third of the time, and two without turns fell into step, softmax with softmax.
// The accumulator is rescaled
// only when a row's maximum has grown by more than 2^8: until then weights are relative to
// an older maximum, at most 256, which costs no precision in either float type.
//
// Few rows.  128 rows or fewer go to both blocks, every other tile each, so that one's
// softmax still hides behind the other's products; and where that pays, 2, 4 or 8 CTAs of a
// cluster share a piece's key tiles (choose_cluster in attend_plan.h).  The parts
// join their sums through shared memory, each other's in a cluster:
// out = sum_k 2^(m_k - m) O_k / sum_k 2^(m_k - m) l_k.
//
// 8-bit pages.  Warps 14 and 15 fetch the codes, warps 8-11 widen them to f16, exactly, into
// the tiles the products read; queries and weights are f16 as well.  Scales per head are
// constants of the CTA.  Scales per block go where a float32 value is at hand anyway, K's on
// the scores and V's into the exponent of the weights (the row's sum takes them out again):
// multiplied into V while it is widened they cost 5% of the whole (2048 of 8192 tokens, 64/8
// heads: 489 against 465 us; now 446, 396 with scales per head, 338 over bfloat16).
//
// What bounds it.  At D = 128 a tile of one block is 2 x 8 products of 64 cycles (1024), and
// each of its four softmax warps, one in every quarter of the SM, has 128 exponentials of
// 4.07 cycles (521), about 900 cycles with the maxima, sums and conversions; the two blocks'
// warps of a quarter together take 1500.  So the softmax hides behind the products of both
// blocks (2048 cycles) with little to spare.  Measured (bfloat16, 64/8 heads, 2048 queries):
// of 32768 tokens 1364 us, 1.56 PFLOP/s, 81% of a library product's burst (1265 us and 87%
// before the clock drops under the load); of 8192 tokens 338 us with the tensor cores busy 61%
// of the time, since a CTA's search, query load, first tile and epilogue (some 10 us) are not
// hidden and causal pieces end unevenly.  Over 8-bit pages the widening warps share the issue slots
// with the softmax: 44% (scales per block).  ptxas spills 104 bytes of stores and 248 of loads
// over bfloat16 pages, 180 and 416 to 200 and 464 over 8-bit ones.
//
// Every wait is bounded; one that gives up latches PGD_ERR_TIMEOUT and ends the CTA.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <type_traits>

#include "attend_plan.h"
#include "page_ops.h"
#include "ragged.cuh"
#include "umma.cuh"

namespace pgd {
namespace attend {

using namespace umma;

constexpr int kBlock = 128;     // rows of a block
constexpr int kThreads = 512;
// Registers a thread: launched with 128, then the 256 threads of the softmax take 200, the
// 128 producers or widening warps keep 64 and the last 128 keep 48, which is the launch's
// 65536 again (192, 80 and 48 with scales per block: 460 against 445 us at 2048 of 8192
// tokens, 64/8 heads).
constexpr int kSoftmaxRegs = 200, kProducerRegs = 64, kIssuerRegs = 48;
static_assert(256 * kSoftmaxRegs + 128 * (kProducerRegs + kIssuerRegs) == kThreads * 128,
              "registers of the launch");
constexpr float kGrow = 8.f;    // base-2 growth of a maximum that is let pass
// Base-2 lift of f16 weights over 8-bit pages with scales per head: up to 2^(kGrow + kLift) they
// stay below 65504, and keep 11 bits down to 2^-21 of the running maximum's, then steps of 2^-31
// of it (without: 2^-14 and 2^-24, so that a long tail of weights below 2^-25 vanished in P V,
// though not in their sum).  The sum and the accumulator have the same factor.
constexpr float kLift = 7.f;

struct Args {
    Ragged r;
    int hq, hkv, group;
    const __nv_bfloat16* q;
    int64_t q_stride;
    __nv_bfloat16* out;
    int causal;
    int window;
    float scale_log2;       // positive: queries take the sign of the scale
    uint32_t q_and, q_xor;  // applied to pairs of query elements (a scale below or of zero)
    int pieces;             // row pieces of the grid (each with every KV head)
    int cluster;            // CTAs sharing a piece's keys
    const float* k_scale;   // 8-bit pages: [hkv], or [num_blocks][hkv]
    const float* v_scale;
};

template <int D, int PAGE, bool PB>
struct Layout {
    static constexpr bool kQ8 = PAGE != PGD_BF16;
    static constexpr int kHalves = D / 64;                 // 128-byte columns of a 16-bit tile
    static constexpr int kSlot = kTile * D * 2;            // bytes of a K or V tile
    static constexpr int kSlots = kQ8 ? 4 : D == 128 ? 5 : 8;
    static constexpr int kQ = kBlock * D * 2;              // bytes of a block of queries
    static constexpr int kRing = 2 * kQ;
    // 8-bit pages: tiles as they are stored, and the scales of the tiles in flight (those of
    // tile j + 1 are written when V of j has a slot, so when V of j - 3 is done with, and the
    // weights that it was multiplied with before that): for each 8 tokens K's,
    // log2 of V's and 1 over V's, then V's gain.
    static constexpr int kRawSlot = kTile * 128;
    static constexpr int kRawSlots = 2;
    static constexpr int kRaw = kRing + kSlots * kSlot;
    static constexpr int kScaleTiles = 6;
    static constexpr int kScales = kRaw + (kQ8 ? kRawSlots * kRawSlot : 0);
    static constexpr int kScaleBytes = 272;
    static constexpr int kBars = kScales + (PB ? kScaleTiles * kScaleBytes : 0);
    static constexpr int kBytes = kBars + 320 + 1024;      // and room to align to 1024
    // warps that issue copies, and the tiles' 128-byte columns they fetch one by one
    static constexpr int kProducers = kQ8 ? 2 : 4;
    static constexpr int kColumns = kQ8 ? 1 : kHalves;
};

// The keys a block of rows sees: tiles [t0, t1), and which of them every row sees whole.
struct Span {
    int t0, t1;
    int lo, hi;         // first visible token, one past the last
    int lo_all, hi_all; // tokens in [lo_all, hi_all) are visible to every row
};

// Rows [first, last] of a sequence, counted (token, head of the group).
__device__ __forceinline__ Span span_of(const Args& a, const Seq& s, int first, int last) {
    Span p = {0, 0, 0, 0, 0, 0};
    if (last < first || !s.ok) return p;
    const int p0 = s.len - s.n + first / a.group, p1 = s.len - s.n + last / a.group;
    p.hi = a.causal ? max(0, p1 + 1) : s.len;
    p.hi_all = a.causal ? p0 + 1 : s.len;
    if (a.window > 0) {
        p.lo = max(0, p0 - a.window + 1);
        p.lo_all = max(0, p1 - a.window + 1);
    }
    if (p.hi > p.lo) {
        p.t0 = p.lo / kTile;
        p.t1 = (p.hi - 1) / kTile + 1;
    } else {
        p.lo = p.hi = 0;
    }
    return p;
}

__device__ __forceinline__ bool valid(const Ragged& r, int id) {
    return id >= 0 && id < r.num_blocks;
}

// A page, tokens [t, t + n), has a block id out of range: the rows of the piece that see it are
// marked in `lost`, a bit a row, to become NaN.  Apart from the kernel's own code, whose loops it
// would slow down (2048 of 8192 tokens over bfloat16 pages, 64/8 heads: 337 -> 356 us).
__device__ __noinline__ void mark_lost(const Args& a, const Seq& s, int row0, int t, int n,
                                       uint32_t* lost) {
    for (int r = 0; r < 1 << kRowShift; ++r) {
        const int pos = s.len - s.n + (row0 + r) / a.group;
        const int lo = a.window > 0 ? max(0, pos - a.window + 1) : 0;
        const int hi = a.causal ? pos + 1 : s.len;
        if (lo < t + n && hi > t) atomicOr(lost + r / 32, 1u << r % 32);
    }
}

// Token and head of the group of row r, r + step, r + 2 step, ..: one division for all.
struct Rows {
    int64_t token;
    uint32_t head, group, dt, dh;
    __device__ __forceinline__ Rows(uint32_t r, uint32_t g, uint32_t step)
        : token(r / g), head(r % g), group(g), dt(step / g), dh(step % g) {}
    __device__ __forceinline__ void next() {
        token += dt;
        head += dh;
        if (head >= group) head -= group, ++token;
    }
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float m;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(a), "f"(b), "f"(c));
    return m;
}
__device__ __forceinline__ float max8(const uint32_t* x) {
    const float a = max3(__uint_as_float(x[0]), __uint_as_float(x[1]), __uint_as_float(x[2]));
    const float b = max3(__uint_as_float(x[3]), __uint_as_float(x[4]), __uint_as_float(x[5]));
    return max3(a, b, fmaxf(__uint_as_float(x[6]), __uint_as_float(x[7])));
}
__device__ __forceinline__ uint64_t pair(float a, float b) {
    uint64_t p;
    asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(a), "f"(b));
    return p;
}
__device__ __forceinline__ void unpair(uint64_t p, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
// The type of the products' operands: bfloat16, or f16 over 8-bit pages, in which both
// codes are exact.
template <int PAGE>
__device__ __forceinline__ uint32_t operand2(float lo, float hi) {
    return PAGE == PGD_BF16 ? bf16x2(lo, hi) : f16x2(lo, hi);
}
// Four codes to two pairs of f16.
template <int PAGE>
__device__ __forceinline__ void widen4(uint32_t w, uint32_t& a, uint32_t& b) {
    if (PAGE == PGD_INT8) {
        // a code with its sign bit turned is code + 128; under the high byte 0x64 it is the
        // f16 1024 + code + 128
        const __half2 off = __half2half2(__float2half(1152.f));
        w ^= 0x80808080u;
        const uint32_t lo = __byte_perm(w, 0x64646464u, 0x4140);
        const uint32_t hi = __byte_perm(w, 0x64646464u, 0x4342);
        const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&lo), off);
        const __half2 y = __hsub2(*reinterpret_cast<const __half2*>(&hi), off);
        a = *reinterpret_cast<const uint32_t*>(&x);
        b = *reinterpret_cast<const uint32_t*>(&y);
    } else {
        asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.rn.f16x2.e4m3x2 %0, l;\n"
            " cvt.rn.f16x2.e4m3x2 %1, h;\n}"
            : "=r"(a), "=r"(b)
            : "r"(w));
    }
}

template <int D, int PAGE, bool PB>
__global__ void __launch_bounds__(kThreads, 1)
    attend_kernel(const __grid_constant__ Args a, const __grid_constant__ CUtensorMap map_k,
                  const __grid_constant__ CUtensorMap map_v) {
    using L = Layout<D, PAGE, PB>;
    constexpr bool kQ8 = L::kQ8;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = (smem_addr(smem_raw) + 1023) & ~1023u;
    uint8_t* const smem = smem_raw + (base - smem_addr(smem_raw));
    const uint32_t bars = base + L::kBars;
    const uint32_t bar_q = bars, bar_s = bars + 16, bar_p = bars + 32, bar_o = bars + 64;
    // bar_patch: one of each producer (bfloat16), bar_raw: full and empty raw slots (8-bit)
    const uint32_t bar_turn = bars + 80, bar_patch = bars + 96, bar_full = bars + 128;
    const uint32_t bar_raw = bars + 192, bar_raw_empty = bar_raw + 8 * L::kRawSlots;
    const uint32_t bar_empty = bar_full + 8 * L::kSlots;
    volatile int* const gave_up = reinterpret_cast<int*>(smem + L::kBars + 272);
    uint32_t* const lost = reinterpret_cast<uint32_t*>(smem + L::kBars + 288);  // of 256 rows
    uint32_t* const tmem_at = reinterpret_cast<uint32_t*>(smem + L::kBars + 280);

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int share = a.cluster > 1 ? (int)cluster_rank() : 0;
    if (blockIdx.x == 0) check_all(a.r, false);

    // one thread sets the barriers up while the other warps look for their sequence
    if (threadIdx.x == 416) {
        for (int i = 0; i < 2; ++i) {
            bar_init(bar_q + 8 * i, 4);  // warps of a block
            bar_init(bar_s + 8 * i, 1);
            bar_init(bar_p + 16 * i, 4);
            bar_init(bar_p + 16 * i + 8, 4);
            bar_init(bar_o + 8 * i, 1);
            bar_init(bar_turn + 8 * i, 1);
        }
        if (kQ8) {
            for (int i = 0; i < L::kRawSlots; ++i) {
                bar_init(bar_raw + 8 * i, L::kProducers);
                bar_init(bar_raw_empty + 8 * i, 4);
            }
        } else {
            for (int i = 0; i < L::kProducers; ++i) bar_init(bar_patch + 8 * i, 1);
        }
        for (int i = 0; i < L::kSlots; ++i) {
            bar_init(bar_full + 8 * i, 4);  // producer or widening warps
            bar_init(bar_empty + 8 * i, 2);
        }
        *gave_up = 0;
        for (int i = 0; i < 8; ++i) lost[i] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }

    // the piece of rows: the longest walks first, which for causal rows are the last ones
    const int64_t unit = blockIdx.x / a.cluster;
    const int piece = a.pieces - 1 - int(unit % a.pieces);
    const int head = int(unit / a.pieces);
    const int b = find_seq(a.r, piece, a.group, kRowShift, 1);
    if (b >= a.r.B) return;  // the same for the whole cluster
    const Seq s = load_seq(a.r, b);
    const uint32_t group = a.group;
    const int row0 = int(piece - first_piece(a.r, b, a.group, kRowShift, 1)) << kRowShift;
    // rows of the piece (an impossible sequence's only become NaN)
    const int n = s.ok ? s.n : min(__ldg(a.r.cu + b + 1), a.r.total) - s.row0;
    if (row0 < 0 || s.row0 < 0 || n <= 0) return;
    const int rows = min(n * a.group - row0, 1 << kRowShift);
    if (rows <= 0) return;

    Span sp[2];
    sp[0] = span_of(a, s, row0, row0 + min(rows, kBlock) - 1);
    sp[1] = span_of(a, s, row0 + kBlock, row0 + rows - 1);
    const bool some0 = sp[0].t1 > sp[0].t0, some1 = sp[1].t1 > sp[1].t0;
    // tokens and tiles of the CTA
    const int lo = some0 ? (some1 ? min(sp[0].lo, sp[1].lo) : sp[0].lo) : sp[1].lo;
    const int hi = max(sp[0].hi, sp[1].hi);
    int T0 = lo / kTile, T1 = hi > lo ? (hi - 1) / kTile + 1 : T0;
    // 128 rows or fewer: both blocks take them, and every other tile each, where every CTA of
    // the cluster has two (all of them decide alike)
    const bool paired = rows <= kBlock && T1 - T0 >= 2 * a.cluster;
    if (a.cluster > 1) {  // this CTA's share of the tiles
        const int tiles = T1 - T0, t = T0;
        T0 = t + tiles * share / a.cluster;
        T1 = t + tiles * (share + 1) / a.cluster;
    }
    if (paired) sp[1] = sp[0];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        sp[i].t0 = max(sp[i].t0, T0);
        sp[i].t1 = max(sp[i].t0, min(sp[i].t1, T1));
    }

    if (warp == 12) tmem_alloc(smem_addr(tmem_at), 512);
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = *tmem_at;

    float m = -INFINITY, l = 0.f;  // of the thread's row, in the units of exp2
    float vgain = 0.f;             // of the accumulator, with a V scale per block
    const int blk = warp / 4;      // block of rows of a softmax warp
    const int my_row = threadIdx.x % kBlock;
    const int at_row = (paired ? 0 : blk * kBlock) + my_row;  // in the piece

    if (warp < 8) {
        // ---------------------------------------------------------------- softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
        const Span p = blk ? sp[1] : sp[0];
        if (p.t1 > p.t0) {
            // the block's queries into shared memory, swizzled
            constexpr int kVecs = D / 8, kStep = kBlock / kVecs;  // 16-byte pieces; rows at once
            const int c = my_row % kVecs;
            const __nv_bfloat16* q =
                a.q + (int64_t)s.row0 * a.q_stride + (int64_t)head * a.group * D + c * 8;
            const int first_row = at_row - my_row + my_row / kVecs;
            Rows at(row0 + first_row, group, kStep);
            uint4 x[kVecs];
#pragma unroll
            for (int i = 0; i < kVecs; ++i, at.next()) {  // all loads, then all stores
                x[i] = make_uint4(0, 0, 0, 0);
                if (first_row + i * kStep < rows)
                    x[i] = __ldg(reinterpret_cast<const uint4*>(q + at.token * a.q_stride +
                                                                at.head * D));
            }
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                const int r = my_row / kVecs + i * kStep;
                auto operand = [&](uint32_t two) {
                    two = (two & a.q_and) ^ a.q_xor;
                    return kQ8 ? f16x2(__uint_as_float(two << 16),
                                       __uint_as_float(two & 0xffff0000u))
                               : two;
                };
                *reinterpret_cast<uint4*>(smem + blk * L::kQ + c / 8 * (kBlock * 128) + r * 128 +
                                          ((c ^ r) & 7) * 16) =
                    make_uint4(operand(x[i].x), operand(x[i].y), operand(x[i].z),
                               operand(x[i].w));
            }
            fence_smem_async();
            warp_arrive(bar_q + 8 * blk);

            const uint32_t R = row0 + at_row;
            int my_lo = 0, my_hi = 0;
            if (at_row < rows) {
                const int pos = s.len - s.n + int(R / group);
                my_hi = a.causal ? pos + 1 : s.len;
                if (a.window > 0) my_lo = max(0, pos - a.window + 1);
            }
            const uint32_t lanes = uint32_t(warp % 4 * 32) << 16;
            const uint32_t ts = tmem + lanes + blk * kTile;
            const uint32_t to = tmem + lanes + 2 * kTile + blk * D;
            // a scale of 0 still has to leave masked scores at -infinity
            const float scale =
                kQ8 && !PB ? fmaxf(a.scale_log2 * __ldg(a.k_scale + head), 1e-30f) : a.scale_log2;
            auto rescale = [&](float keep) {  // the block's accumulator
#pragma unroll
                for (int i = 0; i < D; i += 32) {
                    uint32_t o[32];
                    tmem_ld32(to + i, o);
                    wait_ld();
                    keep32(o);
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        o[e] = __float_as_uint(__uint_as_float(o[e]) * keep);
                    tmem_st32(to + i, o);
                }
                if (PB) wait_st();  // a tile may rescale twice, for the gain and for the maximum
            };
            const int first = p.t0 + (paired ? blk : 0), by = paired ? 2 : 1;  // its tiles
            // One tile of scores; `edge`: some row does not see all of it.
            auto tile = [&](int j, auto edge) {
                uint32_t x[kTile], w[kTile / 4];
                uint64_t sum[2];
                float top[8];
                // Scales of each 8 tokens: K's (times the logit multiplier) go on the scores, V's,
                // times a gain that the accumulator follows, on the weights: as a term of the
                // exponent, divided out again for the sum of the weights alone
                const float4* const sc = reinterpret_cast<const float4*>(
                    smem + L::kScales + (PB ? (j - T0) % L::kScaleTiles * L::kScaleBytes : 0));
                if (PB) {
                    const float gain = sc[kTile / 8].x;
                    if (gain != vgain) {
                        if (j > first) rescale(gain / vgain);
                        vgain = gain;
                    }
                }
                // weights of elements [64 h, 64 h + 64) relative to the maximum m, in the
                // scores' registers and 8 at a time; along with the first half the largest of
                // all 128 scores: the exponentials set the pace, the rest is issued in between
                auto weigh = [&](int h) {
                    float off = m == -INFINITY ? 0.f : -m;
                    if (kQ8 && !PB) off += kLift;
#pragma unroll
                    for (int g = 0; g <= 8; ++g) {
                        const int at = h * (kTile / 2) + g * 8;
                        const float mul = PB && g < 8 ? sc[h * 8 + g].x : scale;
                        const float add = PB && g < 8 ? off + sc[h * 8 + g].y : off;
                        const uint64_t cc = pair(mul, mul), mm = pair(add, add);
                        if (g < 8) {
                            if (h == 0 && PB) {
                                float u = max8(x + g * 8) * sc[g].x;
                                float v = max8(x + kTile / 2 + g * 8) * sc[8 + g].x;
                                top[0] = g == 0 ? fmaxf(u, v) : max3(top[0], u, v);
                            } else if (h == 0) {
#pragma unroll
                                for (int i = 0; i < 8; ++i) {
                                    const float u = __uint_as_float(x[g * 8 + i]);
                                    const float v = __uint_as_float(x[kTile / 2 + g * 8 + i]);
                                    top[i] = g == 0 ? fmaxf(u, v) : max3(top[i], u, v);
                                }
                            }
#pragma unroll
                            for (int i = 0; i < 8; i += 2) {
                                float e0, e1;
                                unpair(fma2(pair(__uint_as_float(x[at + i]),
                                                 __uint_as_float(x[at + i + 1])),
                                            cc, mm),
                                       e0, e1);
                                x[at + i] = __float_as_uint(ex2(e0));
                                x[at + i + 1] = __float_as_uint(ex2(e1));
                            }
                        }
                        if (g > 0) {
                            uint64_t part = 0;  // of these 8 weights, with V's scale
#pragma unroll
                            for (int i = -8; i < 0; i += 2) {
                                const float e0 = __uint_as_float(x[at + i]);
                                const float e1 = __uint_as_float(x[at + i + 1]);
                                if (PB)
                                    part = i == -8 ? pair(e0, e1) : add2(part, pair(e0, e1));
                                else
                                    sum[i / 2 & 1] = add2(sum[i / 2 & 1], pair(e0, e1));
                                w[g * 4 + i / 2] = operand2<PAGE>(e0, e1);
                            }
                            if (PB) {
                                const float over = sc[h * 8 + g - 1].z;
                                sum[g & 1] = fma2(part, pair(over, over), sum[g & 1]);
                            }
                        }
                    }
                };
                // The first half's weights are relative to the old maximum while the new one is
                // found; the tile is read again where that has grown too far.
                bool grown;
                do {
#pragma unroll
                    for (int i = 0; i < kTile; i += 32) tmem_ld32(ts + i, x + i);
                    wait_ld();
#pragma unroll
                    for (int i = 0; i < kTile; i += 32) keep32(x + i);
                    if (decltype(edge)::value) {
                        const int from = my_lo - j * kTile, until = my_hi - j * kTile;
#pragma unroll
                        for (int i = 0; i < kTile; ++i)
                            if (i < from || i >= until) x[i] = 0xff800000u;  // -infinity
                    }
                    sum[0] = sum[1] = 0;
                    weigh(0);
                    if (!PB)
                        top[0] = fmaxf(max3(max3(top[0], top[1], top[2]), top[3], top[4]),
                                       max3(top[5], top[6], top[7]));
                    const float now = PB ? top[0] : top[0] * scale;
                    const bool over = now > m + kGrow;
                    grown = __any_sync(0xffffffffu, over);
                    if (grown) {
                        float keep = 1.f;
                        if (over) {
                            keep = m == -INFINITY ? 0.f : ex2(m - now);
                            l *= keep;
                            m = now;
                        }
                        // the block's last products are done: its scores came after them
                        if (j > first) rescale(keep);
                    }
                } while (grown);
                // the first half's product runs while the second half is computed
                tmem_st32(ts, w);
                wait_st();
                fence_before();
                warp_arrive(bar_p + 16 * blk);
                weigh(1);
                tmem_st32(ts + kTile / 4, w);
                wait_st();
                fence_before();
                warp_arrive(bar_p + 16 * blk + 8);
                float s0, s1;
                unpair(add2(sum[0], sum[1]), s0, s1);
                l += s0 + s1;
            };
            uint32_t phase = 0;
            for (int j = first; j < p.t1; j += by, phase ^= 1) {
                if (!warp_wait(bar_s + 8 * blk, phase, gave_up)) break;
                fence_after();
                if (j * kTile < p.lo_all || p.hi_all - j * kTile < kTile)
                    tile(j, std::true_type());
                else
                    tile(j, std::false_type());
            }
            warp_wait(bar_o + 8 * blk, 0, gave_up);
        }
    } else if (kQ8 && warp < 12) {
        // ---------------------------------------------------------- widening (8-bit pages)
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kProducerRegs));
        // A warp reads 64 of the 128 codes of 8 rows at a time and stores them as f16.  Its
        // lanes take rows r and r ^ 5 in pairs, so that neither the reads (in 16-byte pieces
        // swizzled by r) nor the writes (every other piece, swizzled alike) share a bank.
        const int c = lane % 4, r8 = lane / 8 ^ (lane / 4 % 2 * 5);
        uint32_t slot = 0, turn = 0, raw = 0, raw_turn = 0;
        bool live = true;
        for (int j = T0; j < T1 && live; ++j) {
#pragma unroll
            for (int side = 0; side < 2; ++side) {
                if (live) live = warp_wait(bar_raw + 8 * raw, raw_turn, gave_up);
                if (live) live = warp_wait(bar_empty + 8 * slot, turn ^ 1, gave_up);
                if (!live) break;
                const uint8_t* const src = smem + L::kRaw + raw * L::kRawSlot;
                uint8_t* const dst = smem + L::kRing + slot * L::kSlot;
                const bool edge = side == 1 && (j * kTile < lo || hi - j * kTile < kTile);
                uint4 x[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int u = (warp - 8) * 8 + i, r = u / 2 * 8 + r8, h = u % 2;
                    x[i] = *reinterpret_cast<const uint4*>(src + r * 128 +
                                                           (((h * 4 + c) ^ r) & 7) * 16);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int u = (warp - 8) * 8 + i, r = u / 2 * 8 + r8, h = u % 2;
                    uint32_t y[8];
                    widen4<PAGE>(x[i].x, y[0], y[1]);
                    widen4<PAGE>(x[i].y, y[2], y[3]);
                    widen4<PAGE>(x[i].z, y[4], y[5]);
                    widen4<PAGE>(x[i].w, y[6], y[7]);
                    const int t = j * kTile + r;
                    if (edge && (t < lo || t >= hi)) {  // V rows no query sees
#pragma unroll
                        for (int e = 0; e < 8; ++e) y[e] = 0;
                    }
                    uint8_t* const row = dst + h * (kTile * 128) + r * 128;
                    *reinterpret_cast<uint4*>(row + ((2 * c ^ r) & 7) * 16) =
                        make_uint4(y[0], y[1], y[2], y[3]);
                    *reinterpret_cast<uint4*>(row + (((2 * c + 1) ^ r) & 7) * 16) =
                        make_uint4(y[4], y[5], y[6], y[7]);
                }
                fence_smem_async();
                warp_arrive(bar_full + 8 * slot);
                warp_arrive(bar_raw_empty + 8 * raw);
                if (++slot == L::kSlots) slot = 0, turn ^= 1;
                if (++raw == L::kRawSlots) raw = 0, raw_turn ^= 1;
            }
        }
    } else if (!kQ8 && warp < 12) {
        // -------------------------------------------------------------- producers
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kProducerRegs));
        // Copy k of a tile (page k / kHalves, column k % kHalves) is issued by warp k % 4,
        // lane k / 4: the lanes of one warp take turns, 54 cycles each.
        const int bs = a.r.block_size, me = warp - 8;
        const int box = min(bs, kTile);               // slots of a copy
        const int copies = kTile / box * L::kHalves;  // of a tile
        const int k = lane * L::kProducers + me, my_page = k / L::kHalves, my_half = k % L::kHalves;
        const bool mine = k < copies;
        const int32_t* table = a.r.table + (int64_t)b * a.r.max_blocks;
        auto seen = [&](int j) {
            const int t = j * kTile + my_page * box;
            return mine && j < T1 && t < hi && t + box > lo;
        };
        auto id_of = [&](int j) {
            return seen(j) ? __ldg(table + (j * kTile + my_page * box) / bs) : -1;
        };
        const uint32_t at = my_half * (kTile * 128) + my_page * box * 128;
        int id = id_of(T0);
        uint32_t slot = 0, turn = 0, patches = 0, n = 0;  // n: tiles into the ring so far
        bool live = true;
        for (int j = T0; j < T1 && live; ++j) {
            const int next = id_of(j + 1);
            const bool ok = valid(a.r, id);
            const unsigned which = __ballot_sync(0xffffffffu, ok);
            const bool gone = seen(j) && !ok;
            if (__any_sync(0xffffffffu, gone)) {  // rare: the warp stays together beside it
                if (gone) {
                    latch(a.r.err, PGD_ERR_BLOCK_ID);
                    mark_lost(a, s, row0, j * kTile + my_page * box, box, lost);
                }
                __syncwarp();
            }
            const uint32_t bytes = __popc(which) * box * 128;
            // rows no query sees, or that have no page, among this warp's copies
            const bool patch = j * kTile < lo || hi - j * kTile < kTile ||
                               __any_sync(0xffffffffu, mine && !ok);
            const int row = (j * kTile + my_page * box) % bs;
#pragma unroll
            for (int side = 0; side < 2; ++side) {
                if (live) live = warp_wait(bar_empty + 8 * slot, turn ^ 1, gave_up);
                if (!live) break;
                const bool hold = side == 1 && patch;
                const uint32_t full = bar_full + 8 * slot;
                const uint32_t bar = hold ? bar_patch + 8 * me : full;
                if (lane == 0) {
                    if (bytes)
                        bar_arrive_tx(bar, bytes);
                    else
                        bar_arrive(bar);
                }
                __syncwarp();
                if (ok)
                    tma_load_4d(base + L::kRing + slot * L::kSlot + at, side ? &map_v : &map_k, bar,
                                0, row, head * L::kHalves + my_half, id);
                if (hold) {
                    // V: zero those rows once the copies are there, then hand the tile over
                    live = warp_wait(bar_patch + 8 * me, patches++ & 1, gave_up);
                    if (!live) break;
                    for (int c = me; c < copies; c += L::kProducers) {
                        const int first = c / L::kHalves * box;
                        uint8_t* const col = smem + L::kRing + slot * L::kSlot +
                                             c % L::kHalves * (kTile * 128) + lane % 8 * 16;
                        for (int r = first + lane / 8; r < first + box; r += 4) {
                            const int t = j * kTile + r;
                            if (t < lo || t >= hi || !(which >> (c / L::kProducers) & 1))
                                *reinterpret_cast<uint4*>(col + r * 128) = make_uint4(0, 0, 0, 0);
                        }
                    }
                    fence_smem_async();
                    __syncwarp();
                    if (lane == 0) bar_arrive(full);
                }
                if (++slot == L::kSlots) slot = 0, turn ^= 1;
                ++n;
            }
            id = next;
        }
        if (!live) {  // no copy of this warp may land after the CTA has ended
            volatile int never = 0;
            if (patches) bar_wait(bar_patch + 8 * me, (patches - 1) & 1, &never);
            for (uint32_t i = n > L::kSlots ? n - L::kSlots : 0; i < n; ++i)
                bar_wait(bar_full + 8 * (i % L::kSlots), i / L::kSlots & 1, &never);
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssuerRegs));
    }
    if (kQ8 && warp >= 14) {
        // -------------------------------------------------------- producers (8-bit pages)
        // One copy a page, issued by warp 14 + page % 2, lane page / 2.  Warp 14 also brings the
        // scales, lane by page, one tile ahead, and V's gain: a power of two that puts the
        // first tile's largest V scale in [8, 16) and falls when one grows past 128: a weight,
        // up to 2^kGrow, times its scale stays within f16 and keeps its 11 bits down to
        // 2^-17 of the largest.
        const int bs = a.r.block_size, me = warp - 14;
        const int box = min(bs, kTile), pages = kTile / box;
        const int page = lane * L::kProducers + me;
        const int32_t* table = a.r.table + (int64_t)b * a.r.max_blocks;
        auto seen = [&](int j, int pg) {
            const int t = j * kTile + pg * box;
            return pg < pages && j < T1 && t < hi && t + box > lo;
        };
        auto id_of = [&](int j, int pg) {
            return seen(j, pg) ? __ldg(table + (j * kTile + pg * box) / bs) : -1;
        };
        auto scale_of = [&](const float* scales, int id, float none) {
            return valid(a.r, id) ? __ldg(scales + (int64_t)id * a.hkv + head) : none;
        };
        int id = id_of(T0, page), id_s = -1;
        float ks = 1.f, vs = 0.f, gain = 0.f;
        const bool scaling = PB && me == 0;
        if (scaling) {
            id_s = id_of(T0, lane);
            ks = scale_of(a.k_scale, id_s, 1.f);
            vs = scale_of(a.v_scale, id_s, 0.f);
            id_s = id_of(T0 + 1, lane);
        }
        // The scales of tile j; warp 14's arrival at the tile's keys hands them over.  That of
        // kScaleTiles before is done with: its values were used before the keys after it.
        auto put_scales = [&](int j) {
            float4* const to = reinterpret_cast<float4*>(
                smem + L::kScales + (j - T0) % L::kScaleTiles * L::kScaleBytes);
            // scales are not negative, so their bits are ordered alike
            const float most = __uint_as_float(
                __reduce_max_sync(0xffffffffu, __float_as_uint(vs) & 0x7fffffffu));
            if (most * gain > 128.f || gain == 0.f) {
                const int e = min(max((__float_as_int(most) >> 23) & 255, 5), 252);
                gain = __int_as_float((257 - e) << 23);
            }
            // a scale of 0 stays above 0: masked scores times K's are still -infinity,
            // and weights times V's (0 in f16) can be summed without it
            const float by = vs * gain < 1e-20f ? 1e-20f : vs * gain;
            const float on = ks * a.scale_log2;
            const float4 e =
                make_float4(on < 1e-30f ? 1e-30f : on, __log2f(by), __fdividef(1.f, by), 0.f);
            if (lane < pages)
                for (int g = lane * box / 8; g < (lane + 1) * box / 8; ++g) to[g] = e;
            if (lane == 0) to[kTile / 8].x = gain;
        };
        if (scaling) put_scales(T0);
        uint32_t raw = 0, turn = 0, n = 0;
        bool live = true;
        for (int j = T0; j < T1 && live; ++j) {
            const int next = id_of(j + 1, page);
            float next_ks = 1.f, next_vs = 0.f;
            if (scaling) {
                next_ks = scale_of(a.k_scale, id_s, 1.f);
                next_vs = scale_of(a.v_scale, id_s, 0.f);
                id_s = id_of(j + 2, lane);
            }
            const bool ok = seen(j, page);
            if (ok && !valid(a.r, id)) {
                latch(a.r.err, PGD_ERR_BLOCK_ID);
                mark_lost(a, s, row0, j * kTile + page * box, box, lost);
                id = -1;  // outside the tensor: zeros
            }
            const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, ok)) * box * 128;
            const int row = (j * kTile + page * box) % bs;
#pragma unroll
            for (int side = 0; side < 2; ++side) {
                if (live) live = warp_wait(bar_raw_empty + 8 * raw, turn ^ 1, gave_up);
                if (!live) break;
                __syncwarp();
                if (lane == 0) {
                    if (bytes)
                        bar_arrive_tx(bar_raw + 8 * raw, bytes);
                    else
                        bar_arrive(bar_raw + 8 * raw);
                }
                __syncwarp();
                if (ok)
                    tma_load_4d(base + L::kRaw + raw * L::kRawSlot + page * box * 128,
                                side ? &map_v : &map_k, bar_raw + 8 * raw, 0, row, head, id);
                if (++raw == L::kRawSlots) raw = 0, turn ^= 1;
                ++n;
            }
            id = next;
            ks = next_ks;
            vs = next_vs;
            // behind this tile's copies, which it would hold up
            if (scaling && live && j + 1 < T1) put_scales(j + 1);
        }
        if (!live) {  // no copy of this warp may land after the CTA has ended
            volatile int never = 0;
            for (uint32_t i = n > L::kRawSlots ? n - L::kRawSlots : 0; i < n; ++i)
                bar_wait(bar_raw + 8 * (i % L::kRawSlots), i / L::kRawSlots & 1, &never);
        }
    }
    if ((warp == 12 || warp == 13) && T1 > T0) {
        // --------------------------------------------------------------- products
        constexpr uint32_t kQK = instruction(kBlock, kTile, !kQ8, 0);
        constexpr uint32_t kPV = instruction(kBlock, D, !kQ8, 1);
        constexpr uint32_t kHi = operand_hi(1024);
        const int i = warp - 12;  // the block whose products this warp issues
        const int t0 = i ? sp[1].t0 : sp[0].t0, t1 = i ? sp[1].t1 : sp[0].t1;
        const int first = t0 + (paired ? i : 0);
        auto sees = [&](int j) { return j >= first && j < t1 && (!paired || !((j - first) & 1)); };
        const uint32_t acc = __shfl_sync(0xffffffffu, tmem, 0);
        const uint32_t acc_s = acc + i * kTile, acc_o = acc + 2 * kTile + i * D;
        const uint32_t q_lo = operand_lo(base, 16) + i * (L::kQ / 16);
        const uint32_t k_lo = operand_lo(base + L::kRing, 16);
        const uint32_t v_lo = operand_lo(base + L::kRing, kTile * 128);
        auto wait = [&](uint32_t bar, uint32_t parity) {
            return warp_wait(bar, parity, gave_up);
        };
        auto scores = [&](uint32_t slot, bool turn) {
            fence_after();
            if (elected()) {
#pragma unroll
                for (int e = 0; e < D / 16; ++e) {
                    const uint32_t at = (e / 4 * (kTile * 128) + e % 4 * 32) / 16;
                    mma_ss(acc_s, q_lo + at, k_lo + slot * (L::kSlot / 16) + at, kHi, kQK, e > 0);
                }
                // the commits wait for the queue of products, so the turn goes first
                if (turn) bar_arrive(bar_turn + 8 * (1 - i));
                mma_commit(bar_s + 8 * i);
                mma_commit(bar_empty + 8 * slot);
            }
        };
        auto values = [&](int half, uint32_t slot, bool add) {
            fence_after();
            if (elected()) {
#pragma unroll
                for (int k = 0; k < kTile / 32; ++k) {
                    const int e = half * (kTile / 32) + k;
                    mma_ts(acc_o, acc_s + e * 8, v_lo + slot * (L::kSlot / 16) + e * 128, kHi, kPV,
                           add || e > 0);
                }
                if (half) mma_commit(bar_empty + 8 * slot);
            }
        };
        auto pass = [&](uint32_t slot) {  // a tile this block does not see
            warp_arrive(bar_empty + 8 * slot);
        };
        // tiles lie in the ring as K(T0), V(T0), K(T0 + 1), ..: `at` is the next one's slot
        uint32_t at = 0, turn = 0, weights = 0;
        auto step = [&]() {
            if (++at == L::kSlots) at = 0, turn ^= 1;
        };
        bool live = wait(bar_full, 0);
        if (live && sees(T0)) live = wait(bar_q + 8 * i, 0);
        if (live) {
            if (sees(T0))
                scores(0, false);
            else
                pass(0);
        }
        step();
        for (int j = T0; j < T1 && live; ++j) {
            const uint32_t v_at = at, v_turn = turn;
            step();
            // all that can be waited for is there before the turn is taken
            const bool now = sees(j), next = sees(j + 1);
            live = wait(bar_full + 8 * v_at, v_turn);
            if (live && j + 1 < T1) live = wait(bar_full + 8 * at, turn);
            if (live && j + 1 == first && next) live = wait(bar_q + 8 * i, 0);
            if (live && now) live = wait(bar_p + 16 * i, weights);
            if (live && (i || j > T0)) live = wait(bar_turn + 8 * i, (j - T0 + 1 - i) & 1);
            if (!live) break;
            if (now) {
                values(0, v_at, j > first);
                live = wait(bar_p + 16 * i + 8, weights);
                if (!live) break;
                values(1, v_at, true);
                weights ^= 1;
            } else {
                pass(v_at);
            }
            if (j + 1 < T1 && next) {
                scores(at, true);
            } else {
                if (j + 1 < T1) pass(at);
                warp_arrive(bar_turn + 8 * (1 - i));
            }
            step();
        }
        // every product and its arrivals are over before their memory is given up
        if (elected()) {
            mma_commit(bar_o + 8 * i);
        }
        volatile int never = 0;
        bar_wait(bar_o + 8 * i, 0, &never);
    }
    __syncwarp();
    fence_before();
    __syncthreads();
    fence_after();
    const bool failed = *gave_up || !s.ok || (warp < 8 && lost[at_row / 32] >> lane & 1);
    if (*gave_up && threadIdx.x == 0) latch(a.r.err, PGD_ERR_TIMEOUT);

    // -------------------------------------------------------------------- results
    const int64_t out_at = (int64_t)s.row0 * a.hq + (int64_t)head * a.group;  // head vectors
    // what the accumulator is to be multiplied with beside 1 / l
    const float by = !kQ8 ? 1.f : PB ? 1.f / vgain : __ldg(a.v_scale + head);
    if (a.cluster == 1 && !paired) {
        if (warp < 8) {
            const uint32_t to = tmem + (uint32_t(warp % 4 * 32) << 16) + 2 * kTile + blk * D;
            const float inv = failed ? NAN : l > 0.f ? by / l : l == 0.f ? 0.f : NAN;
            const bool have = blk ? sp[1].t1 > sp[1].t0 : sp[0].t1 > sp[0].t0;
            uint8_t* const rowp = smem + (blk * kBlock + my_row) * (D * 2);
#pragma unroll
            for (int i = 0; i < D; i += 32) {
                uint32_t o[32];
                if (have) {
                    tmem_ld32(to + i, o);
                    wait_ld();
                    keep32(o);
                }
#pragma unroll
                for (int e = 0; e < 32; e += 8) {
                    uint32_t w[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float y0 = __uint_as_float(o[e + 2 * k]) * inv;
                        const float y1 = __uint_as_float(o[e + 2 * k + 1]) * inv;
                        w[k] = l == 0.f && !failed ? 0u : inv != inv ? 0x7fc07fc0u : bf16x2(y0, y1);
                    }
                    const int c = (i + e) / 8;
                    *reinterpret_cast<uint4*>(rowp + ((c ^ my_row) & (D / 8 - 1)) * 16) =
                        make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
            __syncwarp();
            constexpr int kVecs = D / 8, kStep = 32 / kVecs;
            const int c = lane % kVecs;
            Rows at(row0 + warp * 32 + lane / kVecs, group, kStep);
#pragma unroll
            for (int i = 0; i < kVecs; ++i, at.next()) {
                const int r = warp * 32 + lane / kVecs + i * kStep;
                if (r < rows)
                    *reinterpret_cast<uint4*>(
                        a.out + (out_at + at.token * a.hq + at.head) * D + c * 8) =
                        *reinterpret_cast<const uint4*>(smem + r * (D * 2) +
                                                        ((c ^ r) & (kVecs - 1)) * 16);
            }
        }
    } else {
        // unnormalised rows, maxima and sums to shared memory, then every CTA of the
        // cluster joins a share of the rows
        float2* const stat = reinterpret_cast<float2*>(smem);  // of the 256 rows
        if (warp < 8) {
            const uint32_t to = tmem + (uint32_t(warp % 4 * 32) << 16) + 2 * kTile + blk * D;
            const bool have = blk ? sp[1].t1 > sp[1].t0 : sp[0].t1 > sp[0].t0;
            const int r = blk * kBlock + my_row;
            stat[r] = make_float2(m, failed ? NAN : l);
            if (have && at_row - lane < rows) {
#pragma unroll
                for (int i = 0; i < D; i += 32) {
                    uint32_t o[32];
                    tmem_ld32(to + i, o);
                    wait_ld();
                    keep32(o);
#pragma unroll
                    for (int e = 0; e < 32; e += 4) {
                        const int c = (i + e) / 4;
                        *reinterpret_cast<uint4*>(smem + L::kRing + r * (D * 4) +
                                                  ((c ^ r) & (D / 4 - 1)) * 16) =
                            make_uint4(__float_as_uint(__uint_as_float(o[e]) * by),
                                       __float_as_uint(__uint_as_float(o[e + 1]) * by),
                                       __float_as_uint(__uint_as_float(o[e + 2]) * by),
                                       __float_as_uint(__uint_as_float(o[e + 3]) * by));
                    }
                }
            }
        }
        cluster_sync();
        if (warp < 8) {
            // part k of a row: CTA k of the cluster, or with paired blocks block k % 2 of CTA k / 2
            const int parts = paired ? 2 * a.cluster : a.cluster;
            auto cta_of = [&](int k) { return paired ? k / 2 : k; };
            auto row_of = [&](int r, int k) { return paired ? r + k % 2 * kBlock : r; };
            // four columns a thread, kLines rows of a warp at once
            constexpr int kQuads = D / 4, kLines = 32 / kQuads;
            const int step = a.cluster * 8 * kLines;
            const int c = lane % kQuads, line = lane / kQuads;
            const int from = (share * 8 + warp) * kLines;
            Rows at(row0 + from + line, group, step);
            // kR rows with kP parts each are on their way together: four loads, and none for a
            // part that is not there (two parts loaded as four: 481 against 462 us for two
            // chunks of 1400 tokens, 10k cached each; four rows of two spill, 513)
            auto join = [&](auto some_rows, auto some_parts) {
                constexpr int kR = decltype(some_rows)::value, kP = decltype(some_parts)::value;
                for (int r0 = from; r0 < rows; r0 += kR * step) {
                    float o[kR][4], sum[kR], top[kR];
#pragma unroll
                    for (int u = 0; u < kR; ++u) {
                        o[u][0] = o[u][1] = o[u][2] = o[u][3] = sum[u] = 0.f;
                        top[u] = -INFINITY;
                    }
                    for (int k0 = 0; k0 < parts; k0 += kP) {
                        float2 st[kR][kP];
                        float4 v[kR][kP];
#pragma unroll
                        for (int u = 0; u < kR; ++u)
#pragma unroll
                            for (int k = 0; k < kP; ++k) {
                                const int part = min(k0 + k, parts - 1);
                                const int r = row_of(min(r0 + u * step + line, rows - 1), part);
                                st[u][k] = peer_ld2(peer_addr(base + r * 8, cta_of(part)));
                                v[u][k] = peer_ld4(peer_addr(
                                    base + L::kRing + r * (D * 4) + ((c ^ r) & (kQuads - 1)) * 16,
                                    cta_of(part)));
                            }
#pragma unroll
                        for (int u = 0; u < kR; ++u)
#pragma unroll
                            for (int k = 0; k < kP; ++k) {
                                // a part without a tile of the row left nothing there
                                const float2 x = st[u][k];
                                if (k0 + k >= parts || x.y == 0.f) continue;
                                const float now = fmaxf(top[u], x.x);
                                const float keep = ex2(top[u] - now), w = ex2(x.x - now);
                                top[u] = now;
                                sum[u] = fmaf(w, x.y, sum[u] * keep);
                                o[u][0] = fmaf(w, v[u][k].x, o[u][0] * keep);
                                o[u][1] = fmaf(w, v[u][k].y, o[u][1] * keep);
                                o[u][2] = fmaf(w, v[u][k].z, o[u][2] * keep);
                                o[u][3] = fmaf(w, v[u][k].w, o[u][3] * keep);
                            }
                    }
#pragma unroll
                    for (int u = 0; u < kR; ++u, at.next()) {
                        if (r0 + u * step + line >= rows) continue;
                        // a row that sees a token has a sum of 1 or more; NaN where a part failed
                        const float inv = sum[u] == 0.f ? 0.f : __fdividef(1.f, sum[u]);
                        *reinterpret_cast<uint2*>(
                            a.out + (out_at + at.token * a.hq + at.head) * D + c * 4) =
                            make_uint2(bf16x2(o[u][0] * inv, o[u][1] * inv),
                                       bf16x2(o[u][2] * inv, o[u][3] * inv));
                    }
                }
            };
            using std::integral_constant;
            if (parts > 2)
                join(integral_constant<int, 1>(), integral_constant<int, 4>());
            else
                join(integral_constant<int, 2>(), integral_constant<int, 2>());
        }
        cluster_sync();  // shared memory stays until every CTA has read it
    }
    __syncthreads();
    if (warp == 12) tmem_free(tmem, 512);
}

}  // namespace attend
}  // namespace pgd
