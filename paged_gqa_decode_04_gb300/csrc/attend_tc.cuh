// The attention of many query tokens on the asynchronous tensor cores.
//
//     S = q K^T,  m = running maximum of a row's scores,  P = exp2(c S - m),
//     O += P V,   l += sum of P,   out = O / l
//
// with S and O in float32 in TMEM, m and l in float32 in registers and P rounded to 16
// bits, the type the product takes (at most half a step, 2^-8 in bfloat16, of each weight).
//
// Rows.  The G query heads of a KV head see the same keys, so a CTA takes 256 consecutive
// rows (token, head of the group) of one sequence and KV head: a key tile is fetched once
// for all of them, and a few tokens still fill rows.  They are two blocks of 128 rows,
// the height of the tensor cores' accumulator, each with one thread a row for its softmax
// (no shuffles): while one block's weights are computed, the tensor cores run the other's
// products.
//
// Keys.  Tiles of 128 tokens.  A producer warp walks the block table and fetches each page
// of the tile with one TMA copy for every 64 elements of the head, so that pages land as
// one tile in the swizzled layout both products read: K with its head dimension contiguous,
// V with its tokens as rows (the transposed operand).  Pages no query of the CTA sees are
// not fetched, and V rows outside the visible range are zeroed, so that nothing in an
// unused slot is multiplied.
//
// Warps: 0-3 and 4-7 the softmax of the two blocks, 8 the producer, 9 issues products.
// Weights take the place of the scores they came from in TMEM.  The order of products,
// P0 V(j), q0 K(j+1), P1 V(j), q1 K(j+1), keeps the tensor cores busy as long as a block's
// softmax takes no longer than two products of the other.  The accumulator is rescaled
// only when a row's maximum has grown by more than 2^8: until then weights are relative to
// an older maximum, at most 256, which costs no precision in either float type.
//
// Few rows.  Where the batch has fewer blocks of rows than the GPU has SMs, up to 8 CTAs
// of a cluster share a block's key tiles and join their sums through each other's shared
// memory: out = sum_c 2^(m_c - m) O_c / sum_c 2^(m_c - m) l_c.
//
// Every wait is bounded; one that gives up latches PGD_ERR_TIMEOUT and ends the CTA.
#pragma once

#include <cuda_bf16.h>

#include "page_ops.h"
#include "ragged.cuh"
#include "umma.cuh"

namespace pgd {
namespace attend {

using namespace umma;

constexpr int kTile = 128;      // tokens of a key tile
constexpr int kBlock = 128;     // rows of a block
constexpr int kRowShift = 8;    // log2 of the rows of a CTA
constexpr int kThreads = 320;
constexpr float kGrow = 8.f;    // base-2 growth of a maximum that is let pass

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
};

template <int D>
struct Layout {
    static constexpr int kHalves = D / 64;                 // 128-byte columns of a head
    static constexpr int kSlot = kTile * D * 2;            // bytes of a K or V tile
    static constexpr int kSlots = D == 128 ? 5 : 8;
    static constexpr int kQ = kBlock * D * 2;              // bytes of a block of queries
    static constexpr int kRing = 2 * kQ;
    static constexpr int kBars = kRing + kSlots * kSlot;
    static constexpr int kBytes = kBars + 256 + 1024;      // and room to align to 1024
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
        p.t1 = (p.hi + kTile - 1) / kTile;
    } else {
        p.lo = p.hi = 0;
    }
    return p;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
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

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    attend_kernel(const __grid_constant__ Args a, const __grid_constant__ CUtensorMap map_k,
                  const __grid_constant__ CUtensorMap map_v) {
    using L = Layout<D>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = (smem_addr(smem_raw) + 1023) & ~1023u;
    uint8_t* const smem = smem_raw + (base - smem_addr(smem_raw));
    const uint32_t bars = base + L::kBars;
    const uint32_t bar_q = bars, bar_s = bars + 16, bar_p = bars + 32, bar_o = bars + 48;
    const uint32_t bar_patch = bars + 64, bar_full = bars + 72;
    const uint32_t bar_empty = bar_full + 8 * L::kSlots, bar_end = bars + 208;
    volatile int* const gave_up = reinterpret_cast<int*>(smem + L::kBars + 240);
    volatile int* const bad = reinterpret_cast<int*>(smem + L::kBars + 244);
    uint32_t* const tmem_at = reinterpret_cast<uint32_t*>(smem + L::kBars + 248);

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int share = a.cluster > 1 ? (int)cluster_rank() : 0;
    if (blockIdx.x == 0) check_all(a.r, false);

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
    int T0 = lo / kTile, T1 = hi > lo ? (hi + kTile - 1) / kTile : T0;
    if (a.cluster > 1) {  // this CTA's share of the tiles
        const int tiles = T1 - T0, t = T0;
        T0 = t + tiles * share / a.cluster;
        T1 = t + tiles * (share + 1) / a.cluster;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        sp[i].t0 = max(sp[i].t0, T0);
        sp[i].t1 = max(sp[i].t0, min(sp[i].t1, T1));
    }

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            bar_init(bar_q + 8 * i, kBlock);
            bar_init(bar_s + 8 * i, 1);
            bar_init(bar_p + 8 * i, kBlock);
            bar_init(bar_o + 8 * i, 1);
        }
        bar_init(bar_patch, 1);
        bar_init(bar_end, 1);
        for (int i = 0; i < L::kSlots; ++i) {
            bar_init(bar_full + 8 * i, 1);
            bar_init(bar_empty + 8 * i, 1);
        }
        *gave_up = 0;
        *bad = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 9) tmem_alloc(smem_addr(tmem_at), 512);
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = *tmem_at;

    float m = -INFINITY, l = 0.f;  // of the thread's row, in the units of exp2
    const int blk = warp / 4;      // block of rows of a softmax warp
    const int my_row = threadIdx.x % kBlock;

    if (warp < 8) {
        // ---------------------------------------------------------------- softmax
        const Span p = blk ? sp[1] : sp[0];
        if (p.t1 > p.t0) {
            // the block's queries into shared memory, swizzled
            constexpr int kVecs = D / 8;
            const __nv_bfloat16* q = a.q + (int64_t)s.row0 * a.q_stride + (int64_t)head * a.group * D;
#pragma unroll 8
            for (int i = my_row; i < kBlock * kVecs; i += kBlock) {
                const int r = i / kVecs, c = i % kVecs;
                const uint32_t R = row0 + blk * kBlock + r;
                uint4 x = make_uint4(0, 0, 0, 0);
                if (blk * kBlock + r < rows) {
                    x = __ldg(reinterpret_cast<const uint4*>(
                        q + (int64_t)(R / group) * a.q_stride + R % group * D + c * 8));
                    x.x = (x.x & a.q_and) ^ a.q_xor;
                    x.y = (x.y & a.q_and) ^ a.q_xor;
                    x.z = (x.z & a.q_and) ^ a.q_xor;
                    x.w = (x.w & a.q_and) ^ a.q_xor;
                }
                *reinterpret_cast<uint4*>(smem + blk * L::kQ + c / 8 * (kBlock * 128) + r * 128 +
                                          ((c ^ r) & 7) * 16) = x;
            }
            fence_smem_async();
            bar_arrive(bar_q + 8 * blk);

            const uint32_t R = row0 + blk * kBlock + my_row;
            int my_lo = 0, my_hi = 0;
            if (blk * kBlock + my_row < rows) {
                const int pos = s.len - s.n + int(R / group);
                my_hi = a.causal ? pos + 1 : s.len;
                if (a.window > 0) my_lo = max(0, pos - a.window + 1);
            }
            const uint32_t lanes = uint32_t(warp % 4 * 32) << 16;
            const uint32_t ts = tmem + lanes + blk * kTile;
            const uint32_t to = tmem + lanes + 2 * kTile + blk * D;
            const float c = a.scale_log2;
            uint32_t phase = 0;
            for (int j = p.t0; j < p.t1; ++j, phase ^= 1) {
                if (!__all_sync(0xffffffffu, bar_wait(bar_s + 8 * blk, phase, gave_up))) break;
                fence_after();
                uint32_t x[kTile];
#pragma unroll
                for (int i = 0; i < kTile; i += 32) tmem_ld32(ts + i, x + i);
                wait_ld();
#pragma unroll
                for (int i = 0; i < kTile; i += 32) keep32(x + i);
                const int t = j * kTile;
                if (t < p.lo_all || t + kTile > p.hi_all) {
                    const int from = my_lo - t, to_ = my_hi - t;
#pragma unroll
                    for (int i = 0; i < kTile; ++i)
                        if (i < from || i >= to_) x[i] = 0xff800000u;  // -infinity
                }
                float top[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) top[i] = __uint_as_float(x[i]);
#pragma unroll
                for (int i = 4; i < kTile; ++i)
                    top[i % 4] = fmaxf(top[i % 4], __uint_as_float(x[i]));
                const float now = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * c;
                float keep = 1.f;
                if (now > m + kGrow || m == -INFINITY) {
                    keep = m == -INFINITY ? 0.f : ex2(m - now);
                    l *= keep;
                    m = now;
                }
                if (j > p.t0 && __any_sync(0xffffffffu, keep != 1.f)) {
                    // the block's last products are done: its scores came after them
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
                }
                const float off = m == -INFINITY ? 0.f : -m;
                const uint64_t cc = pair(c, c), mm = pair(off, off);
                uint64_t sum[2] = {0, 0};
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t w[kTile / 4];
#pragma unroll
                    for (int i = 0; i < kTile / 2; i += 2) {
                        const int at = h * (kTile / 2) + i;
                        float e0, e1;
                        unpair(fma2(pair(__uint_as_float(x[at]), __uint_as_float(x[at + 1])), cc,
                                    mm),
                               e0, e1);
                        e0 = ex2(e0);
                        e1 = ex2(e1);
                        sum[i / 2 % 2] = add2(sum[i / 2 % 2], pair(e0, e1));
                        w[i / 2] = bf16x2(e0, e1);
                    }
                    tmem_st32(ts + h * (kTile / 4), w);
                }
                wait_st();
                fence_before();
                bar_arrive(bar_p + 8 * blk);
                float s0, s1;
                unpair(add2(sum[0], sum[1]), s0, s1);
                l += s0 + s1;
            }
            bar_wait(bar_o + 8 * blk, 0, gave_up);
        }
    } else if (warp == 8) {
        // --------------------------------------------------------------- producer
        const int bs = a.r.block_size;
        const int box = min(bs, kTile);               // slots of a copy
        const int pages = kTile / box;                // copies of a tile and column
        const uint32_t box_bytes = box * 128;
        const int my_page = lane / L::kHalves, my_half = lane % L::kHalves;
        const bool mine = my_page < pages;
        const int64_t table_row = (int64_t)b * a.r.max_blocks;
        // block id of this lane's page of tile j; -1 where no query sees it
        auto id_of = [&](int j) -> int {
            const int t = j * kTile + my_page * box;
            if (!mine || j >= T1 || t >= hi || t + box <= lo) return -1;
            return __ldg(a.r.table + table_row + t / bs);
        };
        auto seen = [&](int j) {
            const int t = j * kTile + my_page * box;
            return mine && t < hi && t + box > lo;
        };
        int id = T0 < T1 ? id_of(T0) : -1;
        uint32_t n = 0, patches = 0;                  // tiles into the ring so far
        bool stop = false;
        for (int j = T0; j < T1 && !stop; ++j) {
            const int next = id_of(j + 1);
            const bool ok = id >= 0 && id < a.r.num_blocks;
            if (seen(j) && !ok) {
                latch(a.r.err, PGD_ERR_BLOCK_ID);
                *bad = 1;
            }
            const uint32_t copies = __popc(__ballot_sync(0xffffffffu, ok));
            const bool patch = j * kTile < lo || (j + 1) * kTile > hi ||
                               copies < uint32_t(pages * L::kHalves);
            for (int side = 0; side < 2; ++side, ++n) {
                const uint32_t slot = n % L::kSlots, use = n / L::kSlots;
                if (use > 0 &&
                    !__all_sync(0xffffffffu,
                                bar_wait(bar_empty + 8 * slot, (use - 1) & 1, gave_up))) {
                    stop = true;
                    break;
                }
                const bool hold = side == 1 && patch;
                const uint32_t bar = hold ? bar_patch : bar_full + 8 * slot;
                const uint32_t dst = base + L::kRing + slot * L::kSlot;
                if (lane == 0) {
                    if (copies)
                        bar_arrive_tx(bar, copies * box_bytes);
                    else
                        bar_arrive(bar);
                }
                __syncwarp();
                if (ok)
                    tma_load_4d(dst + my_half * (kTile * 128) + my_page * box_bytes,
                                side ? &map_v : &map_k, bar, 0, (j * kTile + my_page * box) % bs,
                                head * L::kHalves + my_half, id);
                if (hold) {
                    // zero the rows no query sees, then hand the tile over
                    if (!__all_sync(0xffffffffu, bar_wait(bar_patch, patches & 1, gave_up))) {
                        stop = true;
                        break;
                    }
                    ++patches;
                    const unsigned there = __ballot_sync(0xffffffffu, ok);
                    for (int r = 0; r < kTile; ++r) {
                        const int t = j * kTile + r;
                        const bool keep = t >= lo && t < hi &&
                                          (there >> (r / box * L::kHalves) & 1);
                        if (!keep && lane < L::kHalves * 8)
                            *reinterpret_cast<uint4*>(smem + L::kRing + slot * L::kSlot +
                                                      lane / 8 * (kTile * 128) + r * 128 +
                                                      lane % 8 * 16) = make_uint4(0, 0, 0, 0);
                    }
                    fence_smem_async();
                    __syncwarp();
                    if (lane == 0) bar_arrive(bar_full + 8 * slot);
                }
            }
            id = next;
        }
        if (stop) {  // no copy may land after the CTA has ended
            const uint32_t from = n > L::kSlots ? n - L::kSlots : 0;
            for (uint32_t i = from; i < n; ++i) {
                volatile int never = 0;
                bar_wait(bar_full + 8 * (i % L::kSlots), i / L::kSlots & 1, &never);
            }
        }
    } else if (lane == 0 && T1 > T0) {
        // --------------------------------------------------------------- products
        constexpr uint32_t kQK = instruction(kBlock, kTile, 1, 0);
        constexpr uint32_t kPV = instruction(kBlock, D, 1, 1);
        uint32_t n = 0;                               // tiles of the ring taken so far
        auto ready = [&](uint32_t i) {
            return bar_wait(bar_full + 8 * (i % L::kSlots), i / L::kSlots & 1, gave_up);
        };
        auto tile = [&](uint32_t i) { return base + L::kRing + i % L::kSlots * L::kSlot; };
        auto scores = [&](int i, uint32_t k) {
            fence_after();
#pragma unroll
            for (int e = 0; e < D / 16; ++e) {
                const uint32_t at = e / 4 * (kTile * 128) + e % 4 * 32;
                mma_ss(tmem + i * kTile, operand(base + i * L::kQ + at, 16, 1024),
                       operand(k + at, 16, 1024), kQK, e > 0);
            }
            mma_commit(bar_s + 8 * i);
        };
        auto values = [&](int i, uint32_t v, bool add) {
            fence_after();
#pragma unroll
            for (int e = 0; e < kTile / 16; ++e)
                mma_ts(tmem + 2 * kTile + i * D, tmem + i * kTile + e * 8,
                       operand(v + e * 2048, kTile * 128, 1024), kPV, add || e > 0);
        };
        uint32_t done[2] = {0, 0};                    // tiles whose weights were taken
        bool live = ready(0);
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (live && T0 >= sp[i].t0 && T0 < sp[i].t1) {
                live = bar_wait(bar_q + 8 * i, 0, gave_up);
                if (live) scores(i, tile(0));
            }
        if (live) mma_commit(bar_empty + 8 * 0);
        n = 1;
        for (int j = T0; j < T1 && live; ++j, n += 2) {
            const bool more = j + 1 < T1;
            live = ready(n) && (!more || ready(n + 1));
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (live && j >= sp[i].t0 && j < sp[i].t1)
                    live = bar_wait(bar_p + 8 * i, done[i]++ & 1, gave_up);
                if (!live) break;
                if (j >= sp[i].t0 && j < sp[i].t1) {
                    values(i, tile(n), j > sp[i].t0);
                    if (j + 1 == sp[i].t1) mma_commit(bar_o + 8 * i);
                }
                if (i == 1) mma_commit(bar_empty + 8 * (n % L::kSlots));
                if (more && j + 1 >= sp[i].t0 && j + 1 < sp[i].t1) {
                    if (j + 1 == sp[i].t0) live = bar_wait(bar_q + 8 * i, 0, gave_up);
                    if (live) scores(i, tile(n + 1));
                }
                if (i == 1 && more) mma_commit(bar_empty + 8 * ((n + 1) % L::kSlots));
            }
        }
        // every product and its arrivals are over before their memory is given up
        volatile int never = 0;
        mma_commit(bar_end);
        bar_wait(bar_end, 0, &never);
    }
    __syncwarp();
    fence_before();
    __syncthreads();
    fence_after();
    const bool failed = *gave_up || *bad || !s.ok;
    if (*gave_up && threadIdx.x == 0) latch(a.r.err, PGD_ERR_TIMEOUT);

    // -------------------------------------------------------------------- results
    const int64_t out_at = (int64_t)s.row0 * a.hq + (int64_t)head * a.group;  // head vectors
    if (a.cluster == 1) {
        if (warp < 8) {
            const uint32_t to = tmem + (uint32_t(warp % 4 * 32) << 16) + 2 * kTile + blk * D;
            const float inv = failed ? NAN : l > 0.f ? 1.f / l : l == 0.f ? 0.f : NAN;
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
                        w[k] = inv == 0.f ? 0u : inv != inv ? 0x7fc07fc0u : bf16x2(y0, y1);
                    }
                    const int c = (i + e) / 8;
                    *reinterpret_cast<uint4*>(rowp + ((c ^ my_row) & (D / 8 - 1)) * 16) =
                        make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
            __syncwarp();
            constexpr int kVecs = D / 8;
            for (int i = lane; i < 32 * kVecs; i += 32) {
                const int r = warp * 32 + i / kVecs, c = i % kVecs;
                if (r >= rows) continue;
                const uint32_t R = row0 + r;
                const uint4 x = *reinterpret_cast<const uint4*>(
                    smem + r * (D * 2) + ((c ^ r) & (kVecs - 1)) * 16);
                *reinterpret_cast<uint4*>(
                    a.out + (out_at + (int64_t)(R / group) * a.hq + R % group) * D + c * 8) = x;
            }
        }
    } else {
        // unnormalised rows, maxima and sums to shared memory, then every CTA of the
        // cluster joins a share of the rows
        float* const stat = reinterpret_cast<float*>(smem);  // [256][2], and a flag
        if (warp < 8) {
            const uint32_t to = tmem + (uint32_t(warp % 4 * 32) << 16) + 2 * kTile + blk * D;
            const bool have = blk ? sp[1].t1 > sp[1].t0 : sp[0].t1 > sp[0].t0;
            const int r = blk * kBlock + my_row;
            stat[2 * r] = m;
            stat[2 * r + 1] = l;
            if (have) {
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
                            make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                    }
                }
            }
        }
        if (threadIdx.x == 0) reinterpret_cast<int*>(stat)[512] = failed;
        cluster_sync();
        bool any_failed = false;
        for (int k = 0; k < a.cluster; ++k)
            any_failed |= __float_as_int(peer_ld4(peer_addr(base + 2048, k)).x) != 0;
        constexpr int kVecs = D / 4;  // four columns a thread
        for (int i = threadIdx.x + share * kThreads; i < rows * kVecs; i += a.cluster * kThreads) {
            const int r = i / kVecs, c = i % kVecs;
            float top = -INFINITY;
            float2 st[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (k < a.cluster) {
                    const float4 v = peer_ld4(peer_addr(base + r / 2 * 16, k));
                    st[k] = r % 2 ? make_float2(v.z, v.w) : make_float2(v.x, v.y);
                    top = fmaxf(top, st[k].x);
                }
            float o[4] = {0.f, 0.f, 0.f, 0.f}, sum = 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (k < a.cluster && st[k].y != 0.f) {
                    const float w = ex2(st[k].x - top);
                    const float4 v = peer_ld4(peer_addr(
                        base + L::kRing + r * (D * 4) + ((c ^ r) & (kVecs - 1)) * 16, k));
                    sum = fmaf(w, st[k].y, sum);
                    o[0] = fmaf(w, v.x, o[0]);
                    o[1] = fmaf(w, v.y, o[1]);
                    o[2] = fmaf(w, v.z, o[2]);
                    o[3] = fmaf(w, v.w, o[3]);
                }
            const float inv = any_failed ? NAN : sum == 0.f ? 0.f : 1.f / sum;
            const uint32_t R = row0 + r;
            *reinterpret_cast<uint2*>(a.out + (out_at + (int64_t)(R / group) * a.hq + R % group) * D +
                                      c * 4) =
                make_uint2(bf16x2(o[0] * inv, o[1] * inv), bf16x2(o[2] * inv, o[3] * inv));
        }
        cluster_sync();  // shared memory stays until every CTA has read it
    }
    __syncthreads();
    if (warp == 9) tmem_free(tmem, 512);
}

}  // namespace attend
}  // namespace pgd
