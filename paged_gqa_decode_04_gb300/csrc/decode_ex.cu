// Decode with shaped scores (soft cap, distance bias) or over what lies behind shared
// prefixes: the choice of the instantiation, and the join of partial results.
#include <cuda_bf16.h>

#include "attend_plan.h"
#include "decode_tma.cuh"

namespace pgd {
namespace tma {
#define PGD_EX(...)                                                                            \
    extern template cudaError_t launch_tma_d<__VA_ARGS__>(const DecodeArgs&, const Pool&,      \
                                                          cudaStream_t);
PGD_EX(64, false, 0, false, false, true)
PGD_EX(128, false, 0, false, false, true)
PGD_EX(128, true, 0, false, false, true)
PGD_EX(128, true, 0, false, true, true)
PGD_EX(128, true, 0, true, false, true)
PGD_EX(128, true, 0, true, true, true)
#undef PGD_EX
}  // namespace tma

cudaError_t launch_decode_ex(const DecodeArgs& a, const Pool& p, cudaStream_t s) {
    using tma::launch_tma_d;
    const int idx = a.hg == 1 ? 0 : a.hg == 2 ? 1 : a.hg == 4 ? 2 : 3;
    if (!p.tmap_ok[idx]) return cudaErrorInvalidValue;
    if (p.dtype == PGD_BF16)
        return a.d == 64 ? launch_tma_d<64, false, 0, false, false, true>(a, p, s)
                         : launch_tma_d<128, false, 0, false, false, true>(a, p, s);
    if (p.dtype == PGD_FP8_E4M3)
        return a.scale_per_block ? launch_tma_d<128, true, 0, false, true, true>(a, p, s)
                                 : launch_tma_d<128, true, 0, false, false, true>(a, p, s);
    return a.scale_per_block ? launch_tma_d<128, true, 0, true, true, true>(a, p, s)
                             : launch_tma_d<128, true, 0, true, false, true>(a, p, s);
}

namespace {

constexpr int kJoinThreads = 128;
constexpr int kJoinBatch = 4;  // parts whose loads are on their way together

// One row (sequence, query token, head) by D / 4 threads, four columns each.  Its parts are
// those of the shared prefix and those of the sequence's own run (the row arrays where the
// run was not split, else the pieces' slots, which follow from the spans as in the decode
// kernel):
//     out = sum_k 2^(lse_k - M) o_k / sum_k 2^(lse_k - M),  M = max_k lse_k.
// A part that saw nothing has lse = -infinity, and its o is not used (it may not be written).
template <int D>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(DecodeArgs a) {
    constexpr int kQuads = D / 4;
    const int64_t rows = (int64_t)a.B * a.q_len * a.hq;
    const int64_t row = (int64_t)blockIdx.x * (kJoinThreads / kQuads) + threadIdx.x / kQuads;
    const int col = threadIdx.x % kQuads * 4;
    if (row >= rows) return;
    const int h = int(row % a.hq), token = int(row / a.hq);
    const int b = token / a.q_len, i = token % a.q_len;
    const int L = a.seq_lens[b];
    if (L == 0 || !seq_len_ok(L, a.max_blocks, a.block_size)) return;  // the decode wrote it
    const int kvh = h / a.group, u = kvh / a.hg, hgi = kvh % a.hg;
    const int prefix = a.starts ? attend::prefix_parts(start_of(a.starts, b, L), a.prefix_splits)
                                : 0;
    // the sequence's own run
    const int64_t N = a.tile_base[a.B], P = a.tile_base[a.B + 1];
    const int W = (int)a.tile_base[a.B + 2];
    const int64_t slots = a.tile_base[b + 1] - a.tile_base[b];
    const int n_b = slots ? int(slots / a.units) - W : 0;
    int own = 0;
    int64_t t0 = 0, c0 = 0;
    bool whole = false, dense = false, first_is_tail = false;
    if (n_b > 0) {
        t0 = a.tile_base[b] + (int64_t)u * (n_b + W) + W;
        c0 = span_owner(t0, N, P);
        const int64_t c1 = span_owner(t0 + n_b - 1, N, P);
        whole = c0 == c1;
        if (whole && !a.row_o) return;  // the decode wrote it
        dense = P <= N;
        own = whole ? 1 : dense ? int(c1 - c0 + 1) : n_b;
        first_is_tail = dense && span_begin(c0, N, P) < t0;
    }
    const int piece_rows = a.hg * a.q_len * a.group;
    const int prow = hgi * a.q_len * a.group + i * a.group + h % a.group;
    float M = -INFINITY, sum = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k0 = 0; k0 < prefix + own; k0 += kJoinBatch) {
        float e[kJoinBatch];
        float4 v[kJoinBatch];
#pragma unroll
        for (int j = 0; j < kJoinBatch; ++j) {
            const int k = k0 + j;
            const float* lse = nullptr;
            const float* o = nullptr;
            if (k < prefix) {
                lse = a.pre_lse + (int64_t)k * rows + row;
                o = a.pre_o + ((int64_t)k * rows + row) * D;
            } else if (k < prefix + own) {
                if (whole) {
                    lse = a.row_lse + row;
                    o = a.row_o + row * D;
                } else {
                    const int piece = k - prefix;
                    const int64_t c = dense ? c0 + piece : span_owner(t0 + piece, N, P);
                    const int64_t r =
                        (c * 2 + (first_is_tail && piece == 0 ? 1 : 0)) * piece_rows + prow;
                    lse = a.part_lse + r;
                    o = a.part_o + r * D;
                }
            }
            e[j] = lse ? __ldcg(lse) : -INFINITY;
            v[j] = lse ? __ldcg(reinterpret_cast<const float4*>(o + col))
                       : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int j = 0; j < kJoinBatch; ++j) {
            if (e[j] == -INFINITY) continue;
            const float now = fmaxf(M, e[j]);
            const float keep = fast_exp2(M - now), w = fast_exp2(e[j] - now);
            M = now;
            sum = fmaf(sum, keep, w);
            acc.x = fmaf(acc.x, keep, w * v[j].x);
            acc.y = fmaf(acc.y, keep, w * v[j].y);
            acc.z = fmaf(acc.z, keep, w * v[j].z);
            acc.w = fmaf(acc.w, keep, w * v[j].w);
        }
    }
    const float by = sum > 0.f ? 1.f / sum : 0.f;  // nothing seen: zeros
    const __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x * by, acc.y * by);
    const __nv_bfloat162 hi = __floats2bfloat162_rn(acc.z * by, acc.w * by);
    uint2 y;
    y.x = *reinterpret_cast<const uint32_t*>(&lo);
    y.y = *reinterpret_cast<const uint32_t*>(&hi);
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + row * D + col) = y;
}

}  // namespace

cudaError_t launch_join(const DecodeArgs& a, cudaStream_t s) {
    const int per = kJoinThreads / (a.d / 4);
    const int64_t blocks = ((int64_t)a.B * a.q_len * a.hq + per - 1) / per;
    if (blocks == 0) return cudaSuccess;
    if (a.d == 64)
        join_kernel<64><<<(unsigned)blocks, kJoinThreads, 0, s>>>(a);
    else
        join_kernel<128><<<(unsigned)blocks, kJoinThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace pgd
