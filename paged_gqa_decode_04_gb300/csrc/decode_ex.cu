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

// The sum of weighted parts so far: acc = sum_k 2^(lse_k - M) o_k, sum = sum_k 2^(lse_k - M).
struct Joined {
    float M, sum;
    float4 acc;
    __device__ __forceinline__ void add(float lse, float w0, float4 o) {
        if (lse == -INFINITY) return;  // saw nothing; its o may not have been written
        const float now = fmaxf(M, lse);
        const float keep = fast_exp2(M - now), w = fast_exp2(lse - now);
        M = now;
        sum = fmaf(sum, keep, w * w0);
        acc.x = fmaf(acc.x, keep, w * o.x);
        acc.y = fmaf(acc.y, keep, w * o.y);
        acc.z = fmaf(acc.z, keep, w * o.z);
        acc.w = fmaf(acc.w, keep, w * o.w);
    }
};

// One row (sequence, query token, head) by D / 4 threads, four columns each, or by PHASES times
// as many that take every PHASES-th part.  Its parts are those of the shared prefix and those of
// the sequence's own run (the row arrays where the run was not split, else the pieces' slots,
// which follow from the spans as in the decode kernel):
//     out = sum_k 2^(lse_k - M) o_k / sum_k 2^(lse_k - M),  M = max_k lse_k.
// A round of loads costs their way to memory and back, about 1 us, whatever their number.
template <int D, int PHASES>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(DecodeArgs a) {
    constexpr int kQuads = D / 4, kRows = kJoinThreads / (kQuads * PHASES);
    const int64_t rows = (int64_t)a.B * a.q_len * a.hq;
    const int phase = threadIdx.x / kQuads % PHASES, mine = threadIdx.x / (kQuads * PHASES);
    const int64_t row = (int64_t)blockIdx.x * kRows + mine;
    const int col = threadIdx.x % kQuads * 4;
    Joined s = {-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
    bool write = false;
    if (row < rows) {
        const int h = int(row % a.hq), token = int(row / a.hq);
        const int b = token / a.q_len, i = token % a.q_len;
        const int L = a.seq_lens[b];
        const int kvh = h / a.group, u = kvh / a.hg, hgi = kvh % a.hg;
        const int prefix =
            a.starts ? attend::prefix_parts(start_of(a.starts, b, L), a.prefix_splits) : 0;
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
            dense = P <= N;
            own = whole ? 1 : dense ? int(c1 - c0 + 1) : n_b;
            first_is_tail = dense && span_begin(c0, N, P) < t0;
        }
        // sequences without tokens or of an impossible length, and runs that were not split
        // where there are no row arrays, were written by the decode
        write = L != 0 && seq_len_ok(L, a.max_blocks, a.block_size) && !(whole && !a.row_o);
        const int piece_rows = a.hg * a.q_len * a.group;
        const int prow = hgi * a.q_len * a.group + i * a.group + h % a.group;
        const int parts = write ? prefix + own : 0;
        for (int k0 = phase; k0 < parts; k0 += kJoinBatch * PHASES) {
            float e[kJoinBatch];
            float4 v[kJoinBatch];
#pragma unroll
            for (int j = 0; j < kJoinBatch; ++j) {
                const int k = k0 + j * PHASES;
                const float* lse = nullptr;
                const float* o = nullptr;
                if (k < prefix) {
                    lse = a.pre_lse + (int64_t)k * rows + row;
                    o = a.pre_o + ((int64_t)k * rows + row) * D;
                } else if (k < parts) {
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
            for (int j = 0; j < kJoinBatch; ++j) s.add(e[j], 1.f, v[j]);
        }
    }
    if constexpr (PHASES > 1) {
        __shared__ Joined of_phase[kJoinThreads];
        of_phase[threadIdx.x] = s;
        __syncthreads();
        if (phase) return;
#pragma unroll
        for (int p = 1; p < PHASES; ++p) {
            const Joined t = of_phase[threadIdx.x + p * kQuads];
            s.add(t.M, t.sum, t.acc);
        }
    }
    if (!write) return;
    const float by = s.sum > 0.f ? 1.f / s.sum : s.sum == 0.f ? 0.f : NAN;  // nothing seen: zeros
    const __nv_bfloat162 lo = __floats2bfloat162_rn(s.acc.x * by, s.acc.y * by);
    const __nv_bfloat162 hi = __floats2bfloat162_rn(s.acc.z * by, s.acc.w * by);
    uint2 y;
    y.x = *reinterpret_cast<const uint32_t*>(&lo);
    y.y = *reinterpret_cast<const uint32_t*>(&hi);
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + row * D + col) = y;
}

template <int D, int PHASES>
cudaError_t launch_join_d(const DecodeArgs& a, cudaStream_t s) {
    constexpr int kRows = kJoinThreads / (D / 4 * PHASES);
    const int64_t blocks = ((int64_t)a.B * a.q_len * a.hq + kRows - 1) / kRows;
    join_kernel<D, PHASES><<<(unsigned)blocks, kJoinThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_join(const DecodeArgs& a, cudaStream_t s) {
    if (a.B == 0) return cudaSuccess;
    // More than two rounds of loads a row and few rows: its parts to four times the threads.  It
    // turns between 1280 and 1536 rows (us of a whole call in a graph, one and four times the
    // threads: behind 8192 tokens, 20 query heads of one KV head, 160 rows 50 and 46, 960 57 and
    // 52, 1280 54 and 50, 2560 54 and 56; 32/8 heads behind 16384, 1024 rows 67 and 63, 1536 69
    // both; a capped step of one sequence of 32768, 32 rows, 75 and 48).
    const int pieces = a.num_parts / (a.B * a.units) + 1;
    const bool many = (a.starts ? a.prefix_splits : 0) + pieces > 2 * kJoinBatch &&
                      (int64_t)a.B * a.q_len * a.hq <= 1024;
    if (a.d == 64) return many ? launch_join_d<64, 4>(a, s) : launch_join_d<64, 1>(a, s);
    return many ? launch_join_d<128, 4>(a, s) : launch_join_d<128, 1>(a, s);
}

}  // namespace pgd
