// Ragged batches over the paged cache: which sequence a packed row or a piece of
// a sequence belongs to, found on the device from cu_seqlens, and the checks a
// sequence has to pass before anything is read or written for it.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "pgd_internal.h"

namespace pgd {

// The tables of a ragged call.  Sequence b owns rows cu[b] .. cu[b+1] - 1 of the
// packed tensors: its last n_b = cu[b+1] - cu[b] cached tokens.
struct Ragged {
    const int32_t* cu;     // [B + 1]
    const int32_t* table;  // [B][max_blocks]
    const int32_t* lens;   // [B]
    int B;
    int total;             // rows of the packed tensors
    int max_blocks;
    int block_size;
    int64_t num_blocks;
    int max_len;           // largest length of a sequence with rows (blocks, rotation table)
    int* err;
};

struct Seq {
    int b;      // sequence
    int row0;   // its first packed row
    int n;      // its rows
    int len;    // its cached tokens
    bool ok;
};

__device__ __forceinline__ void latch(int* err, int status) { atomicCAS(err, 0, status); }

__device__ __forceinline__ Seq load_seq(const Ragged& r, int b) {
    Seq s;
    s.b = b;
    s.row0 = __ldg(r.cu + b);
    const int end = __ldg(r.cu + b + 1);
    s.len = __ldg(r.lens + b);
    s.ok = s.row0 >= 0 && end >= s.row0 && end <= r.total && s.len >= 0 && s.len <= r.max_len;
    s.n = s.ok ? end - s.row0 : 0;
    return s;
}

// Pieces of at most 2^shift units each: sequence b owns the piece numbers
// [first(b), first(b+1)), first(b) = (cu[b] * mul >> shift) + slack * b, which holds
// at least the pieces its cu[b+1] - cu[b] rows of `mul` units can need: one more
// than the difference of the floors when pieces start at the sequence (slack 1),
// two more when they start at multiples of the piece size within it (slack 2).
// One load per probe and no prefix sum; the unused numbers find nothing to do.
__device__ __forceinline__ int64_t first_piece(const Ragged& r, int b, int mul, int shift,
                                               int slack) {
    return ((int64_t)__ldg(r.cu + b) * mul >> shift) + (int64_t)slack * b;
}

__host__ __device__ __forceinline__ int64_t max_pieces(int total, int B, int mul, int shift,
                                                       int slack) {
    return ((int64_t)total * mul >> shift) + (int64_t)slack * B;
}

// The sequence that owns piece `x`: the number of b in [1, B] with first(b) <= x, by a
// warp that probes 32 at a time.  For cu that is not ascending it is some b in [0, B].
__device__ __forceinline__ int find_seq(const Ragged& r, int64_t x, int mul, int shift, int slack) {
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = r.B;  // the answer is in [lo, hi]
    while (hi > lo) {
        const int step = (hi - lo + 31) / 32;
        const int i = lo + step * (lane + 1);
        const bool le = i <= hi && first_piece(r, i, mul, shift, slack) <= x;
        const int c = __popc(__ballot_sync(0xffffffffu, le));
        lo += step * c;
        hi = min(hi, lo + step - 1);
    }
    return lo;
}

// Latch the error of every sequence that fails its checks (one CTA of a launch calls
// this, so that none is missed however cu is laid out).  One without rows asks for no
// position: it may be as long as its blocks.
__device__ __forceinline__ void check_all(const Ragged& r, bool rows_within_len) {
    for (int b = threadIdx.x; b < r.B; b += blockDim.x) {
        const Seq s = load_seq(r, b);
        const int end = __ldg(r.cu + b + 1);
        const bool idle = s.row0 >= 0 && end == s.row0 && end <= r.total && s.len >= 0 &&
                          s.len <= r.max_blocks * r.block_size;
        if ((!s.ok && !idle) || (rows_within_len && s.n > s.len)) latch(r.err, PGD_ERR_SEQ_LEN);
    }
}

// Physical block of logical block i of sequence b, or -1 (error latched) when its id
// is out of range.
__device__ __forceinline__ int64_t block_of(const Ragged& r, int b, int i) {
    const int64_t id = __ldg(r.table + (int64_t)b * r.max_blocks + i);
    if (id >= 0 && id < r.num_blocks) return id;
    latch(r.err, PGD_ERR_BLOCK_ID);
    return -1;
}

}  // namespace pgd
