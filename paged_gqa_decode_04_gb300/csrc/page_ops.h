// Internal declarations of the ragged page operators (write, read, norm and
// rotation, attention of many query tokens).
#pragma once

#include "pgd_internal.h"

namespace pgd {

// Make `dev` current for the scope of a call; restore the caller's device.
struct OnDevice {
    int prev = -1;
    bool ok = true, changed = false;
    explicit OnDevice(int dev) {
        ok = cudaGetDevice(&prev) == cudaSuccess;
        if (ok && prev != dev) {
            ok = cudaSetDevice(dev) == cudaSuccess;
            changed = ok;
        }
    }
    ~OnDevice() {
        if (changed) cudaSetDevice(prev);
    }
};

inline bool is_aligned(const void* p, uintptr_t a) {
    return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

inline bool is_q8(int dtype) { return dtype == PGD_FP8_E4M3 || dtype == PGD_INT8; }

// Bytes of an element of activations (q, k, v rows, out) for a pool.
inline int act_bytes(const Pool& p) { return p.dtype == PGD_F32 ? 4 : 2; }

// The checks of the tables that every ragged entry point shares.  PGD_OK, or the
// status to return.
inline int check_ragged(const Pool& p, int total, const int32_t* cu, int B, const int32_t* table,
                        int max_blocks, const int32_t* lens) {
    if (total < 0 || B < 0 || max_blocks < 0) return PGD_ERR_ARG;
    // token positions plus a tile stay within 31 bits
    if ((int64_t)max_blocks * p.block_size > INT32_MAX - 1024) return PGD_ERR_SHAPE;
    if (B == 0 || total == 0) return PGD_OK;
    if (!cu || !table || !lens) return PGD_ERR_ARG;
    if (max_blocks < 1) return PGD_ERR_SHAPE;
    if (!is_aligned(cu, 4) || !is_aligned(table, 4) || !is_aligned(lens, 4)) return PGD_ERR_ALIGN;
    return PGD_OK;
}

constexpr float kLog2e = 1.4426950408889634f;

// The soft cap and the slopes of a call with shaped scores.  The cap and its inverse stay far
// inside float32's range.
inline int check_shaping(float softcap, const float* slopes) {
    if (softcap != 0.f && !(softcap >= 0x1p-64f && softcap <= 0x1p64f)) return PGD_ERR_ARG;
    return is_aligned(slopes, 4) ? PGD_OK : PGD_ERR_ALIGN;
}

// A packed tensor of rows of `width` elements, `stride` elements apart.
inline int check_rows(const void* p, int64_t stride, int64_t width, int elt) {
    if (!p) return PGD_ERR_ARG;
    if (stride < width) return PGD_ERR_SHAPE;
    if (!is_aligned(p, 16) || stride * elt % 16 != 0) return PGD_ERR_ALIGN;
    return PGD_OK;
}

}  // namespace pgd
