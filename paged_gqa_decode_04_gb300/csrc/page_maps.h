// Tensor maps of a pool's pages for kernels that fetch one KV head at a time.
#pragma once

#include "pgd_internal.h"

namespace pgd {

// bfloat16 and 8-bit pools as 128-byte rows: coordinates (element of the row, slot, row of
// the token's KV heads, block), box (whole row, min(block_size, 128) slots, 1, 1), in the
// 128-byte swizzle.
struct PageMaps {
    CUtensorMap k, v;
};

const PageMaps& page_maps(pgd_pool_t h);

}  // namespace pgd
