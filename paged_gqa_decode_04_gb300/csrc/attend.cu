// paged_gqa_attend, paged_gqa_attend_shaped: attention of a ragged batch of query tokens over
// the pages, causal (prompts, chunks of prompts) or over all cached tokens (cross attention), with
// plain scores or with capped and biased ones and ranges of visible tokens.
// See include/paged_gqa.h for the contract.
//
//     out = sum_t p_t v_t / sum_t p_t,  p_t = exp(scale <q, k_t> - m), m = max_t,
//
// in one pass over the tokens with a running maximum and sum in float32, on the tensor
// cores: attend_tc.cuh.  This file checks the arguments and chooses the launch.
#include "attend_launch.cuh"
#include "page_ops.h"
#include "ragged.cuh"

namespace pgd {
namespace attend {
#define PGD_EXTERN(D, PAGE, PB)                                                              \
    extern template cudaError_t launch_shaped<D, PAGE, PB>(Args&, const Pool&, const PageMaps&, \
                                                           cudaStream_t);
PGD_ATTEND_PAGES(PGD_EXTERN)
#undef PGD_EXTERN

cudaError_t launch_attend(Args& a, const Pool& p, const PageMaps& maps, bool shaped,
                          cudaStream_t s) {
#define PGD_LAUNCH(D, PAGE, PB)                                                              \
    if (p.d == D && p.dtype == PAGE && (p.dtype == PGD_BF16 || (p.scale_per_block != 0) == PB)) \
        return shaped ? launch_shaped<D, PAGE, PB>(a, p, maps, s)                            \
                      : launch<D, PAGE, PB, 0>(a, p, maps, s);
    PGD_ATTEND_PAGES(PGD_LAUNCH)
#undef PGD_LAUNCH
    return cudaErrorInvalidValue;
}
}  // namespace attend
}  // namespace pgd

using namespace pgd;

extern "C" int paged_gqa_attend_shaped(pgd_pool_t pool, const void* q, int64_t q_stride,
                                       int total, int Hq, const int32_t* cu_seqlens, int B,
                                       const int32_t* block_table, int max_blocks,
                                       const int32_t* seq_lens, int causal, int window,
                                       float scale, float softcap, const float* slopes,
                                       const int32_t* visible, void* out, void* stream) {
    const float scale_log2 = fabsf(scale) * 1.4426950408889634f;
    if (!pool || Hq < 1 || window < 0 || (causal != 0 && causal != 1) || !isfinite(scale_log2))
        return PGD_ERR_ARG;
    if (window > 0 && !causal) return PGD_ERR_ARG;
    int rc = check_shaping(softcap, slopes);
    if (rc != PGD_OK) return rc;
    const Pool& p = pool_desc(pool);
    if (Hq % p.hkv != 0) return PGD_ERR_SHAPE;
    if (p.dtype == PGD_F32) return PGD_ERR_UNSUPPORTED;
    rc = check_ragged(p, total, cu_seqlens, B, block_table, max_blocks, seq_lens);
    if (rc != PGD_OK || B == 0 || total == 0) return rc;
    const int64_t width = (int64_t)Hq * p.d;
    rc = check_rows(q, q_stride, width, 2);
    if (rc == PGD_OK) rc = check_rows(out, width, width, 2);
    if (rc != PGD_OK) return rc;
    if (visible && !is_aligned(visible, 8)) return PGD_ERR_ALIGN;
    {
        const char* q0 = static_cast<const char*>(q);
        const char* o0 = static_cast<char*>(out);
        if (q0 < o0 + width * 2 * total && o0 < q0 + (q_stride * (total - 1) + width) * 2)
            return PGD_ERR_ARG;  // out aliases q
    }
    const int cap = max_blocks * p.block_size;
    const int group = Hq / p.hkv;
    // a window that no length exceeds is none; the lower ends of the others, down to
    // 1 - total - window, stay within 31 bits
    if (window >= cap) window = 0;
    if (window > 0 && (int64_t)total + cap > INT32_MAX) return PGD_ERR_SHAPE;
    if ((int64_t)total * group > INT32_MAX / 2) return PGD_ERR_SHAPE;
    const bool shaped = softcap > 0.f || slopes || visible;
    if (shaped && group > attend::kMostGroup) return PGD_ERR_SHAPE;
    const int64_t pieces = max_pieces(total, B, group, attend::kRowShift, 1);
    if (pieces * p.hkv * 8 > INT32_MAX) return PGD_ERR_SHAPE;
    OnDevice dev(p.device);
    if (!dev.ok) return PGD_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    attend::Args t = {};
    t.r = {cu_seqlens, block_table, seq_lens, B, total, max_blocks, p.block_size,
           p.num_blocks, cap, p.err};
    t.hq = Hq;
    t.hkv = p.hkv;
    t.group = group;
    t.q = static_cast<const __nv_bfloat16*>(q);
    t.q_stride = q_stride;
    t.out = static_cast<__nv_bfloat16*>(out);
    t.causal = causal;
    t.window = window;
    // a scale below zero turns the queries' sign, one of zero leaves no query
    t.scale_log2 = scale != 0.f ? scale_log2 : 1.f;
    t.q_and = scale != 0.f ? 0xffffffffu : 0u;
    t.q_xor = scale < 0.f ? 0x80008000u : 0u;
    t.pieces = int(pieces);
    t.k_scale = p.k_scale;
    t.v_scale = p.v_scale;
    attend::set_cap(t, softcap * kLog2e);
    t.slopes = slopes;
    t.visible = reinterpret_cast<const int2*>(visible);
    const cudaError_t e = attend::launch_attend(t, p, page_maps(pool), shaped, s);
    return e == cudaSuccess ? PGD_OK : PGD_ERR_CUDA;
}

extern "C" int paged_gqa_attend(pgd_pool_t pool, const void* q, int64_t q_stride, int total,
                                int Hq, const int32_t* cu_seqlens, int B,
                                const int32_t* block_table, int max_blocks,
                                const int32_t* seq_lens, int causal, int window, float scale,
                                void* out, void* stream) {
    return paged_gqa_attend_shaped(pool, q, q_stride, total, Hq, cu_seqlens, B, block_table,
                                   max_blocks, seq_lens, causal, window, scale, 0.f, nullptr,
                                   nullptr, out, stream);
}
