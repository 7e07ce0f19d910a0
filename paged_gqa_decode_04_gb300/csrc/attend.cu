// paged_gqa_attend: attention of a ragged batch of query tokens over the pages,
// causal (prompts, chunks of prompts) or over all cached tokens (cross attention).
// See include/paged_gqa.h for the contract.
//
//     out = sum_t p_t v_t / sum_t p_t,  p_t = exp(scale <q, k_t> - m), m = max_t,
//
// in one pass over the tokens with a running maximum and sum in float32, on the tensor
// cores: attend_tc.cuh.  This file checks the arguments and chooses the launch.
#include <atomic>

#include "attend_plan.h"
#include "attend_tc.cuh"
#include "page_maps.h"
#include "page_ops.h"
#include "ragged.cuh"

namespace pgd {
namespace {

template <int D, int PAGE, bool PB>
cudaError_t launch(attend::Args& a, const Pool& p, const PageMaps& maps, cudaStream_t s) {
    using namespace attend;
    constexpr int kDevices = 64;
    static std::atomic<uint64_t> fits[kDevices];  // 16 bits a cluster size, 0: not asked yet
    if (p.device < 0 || p.device >= kDevices) return cudaErrorInvalidDevice;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Layout<D, PAGE, PB>::kBytes;
    cfg.stream = s;
    cfg.attrs = attr;
    uint64_t known = fits[p.device].load();
    if (!known) {
        cudaError_t e = cudaFuncSetAttribute(attend_kernel<D, PAGE, PB>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             Layout<D, PAGE, PB>::kBytes);
        if (e != cudaSuccess) return e;
        known = p.num_sms;
        for (int i = 1; i < 4; ++i) {
            int n = 0;
            attr[0].val.clusterDim.x = 1 << i;
            cfg.gridDim = dim3(1 << i);
            cfg.numAttrs = 1;
            e = cudaOccupancyMaxActiveClusters(&n, attend_kernel<D, PAGE, PB>, &cfg);
            if (e != cudaSuccess) return e;
            known |= uint64_t(n) << (16 * i);
        }
        fits[p.device].store(known);
    }
    int fit[4];
    for (int i = 0; i < 4; ++i) fit[i] = int(known >> (16 * i) & 0xffff);
    const bool few = (int64_t)a.r.total * a.group <= (int64_t)a.pieces * kBlock;
    // us of a key tile of 256 rows (measured at D = 128)
    const double tile = PAGE == PGD_BF16 ? 1.2 : PB ? 1.75 : 1.5;
    a.cluster = choose_cluster(fit, (int64_t)a.pieces * a.hkv,
                               piece_tiles(a.r.max_len, a.window, a.group), few, tile);
    attr[0].val.clusterDim.x = a.cluster;
    cfg.gridDim = dim3(unsigned(a.pieces) * a.hkv * a.cluster);
    cfg.numAttrs = a.cluster > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, attend_kernel<D, PAGE, PB>, a, maps.k, maps.v);
}

}  // namespace
}  // namespace pgd

using namespace pgd;

extern "C" int paged_gqa_attend(pgd_pool_t pool, const void* q, int64_t q_stride, int total,
                                int Hq, const int32_t* cu_seqlens, int B,
                                const int32_t* block_table, int max_blocks,
                                const int32_t* seq_lens, int causal, int window, float scale,
                                void* out, void* stream) {
    const float scale_log2 = fabsf(scale) * 1.4426950408889634f;
    if (!pool || Hq < 1 || window < 0 || (causal != 0 && causal != 1) || !isfinite(scale_log2))
        return PGD_ERR_ARG;
    if (window > 0 && !causal) return PGD_ERR_ARG;
    const Pool& p = pool_desc(pool);
    if (Hq % p.hkv != 0) return PGD_ERR_SHAPE;
    if (p.dtype == PGD_F32) return PGD_ERR_UNSUPPORTED;
    int rc = check_ragged(p, total, cu_seqlens, B, block_table, max_blocks, seq_lens);
    if (rc != PGD_OK || B == 0 || total == 0) return rc;
    const int64_t width = (int64_t)Hq * p.d;
    rc = check_rows(q, q_stride, width, 2);
    if (rc == PGD_OK) rc = check_rows(out, width, width, 2);
    if (rc != PGD_OK) return rc;
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
    const PageMaps& maps = page_maps(pool);
    cudaError_t e;
    if (p.dtype == PGD_BF16)
        e = p.d == 64 ? launch<64, PGD_BF16, false>(t, p, maps, s)
                      : launch<128, PGD_BF16, false>(t, p, maps, s);
    else if (p.dtype == PGD_FP8_E4M3)
        e = p.scale_per_block ? launch<128, PGD_FP8_E4M3, true>(t, p, maps, s)
                              : launch<128, PGD_FP8_E4M3, false>(t, p, maps, s);
    else
        e = p.scale_per_block ? launch<128, PGD_INT8, true>(t, p, maps, s)
                              : launch<128, PGD_INT8, false>(t, p, maps, s);
    return e == cudaSuccess ? PGD_OK : PGD_ERR_CUDA;
}
