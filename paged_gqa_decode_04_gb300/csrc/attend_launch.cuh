// The launch of an attention kernel: its shared memory, its cluster size and its grid.
#pragma once

#include <atomic>

#include "attend_plan.h"
#include "attend_tc.cuh"
#include "page_maps.h"

namespace pgd {
namespace attend {

template <int D, int PAGE, bool PB, int MOD>
cudaError_t launch(Args& a, const Pool& p, const PageMaps& maps, cudaStream_t s) {
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
        cudaError_t e = cudaFuncSetAttribute(attend_kernel<D, PAGE, PB, MOD>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             Layout<D, PAGE, PB>::kBytes);
        if (e != cudaSuccess) return e;
        known = p.num_sms;
        for (int i = 1; i < 4; ++i) {
            int n = 0;
            attr[0].val.clusterDim.x = 1 << i;
            cfg.gridDim = dim3(1 << i);
            cfg.numAttrs = 1;
            e = cudaOccupancyMaxActiveClusters(&n, attend_kernel<D, PAGE, PB, MOD>, &cfg);
            if (e != cudaSuccess) return e;
            known |= uint64_t(n) << (16 * i);
        }
        fits[p.device].store(known);
    }
    auto step = [&](int rows) { return make_int2(rows / a.group, rows % a.group); };
    a.inv_group = 1.f / float(a.group);
    a.q_step = step(kBlock / (D / 8));
    a.o_step = step(32 / (D / 8));
    a.part_step = step(32 / (D / 8));
    auto join_step = [&]() { return step(a.cluster * 8 * (32 / (D / 4))); };
    if (MOD != 0 && a.shared) {  // one more CTA for the starts
        a.cluster = 1;
        a.join_step = join_step();
        cfg.gridDim = dim3(1 + unsigned(a.pieces) * a.hkv * a.splits);
        cfg.numAttrs = 0;
        return cudaLaunchKernelEx(&cfg, attend_kernel<D, PAGE, PB, MOD>, a, maps.k, maps.v);
    }
    int fit[4];
    for (int i = 0; i < 4; ++i) fit[i] = int(known >> (16 * i) & 0xffff);
    const bool few = (int64_t)a.r.total * a.group <= (int64_t)a.pieces * kBlock;
    // us of a key tile of 256 rows (measured at D = 128)
    const double tile = PAGE == PGD_BF16 ? 1.2 : PB ? 1.75 : 1.5;
    a.cluster = choose_cluster(fit, (int64_t)a.pieces * a.hkv,
                               piece_tiles(a.r.max_len, a.window, a.group), few, tile);
    a.join_step = join_step();
    attr[0].val.clusterDim.x = a.cluster;
    cfg.gridDim = dim3(unsigned(a.pieces) * a.hkv * a.cluster);
    cfg.numAttrs = a.cluster > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, attend_kernel<D, PAGE, PB, MOD>, a, maps.k, maps.v);
}

// The kernels with kShaped and what of kCap and kBias is asked for, one page type a file.
template <int D, int PAGE, bool PB>
cudaError_t launch_shaped(Args& a, const Pool& p, const PageMaps& maps, cudaStream_t s) {
    if (a.slopes)
        return a.cap > 0.f ? launch<D, PAGE, PB, kShaped | kCap | kBias>(a, p, maps, s)
                           : launch<D, PAGE, PB, kShaped | kBias>(a, p, maps, s);
    if (a.cap == 0.f) return launch<D, PAGE, PB, kShaped>(a, p, maps, s);
    if constexpr (PAGE == PGD_BF16)
        if (a.cap <= kFixedMost) return launch<D, PAGE, PB, kShaped | kCap | kFixed>(a, p, maps, s);
    return launch<D, PAGE, PB, kShaped | kCap>(a, p, maps, s);
}

// launch or launch_shaped for the pool's pages.
cudaError_t launch_attend(Args& a, const Pool& p, const PageMaps& maps, bool shaped,
                          cudaStream_t s);

#define PGD_ATTEND_PAGES(F)   \
    F(64, PGD_BF16, false)    \
    F(128, PGD_BF16, false)   \
    F(128, PGD_FP8_E4M3, false) \
    F(128, PGD_FP8_E4M3, true)  \
    F(128, PGD_INT8, false)   \
    F(128, PGD_INT8, true)

}  // namespace attend
}  // namespace pgd
