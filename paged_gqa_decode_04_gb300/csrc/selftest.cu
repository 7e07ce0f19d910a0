// Diagnostic: exercise the bounded-wait path of the pipeline kernels without
// faulting anything.  One warp initialises an mbarrier that nothing will
// ever arrive on and waits on it with the same helpers the decode and the
// attention kernels use, but with a caller-chosen limit for each; when all of
// them have given up it latches PGD_ERR_TIMEOUT in the pool's error word and
// returns, so the context stays usable and the host reads the status with
// paged_gqa_get_error.
#include "decode_tma.cuh"
#include "umma.cuh"

namespace pgd {
namespace {

__global__ void wait_timeout_kernel(uint64_t limit_ns, int* err) {
    __shared__ __align__(8) uint64_t bar;
    __shared__ int gave_up[3];
    const uint32_t b = tma::smem_u32(&bar);
    if (threadIdx.x == 0) {
        tma::mbar_init(b, 1);
        tma::fence_barrier_init();
        gave_up[0] = gave_up[1] = 0;
        gave_up[2] = 1;  // as if another thread of the CTA had given up
    }
    __syncwarp();
    bool came = false;
    if (threadIdx.x == 0) {
        came |= tma::mbar_wait(b, 0, limit_ns);
        came |= umma::bar_wait(b, 0, &gave_up[0], limit_ns);
        came |= umma::bar_wait(b, 0, &gave_up[2]);
    }
    __syncwarp();
    came |= umma::warp_wait(b, 0, &gave_up[1], limit_ns);
    came |= umma::warp_wait(b, 0, &gave_up[2]);
    came |= !gave_up[0] || !gave_up[1];
    if (!__any_sync(0xffffffffu, came) && threadIdx.x == 0) latch_error(err, PGD_ERR_TIMEOUT);
}

}  // namespace
}  // namespace pgd

extern "C" int paged_gqa_selftest_wait_timeout(pgd_pool_t pool, int64_t limit_us, void* stream) {
    if (!pool || limit_us < 1 || limit_us > 1000000) return PGD_ERR_ARG;
    const pgd::Pool& p = pgd::pool_desc(pool);
    int prev = -1;
    if (cudaGetDevice(&prev) != cudaSuccess) return PGD_ERR_CUDA;
    if (prev != p.device && cudaSetDevice(p.device) != cudaSuccess) return PGD_ERR_CUDA;
    pgd::wait_timeout_kernel<<<1, 32, 0, static_cast<cudaStream_t>(stream)>>>(
        (uint64_t)limit_us * 1000ull, p.err);
    const cudaError_t e = cudaGetLastError();
    if (prev != p.device) cudaSetDevice(prev);
    return e == cudaSuccess ? PGD_OK : PGD_ERR_CUDA;
}
