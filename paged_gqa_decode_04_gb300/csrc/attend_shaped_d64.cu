// The attention kernels with shaped scores and shared prefixes:
// bfloat16 pages, head_dim 64.
#include "attend_launch.cuh"

namespace pgd {
namespace attend {
template cudaError_t launch_shaped<64, PGD_BF16, false>(Args&, const Pool&, const PageMaps&,
                                                        cudaStream_t);
}  // namespace attend
}  // namespace pgd
