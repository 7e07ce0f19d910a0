// The attention kernels with shaped scores and shared prefixes:
// e4m3 pages with a scale per KV head.
#include "attend_launch.cuh"

namespace pgd {
namespace attend {
template cudaError_t launch_shaped<128, PGD_FP8_E4M3, false>(Args&, const Pool&, const PageMaps&,
                                                             cudaStream_t);
}  // namespace attend
}  // namespace pgd
