// The attention kernels with shaped scores and shared prefixes:
// int8 pages with a scale per block.
#include "attend_launch.cuh"

namespace pgd {
namespace attend {
template cudaError_t launch_shaped<128, PGD_INT8, true>(Args&, const Pool&, const PageMaps&,
                                                        cudaStream_t);
}  // namespace attend
}  // namespace pgd
