// The TMA decode kernel for e4m3 pages with a scale per KV head,
// with shaped scores (softcap, distance bias), sequences walked from a start and results
// left for a join.
#include "decode_tma.cuh"

namespace pgd {
namespace tma {
template cudaError_t launch_tma_d<128, true, 0, false, false, true>(const DecodeArgs&, const Pool&,
                                                                    cudaStream_t);
}  // namespace tma
}  // namespace pgd
