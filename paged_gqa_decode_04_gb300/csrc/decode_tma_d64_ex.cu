// The TMA decode kernel for head_dim 64,
// with shaped scores (softcap, distance bias), sequences walked from a start and results
// left for a join.
#include "decode_tma.cuh"

namespace pgd {
namespace tma {
template cudaError_t launch_tma_d<64, false, 0, false, false, true>(const DecodeArgs&, const Pool&,
                                                                    cudaStream_t);
}  // namespace tma
}  // namespace pgd
