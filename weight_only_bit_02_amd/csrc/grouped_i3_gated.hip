// 3-bit instantiations of the ragged-row GEMM (kGated), in a file of their own so that the
// build compiles the variants in parallel.
#include "grouped_gemm.hpp"

namespace awq {

void launch_grouped3_gated(const GroupedArgs& g, bool big, dim3 grid, hipStream_t stream) {
  if (big)
    hipLaunchKernelGGL((k_grouped<kGated, 8, 3>), grid, dim3(256), 0, stream, g);
  else
    hipLaunchKernelGGL((k_grouped<kGated, 2, 3>), grid, dim3(256), 0, stream, g);
}

}  // namespace awq
