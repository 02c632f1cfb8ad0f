// 8-bit instantiations of the ragged-row GEMM (kGated), in a file of their own so that the
// build compiles the variants in parallel.
#include "grouped_gemm.hpp"

namespace awq {

void launch_grouped8_gated(const GroupedArgs& g, int row_tiles, int k_waves, dim3 grid, hipStream_t stream) {
  launch_grouped_t<kGated, 8>(g, row_tiles, k_waves, grid, stream);
}

}  // namespace awq
