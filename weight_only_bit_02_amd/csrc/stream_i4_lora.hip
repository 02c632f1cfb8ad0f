// 4-bit instantiations of the ragged-row streaming linear (kLora), in a file of their own so
// that the build compiles the variants in parallel.
#include "grouped_stream.hpp"

namespace awq {

void launch_stream4_lora(const GroupedArgs& g, bool narrow, int s, dim3 grid, hipStream_t stream) {
  launch_stream_t<kLora, 4>(g, narrow, s, grid, stream);
}

}  // namespace awq
