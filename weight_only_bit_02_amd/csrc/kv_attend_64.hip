// Attention over the 4-bit cache, heads of 64 channels (kv_attend.hpp, kv_attend_tiles.hpp).
#include "kv_attend_tiles.hpp"

namespace awq {

hipError_t attend_stream_64(const KvView& v, const AttendArgs& a, const AttendList& list, hipStream_t stream) {
  switch (v.group) {
    case 64: return attend_stream<64, 1>(v, a, list, stream);
    case 32: return attend_stream<64, 2>(v, a, list, stream);
  }
  return hipErrorInvalidValue;
}

hipError_t attend_tiles_64(const KvView& v, const AttendArgs& a, const AttendList& list, hipStream_t stream) {
  switch (v.group) {
    case 64: return attend_tiles<64, 1>(v, a, list, stream);
    case 32: return attend_tiles<64, 2>(v, a, list, stream);
  }
  return hipErrorInvalidValue;
}

hipError_t attend_join_64(const AttendArgs& a, int tile, hipStream_t stream) {
  hipLaunchKernelGGL(k_attend_join<64>, dim3(a.blocks, tile / kJoinRows), dim3(kJoinThreads), 0, stream, a, tile);
  return hipGetLastError();
}

}  // namespace awq
