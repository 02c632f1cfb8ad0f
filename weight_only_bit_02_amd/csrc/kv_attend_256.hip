// Attention over the 4-bit cache, heads of 256 channels (kv_attend.hpp, kv_attend_tiles.hpp).
#include "kv_attend_tiles.hpp"

namespace awq {

hipError_t attend_stream_256(const KvView& v, const AttendArgs& a, const AttendList& list, hipStream_t stream) {
  switch (v.group) {
    case 128: return attend_stream<256, 2>(v, a, list, stream);
    case 64: return attend_stream<256, 4>(v, a, list, stream);
    case 32: return attend_stream<256, 8>(v, a, list, stream);
  }
  return hipErrorInvalidValue;
}

hipError_t attend_tiles_256(const KvView& v, const AttendArgs& a, const AttendList& list, hipStream_t stream) {
  switch (v.group) {
    case 128: return attend_tiles<256, 2>(v, a, list, stream);
    case 64: return attend_tiles<256, 4>(v, a, list, stream);
    case 32: return attend_tiles<256, 8>(v, a, list, stream);
  }
  return hipErrorInvalidValue;
}

hipError_t attend_join_256(const AttendArgs& a, int tile, hipStream_t stream) {
  hipLaunchKernelGGL(k_attend_join<256>, dim3(a.blocks, tile / kJoinRows), dim3(kJoinThreads), 0, stream, a, tile);
  return hipGetLastError();
}

}  // namespace awq
