// Attention over the 4-bit cache, heads of 128 channels (kv_attend.hpp, kv_attend_tiles.hpp).
#include "kv_attend_tiles.hpp"

namespace awq {

hipError_t attend_stream_128(const KvView& v, const AttendArgs& a, const AttendList& list, hipStream_t stream) {
  switch (v.group) {
    case 128: return attend_stream<128, 1>(v, a, list, stream);
    case 64: return attend_stream<128, 2>(v, a, list, stream);
    case 32: return attend_stream<128, 4>(v, a, list, stream);
  }
  return hipErrorInvalidValue;
}

hipError_t attend_tiles_128(const KvView& v, const AttendArgs& a, const AttendList& list, hipStream_t stream) {
  switch (v.group) {
    case 128: return attend_tiles<128, 1>(v, a, list, stream);
    case 64: return attend_tiles<128, 2>(v, a, list, stream);
    case 32: return attend_tiles<128, 4>(v, a, list, stream);
  }
  return hipErrorInvalidValue;
}

hipError_t attend_join_128(const AttendArgs& a, int tile, hipStream_t stream) {
  hipLaunchKernelGGL(k_attend_join<128>, dim3(a.blocks, tile / kJoinRows), dim3(kJoinThreads), 0, stream, a, tile);
  return hipGetLastError();
}

}  // namespace awq
