// Attention over the 4-bit cache, heads of 256 channels (kv_attend.hpp).
#include "kv_attend.hpp"

namespace awq {

hipError_t attend_stream_256(const KvView& v, const AttendArgs& a, int tiles, hipStream_t stream) {
  switch (v.group) {
    case 128: return attend_stream<256, 2>(v, a, tiles, stream);
    case 64: return attend_stream<256, 4>(v, a, tiles, stream);
    case 32: return attend_stream<256, 8>(v, a, tiles, stream);
  }
  return hipErrorInvalidValue;
}

hipError_t attend_join_256(const KvView& v, const AttendArgs& a, int tile, hipStream_t stream) {
  hipLaunchKernelGGL(k_attend_join<256>, dim3((unsigned)(v.n_rows * a.q_heads)), dim3(kAttendWaves * kWave), 0,
                     stream, v, a, tile);
  return hipGetLastError();
}

}  // namespace awq
