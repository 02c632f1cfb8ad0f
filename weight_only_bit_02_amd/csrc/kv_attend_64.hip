// Attention over the 4-bit cache, heads of 64 channels (kv_attend.hpp).
#include "kv_attend.hpp"

namespace awq {

hipError_t attend_stream_64(const KvView& v, const AttendArgs& a, int tiles, hipStream_t stream) {
  switch (v.group) {
    case 64: return attend_stream<64, 1>(v, a, tiles, stream);
    case 32: return attend_stream<64, 2>(v, a, tiles, stream);
  }
  return hipErrorInvalidValue;
}

hipError_t attend_join_64(const KvView& v, const AttendArgs& a, int tile, hipStream_t stream) {
  hipLaunchKernelGGL(k_attend_join<64>, dim3((unsigned)(v.n_rows * a.q_heads)), dim3(kAttendWaves * kWave), 0,
                     stream, v, a, tile);
  return hipGetLastError();
}

}  // namespace awq
