// Launcher of the ragged-row streaming linear (the kernel is in grouped_stream.hpp).
#include "grouped_stream.hpp"

namespace awq {

#define AWQ_STREAM(B)                                                                                     \
  void launch_stream##B##_plain(const GroupedArgs& g, int s, dim3 grid, hipStream_t stream); \
  void launch_stream##B##_gated(const GroupedArgs& g, int s, dim3 grid, hipStream_t stream); \
  void launch_stream##B##_lora(const GroupedArgs& g, int s, dim3 grid, hipStream_t stream);
AWQ_STREAM(3)
AWQ_STREAM(4)
AWQ_STREAM(8)
#undef AWQ_STREAM

// Scales and zeros are read eight bytes at a time.
bool grouped_stream_supported(int64_t weights, int64_t N, int64_t K, int group, int w_bit) {
  const int64_t Gs = K / group, zb = w_bit == 8 ? Gs : (Gs + 1) / 2;
  return weights * N * Gs * 2 >= 8 && weights * N * zb >= 8;
}

hipError_t launch_grouped_stream(GroupedArgs g, int mode, int w_bit, hipStream_t stream) {
  const int64_t outs = mode == kGated ? g.N / 2 : g.N;
  const int64_t parts = mode == kLora ? 1 : g.groups < g.n ? g.groups : g.n;
  const int64_t mt = (g.n + 15 * parts) / 16;  // the most row tiles
  const int cols = stream_cols(w_bit) / (mode == kGated ? 2 : 1);
  g.nt = (int)((outs + cols - 1) / cols);
  // the fewest waves that hold all of K: each item then costs the fewest sums
  const int64_t waves = (g.K / kGroup + kStreamSteps - 1) / kStreamSteps;
  const int s = waves <= 2 ? 2 : waves <= 4 ? 4 : 8;
  const int64_t items = mt * g.nt, blocks = kStreamSlots / s;
  const dim3 grid((unsigned)(items < blocks ? items : blocks));
  auto* const f = w_bit == 8   ? (mode == kPlain ? launch_stream8_plain : mode == kGated ? launch_stream8_gated : launch_stream8_lora)
                  : w_bit == 3 ? (mode == kPlain ? launch_stream3_plain : mode == kGated ? launch_stream3_gated : launch_stream3_lora)
                               : (mode == kPlain ? launch_stream4_plain : mode == kGated ? launch_stream4_gated : launch_stream4_lora);
  f(g, s, grid, stream);
  return hipGetLastError();
}

}  // namespace awq
