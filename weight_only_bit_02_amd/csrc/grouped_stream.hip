// Launcher of the ragged-row streaming linear (the kernel is in grouped_stream.hpp).
#include "grouped_stream.hpp"

namespace awq {

#define AWQ_STREAM(B)                                                                                     \
  void launch_stream##B##_plain(const GroupedArgs& g, bool narrow, int s, dim3 grid, hipStream_t stream); \
  void launch_stream##B##_gated(const GroupedArgs& g, bool narrow, int s, dim3 grid, hipStream_t stream); \
  void launch_stream##B##_lora(const GroupedArgs& g, bool narrow, int s, dim3 grid, hipStream_t stream);
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
  // the fewest waves that hold all of K: each item then costs the fewest sums
  const int64_t waves = (g.K / kGroup + kStreamSteps - 1) / kStreamSteps;
  const int s = waves <= 2 ? 2 : waves <= 4 ? 4 : 8;
  const int64_t blocks = kStreamSlots / s;
  auto chunks = [&](bool narrow) -> int64_t {
    const int cols = stream_cols(w_bit, narrow) / (mode == kGated ? 2 : 1);
    return (outs + cols - 1) / cols;
  };
  // items for half the blocks or fewer: narrower ones (4096 x 4096 with adapters, one row: 13.1 us
  // with whole items, 11.2 so; with items for more blocks, 11008 rows of weights, 13.5 and 13.9)
  const bool narrow = w_bit != 8 && mt * chunks(false) * 2 <= blocks;
  g.nt = (int)chunks(narrow);
  const int64_t items = mt * g.nt;
  const dim3 grid((unsigned)(items < blocks ? (items + 7) / 8 * 8 : blocks));  // a multiple of the XCDs
  auto* const f = w_bit == 8   ? (mode == kPlain ? launch_stream8_plain : mode == kGated ? launch_stream8_gated : launch_stream8_lora)
                  : w_bit == 3 ? (mode == kPlain ? launch_stream3_plain : mode == kGated ? launch_stream3_gated : launch_stream3_lora)
                               : (mode == kPlain ? launch_stream4_plain : mode == kGated ? launch_stream4_gated : launch_stream4_lora);
  f(g, narrow, s, grid, stream);
  return hipGetLastError();
}

}  // namespace awq
