// Launcher of the ragged-row GEMM (the kernel is in grouped_gemm.hpp).
#include "grouped_gemm.hpp"

namespace awq {

#define AWQ_GROUPED(B)                                                                        \
  void launch_grouped##B##_plain(const GroupedArgs& g, bool big, dim3 grid, hipStream_t stream); \
  void launch_grouped##B##_gated(const GroupedArgs& g, bool big, dim3 grid, hipStream_t stream); \
  void launch_grouped##B##_lora(const GroupedArgs& g, bool big, dim3 grid, hipStream_t stream);
AWQ_GROUPED(3)
AWQ_GROUPED(4)
AWQ_GROUPED(8)
#undef AWQ_GROUPED

hipError_t launch_grouped_gemm(GroupedArgs g, int mode, int w_bit, bool big, hipStream_t stream) {
  const int64_t bm = !big ? 64 : w_bit == 8 ? 128 : 256;
  const int64_t outs = mode == kGated ? g.N / 2 : g.N, cols = mode == kGated ? kGN / 2 : kGN;
  // the most row tiles the groups can need: each may leave one partly filled
  const int64_t parts = mode == kLora ? 1 : g.groups < g.n ? g.groups : g.n;
  const int64_t mt = (g.n + (bm - 1) * parts) / bm;
  g.nt = (int)((outs + cols - 1) / cols);
  const int64_t blocks = (mt * g.nt + 7) / 8 * 8;
  if (blocks > 0x7FFFFFFF) return hipErrorInvalidValue;
  const dim3 grid((unsigned)blocks);
  auto* const f = w_bit == 8   ? (mode == kPlain ? launch_grouped8_plain : mode == kGated ? launch_grouped8_gated : launch_grouped8_lora)
                  : w_bit == 3 ? (mode == kPlain ? launch_grouped3_plain : mode == kGated ? launch_grouped3_gated : launch_grouped3_lora)
                               : (mode == kPlain ? launch_grouped4_plain : mode == kGated ? launch_grouped4_gated : launch_grouped4_lora);
  f(g, big, grid, stream);
  return hipGetLastError();
}

}  // namespace awq
