// Launcher of the ragged-row GEMM (the kernel is in grouped_gemm.hpp).
#include "awq.h"
#include "grouped_gemm.hpp"

namespace awq {

#define AWQ_GROUPED(B)\
  void launch_grouped##B##_plain(const GroupedArgs& g, int row_tiles, int k_waves, dim3 grid, hipStream_t stream); \
  void launch_grouped##B##_gated(const GroupedArgs& g, int row_tiles, int k_waves, dim3 grid, hipStream_t stream); \
  void launch_grouped##B##_lora(const GroupedArgs& g, int row_tiles, int k_waves, dim3 grid, hipStream_t stream);
AWQ_GROUPED(3)
AWQ_GROUPED(4)
AWQ_GROUPED(8)
#undef AWQ_GROUPED

namespace {

// Row tiles of 32 in a tile and waves along K.
struct Shape {
  int row_tiles, k_waves;
};
Shape shape_of(int kernel, int w_bit) {
  const bool narrow = w_bit == 8;  // LDS holds fewer rows
  switch (kernel) {
    case AWQ_GROUPED_GEMM64K: return {narrow ? 1 : 2, 4};
    case AWQ_GROUPED_GEMM64: return {2, 1};
    case AWQ_GROUPED_GEMM128: return {4, 1};
    default: return {narrow ? 4 : 8, 1};
  }
}
int columns_of(int mode, int k_waves) { return kGN / k_waves / (mode == kGated ? 2 : 1); }

}  // namespace

// The tile shape that a batch of n rows in `groups` groups should take the least time with.
// Microseconds of a K step measured on full and half-full chips at 4-bit codes, by the rows
// that a block multiplies, and of the rest of a tile (launch, first loads, stores); blocks run
// 256 at a time. The groups' sizes are not known here: a quarter more rows than the mean in the
// largest tiles and half a tile lost per group. What the rule picks between, in us (GEMM64,
// 128, 256, 64K; the first two lines experts by mean rows per group, the others adapters):
//   8 x 4096 x 4096    64: 47 59 61 54     96: 51 61 62 69    512: 236 199 218 285
//   64 x 4096 x 1024   64: 116 96 94 187   96: 146 107 104 259 512: 631 465 402 1107
//   4096 x 4096 rows   65: 54 70 73 24   1024: 60 72 138 84  4096: 219 172 177 302
//   11008 x 4096 rows 192: 54 73 130 61   512: 104 75 139 115
int choose_grouped_gemm(const GroupedArgs& g, int mode, int w_bit) {
  const int kernels[] = {AWQ_GROUPED_GEMM128, AWQ_GROUPED_GEMM64, AWQ_GROUPED_GEMM256, AWQ_GROUPED_GEMM64K};
  const double outs = (double)(mode == kGated ? g.N / 2 : g.N);
  const int parts = g.groups < g.n ? g.groups : g.n;
  const double mean = mode == kLora ? g.n : (double)g.n / parts;
  int best = kernels[0];
  double least = 1e30;
  for (const int k : kernels) {
    const Shape s = shape_of(k, w_bit);
    if (k == AWQ_GROUPED_GEMM256 && s.row_tiles < 8) continue;
    const double bm = 32 * s.row_tiles, cols = columns_of(mode, s.k_waves);
    const double tiles = mode == kLora ? __builtin_ceil(mean / bm)
                                       : parts * (mean / bm + 0.5 > 1 ? mean / bm + 0.5 : 1);
    double rounds = tiles * __builtin_ceil(outs / cols) / 256;
    rounds = mode == kLora ? __builtin_ceil(rounds) : rounds <= 1 ? 1 : rounds + 0.25;
    const double rows = 1.25 * mean < bm ? 1.25 * mean : bm;  // that a tile multiplies
    const double step = s.k_waves > 1 ? (rows <= 32 ? 1.3 : 1.9)
                        : rows <= 32  ? 1.05
                        : rows <= 64  ? 1.3
                        : rows <= 128 ? 1.85
                                      : 2.8;
    const double steps = __builtin_ceil((double)g.K / kGK / s.k_waves);
    const double rest = 3 + (mode == kLora && s.k_waves == 1 ? 0.1 * rows : 1);
    const double t = rounds * (step * steps + rest);
    if (t < least) {
      least = t;
      best = k;
    }
  }
  return best;
}

hipError_t launch_grouped_gemm(GroupedArgs g, int mode, int w_bit, int kernel, hipStream_t stream) {
  const Shape shape = shape_of(kernel, w_bit);
  const int64_t bm = 32 * shape.row_tiles;
  const int64_t outs = mode == kGated ? g.N / 2 : g.N, cols = columns_of(mode, shape.k_waves);
  // the most row tiles the groups can need: each may leave one partly filled
  const int64_t parts = mode == kLora ? 1 : g.groups < g.n ? g.groups : g.n;
  const int64_t mt = (g.n + (bm - 1) * parts) / bm;
  g.nt = (int)((outs + cols - 1) / cols);
  const int64_t blocks = (mt * g.nt + 7) / 8 * 8;
  if (blocks >= (int64_t)1 << 24) return hipErrorInvalidValue;
  const dim3 grid((unsigned)blocks);
  auto* const f = w_bit == 8   ? (mode == kPlain ? launch_grouped8_plain : mode == kGated ? launch_grouped8_gated : launch_grouped8_lora)
                  : w_bit == 3 ? (mode == kPlain ? launch_grouped3_plain : mode == kGated ? launch_grouped3_gated : launch_grouped3_lora)
                               : (mode == kPlain ? launch_grouped4_plain : mode == kGated ? launch_grouped4_gated : launch_grouped4_lora);
  f(g, shape.row_tiles, shape.k_waves, grid, stream);
  return hipGetLastError();
}

}  // namespace awq
