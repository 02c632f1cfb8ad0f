// Attention over the 4-bit cache: workspace and launches (kernels: kv_attend.hpp).
#include "kv_attend.hpp"

namespace awq {

#define AWQ_DECLARE(D)                                                                                    \
  hipError_t attend_stream_##D(const KvView& v, const AttendArgs& a, int tiles, hipStream_t stream);      \
  hipError_t attend_join_##D(const KvView& v, const AttendArgs& a, int tile, hipStream_t stream);
AWQ_DECLARE(64)
AWQ_DECLARE(128)
AWQ_DECLARE(256)
#undef AWQ_DECLARE

namespace {
constexpr int kMostBlocks = 1024;  // four blocks a CU
size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }
}  // namespace

AttendPlan attend_plan(int64_t n_rows, int seqs, int max_rows, int64_t max_tokens, int share, int heads, int dim) {
  AttendPlan p{};
  p.tiles = (int64_t)max_rows * share <= 16 ? 1 : 2;
  const int64_t rows = 16 * p.tiles, chunks = (max_tokens + kAttendChunk - 1) / kAttendChunk;
  const int64_t tiles = n_rows * share / rows + (seqs < n_rows ? seqs : n_rows);  // at most
  const int64_t units = heads * tiles * chunks;
  p.blocks = (int)(units < kMostBlocks ? units : kMostBlocks);
  p.join = chunks > 1;
  p.part = 0;
  if (p.join) {
    p.part_ml = align256((size_t)2 * p.blocks * rows * dim * sizeof(float));
    p.bytes = p.part_ml + align256((size_t)2 * p.blocks * rows * sizeof(float2));
  }
  return p;
}

hipError_t launch_attend(const KvView& v, const AttendArgs& a, const AttendPlan& p, hipStream_t stream) {
  auto* const f = v.dim == 64 ? attend_stream_64 : v.dim == 128 ? attend_stream_128 : attend_stream_256;
  const hipError_t e = f(v, a, p.tiles, stream);
  if (e != hipSuccess || !p.join) return e;
  auto* const g = v.dim == 64 ? attend_join_64 : v.dim == 128 ? attend_join_128 : attend_join_256;
  return g(v, a, 16 * p.tiles, stream);
}

}  // namespace awq
