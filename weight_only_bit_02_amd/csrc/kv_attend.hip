// Attention over the 4-bit cache: workspace and launches (kernels: kv_attend.hpp, kv_attend_tiles.hpp).
#include "kv_attend_tiles.hpp"

namespace awq {

#define AWQ_DECLARE(D)                                                                                        \
  hipError_t attend_stream_##D(const KvView& v, const AttendArgs& a, const AttendList& list, hipStream_t stream); \
  hipError_t attend_tiles_##D(const KvView& v, const AttendArgs& a, const AttendList& list, hipStream_t stream);  \
  hipError_t attend_join_##D(const AttendArgs& a, int tile, hipStream_t stream);
AWQ_DECLARE(64)
AWQ_DECLARE(128)
AWQ_DECLARE(256)
#undef AWQ_DECLARE

namespace {

constexpr int kFew = 64;
constexpr int kCus = 256;
constexpr int64_t kDirectItems = 512;
size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

// Room for the sums of items that are split, `blocks` or fewer of them.
void part_room(AttendPart& p, int blocks, int dim, size_t& bytes) {
  if (!p.join) return;
  const size_t rows = (size_t)2 * blocks * p.tile;
  p.part = bytes;
  bytes += align256(rows * dim * sizeof(float));
  p.part_ml = bytes;
  bytes += align256(rows * sizeof(float2));
  p.split = bytes;
  bytes += align256(blocks * sizeof(AttendSplit));
}

}  // namespace

AttendPlan attend_plan(int64_t n_rows, int seqs, int max_rows, int64_t max_tokens, int share, int heads, int dim,
                       int group) {
  AttendPlan p{};
  const int64_t chunks = (max_tokens + kAttendChunk - 1) / kAttendChunk;
  const int64_t flat = n_rows * share;
  const bool both = (int64_t)max_rows * share > kFew;
  p.few = both ? kFew : 0x7FFFFFFF;
  // items at most: whole tiles, and the last one of each sequence with rows
  p.stream.tile = (int64_t)max_rows * share <= 16 ? 16 : 32;
  const int64_t some = seqs < n_rows ? seqs : n_rows;
  const int64_t units = heads * (flat / p.stream.tile + some) * chunks;
  const auto blocks = [&](int g) {  // one wave's place on every SIMD takes a block per CU
    const int fill = kCus * stream_waves(dim, g, p.stream.tile);
    return (int)(units < fill ? units : fill);
  };
  p.stream.blocks = blocks(group);
  p.stream.join = chunks > 1;
  part_room(p.stream, blocks(32), dim, p.bytes);  // the most of any group: the workspace does not go by it
  if (both) {
    p.tiles.tile = dim == 256 ? TileShape<256>::kRows : TileShape<128>::kRows;
    const int64_t long_ones = flat / (kFew + 1) < some ? flat / (kFew + 1) : some;
    const int64_t n = heads * (flat / p.tiles.tile + long_ones);
    p.tiles.direct = n >= kDirectItems || chunks == 1;
    p.tiles.join = !p.tiles.direct;
    p.tiles.blocks = p.tiles.direct ? (int)n : kCus;
    part_room(p.tiles, kCus, dim, p.bytes);
  }
  return p;
}

hipError_t launch_attend(const KvView& v, AttendArgs a, const AttendPlan& p, void* workspace, hipStream_t stream) {
  const auto take = [&](const AttendPart& s) {
    char* const w = (char*)workspace;
    a.blocks = s.blocks;
    a.direct = s.direct;
    a.part = s.join ? (float*)(w + s.part) : nullptr;
    a.part_ml = s.join ? (float2*)(w + s.part_ml) : nullptr;
    a.split = s.join ? (AttendSplit*)(w + s.split) : nullptr;
  };
  auto* const streaming = v.dim == 64 ? attend_stream_64 : v.dim == 128 ? attend_stream_128 : attend_stream_256;
  auto* const tiles = v.dim == 64 ? attend_tiles_64 : v.dim == 128 ? attend_tiles_128 : attend_tiles_256;
  auto* const join = v.dim == 64 ? attend_join_64 : v.dim == 128 ? attend_join_128 : attend_join_256;
  hipError_t e = hipSuccess;
  if (p.tiles.tile) {
    take(p.tiles);
    e = tiles(v, a, AttendList{p.tiles.tile, p.few, 0x7FFFFFFF}, stream);
    if (e == hipSuccess && p.tiles.join) e = join(a, p.tiles.tile, stream);
    if (e != hipSuccess) return e;
  }
  take(p.stream);
  e = streaming(v, a, AttendList{p.stream.tile, 0, p.few}, stream);
  if (e == hipSuccess && p.stream.join) e = join(a, p.stream.tile, stream);
  return e;
}

}  // namespace awq
