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

constexpr int kCus = 256;

// Rows x share up to which a sequence is streamed: the streaming form widens the codes once per 32
// rows, the tile form once per 256 (D = 256: 128) but takes whole items of one or few blocks. Where
// tiles leave CUs without an item, more rows are streamed (not at D = 256, where it has half the
// waves). 8 heads of keys, D = 128, groups of 128, in us, streamed and tiled:
//   16 sequences of 2000 tokens   8 rows 25, 41; 32: 33, 47; 64: 41, 57; 128: 47, 57; 256: 95, 90
//   32 sequences of 2000 tokens   128: 85, 60
//   64 sequences of 1000 tokens   128: 101, 68
//   1 sequence of 30000 tokens    64: 39, 50; 128: 60, 56
//   16 sequences, D = 256         128: 122, 95
constexpr int kFew = 64, kFewAlone = 128;

// The tile form gives every block one item, or cuts the list of their tokens into equal pieces and
// joins what is cut, some 40 us for the sums (128 KB of a piece). Pieces are taken where items are
// few and their last round leaves CUs idle for longer than that: a tile's 36 tokens take a us at D =
// 64 and 128, half as many at D = 256. 32 heads, D = 128, one item a block and pieces, in us:
//   64 items of 512 tokens    30, 40        64 items of 1024     42, 55      256 of 2048    72, 120
//   64 of 4000               118, 95       128 of 4096          120, 124     256 of 4096   135, 181
//   64 of 16000              420, 191      128 of 8000          219, 180     384 of 9000   495, 458
//   512 of 2048               94, 182     2048 of 2048          385, 471     512 of 9000   552, 585
constexpr int64_t kIdle = 450000;  // tokens x CUs
constexpr int64_t kManyItems = 512;

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
  const int64_t flat = n_rows * share, most = (int64_t)max_rows * share;
  const int64_t some = seqs < n_rows ? seqs : n_rows;
  // items of the tile form, at most: sequences that are not streamed end with a part of a tile
  const int tile = dim == 256 ? TileShape<256>::kRows : TileShape<128>::kRows;
  const auto items = [&](int few) {
    const int64_t long_ones = flat / (few + 1) < some ? flat / (few + 1) : some;
    return heads * ((flat + long_ones * (tile - 1)) / tile);
  };
  const int few = dim < 256 && items(kFew) < kCus ? kFewAlone : kFew;
  // One sequence with many rows is tiled without a look at how many it has: the streaming form finds
  // nothing to do in 10 us (a prompt of 4096 tokens, 32 heads: 165 us with it, 155 without).
  const bool many = most > few, stream = !many || seqs > 1;
  p.few = !many ? 0x7FFFFFFF : stream ? few : 0;
  const int streamed = most <= 16 ? 16 : 32;  // rows of its tile
  if (stream) {
    const int64_t units = heads * (flat / streamed + some) * chunks;
    const auto blocks = [&](int g) {  // one wave's place on every SIMD takes a block per CU
      const int fill = kCus * stream_waves(dim, g, streamed);
      return (int)(units < fill ? units : fill);
    };
    p.stream.tile = streamed;
    p.stream.blocks = blocks(group);
    p.stream.join = chunks > 1;
    part_room(p.stream, blocks(32), dim, p.bytes);  // the most of any group: the workspace does not go by it
  }
  if (many) {
    p.tiles.tile = tile;
    const int64_t n = items(few), idle = (kCus - n % kCus) % kCus;
    const int64_t tokens = max_tokens * (dim == 256 ? 2 : 1);
    p.tiles.direct = n >= kManyItems || chunks == 1 || idle * tokens < kIdle;
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
  }
  if (e == hipSuccess && p.stream.tile) {
    take(p.stream);
    e = streaming(v, a, AttendList{p.stream.tile, 0, p.few}, stream);
    if (e == hipSuccess && p.stream.join) e = join(a, p.stream.tile, stream);
  }
  return e;
}

}  // namespace awq
