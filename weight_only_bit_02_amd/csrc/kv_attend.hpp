// Attention over the 4-bit cache, streaming form: few query rows per sequence and head of keys
// (decoding, drafted tokens), any number in principle.
//
//   o[r] = sum_t softmax_t(scale q[r] . k[t]) v[t]   over the tokens t that row r sees
//
// One pass over the tokens with a running maximum and sum. Rows are (token, query head) pairs of
// one head of keys, 16 to a tile: a lane (h, c) = (lane / 16, lane % 16) keeps row c. With keys as
// the first operand, S = K Q^T leaves a lane the scores of its row's tokens 4 h + i of every 16,
// which is the second operand that O^T = V^T P^T wants if its tokens are taken in that order: the
// probabilities never leave the lane, and the cache holds the values in that order.
//
// The work is the list of (sequence, tile of rows, head of keys, 256 tokens), cut into one equal
// piece per block whatever the sequences' lengths, which only the device knows. A block that holds
// the whole of a (sequence, tile, head) writes its output; pieces of one leave their unnormalised
// sums, which k_attend_join adds in the order of the blocks.
//
// A wave takes every fourth 32 tokens of its block's piece. Their codes and parameters come by DMA
// into one of the wave's own two LDS buffers while the other is worked on: no wave waits for another,
// and no register holds what is under way. Waves take turns at priority (left alone, the oldest one
// wins, and the blocks of a CU end one after the other).
//
// Measured. 24 sequences of 300-4000 tokens, 32 heads, D = 128, groups of 128 (241 MB): 62 us and 5 for
// the join, 3.9 TB/s; one sequence of 131071 tokens, 8 heads of keys (138 MB): 37 and 7, 3.7 TB/s; 64
// sequences, 8 heads of keys, groups of 32 (345 MB): 94 and 6, 3.7 TB/s. Bound by loads (alone 52 us
// in the first case, 4.6 TB/s) and vector instructions (alone 56) that overlap in part only; matrix
// cores are busy for 13% of the time. Short calls are chains of loads: the work list's, the
// page's, the codes', 8 us for one sequence of 77 tokens.
#pragma once

#include "groups.hpp"
#include "kv_cache.hpp"

#include <type_traits>

namespace awq {

#define AWQ_INLINE __attribute__((always_inline))
constexpr int kAttendWaves = 4;
constexpr int kAttendChunk = 256;  // tokens of the work list's unit, a multiple of every kernel's step
constexpr float kLazy = 8.0f;  // the running maximum is renewed when a score passes it by 2^8
// Probabilities go to the second product times 2^7: up to 2^15 (kLazy) they fit fp16, and its smallest
// number, 2^-24, is 2^-31 of the largest probability, not 2^-24. A first token of value zero, 18 nats above 8000
// others: off by 8e-3 (hi + lo) and 3e-2 (one fp16) without the 2^7, by 2e-4 with it, as the output's rounding alone.
constexpr float kLift = 7.0f, kDrop = 0x1p-7f;
// Folded (k_attend_stream), a probability takes the value's scale along, 2^-14 to 2^13, so that the maximum
// that runs is that of their products, for each row and group: the largest one that the row met lies between 2^6
// and 2^15. (One power of two for all rows of a wave, above every scale that it loaded: values 2^25 below others that
// the row does not see were off by 2e-2.)
constexpr float kRoom = 15.0f, kLeastScale = 0x1p-14f;
// A score times the softmax's scale minus the maximum is one instruction, but the maximum was rounded:
// scores from 2^24 on differ from it by more than a unit of log2, from 2^27 on by so much that probabilities are
// infinite in fp16 or all zero. Rows whose maximum passes this have it taken off first (attend_far).
constexpr float kFar = 0x1p22f;

constexpr int kJoinThreads = 256;
constexpr int kJoinRows = 4;  // of a join block, at most

typedef _Float16 half4a __attribute__((ext_vector_type(4)));

// The work list of a kernel: units of kAttendChunk tokens of (sequence, tile of rows, head of
// keys), of the sequences with more than `over` and at most `upto` rows x share.
struct AttendList {
  int tile;  // rows of a tile
  int over, upto;
};

struct AttendSeq {
  KvSeq q;
  int flat;   // rows x share
  int tiles;  // 0: not of this list
  int first;  // first token looked at, a multiple of 64
  int units;
};

// The last token that a row at position p may see, `last` the sequence's: none (-1 or less) for a row before
// position 0, which is no token.
__device__ __forceinline__ int attend_last(const AttendArgs& a, int p, int last) {
  return p < last && (a.causal || p < 0) ? p : last;
}

// Chunks of tile j of a sequence: as far as its last row sees, one for rows without a token.
__device__ __forceinline__ int attend_chunks(const AttendArgs& a, const AttendList& g, const AttendSeq& w, int j) {
  const int end = (j + 1) * g.tile < w.flat ? (j + 1) * g.tile : w.flat;
  const int p = w.q.length - w.q.rows + (end - 1) / a.share;  // the last row's position
  const int n = attend_last(a, p, w.q.tokens - 1) + 1 - w.first;
  return n <= 0 ? 1 : (n + kAttendChunk - 1) / kAttendChunk;
}

__device__ __forceinline__ AttendSeq attend_seq(const KvView& v, const AttendArgs& a, const AttendList& g, int s) {
  AttendSeq w;
  w.q = kv_sequence(v, s);
  w.flat = w.q.rows * a.share;
  w.tiles = w.flat > g.over && w.flat <= g.upto ? (w.flat + g.tile - 1) / g.tile : 0;
  w.first = 0;
  if (a.window > 0) {
    const int64_t lo = (int64_t)w.q.length - w.q.rows - a.window + 1;
    w.first = lo <= 0 ? 0 : (int)(lo < w.q.tokens ? lo : w.q.tokens) & ~63;
  }
  w.units = 0;
  for (int j = 0; j < w.tiles; ++j) w.units += attend_chunks(a, g, w, j);
  w.units *= v.heads;
  return w;
}

// A unit's place: tile, head and chunk of the item's chunks.
struct AttendItem {
  int tile, head, chunk, chunks;
};
__device__ __forceinline__ AttendItem attend_item(const KvView& v, const AttendArgs& a, const AttendList& g,
                                                  const AttendSeq& w, int at) {
  AttendItem x{0, 0, 0, 1};
  for (; x.tile < w.tiles; ++x.tile) {
    x.chunks = attend_chunks(a, g, w, x.tile);
    const int n = x.chunks * v.heads;
    if (at < n) break;
    at -= n;
  }
  x.head = at / x.chunks;
  x.chunk = at - x.head * x.chunks;
  return x;
}

// The list's `total` units in one piece for each of n blocks (n at most total, so that every block
// has some): the first `more` have one unit more than the rest.
struct AttendCut {
  int each, more;
  __device__ __forceinline__ AttendCut(int total, int n) {
    each = (int)((unsigned)total / (unsigned)n);
    more = total - each * n;
  }
  __device__ __forceinline__ int start(int b) const { return b * each + (b < more ? b : more); }
  __device__ __forceinline__ int block(int x) const {  // of unit x
    const unsigned wide = (unsigned)more * (each + 1);
    return (unsigned)x < wide ? (unsigned)x / (unsigned)(each + 1) : more + ((unsigned)x - wide) / (unsigned)each;
  }
};

// The batch's sequences, 64 at a time, one to a lane: what a wave has once read it finds there.
struct AttendSeqs {
  const KvView& v;
  const AttendArgs& a;
  const AttendList& g;
  int lane, base;
  AttendSeq mine;

  __device__ __forceinline__ AttendSeqs(const KvView& v, const AttendArgs& a, const AttendList& g, int lane)
      : v(v), a(a), g(g), lane(lane), base(-1) {}
  __device__ __forceinline__ void fetch(int i) {
    if (i == base) return;
    base = i;
    mine = AttendSeq{};
    if (i + lane < v.seqs) mine = attend_seq(v, a, g, i + lane);
  }
  // Sequence s (uniform), of those fetched last.
  __device__ __forceinline__ AttendSeq get(int s) const {
    const int at = s & (kWave - 1);
    const auto of = [&](int x) AWQ_INLINE { return __builtin_amdgcn_readlane(x, at); };
    AttendSeq w;
    w.q = KvSeq{of(mine.q.row0), of(mine.q.rows), of(mine.q.length), of(mine.q.tokens)};
    w.flat = of(mine.flat), w.tiles = of(mine.tiles), w.first = of(mine.first), w.units = of(mine.units);
    return w;
  }
  // Units of all sequences.
  __device__ __forceinline__ int units() {
    int total = 0;
    for (int i = 0; i < v.seqs; i += kWave) {
      fetch(i);
      total += __builtin_amdgcn_readlane(wave_scan(mine.units), kWave - 1);
    }
    return total;
  }
  // The sequence that holds unit x (or, tiles = true, tile x of all tiles); the units and tiles
  // before it.
  __device__ __forceinline__ int find(int x, bool tiles, int& units_before, int& tiles_before) {
    units_before = tiles_before = 0;
    for (int i = 0; i < v.seqs; i += kWave) {
      fetch(i);
      const int u = wave_scan(mine.units), t = wave_scan(mine.tiles);
      const uint64_t m = __ballot((tiles ? tiles_before + t : units_before + u) > x);
      if (m) {
        const int at = __ffsll((unsigned long long)m) - 1;
        units_before += __builtin_amdgcn_readlane(u, at) - __builtin_amdgcn_readlane(mine.units, at);
        tiles_before += __builtin_amdgcn_readlane(t, at) - __builtin_amdgcn_readlane(mine.tiles, at);
        return i + at;
      }
      units_before += __builtin_amdgcn_readlane(u, kWave - 1);
      tiles_before += __builtin_amdgcn_readlane(t, kWave - 1);
    }
    return v.seqs;
  }
};

// x as it is, rounded to fp32: no part of an instruction that rounds once for two operations.
__device__ __forceinline__ float attend_rounded(float x) {
  asm("" : "+v"(x));
  return x;
}

// The score that, times scale, is x scale - m with the product rounded, as m was.
__device__ __forceinline__ float attend_far(float x, float m, float scale) {
  return (attend_rounded(x * scale) - m) * __builtin_amdgcn_rcpf(scale);
}

// Parameters of two tokens' values, scales at most 4352 as appending writes them. What no row sees may be
// anything, an infinite scale too, and its probability, zero, must meet a finite value. (Clearing what is seen by
// none, by its position: 1% to 2% of every call with many groups or rows.)
__device__ __forceinline__ uint32_t attend_finite(uint32_t p) {
  typedef uint16_t half_words __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_min(__builtin_bit_cast(half_words, p), half_words{0x6C4F, 0x6C4F}));
}

// What block b leaves for k_attend_join (thread 0): the item that the next block goes on with.
__device__ __forceinline__ void attend_split(const AttendArgs& a, const AttendSplit& d) {
  if (a.split && threadIdx.x == 0) a.split[blockIdx.x] = d;
}

// log of a row's sum of exponentials from its maximum (of log2) and sum; -inf without a token.
__device__ __forceinline__ float attend_lse(float m, float l) { return m * 0.69314718055994531f + __logf(l); }

// (a & mask) | magic in one instruction (with two constants the compiler takes two): the mask in a
// scalar register, the magic in a vector register.
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t mask, uint32_t magic) {
  uint32_t r;
  asm("v_and_or_b32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "s"(mask), "v"(magic));
  return r;
}
struct Magic {  // the exponents under which a nibble at bits 0..3, and at 4..7, counts ones
  uint32_t m64, m54;
};
__device__ __forceinline__ Magic magics() {
  Magic m;
  asm volatile("v_mov_b32 %0, 0x64006400\n\tv_mov_b32 %1, 0x54005400" : "=v"(m.m64), "=v"(m.m54));
  return m;
}

// (code - zero) scale of the four nibbles of each half of w, pairs by nibble: zz = -(1024 + z),
// zz64 = -(64 + z), s2 = scale, of the low and of the high half.
__device__ __forceinline__ void widen4(uint32_t w, half2w zz, half2w zz64, half2w s2, Magic m, half2w (&d)[4]) {
  const uint32_t w8 = w >> 8;
  const uint32_t u0 = and_or(w, 0x000F000Fu, m.m64), u1 = and_or(w, 0x00F000F0u, m.m54);
  const uint32_t u2 = and_or(w8, 0x000F000Fu, m.m64), u3 = and_or(w8, 0x00F000F0u, m.m54);
  d[0] = (__builtin_bit_cast(half2w, u0) + zz) * s2;
  d[1] = (__builtin_bit_cast(half2w, u1) + zz64) * s2;
  d[2] = (__builtin_bit_cast(half2w, u2) + zz) * s2;
  d[3] = (__builtin_bit_cast(half2w, u3) + zz64) * s2;
}

// code - zero of the four nibbles of each half of w.
__device__ __forceinline__ void centre4(uint32_t w, half2w zz, half2w zz64, Magic m, half2w (&d)[4]) {
  const uint32_t w8 = w >> 8;
  d[0] = __builtin_bit_cast(half2w, and_or(w, 0x000F000Fu, m.m64)) + zz;
  d[1] = __builtin_bit_cast(half2w, and_or(w, 0x00F000F0u, m.m54)) + zz64;
  d[2] = __builtin_bit_cast(half2w, and_or(w8, 0x000F000Fu, m.m64)) + zz;
  d[3] = __builtin_bit_cast(half2w, and_or(w8, 0x00F000F0u, m.m54)) + zz64;
}

struct Params2 {  // of two tokens, or of one twice
  half2w zz, zz64, s2;
};
__device__ __forceinline__ Params2 params2(uint32_t p) {
  const uint32_t z = p & 0x000F000Fu;
  return Params2{__builtin_bit_cast(half2w, z | 0xE400E400u), __builtin_bit_cast(half2w, z << 4 | 0xD400D400u),
                 __builtin_bit_cast(half2w, p & 0xFFF0FFF0u)};
}

// Waves of the streaming kernel per SIMD, so blocks per CU: what registers and LDS allow, and where
// that is more than pays. One sequence of 131071 tokens, groups of 128: four a SIMD 46 us, three 43; 24
// sequences of 300-4000 tokens, 32 heads: 62, 63 (two: 74); 64 sequences, shared heads, groups of 32:
// four 97, three 101.
constexpr int stream_waves(int dim, int group, int tile) {
  return tile == 32 ? (dim == 256 ? 1 : 2) : dim == 256 ? 2 : dim / group <= 2 ? 3 : 4;
}

// A wave's buffers of the streaming kernel: one step's codes and parameters each.
template <int D, int G>
struct StreamShape {
  static constexpr int kUnits = 2;   // of 16 tokens, of a step (4: two buffers take half the chip's waves)
  static constexpr int kStages = 2;  // one is worked on (the waits count on it)
  static constexpr int kCodes = 8 * D;    // bytes of a unit's keys, or values
  static constexpr int kParams = 32 * G;  // of their parameters, [group][token]
  static constexpr int kStage = 2 * kUnits * (kCodes + kParams);
  static constexpr int kSends = kUnits * (2 * (D == 256 ? 2 : 1) + 2);  // DMA instructions of a step
  static constexpr int k_codes(int u) { return u * kCodes; }
  static constexpr int v_codes(int u) { return (kUnits + u) * kCodes; }
  static constexpr int k_params(int u) { return 2 * kUnits * kCodes + u * kParams; }
  static constexpr int v_params(int u) { return k_params(kUnits + u); }

  // A lane's words of a unit: D / 32 slices of token c's keys, or of four tokens' values. They lie in
  // the lanes' order, 16 bytes each at a time (D = 64: as in the cache).
  static __device__ __forceinline__ void key_words(const char* p, int lane, uint32_t (&w)[D / 32]) {
    if constexpr (D == 64) {
      const uint2 x = *reinterpret_cast<const uint2*>(p + (lane & 15) * 32 + (lane >> 4) * 8);
      w[0] = x.x, w[1] = x.y;
    } else {
      value_words(p, lane, w);
    }
  }
  static __device__ __forceinline__ void value_words(const char* p, int lane, uint32_t (&w)[D / 32]) {
    if constexpr (D == 64) {
      const uint2 x = *reinterpret_cast<const uint2*>(p + lane * 8);
      w[0] = x.x, w[1] = x.y;
    } else {
#pragma unroll
      for (int i = 0; i < D / 128; ++i) {
        const uint4 x = *reinterpret_cast<const uint4*>(p + 1024 * i + 16 * lane);
        w[4 * i] = x.x, w[4 * i + 1] = x.y, w[4 * i + 2] = x.z, w[4 * i + 3] = x.w;
      }
    }
  }
};

// D channels, G groups of them, R tiles of 16 rows.
template <int D, int G, int R>
__global__ void __launch_bounds__(kAttendWaves* kWave)
    __attribute__((amdgpu_waves_per_eu(stream_waves(D, D / G, 16 * R))))
    k_attend_stream(KvView v, AttendArgs a, AttendList list) {
  constexpr int kSlices = D / 32, kTiles = D / 16, kPerGroup = kSlices / G;  // slices of a group
  using S = StreamShape<D, G>;
  constexpr int kUnits = S::kUnits, kStep = 16 * kUnits, kStages = S::kStages;
  constexpr int kPad = 68;
  using Sums = float[kAttendWaves][16][kPad];
  constexpr int kRing = kAttendWaves * kStages * S::kStage;
  __shared__ __attribute__((aligned(16))) char smem[kRing > (int)sizeof(Sums) ? kRing : (int)sizeof(Sums)];
  Sums& sums = *reinterpret_cast<Sums*>(smem);  // after an item's last step
  // Up to two groups a head, the scale is applied outside the products: operands are code - zero, and a
  // token's scale multiplies its scores and probabilities in fp32: some 220 vector instructions a step
  // instead of 320 at one group. (The zero outside as well takes 208, but then sums of codes and of
  // zeros, up to 15 scales a token, leave a small difference: 131071 tokens with values around zero
  // came out 1e-3 off, relatively, not 2e-4.)
  constexpr bool kFold = G <= 2;
  __shared__ __attribute__((aligned(16))) float folds[kFold ? kAttendWaves : 1][96 * G];
  __shared__ float2 ml[kAttendWaves][16];

  const int lane = threadIdx.x & (kWave - 1), h = lane >> 4, c = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const uint32_t ring = lds_address(reinterpret_cast<uint4*>(smem + wave * kStages * S::kStage));
  const Magic magic = magics();
  float* const mine = folds[kFold ? wave : 0];
  AttendSeqs seqs(v, a, list, lane);
  const int total = seqs.units();
  const int blocks = (int)gridDim.x < total ? (int)gridDim.x : total;
  AttendSplit split{};
  if ((int)blockIdx.x >= blocks) {
    attend_split(a, split);
    return;
  }
  const AttendCut cut(total, blocks);
  const int from = cut.start(blockIdx.x), to = cut.start(blockIdx.x + 1);
  int before, tiles_before;
  int s = seqs.find(from, false, before, tiles_before);
  if (s >= v.seqs) {  // (wrong rows)
    attend_split(a, split);
    return;
  }
  AttendSeq w = seqs.get(s);
  int unit = from;
  while (unit < to) {
    const int at = unit - before;
    if (at < 0) break;  // sums that wrapped (wrong rows)
    if (at >= w.units) {
      before += w.units;
      if (++s >= v.seqs) break;
      w = attend_seq(v, a, list, s);
      continue;
    }
    const AttendItem x = attend_item(v, a, list, w, at);
    const int tile = x.tile, head = x.head, u0 = x.chunk;
    const int u1 = x.chunks - u0 < to - unit ? x.chunks : u0 + (to - unit);

    // the tile's rows: their positions, queries as the second operand
    const int r0 = tile * 16 * R, r1 = (r0 + 16 * R < w.flat ? r0 + 16 * R : w.flat) - 1;
    const int p0 = w.q.length - w.q.rows, last = w.q.tokens - 1;
    int lo[R], hi[R];
    half8w q[R][kSlices];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int row = r0 + 16 * r + c, in = row <= r1 ? row : r1;
      const int token = in / a.share, p = p0 + token;
      hi[r] = attend_last(a, p, last);
      lo[r] = a.window > 0 ? p - a.window + 1 : 0;
      const uint16_t* x = a.q + (w.q.row0 + token) * a.q_ld + (int64_t)(head * a.share + in - token * a.share) * D;
#pragma unroll
      for (int t = 0; t < kSlices; ++t) {
        const uint4 b = row <= r1 ? *reinterpret_cast<const uint4*>(x + 32 * t + 8 * h) : make_uint4(0, 0, 0, 0);
        q[r][t] = __builtin_bit_cast(half8w, b);
      }
    }
    // tokens that every row of the tile sees, and that any does
    const int pa = p0 + r0 / a.share, pb = p0 + r1 / a.share;
    const int all_hi = attend_last(a, pa, last), any_hi = attend_last(a, pb, last);
    const int all_lo = a.window > 0 ? pb - a.window + 1 : 0;
    const int t0 = w.first + u0 * kAttendChunk;
    int t1 = w.first + u1 * kAttendChunk;
    t1 = t1 <= any_hi ? t1 : any_hi + 1;

    f32x4w o[R][kTiles];
    constexpr int kP = kFold ? G : 1;
    // a row's (group's) running maximum; folded: its sums are in units of 2^m[g], products up to limit[g] fit, and
    // rest[g] = 2^(m[0] - m[g])
    float m[R][kP], l[R], limit[R][kP], rest[R][kP];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      l[r] = 0.0f;
#pragma unroll
      for (int g = 0; g < kP; ++g) m[r][g] = limit[r][g] = -__builtin_inff(), rest[r][g] = 1.0f;
#pragma unroll
      for (int n = 0; n < kTiles; ++n) o[r][n] = f32x4w{0, 0, 0, 0};
    }

    // Codes and parameters of a step go to one of the wave's own buffers by DMA, kStages - 1 steps
    // ahead: nobody else waits for them. A unit without a page (or behind t1) takes page 0's.
    const uint32_t code_page = v.heads * (uint32_t)v.code_bytes(), par_page = v.heads * (uint32_t)v.param_words();
    const uint8_t* const kb0 = v.k_codes + head * v.code_bytes();
    const uint8_t* const vb0 = v.v_codes + head * v.code_bytes();
    const uint16_t* const kq0 = v.k_params + head * v.param_words();
    const uint16_t* const vq0 = v.v_params + head * v.param_words();
    int pages = -1;      // lane kUnits k + u: the page of unit u of the wave's step k of 64 / kUnits
    uint64_t gone = 0;   // units without a page of the steps sent, the last one's in the lowest bits
    const auto send = [&](int k) AWQ_INLINE {
      constexpr int kMany = kWave / kUnits;
      const int tb = t0 + (wave + k * kAttendWaves) * kStep;
      if (k % kMany == 0)
        pages = v.page_of(s, (int64_t)tb + lane / kUnits * (kAttendWaves * kStep) + lane % kUnits * 16);
      const uint32_t to = ring + (uint32_t)(k % kStages) * S::kStage;
      u32x4 kb, vb, kq, vq;
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the buffer's last reads
#pragma unroll
      for (int u = 0; u < kUnits; ++u) {
        int page = __builtin_amdgcn_readlane(pages, kUnits * (k % kMany) + u);
        if (tb + 16 * u >= t1) page = -1;
        gone = gone << 1 | (page < 0 ? 1 : 0);
        if (u == 0 || v.page_shift == 4) {  // a step's tokens lie in one page of 32 or more
          const uint32_t in = page < 0 ? 0 : page;
          const uint32_t place = (uint32_t)(tb + 16 * u) & ((1u << v.page_shift) - 1);
          const uint64_t code = (uint64_t)in * code_page + place * (D / 2), par = (uint64_t)in * par_page + place;
          kb = buffer_words(kb0 + code), vb = buffer_words(vb0 + code);
          kq = buffer_words(kq0 + par), vq = buffer_words(vq0 + par);
        }
        const uint32_t on = u == 0 || v.page_shift == 4 ? 0 : u;  // units behind the address
        if constexpr (D == 64) {
          if (lane < 32) {
            dma16_own(kb, to + S::k_codes(u), lane * 16, on * S::kCodes);
            dma16_own(vb, to + S::v_codes(u), lane * 16, on * S::kCodes);
          }
        } else {
#pragma unroll
          for (int i = 0; i < D / 128; ++i) {
            dma16_own(kb, to + S::k_codes(u) + 1024 * i, c * (D / 2) + h * (D / 8) + 16 * i, on * S::kCodes);
            dma16_own(vb, to + S::v_codes(u) + 1024 * i, lane * (D / 8) + 16 * i, on * S::kCodes);
          }
        }
        if (G == 8 || lane < 8 * G) {  // group lane / 8, tokens 2 (lane % 8) and the next
          const uint32_t at = (lane / 8) << (v.page_shift + 1) | 4 * (lane % 8);
          dma4_own(kq, to + S::k_params(u), at, on * 32);
          dma4_own(vq, to + S::v_params(u), at, on * 32);
        }
      }
    };
    // Folded: a lane brings one token's (and group's) scales into fp32 for all lanes that have that token: of keys
    // times the softmax's (in log2), of values, and the latter's log2.
    const auto fold = [&](const char* from) AWQ_INLINE {
      const int u = lane >> 4 & 1, at = 16 * (G == 2 ? lane >> 5 : 0) + (lane & 15);
      const uint32_t kp = reinterpret_cast<const uint16_t*>(from + S::k_params(0) + u * S::kParams)[at];
      uint32_t vp = reinterpret_cast<const uint16_t*>(from + S::v_params(0) + u * S::kParams)[at];
      vp = attend_finite(vp);
      const float ks = h2f(kp & 0xFFF0), vs = h2f(vp & 0xFFF0);
      float* const to = mine + lane;  // (G = 1: lanes from 32 on repeat the others' values)
      to[G == 1 ? -(lane & 32) : 0] = ks * a.scale_log2;
      to[32 * G + (G == 1 ? -(lane & 32) : 0)] = vs;
      to[64 * G + (G == 1 ? -(lane & 32) : 0)] = __builtin_amdgcn_logf(fmaxf(vs, kLeastScale));
    };
    const auto folded = [&](int what, int g, int u) AWQ_INLINE {
      return *reinterpret_cast<const f32x4w*>(mine + 32 * G * what + 32 * g + 16 * u + 4 * h);
    };
    const auto step = [&](int k, int ahead) AWQ_INLINE {
      const int tb = t0 + (wave + k * kAttendWaves) * kStep;
      const char* from = smem + (wave * kStages + k % kStages) * S::kStage;
      const uint32_t none = (uint32_t)(gone >> (kUnits * ahead)) & ((1u << kUnits) - 1);  // unit 0 in the highest bit
      const bool part = tb + kStep > all_hi + 1 || tb < all_lo || tb + kStep > t1 || none != 0;
      if constexpr (kFold) fold(from);
      // scores (folded ones in units of log2)
      f32x4w sc[R][kUnits];
#pragma unroll
      for (int u = 0; u < kUnits; ++u) {
        uint32_t kw[kSlices];
        S::key_words(from + S::k_codes(u), lane, kw);
#pragma unroll
        for (int r = 0; r < R; ++r) sc[r][u] = f32x4w{0, 0, 0, 0};
#pragma unroll
        for (int g = 0; g < G; ++g) {
          f32x4w part_sum[R];
          const uint32_t kp = reinterpret_cast<const uint16_t*>(from + S::k_params(u))[16 * g + c];
          const Params2 p = params2(kp | kp << 16);
          if constexpr (kFold) {
#pragma unroll
            for (int r = 0; r < R; ++r) part_sum[r] = f32x4w{0, 0, 0, 0};
          }
#pragma unroll
          for (int t = g * kPerGroup; t < (g + 1) * kPerGroup; ++t) {
            half2w e[4];
            if constexpr (kFold) centre4(kw[t], p.zz, p.zz64, magic, e);
            else widen4(kw[t], p.zz, p.zz64, p.s2, magic, e);
            const half8w key{e[0][0], e[0][1], e[1][0], e[1][1], e[2][0], e[2][1], e[3][0], e[3][1]};
#pragma unroll
            for (int r = 0; r < R; ++r) {
              f32x4w& x = kFold ? part_sum[r] : sc[r][u];
              x = __builtin_amdgcn_mfma_f32_16x16x32_f16(key, q[r][t], x, 0, 0, 0);
            }
          }
          if constexpr (kFold) {
            const f32x4w by = folded(0, g, u);
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                sc[r][u][i] = __builtin_fmaf(part_sum[r][i], by[i], sc[r][u][i]);
          }
        }
      }
      if (part) {
        asm volatile("");  // nothing of this ahead of the branch
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const int most = hi[r] - tb - 4 * h, least = lo[r] - tb - 4 * h;
#pragma unroll
          for (int u = 0; u < kUnits; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (16 * u + i > most || 16 * u + i < least || (none >> (kUnits - 1 - u) & 1))
                sc[r][u][i] = -__builtin_inff();
        }
        asm volatile("");
      }
      // probabilities, as fp16 hi + lo: rounded to fp16 alone they would add as much to the output's
      // error as its own rounding does
      half8w ph[kP][R][kUnits / 2], pl[kP][R][kUnits / 2];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const auto highest = [&](int g) AWQ_INLINE {  // of the scores; folded: g >= 0 with the values' scales
          float x = -__builtin_inff();
#pragma unroll
          for (int u = 0; u < kUnits; ++u) {
            f32x4w y = sc[r][u];
            if (kFold && g >= 0) y += folded(2, g, u);
#pragma unroll
            for (int i = 0; i < 4; ++i) x = fmaxf(x, y[i]);
          }
          return x;
        };
        const auto of_row = [&](float x) AWQ_INLINE {
          x = fmaxf(x, __shfl_xor(x, 16));
          return fmaxf(x, __shfl_xor(x, 32));
        };
        float base;
        if constexpr (kFold) {
          float top[kP];
          bool over = false;
#pragma unroll
          for (int g = 0; g < kP; ++g) over |= (top[g] = highest(g)) > limit[r][g];
          if (__ballot(over)) {
            asm volatile("");
            // scores beyond kFar lose the scales beside them: their maximum alone, looked at every step
            const float plain = of_row(highest(-1));
            const bool far = __builtin_fabsf(plain) > kFar;
#pragma unroll
            for (int g = 0; g < kP; ++g) {
              const float weighed = of_row(top[g]);
              const float next = far ? plain : __builtin_ceilf(weighed) - kLift;
              const bool renew = (far || weighed > limit[r][g]) && next > m[r][g];
              const float f = renew ? __builtin_amdgcn_exp2f(m[r][g] - next) : 1.0f;
              if (renew) limit[r][g] = far ? -__builtin_inff() : next + kRoom;
              if (renew) m[r][g] = next;
              if (g == 0) l[r] *= f;
#pragma unroll
              for (int n = g * kTiles / kP; n < (g + 1) * kTiles / kP; ++n) o[r][n] *= f;
              rest[r][g] = g == 0 || m[r][g] == -__builtin_inff() ? 1.0f : __builtin_amdgcn_exp2f(m[r][0] - m[r][g]);
            }
          }
          base = m[r][0] == -__builtin_inff() ? 0.0f : m[r][0];
        } else {
          float top = highest(-1) * a.scale_log2;
          if (__ballot(top > m[r][0] + kLazy)) {
            asm volatile("");
            top = fmaxf(of_row(top), m[r][0]);
            const float f = top > m[r][0] ? __builtin_amdgcn_exp2f(m[r][0] - top) : 1.0f;
            m[r][0] = top;
            l[r] *= f;
#pragma unroll
            for (int n = 0; n < kTiles; ++n) o[r][n] *= f;
          }
          base = m[r][0] == -__builtin_inff() ? 0.0f : m[r][0] - kLift;
          if (__ballot(__builtin_fabsf(base) > kFar)) {
            asm volatile("");
            if (__builtin_fabsf(base) > kFar) {
#pragma unroll
              for (int u = 0; u < kUnits; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i) sc[r][u][i] = attend_far(sc[r][u][i], m[r][0], a.scale_log2);
              base = -kLift;
            }
          }
        }
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
          f32x4w e;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            e[i] = __builtin_amdgcn_exp2f(kFold ? sc[r][u][i] - base : __builtin_fmaf(sc[r][u][i], a.scale_log2, -base));
            l[r] += e[i];
          }
#pragma unroll
          for (int g = 0; g < kP; ++g) {
            f32x4w y = e;
            if constexpr (kFold) {
              y *= folded(1, g, u);
              if (g > 0) y *= rest[r][g];
              // before hi is taken of it: one instruction for product and hi would round once, now and then to
              // another hi than the one that lo is the rest of
#pragma unroll
              for (int i = 0; i < 4; ++i) y[i] = attend_rounded(y[i]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const _Float16 hi16 = (_Float16)y[i];
              ph[g][r][u >> 1][4 * (u & 1) + i] = hi16;
              pl[g][r][u >> 1][4 * (u & 1) + i] = (_Float16)__builtin_fmaf(-(float)hi16, 1.0f, y[i]);
            }
          }
        }
      }
      // O^T += V^T P^T, 32 tokens at a time
#pragma unroll
      for (int u = 0; u < kUnits; u += 2) {
        uint32_t vw[2][kSlices];
        S::value_words(from + S::v_codes(u), lane, vw[0]);
        S::value_words(from + S::v_codes(u + 1), lane, vw[1]);
        uint2 vp[2][G];
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int g = 0; g < G; ++g)
            vp[b][g] = *reinterpret_cast<const uint2*>(from + S::v_params(u + b) + 32 * g + 8 * h);
        if (!kFold && part) {
          asm volatile("");  // nothing of this ahead of the branch
#pragma unroll
          for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int g = 0; g < G; ++g) vp[b][g] = make_uint2(attend_finite(vp[b][g].x), attend_finite(vp[b][g].y));
        }
#pragma unroll
        for (int t = 0; t < kSlices / 2; ++t) {  // tiles 4 t .. 4 t + 3, 64 channels
#pragma unroll
          for (int half = 0; half < 2; ++half) {  // tiles 4 t + 2 half and the next: one group of 32 channels
            const int g = (2 * t + half) / kPerGroup;
            half2w e[4][4];
#pragma unroll
            for (int b = 0; b < 4; ++b) {  // token pairs
              const uint32_t word = vw[b >> 1][2 * t + (b & 1)];
              const Params2 p = params2(b & 1 ? vp[b >> 1][g].y : vp[b >> 1][g].x);
              if constexpr (kFold) centre4(word, p.zz, p.zz64, magic, e[b]);
              else widen4(word, p.zz, p.zz64, p.s2, magic, e[b]);
            }
#pragma unroll
            for (int j = 2 * half; j < 2 * half + 2; ++j) {
              const half8w val{e[0][j][0], e[0][j][1], e[1][j][0], e[1][j][1],
                               e[2][j][0], e[2][j][1], e[3][j][0], e[3][j][1]};
#pragma unroll
              for (int r = 0; r < R; ++r) {
                f32x4w& x = o[r][4 * t + j];
                x = __builtin_amdgcn_mfma_f32_16x16x32_f16(val, ph[kFold ? g : 0][r][u >> 1], x, 0, 0, 0);
                x = __builtin_amdgcn_mfma_f32_16x16x32_f16(val, pl[kFold ? g : 0][r][u >> 1], x, 0, 0, 0);
              }
            }
          }
        }
      }
    };
    __syncthreads();  // the item before is done with the buffers
    const int left = t1 - t0 - wave * kStep;
    const int steps = left <= 0 ? 0 : (left + kAttendWaves * kStep - 1) / (kAttendWaves * kStep);
    for (int k = 0; k < kStages - 1 && k < steps; ++k) send(k);
    for (int k = 0; k < steps; ++k) {
      const int ahead = steps - 1 - k < kStages - 1 ? steps - 1 - k : kStages - 1;
      if (ahead == kStages - 1) {
        send(k + kStages - 1);
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"((kStages - 1) * S::kSends) : "memory");
      } else {
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      }
      // Waves of one age share a SIMD's issue slots fairly, of several the oldest takes them: four
      // blocks a CU would end one after the other, the last alone. The turn changes hands.
      switch ((k / 2 + blockIdx.x / 256) % 4) {
        case 0: __builtin_amdgcn_s_setprio(0); break;
        case 1: __builtin_amdgcn_s_setprio(1); break;
        case 2: __builtin_amdgcn_s_setprio(2); break;
        default: __builtin_amdgcn_s_setprio(3);
      }
      step(k, ahead);
    }

    // the waves' sums together
    const bool alone = u0 == 0 && u1 == x.chunks;
    const int slot = 2 * blockIdx.x + (u0 == 0 ? 1 : 0);
    if (u1 < x.chunks) {
      const int b0 = cut.block(unit - u0), b1 = cut.block(unit - u0 + x.chunks - 1);
      split = AttendSplit{w.q.row0, r0, r1, head, b1 - b0 + 1, (int)blockIdx.x - b0};
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      l[r] += __shfl_xor(l[r], 16);
      l[r] += __shfl_xor(l[r], 32);
      if constexpr (!kFold) l[r] *= kDrop;
#pragma unroll
      for (int n = 0; n < kTiles; ++n) {
        const int g = n * kP / kTiles;
        if (!kFold) o[r][n] *= kDrop;
        else if (g > 0) o[r][n] *= 1.0f / rest[r][g];
      }
      __syncthreads();
      if (h == 0) ml[wave][c] = make_float2(m[r][0], l[r]);
      __syncthreads();
      float top = ml[0][c].x;
#pragma unroll
      for (int i = 1; i < kAttendWaves; ++i) top = fmaxf(top, ml[i][c].x);
      const float base = top == -__builtin_inff() ? 0.0f : top;
      const float f = __builtin_amdgcn_exp2f(m[r][0] - base);
      const int row = threadIdx.x >> 4, col = 4 * (threadIdx.x & 15);  // the thread's part of 16 x 64 sums
      float rtop = ml[0][row].x, sum = 0.0f;
#pragma unroll
      for (int i = 1; i < kAttendWaves; ++i) rtop = fmaxf(rtop, ml[i][row].x);
#pragma unroll
      for (int i = 0; i < kAttendWaves; ++i)
        sum += ml[i][row].y * __builtin_amdgcn_exp2f(ml[i][row].x - (rtop == -__builtin_inff() ? 0.0f : rtop));
      const int flat = r0 + 16 * r + row;
      const bool live = flat <= r1;
      const int token = flat / a.share;
      const int64_t q_row = w.q.row0 + token;
      const int q_head = head * a.share + flat - token * a.share;
#pragma unroll
      for (int part = 0; part < D / 64; ++part) {
        if (part) __syncthreads();
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          const f32x4w y = o[r][4 * part + n] * f;
          *reinterpret_cast<f32x4w*>(&sums[wave][c][16 * n + 4 * h]) = y;
        }
        __syncthreads();
        f32x4w y = *reinterpret_cast<const f32x4w*>(&sums[0][row][col]);
#pragma unroll
        for (int i = 1; i < kAttendWaves; ++i) y += *reinterpret_cast<const f32x4w*>(&sums[i][row][col]);
        if (live && alone) {
          const float d = sum == 0.0f ? 0.0f : 1.0f / sum;  // no token: zeros
          half4a b;
#pragma unroll
          for (int i = 0; i < 4; ++i) b[i] = (_Float16)(y[i] * d);
          *reinterpret_cast<half4a*>(a.out + q_row * a.out_ld + (int64_t)q_head * D + 64 * part + col) = b;
        } else if (live) {
          *reinterpret_cast<f32x4w*>(a.part + ((int64_t)slot * (16 * R) + 16 * r + row) * D + 64 * part + col) = y;
        }
      }
      if (col == 0) {
        if (alone) {
          if (live && a.lse)
            a.lse[q_row * a.q_heads + q_head] = attend_lse(rtop, sum);
        } else if (live) {
          a.part_ml[(int64_t)slot * (16 * R) + 16 * r + row] = make_float2(rtop, sum);
        }
      }
    }
    unit += u1 - u0;
  }
  attend_split(a, split);
}

// Items that several blocks took. The join block (b, y) belongs to the item that block b leaves
// unfinished: the blocks of an item share its rows, so that an item cut into many pieces has many
// blocks to add them. D / 4 lanes take 16 bytes each of a piece of a row; the 1024 / D such groups of
// a block are dealt out to its one, two or four rows.
template <int D>
__global__ void __launch_bounds__(kJoinThreads) k_attend_join(AttendArgs a, int tile) {
  constexpr int kLanes = D / 4, kGroups = kJoinThreads / kLanes;
  __shared__ f32x4w part[kGroups][kLanes];
  __shared__ float2 ml[kGroups];
  const AttendSplit d = a.split[blockIdx.x];
  const int joins = (d.blocks - 1) * gridDim.y, id = d.index * gridDim.y + blockIdx.y;
  const int b0 = (int)blockIdx.x - d.index;
  if (d.blocks < 2 || b0 < 0 || d.blocks > (int)gridDim.x - b0 || d.r0 + id > d.r1) return;
  const int per = (tile + joins - 1) / joins, rows = per > 2 ? 4 : per;  // (at most four)
  const int ways = kGroups / rows, group = threadIdx.x / kLanes, lane = threadIdx.x % kLanes;
  const int row = id + group / ways * joins, flat = d.r0 + row;
  float m = -__builtin_inff(), l = 0.0f;
  f32x4w y{0, 0, 0, 0};
  if (row < tile && flat <= d.r1) {
    constexpr int kDeep = 4;
    const auto add = [&](int k, auto many) AWQ_INLINE {  // pieces k, k + ways ..., loaded together
      constexpr int kMany = decltype(many)::value;
      float2 p[kMany];
      f32x4w z[kMany];
#pragma unroll
      for (int i = 0; i < kMany; ++i) {
        const int at = k + i * ways;
        const int64_t slot = ((int64_t)2 * (b0 + at) + (at == 0 ? 1 : 0)) * tile + row;
        p[i] = a.part_ml[slot];
        z[i] = *reinterpret_cast<const f32x4w*>(a.part + slot * D + 4 * lane);
      }
#pragma unroll
      for (int i = 0; i < kMany; ++i) {
        const float top = fmaxf(m, p[i].x), base = top == -__builtin_inff() ? 0.0f : top;
        const float f = __builtin_amdgcn_exp2f(m - base), g = __builtin_amdgcn_exp2f(p[i].x - base);
        l = l * f + p[i].y * g;
        y = y * f + z[i] * g;
        m = top;
      }
    };
    // whole fours and single ones: with pieces beyond the last one, eight at a time and weighed as
    // nothing, calls of 32 and 93 us took 35 and 96
    int k = group % ways;
    for (; k + (kDeep - 1) * ways < d.blocks; k += kDeep * ways) add(k, std::integral_constant<int, kDeep>());
    for (; k < d.blocks; k += ways) add(k, std::integral_constant<int, 1>());
  }
  part[group][lane] = y;
  if (lane == 0) ml[group] = make_float2(m, l);
  __syncthreads();
  if (group % ways != 0 || row >= tile || flat > d.r1) return;
  for (int i = 1; i < ways; ++i) {
    const float2 p = ml[group + i];
    const float top = fmaxf(m, p.x), base = top == -__builtin_inff() ? 0.0f : top;
    const float f = __builtin_amdgcn_exp2f(m - base), g = __builtin_amdgcn_exp2f(p.x - base);
    l = l * f + p.y * g;
    y = y * f + part[group + i][lane] * g;
    m = top;
  }
  const int token = flat / a.share;
  const int64_t q_row = d.row0 + token;
  const int q_head = d.head * a.share + flat - token * a.share;
  const float r = l == 0.0f ? 0.0f : 1.0f / l;  // no token: zeros
  half4a b;
#pragma unroll
  for (int e = 0; e < 4; ++e) b[e] = (_Float16)(y[e] * r);
  *reinterpret_cast<half4a*>(a.out + q_row * a.out_ld + (int64_t)q_head * D + 4 * lane) = b;
  if (a.lse && lane == 0) a.lse[q_row * a.q_heads + q_head] = attend_lse(m, l);
}

template <int D, int G>
hipError_t attend_stream(const KvView& v, const AttendArgs& a, const AttendList& list, hipStream_t stream) {
  auto* const f = list.tile == 16 ? k_attend_stream<D, G, 1> : k_attend_stream<D, G, 2>;
  hipLaunchKernelGGL(f, dim3(a.blocks), dim3(kAttendWaves * kWave), 0, stream, v, a, list);
  return hipGetLastError();
}

}  // namespace awq
