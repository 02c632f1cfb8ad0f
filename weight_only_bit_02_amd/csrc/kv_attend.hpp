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
#pragma once

#include "groups.hpp"
#include "kv_cache.hpp"

namespace awq {

constexpr int kAttendWaves = 4;
constexpr int kAttendStep = 64;                          // tokens of a wave's step
constexpr int kAttendChunk = kAttendStep * kAttendWaves;  // tokens of the work list's unit
constexpr float kLazy = 8.0f;  // the running maximum is renewed when a score passes it by 2^8

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

// Chunks of tile j of a sequence: as far as its last row sees, one for rows without a token.
__device__ __forceinline__ int attend_chunks(const AttendArgs& a, const AttendList& g, const AttendSeq& w, int j) {
  const int end = (j + 1) * g.tile < w.flat ? (j + 1) * g.tile : w.flat;
  const int p = w.q.length - w.q.rows + (end - 1) / a.share + 1;  // tokens up to the last row's own
  const int n = (a.causal && p < w.q.tokens ? p : w.q.tokens) - w.first;
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
    w.first = lo <= 0 ? 0 : (int)(lo < w.q.tokens ? lo : w.q.tokens) & ~(kAttendStep - 1);
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

// First unit of block b of n, of `total` units (n at most total: no block between two others is
// without a unit); and the block that unit x belongs to.
__device__ __forceinline__ int block_start(int b, int n, int total) { return (int)((int64_t)b * total / n); }
__device__ __forceinline__ int block_of(int x, int n, int total) {
  return (int)((((int64_t)x + 1) * n - 1) / total);
}

// Units of all sequences, and of those before sequence s (uniform over the wave).
__device__ __forceinline__ int attend_units(const KvView& v, const AttendArgs& a, const AttendList& g, int s, int lane,
                                            int& before) {
  int total = 0;
  before = 0;
  for (int i = 0; i < v.seqs; i += kWave) {
    const int n = i + lane < v.seqs ? attend_seq(v, a, g, i + lane).units : 0;
    total += __builtin_amdgcn_readlane(wave_scan(n), kWave - 1);
    before += __builtin_amdgcn_readlane(wave_scan(i + lane < s ? n : 0), kWave - 1);
  }
  return total;
}

// The sequence that holds unit x of the list, and the units before it (uniform over the wave).
__device__ __forceinline__ int attend_find(const KvView& v, const AttendArgs& a, const AttendList& g, int x, int lane,
                                           int& before) {
  before = 0;
  for (int i = 0; i < v.seqs; i += kWave) {
    const int n = i + lane < v.seqs ? attend_seq(v, a, g, i + lane).units : 0;
    const int sum = wave_scan(n);
    const uint64_t m = __ballot(before + sum > x);
    if (m) {
      const int at = __ffsll((unsigned long long)m) - 1;
      before += __builtin_amdgcn_readlane(sum, at) - __builtin_amdgcn_readlane(n, at);
      return i + at;
    }
    before += __builtin_amdgcn_readlane(sum, kWave - 1);
  }
  return v.seqs;
}

// The sequence with tile x of all tiles, the units before it, and which of its tiles it is.
__device__ __forceinline__ int attend_find_tile(const KvView& v, const AttendArgs& a, const AttendList& g, int x,
                                                int lane, int& before, int& tile) {
  int tiles = 0;
  before = 0;
  for (int i = 0; i < v.seqs; i += kWave) {
    AttendSeq w{};
    if (i + lane < v.seqs) w = attend_seq(v, a, g, i + lane);
    const int sum = wave_scan(w.tiles), units = wave_scan(w.units);
    const uint64_t m = __ballot(tiles + sum > x);
    if (m) {
      const int at = __ffsll((unsigned long long)m) - 1;
      before += __builtin_amdgcn_readlane(units, at) - __builtin_amdgcn_readlane(w.units, at);
      tile = x - tiles - __builtin_amdgcn_readlane(sum, at) + __builtin_amdgcn_readlane(w.tiles, at);
      return i + at;
    }
    tiles += __builtin_amdgcn_readlane(sum, kWave - 1);
    before += __builtin_amdgcn_readlane(units, kWave - 1);
  }
  return v.seqs;
}

// What block b leaves for k_attend_join (thread 0): the item that the next block goes on with.
__device__ __forceinline__ void attend_split(const AttendArgs& a, const AttendSplit& d) {
  if (a.split && threadIdx.x == 0) a.split[blockIdx.x] = d;
}

// log of a row's sum of exponentials from its maximum (of log2) and sum; -inf without a token.
__device__ __forceinline__ float attend_lse(float m, float l) { return m * 0.69314718055994531f + __logf(l); }

// (code - zero) scale of the four nibbles of each half of w, pairs by nibble: zz = -(1024 + z),
// zz64 = -(64 + z), s2 = scale, of the low and of the high half.
__device__ __forceinline__ void widen4(uint32_t w, half2w zz, half2w zz64, half2w s2, half2w (&d)[4]) {
  const uint32_t w8 = w >> 8;
  const uint32_t u0 = (w & 0x000F000Fu) | 0x64006400u, u1 = (w & 0x00F000F0u) | 0x54005400u;
  const uint32_t u2 = (w8 & 0x000F000Fu) | 0x64006400u, u3 = (w8 & 0x00F000F0u) | 0x54005400u;
  d[0] = (__builtin_bit_cast(half2w, u0) + zz) * s2;
  d[1] = (__builtin_bit_cast(half2w, u1) + zz64) * s2;
  d[2] = (__builtin_bit_cast(half2w, u2) + zz) * s2;
  d[3] = (__builtin_bit_cast(half2w, u3) + zz64) * s2;
}

struct Params2 {  // of two tokens, or of one twice
  half2w zz, zz64, s2;
};
__device__ __forceinline__ Params2 params2(uint32_t p) {
  const uint32_t z = p & 0x000F000Fu;
  return Params2{__builtin_bit_cast(half2w, z | 0xE400E400u), __builtin_bit_cast(half2w, z << 4 | 0xD400D400u),
                 __builtin_bit_cast(half2w, p & 0xFFF0FFF0u)};
}

// D channels, G groups of them, R tiles of 16 rows.
template <int D, int G, int R>
__global__ void __launch_bounds__(kAttendWaves* kWave) k_attend_stream(KvView v, AttendArgs a, AttendList list) {
  constexpr int kSlices = D / 32, kTiles = D / 16, kPerGroup = kSlices / G;  // slices of a group
  constexpr int kPad = 68;
  __shared__ float sums[kAttendWaves][16][kPad];
  __shared__ float2 ml[kAttendWaves][16];

  const int lane = threadIdx.x & (kWave - 1), h = lane >> 4, c = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  int before;
  const int total = attend_units(v, a, list, 0, lane, before);
  const int blocks = (int)gridDim.x < total ? (int)gridDim.x : total;
  AttendSplit split{};
  if ((int)blockIdx.x >= blocks) {
    attend_split(a, split);
    return;
  }
  const int from = block_start(blockIdx.x, blocks, total), to = block_start(blockIdx.x + 1, blocks, total);
  int s = attend_find(v, a, list, from, lane, before);
  int unit = from;
  while (unit < to && s < v.seqs) {
    const AttendSeq w = attend_seq(v, a, list, s);
    const int at = unit - before;
    if (at < 0) break;  // sums that wrapped (wrong rows)
    if (at >= w.units) {
      before += w.units;
      ++s;
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
      hi[r] = a.causal && p < last ? p : last;
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
    const int all_hi = a.causal && pa < last ? pa : last, any_hi = a.causal && pb < last ? pb : last;
    const int all_lo = a.window > 0 ? pb - a.window + 1 : 0;
    const int t0 = w.first + u0 * kAttendChunk;
    int t1 = w.first + u1 * kAttendChunk;
    t1 = t1 <= any_hi ? t1 : any_hi + 1;

    f32x4w o[R][kTiles];
    float m[R], l[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      m[r] = -__builtin_inff();
      l[r] = 0.0f;
#pragma unroll
      for (int n = 0; n < kTiles; ++n) o[r][n] = f32x4w{0, 0, 0, 0};
    }

    const int64_t code_head = v.code_bytes(), par_head = v.param_words();
    int pages = -1;  // lane 4 k + u: the page of unit u of the wave's step k of 16
    for (int tb = t0 + wave * kAttendStep, k = 0; tb < t1; tb += kAttendChunk, ++k) {
      if ((k & 15) == 0) pages = v.page_of(s, (int64_t)tb + (lane >> 2) * kAttendChunk + (lane & 3) * 16);
      // codes and parameters of 64 tokens: units of 16
      uint32_t kc[4][kSlices], vc[4][kSlices];
      uint32_t kp[4][G];
      uint2 vp[4][G];
      int page[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        page[u] = __builtin_amdgcn_readlane(pages, 4 * (k & 15) + u);
        if (tb + 16 * u >= t1) page[u] = -1;
        if (page[u] >= 0) {
          const int place = (tb + 16 * u) & ((1 << v.page_shift) - 1);
          const int64_t at = (int64_t)page[u] * v.heads + head;
          const uint8_t* kb = v.k_codes + at * code_head + (int64_t)place * (D / 2);
          const uint8_t* vb = v.v_codes + at * code_head + (int64_t)place * (D / 2);
          // D / 8 bytes a lane
          if constexpr (kSlices == 2) {
            const uint2 x = *reinterpret_cast<const uint2*>(kb + c * (D / 2) + h * (D / 8));
            const uint2 y = *reinterpret_cast<const uint2*>(vb + lane * (D / 8));
            kc[u][0] = x.x, kc[u][1] = x.y, vc[u][0] = y.x, vc[u][1] = y.y;
          } else {
#pragma unroll
            for (int i = 0; i < kSlices; i += 4) {
              const uint4 x = *reinterpret_cast<const uint4*>(kb + c * (D / 2) + h * (D / 8) + 4 * i);
              const uint4 y = *reinterpret_cast<const uint4*>(vb + lane * (D / 8) + 4 * i);
              kc[u][i] = x.x, kc[u][i + 1] = x.y, kc[u][i + 2] = x.z, kc[u][i + 3] = x.w;
              vc[u][i] = y.x, vc[u][i + 1] = y.y, vc[u][i + 2] = y.z, vc[u][i + 3] = y.w;
            }
          }
          const uint16_t* kpar = v.k_params + at * par_head + place;
          const uint16_t* vpar = v.v_params + at * par_head + place;
#pragma unroll
          for (int g = 0; g < G; ++g) {
            kp[u][g] = kpar[((int64_t)g << v.page_shift) + c];
            vp[u][g] = *reinterpret_cast<const uint2*>(vpar + ((int64_t)g << v.page_shift) + 4 * h);
          }
        } else {
#pragma unroll
          for (int i = 0; i < kSlices; ++i) kc[u][i] = vc[u][i] = 0;
#pragma unroll
          for (int g = 0; g < G; ++g) kp[u][g] = 0, vp[u][g] = make_uint2(0, 0);
        }
      }
      // scores
      f32x4w sc[R][4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
#pragma unroll
        for (int r = 0; r < R; ++r) sc[r][u] = f32x4w{0, 0, 0, 0};
#pragma unroll
        for (int g = 0; g < G; ++g) {
          const Params2 p = params2(kp[u][g] | kp[u][g] << 16);
#pragma unroll
          for (int t = g * kPerGroup; t < (g + 1) * kPerGroup; ++t) {
            half2w d[4];
            widen4(kc[u][t], p.zz, p.zz64, p.s2, d);
            const half8w key{d[0][0], d[0][1], d[1][0], d[1][1], d[2][0], d[2][1], d[3][0], d[3][1]};
#pragma unroll
            for (int r = 0; r < R; ++r)
              sc[r][u] = __builtin_amdgcn_mfma_f32_16x16x32_f16(key, q[r][t], sc[r][u], 0, 0, 0);
          }
        }
      }
      const bool whole = tb + kAttendStep <= all_hi + 1 && tb >= all_lo && tb + kAttendStep <= t1 &&
                         (page[0] | page[1] | page[2] | page[3]) >= 0;
      if (!whole) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int t = tb + 16 * u + 4 * h + i;
#pragma unroll
            for (int r = 0; r < R; ++r)
              if (!(t >= lo[r] && t <= hi[r] && page[u] >= 0)) sc[r][u][i] = -__builtin_inff();
            // what lies behind the sequence's last token may be anything, an infinite scale too
            if (t > last) {
#pragma unroll
              for (int g = 0; g < G; ++g) {
                uint32_t& p = i < 2 ? vp[u][g].x : vp[u][g].y;
                p &= i & 1 ? 0x0000FFFFu : 0xFFFF0000u;
              }
            }
          }
        }
      }
      // probabilities, as fp16 hi + lo: rounded to fp16 alone they would add as much to the output's
      // error as its own rounding does
      half8w ph[R][2], pl[R][2];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float top = sc[r][0][0];
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
          for (int i = 0; i < 4; ++i) top = fmaxf(top, sc[r][u][i]);
        top *= a.scale_log2;
        if (__ballot(top > m[r] + kLazy)) {
          top = fmaxf(top, __shfl_xor(top, 16));
          top = fmaxf(fmaxf(top, __shfl_xor(top, 32)), m[r]);
          const float f = top > m[r] ? __builtin_amdgcn_exp2f(m[r] - top) : 1.0f;
          m[r] = top;
          l[r] *= f;
#pragma unroll
          for (int n = 0; n < kTiles; ++n) o[r][n] *= f;
        }
        const float base = m[r] == -__builtin_inff() ? 0.0f : m[r];
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[r][u][i], a.scale_log2, -base));
            l[r] += e;
            const _Float16 hi16 = (_Float16)e;
            ph[r][u >> 1][4 * (u & 1) + i] = hi16;
            pl[r][u >> 1][4 * (u & 1) + i] = (_Float16)(e - (float)hi16);
          }
      }
      // O^T += V^T P^T, 32 tokens at a time
#pragma unroll
      for (int u = 0; u < 4; u += 2) {
#pragma unroll
        for (int t = 0; t < kSlices / 2; ++t) {  // tiles 4 t .. 4 t + 3, 64 channels
#pragma unroll
          for (int half = 0; half < 2; ++half) {  // tiles 4 t + 2 half and the next: one group of 32 channels
            const int g = (2 * t + half) / kPerGroup;
            half2w d[4][4];
#pragma unroll
            for (int b = 0; b < 4; ++b) {  // token pairs
              const uint2 two = vp[u + (b >> 1)][g];
              const Params2 p = params2(b & 1 ? two.y : two.x);
              widen4(vc[u + (b >> 1)][2 * t + (b & 1)], p.zz, p.zz64, p.s2, d[b]);
            }
#pragma unroll
            for (int j = 2 * half; j < 2 * half + 2; ++j) {
              const half8w val{d[0][j][0], d[0][j][1], d[1][j][0], d[1][j][1],
                               d[2][j][0], d[2][j][1], d[3][j][0], d[3][j][1]};
#pragma unroll
              for (int r = 0; r < R; ++r) {
                o[r][4 * t + j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(val, ph[r][u >> 1], o[r][4 * t + j], 0, 0, 0);
                o[r][4 * t + j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(val, pl[r][u >> 1], o[r][4 * t + j], 0, 0, 0);
              }
            }
          }
        }
      }
    }

    // the waves' sums together
    const bool alone = u0 == 0 && u1 == x.chunks;
    const int slot = 2 * blockIdx.x + (u0 == 0 ? 1 : 0);
    if (u1 < x.chunks) {
      const int b0 = block_of(unit - u0, blocks, total), b1 = block_of(unit - u0 + x.chunks - 1, blocks, total);
      split = AttendSplit{w.q.row0, r0, r1, head, b1 - b0 + 1, (int)blockIdx.x - b0};
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      l[r] += __shfl_xor(l[r], 16);
      l[r] += __shfl_xor(l[r], 32);
      __syncthreads();
      if (h == 0) ml[wave][c] = make_float2(m[r], l[r]);
      __syncthreads();
      float top = ml[0][c].x;
#pragma unroll
      for (int i = 1; i < kAttendWaves; ++i) top = fmaxf(top, ml[i][c].x);
      const float base = top == -__builtin_inff() ? 0.0f : top;
      const float f = __builtin_amdgcn_exp2f(m[r] - base);
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
    for (int k = group % ways; k < d.blocks; k += kDeep * ways) {
      float2 p[kDeep];
      f32x4w z[kDeep];
#pragma unroll
      for (int i = 0; i < kDeep; ++i) {
        const int kk = k + i * ways;
        const int64_t slot = ((int64_t)2 * (b0 + kk) + (kk == 0 ? 1 : 0)) * tile + row;
        p[i] = kk < d.blocks ? a.part_ml[slot] : make_float2(-__builtin_inff(), 0.0f);
        z[i] = kk < d.blocks ? *reinterpret_cast<const f32x4w*>(a.part + slot * D + 4 * lane) : f32x4w{0, 0, 0, 0};
      }
#pragma unroll
      for (int i = 0; i < kDeep; ++i) {
        const float top = fmaxf(m, p[i].x), base = top == -__builtin_inff() ? 0.0f : top;
        const float f = __builtin_amdgcn_exp2f(m - base), g = __builtin_amdgcn_exp2f(p[i].x - base);
        l = l * f + p[i].y * g;
        y = y * f + z[i] * g;
        m = top;
      }
    }
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
