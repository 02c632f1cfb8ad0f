// Ragged-row linear for few rows per group (decoding): the products of grouped_gemm.hpp on
// tiles of 16 rows. Decoding streams every active weight once and multiplies it with a
// handful of rows, so the design is about bytes in flight, cache-line requests per byte and
// instructions per byte.
//
//   - A work item is one row tile x 16 R weight rows over all of K, split over the S waves of a
//     block, which meet in LDS in a fixed order. Blocks are persistent: the launch fills the
//     chip once, each block takes a contiguous run of the items there are (counted on the
//     device from the offsets).
//   - A wave owns L K steps (128 channels each) of every item, so its part of X stays in
//     registers for as long as the tile does: nothing but codes, scales and zeros is loaded per
//     item. (K beyond S L steps is walked in parts, which reload X.)
//   - Codes go global -> LDS by 16-byte DMA, eight neighbouring lanes on 128 contiguous bytes of
//     a weight row, a whole cache line per request: the matrix cores want neighbouring lanes on
//     neighbouring rows, and loading in that order straight into registers costs an L1 access
//     per lane (this way 64 experts x 4096 x 1024 on 384 rows, 145 MB, take 4.1 M in all), loading
//     64 bytes per row twice the requests in flight for the same bytes. The buffers belong to one
//     wave, so there is no barrier: a buffer is refilled as soon as its codes are in registers,
//     and a wave keeps 16 KB in flight. Pieces are stored so that the reads have no bank
//     conflicts. The waits are written out (take_codes, meet): left to itself the compiler
//     drains every load in flight before each read, barrier and loop end.
//   - v_mfma_f32_16x16x32_f16: lane l works on weight row l % 16 and on 32 channels of a step, by
//     kg = l / 16: with 128-channel groups on [32 kg, 32 kg + 32), 16 bytes of 4-bit codes per weight
//     row; with smaller ones on [32 i + 8 kg, 32 i + 8 kg + 8), i = 0 .. 3, so that the channels of
//     a product (slice i) lie in one group. The codes are widened 8 channels at a time.
//   - Scales and zeros of the L steps are loaded one weight row per lane, all steps at once
//     (2 bytes per group would ask for a cache line each), and handed to the lanes that need
//     them by ds_bpermute. Their addresses have the alignment of their type only.
//   - The operand is q - z, exact in fp16, and the scale multiplies a group's partial tile in fp32.
//     (Codes under the bias of their exponent, with the bias and z taken off in the fp32 sums, would
//     save the subtraction of two channels at a time, but then a channel whose code equals its zero
//     leaves the rounding of 1024 |x| in a sum that it is no part of; operands that carry the scale,
//     fp16((q - z) sc), have a rounding more than the plain linear for few rows.)
//   - A chunk that would pass the last weight row starts earlier instead and computes some
//     columns twice, to the same values.
//
// What bounds it: the widening and the stream together; large launches reach three quarters of
// what a copy reaches, more with 8-bit codes. 64 experts x 4096 x 1024, 384 rows: 36.3 us, 4.0
// TB/s; 8 experts x 22016 x 4096 gated, 64 rows: 81 us, 4.6 TB/s; 8 experts x 2048 x 2048 gated, a
// row each: 9.3 us, of which the chain offsets, row, first codes, sums is most. 3-bit codes cost
// more instructions per byte: 64 x 2048 x 2048, 512 rows, 37 us. Groups of 64 and 32 cost more scales
// and partial tiles: 64 x 4096 x 1024, 512 rows, 4-bit, 34, 37 and 41 us.
//
// Gated: tiles 0 .. R / 2 - 1 are gate rows, the rest their up rows, so a lane's sums hold
// both and the epilogue needs no exchange. Adapters: as in grouped_gemm.hpp; the waves share
// the adapters among a tile's rows.
#pragma once

#include "common.hpp"
#include "groups.hpp"
#include "launch.hpp"
#include "widen.hpp"

namespace awq {


#define AWQ_INLINE __attribute__((always_inline))

constexpr int kStreamWaves = 8;     // S at most
constexpr int kStreamSlots = 2048;  // resident waves: two per SIMD

constexpr int kStreamSteps = 4;     // L
constexpr int kStreamSplit = 64;    // chunks from which on each XCD takes an eighth of them

// Columns of an item: 8-bit codes take twice the LDS; half where whole ones would leave blocks
// without an item.
constexpr int stream_cols(int w_bit, bool narrow) { return w_bit == 8 || narrow ? 32 : 64; }

// Eight bytes at byte `at` of [p, p + bytes), bytes >= 8, at any alignment; those past the end
// are not read: the load moves back, and the value is shifted when it is used (shifting it here
// would wait for the load).
struct Eight {
  uint64_t v;
  uint32_t shift;
  __device__ __forceinline__ uint64_t value() const { return v >> (shift & 63); }
};
__device__ __forceinline__ Eight load8(const void* p, int64_t at, int64_t bytes) {
  const int64_t from = at < bytes - 8 ? at : bytes - 8;
  Eight e;
  __builtin_memcpy(&e.v, (const char*)p + from, 8);
  e.shift = (uint32_t)(8 * (at - from));
  return e;
}

// A zero point as the subtrahends of widened codes: -(1024 + z) twice, and -(64 + z) twice.
struct ZeroPair {
  half2w z1024, z64;
};
__device__ __forceinline__ ZeroPair zero_pair(uint32_t z) {
  const uint32_t a = 0xE400u + z, b = 0xD400u + (z << 4);  // negative fp16
  return ZeroPair{__builtin_bit_cast(half2w, a | (a << 16)), __builtin_bit_cast(half2w, b | (b << 16))};
}

// A lane's code words of a step: its 32 channels in order; 3-bit codes in slices of their own
// (small groups): per slice the low planes' fields in bits 0-7 of each half, the high plane's in
// bits 8-11.
constexpr int stream_words(int bits, int groups) { return bits == 3 && groups > 1 ? 4 : bits; }

// Codes of 8 channels (slice s of a lane's 32) as exact q - z.
template <int BITS, int W>
__device__ __forceinline__ half8w centered(const uint32_t (&w)[W], int s, const ZeroPair& z,
                                           uint32_t magic) {
  half2w d[4];
  if constexpr (BITS == 4) {
    const uint32_t w0 = w[s], w8 = w[s] >> 8;
    d[0] = __builtin_bit_cast(half2w, (w0 & 0x000F000Fu) | magic) + z.z1024;
    d[1] = __builtin_bit_cast(half2w, (w0 & 0x00F000F0u) | 0x54005400u) + z.z64;
    d[2] = __builtin_bit_cast(half2w, (w8 & 0x000F000Fu) | magic) + z.z1024;
    d[3] = __builtin_bit_cast(half2w, (w8 & 0x00F000F0u) | 0x54005400u) + z.z64;
  } else if constexpr (BITS == 8) {
    const uint32_t m8 = 0x64646464u;
#pragma unroll
    for (int p = 0; p < 4; ++p)
      d[p] = __builtin_bit_cast(half2w, __builtin_amdgcn_perm(m8, w[2 * s + (p >> 1)], p & 1 ? 0x04030402u : 0x04010400u)) + z.z1024;
  } else {
#pragma unroll
    for (int p = 0; p < 4; ++p)
      d[p] = __builtin_bit_cast(half2w, W == 4 ? widen3_pair(w[s], w[s], p, 8 + p, magic)
                                               : widen3_pair(w[s >> 1], w[2], 4 * (s & 1) + p, 4 * s + p, magic)) +
             z.z1024;
  }
  return half8w{d[0][0], d[0][1], d[1][0], d[1][1], d[2][0], d[2][1], d[3][0], d[3][1]};
}

// A position of the walk: an item (row tile x column chunk) and a part of K. Uniform.
struct StreamItem {
  int tile, chunk, part, row0, rows;
};

// GS: groups of a step of 128 channels (1, 2, 4).
template <int MODE, int BITS, int GS, int R, int L, int S>
__global__ void __launch_bounds__(S * 64) __attribute__((amdgpu_waves_per_eu(2)))
    k_stream(GroupedArgs g) {
  constexpr int BM = 16, kCols = MODE == kGated ? 8 * R : 16 * R;
  constexpr int H = BITS == 8 ? 1 : 2;        // steps of a buffer: 128 bytes of a row (3-bit: 96)
  constexpr int NB = L / H;                   // buffers, one position's codes
  constexpr int P = BITS * H;                 // 16-byte pieces of a row in a buffer
  constexpr int kBuf = R * 2 * 64;            // slots of a wave's buffer: two DMA instructions a tile
  __shared__ __attribute__((aligned(16))) uint4 st0[S][kBuf];
  __shared__ __attribute__((aligned(16))) uint4 st1[S][kBuf];
  __shared__ __attribute__((aligned(16))) uint4 st2[NB > 2 ? S : 1][NB > 2 ? kBuf : 1];
  __shared__ __attribute__((aligned(16))) uint4 st3[NB > 2 ? S : 1][NB > 2 ? kBuf : 1];
  __shared__ __attribute__((aligned(16))) f32x4w red[S * R * 64];
  static_assert(L == 4, "the scales and zeros of four steps are loaded eight bytes at a time");
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c16 = lane & 15, kg = lane >> 4;
  const int64_t N = g.N, K = g.K, nh = N / 2;
  const int outs = (int)(MODE == kGated ? nh : N);
  const int nsteps = (int)(K / kGroup), nt = g.nt, parts = (nsteps + S * L - 1) / (S * L);
  constexpr int W = stream_words(BITS, GS);
  const int64_t Gs = K / g.group, zbw = BITS == 8 ? Gs : (Gs + 1) / 2, words = K * BITS / 32;
  const int64_t sbytes = (MODE == kLora ? 1 : g.groups) * N * Gs * 2;
  const int64_t zbytes = (MODE == kLora ? 1 : g.groups) * N * zbw;
  const uint32_t magic = wide_magic();

  // ---- this block's run of items: row tiles by column chunks, tile after tile. XCD blockIdx % 8
  // takes an eighth of the chunks (kStreamSplit or more), for all tiles, so that the tiles of
  // one weight find it in its L2 (3 tiles of 8-bit 4096 x 4096, with adapters: 28 us without, 21).
  const int mt = MODE == kLora ? (g.n + BM - 1) / BM
                               : __builtin_amdgcn_readfirstlane(count_tiles<BM>(g.offsets, g.groups, g.n, lane));
  const int xcds = nt >= kStreamSplit ? 8 : 1, xcd = blockIdx.x % xcds;
  const int c0 = nt * xcd / xcds, c1 = nt * (xcd + 1) / xcds, nc = c1 - c0;
  const int64_t items = (int64_t)mt * nc, slots = gridDim.x / xcds, slot = blockIdx.x / xcds;
  const int64_t i0 = items * slot / slots, i1 = items * (slot + 1) / slots;
  if (i0 >= i1) return;  // uniform over the block
  int todo = (int)(i1 - i0) * parts;  // positions

  // ---- addresses: a lane's offsets in the weight rows, and the rest uniform
  const uint32_t rowq = (uint32_t)(words * 4);
  auto weight_row = [&](int c) AWQ_INLINE -> uint32_t {  // of column c of a chunk, less the first's
    int o = MODE == kGated ? c % (8 * R) : c;
    o = o < outs ? o : outs - 1;
    return (uint32_t)o + (MODE == kGated && c >= 8 * R ? (uint32_t)nh : 0u);
  };
  // (K of a single step: a row's bytes end inside the buffer; the rest repeats its first piece)
  const int pieces = BITS * (nsteps < H ? nsteps : H);
  // DMA slot of a weight tile's buffer: piece (slot % P) ^ swizzle of row slot / P (3-bit: not
  // swizzled; slots past the last row repeat it)
  uint32_t vq[R][2];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int d = 0; d < 2; ++d) {
      const int slot = d * 64 + lane, row = slot / P < 16 ? slot / P : 15;
      const int piece = BITS == 3 ? slot % P : (slot & 7) ^ (row >> 1);
      vq[r][d] = weight_row(r * 16 + row) * rowq + (piece < pieces ? piece * 16 : 0);
    }
  const uint32_t my_row = weight_row(lane % (16 * R));  // scales and zeros: one weight row per lane
  __amdgpu_buffer_rsrc_t codes;
  int64_t expert_row = 0;  // first weight row of the loads' expert
  auto first = [&](int chunk) AWQ_INLINE -> int {  // first output column of a chunk
    const int c = chunk * kCols, last = outs > kCols ? outs - kCols : 0;
    return c < last ? c : last;
  };
  auto source = [&](int p) AWQ_INLINE -> int {  // the row that order names (out of range: row 0)
    if (!g.order) return p;
    const int o = g.order[p];
    return (unsigned)o < (unsigned)g.n ? o : 0;
  };
  auto step_of = [&](int part, int j) AWQ_INLINE -> int { return (part * S + wave) * L + j; };

  StreamItem ld{(int)(i0 / nc), c0 + (int)(i0 % nc), 0, 0, 0};  // the position being loaded
  auto open_tile = [&]() AWQ_INLINE {
    const RowTile rt = MODE == kLora ? RowTile{0, ld.tile * BM, g.n - ld.tile * BM < BM ? g.n - ld.tile * BM : BM}
                                     : find_tile<BM>(g.offsets, g.groups, g.n, ld.tile, lane);
    ld.row0 = __builtin_amdgcn_readfirstlane(rt.row0);
    ld.rows = __builtin_amdgcn_readfirstlane(rt.rows);
    const int64_t e = MODE == kLora ? 0 : __builtin_amdgcn_readfirstlane(rt.e);
    expert_row = e * N;
    codes = buffer_at(g.qweight + e * N * words);
  };
  auto next = [&]() AWQ_INLINE {
    if (++ld.part < parts) return;
    ld.part = 0;
    if (++ld.chunk < c1) return;
    ld.chunk = c0;
    ++ld.tile;
    open_tile();
  };

  auto buffer = [&](int b) AWQ_INLINE -> uint4* {
    return b == 0 ? st0[wave] : b == 1 ? st1[wave] : b == 2 ? st2[NB > 2 ? wave : 0] : st3[NB > 2 ? wave : 0];
  };
  // steps H i .. of the position being loaded into buffer b (those past the last step: the last
  // ones, not multiplied)
  auto load_codes = [&](int b, int i) AWQ_INLINE {
    int s = step_of(ld.part, H * i);
    s = s + H <= nsteps ? s : nsteps - H;
    const uint32_t at = (uint32_t)first(ld.chunk) * rowq + (s < 0 ? 0 : s) * (16 * BITS);
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int d = 0; d < 2; ++d)
        dma16(codes, buffer(b) + (r * 2 + d) * 64, vq[r][d], at);
  };
  // Buffer b's codes into registers: this lane's 32 channels of weight row c16 of every tile and
  // step (stream_words). The DMAs sent after buffer b's are those of the other buffers, so
  // vmcnt(their number) covers buffer b whatever else was sent in between; the LDS reads end before
  // the block does.
  constexpr int kLater = (NB - 1) * R * 2;
  const int swz = c16 >> 1;
  auto take_codes = [&](int b, bool more, uint32_t (&w)[H][R][W]) AWQ_INLINE {
    if (more)
      asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kLater) : "memory");
    else  // nothing is sent behind the last position's
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    const uint32_t at = (uint32_t)(uintptr_t)(lds_void*)buffer(b);
    if constexpr (BITS == 3) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const uint32_t row = at + r * 2048 + c16 * 96;
        if constexpr (GS == 1) {
#pragma unroll
          for (int h = 0; h < H; ++h) {
            uint2 lo;
            asm volatile("ds_read_b64 %0, %2\n\tds_read_b32 %1, %3\n\ts_waitcnt lgkmcnt(0)"
                         : "=&v"(lo), "=&v"(w[h][r][2])
                         : "v"(row + h * 48 + kg * 8), "v"(row + h * 48 + 32 + kg * 4)
                         : "memory");
            w[h][r][0] = lo.x;
            w[h][r][1] = lo.y;
          }
        } else {
          // slice i of a step: half of low word 2 i + kg / 2 and a quarter of high word i
          uint2 lo[4];
          u32x4 hi[2];
          asm volatile(
              "ds_read2_b32 %0, %6 offset0:0 offset1:2\n\tds_read2_b32 %1, %6 offset0:4 offset1:6\n\t"
              "ds_read2_b32 %2, %6 offset0:12 offset1:14\n\tds_read2_b32 %3, %6 offset0:16 offset1:18\n\t"
              "ds_read_b128 %4, %7\n\tds_read_b128 %5, %7 offset:48\n\ts_waitcnt lgkmcnt(0)"
              : "=&v"(lo[0]), "=&v"(lo[1]), "=&v"(lo[2]), "=&v"(lo[3]), "=&v"(hi[0]), "=&v"(hi[1])
              : "v"(row + (kg >> 1) * 4), "v"(row + 32)
              : "memory");
#pragma unroll
          for (int h = 0; h < H; ++h)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t low = (i & 1 ? lo[2 * h + (i >> 1)].y : lo[2 * h + (i >> 1)].x) >> (8 * (kg & 1));
              const uint32_t high = __builtin_amdgcn_alignbit(hi[h][i], hi[h][i], (4 * kg - 8) & 31);
              w[h][r][i] = (low & 0xF0FFF0FFu) | (high & 0x0F000F00u);
            }
        }
      }
    } else {
      // both steps (8-bit: the step) of two tiles per block: their reads in flight together
#pragma unroll
      for (int r = 0; r < R; r += 2) {
        const uint32_t row = at + r * 2048 + c16 * 128;
        if constexpr (BITS == 8 && GS == 1) {
          u32x4 v[4];
          asm volatile(
              "ds_read_b128 %0, %4\n\tds_read_b128 %1, %5\n\tds_read_b128 %2, %4 offset:2048\n\t"
              "ds_read_b128 %3, %5 offset:2048\n\ts_waitcnt lgkmcnt(0)"
              : "=&v"(v[0]), "=&v"(v[1]), "=&v"(v[2]), "=&v"(v[3])
              : "v"(row + ((2 * kg) ^ swz) * 16), "v"(row + ((2 * kg + 1) ^ swz) * 16)
              : "memory");
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) w[0][r + (i >> 1)][4 * (i & 1) + k] = v[i][k];
        } else if constexpr (BITS == 8) {
          // slice i: 8 bytes of piece 2 i + kg / 2
          const uint32_t half = row + (kg & 1) * 8;
          u32x4 v[4];
          asm volatile(
              "ds_read2st64_b64 %0, %4 offset0:0 offset1:4\n\tds_read2st64_b64 %1, %5 offset0:0 offset1:4\n\t"
              "ds_read2st64_b64 %2, %6 offset0:0 offset1:4\n\tds_read2st64_b64 %3, %7 offset0:0 offset1:4\n\t"
              "s_waitcnt lgkmcnt(0)"
              : "=&v"(v[0]), "=&v"(v[1]), "=&v"(v[2]), "=&v"(v[3])
              : "v"(half + ((kg >> 1) ^ swz) * 16), "v"(half + ((2 + (kg >> 1)) ^ swz) * 16),
                "v"(half + ((4 + (kg >> 1)) ^ swz) * 16), "v"(half + ((6 + (kg >> 1)) ^ swz) * 16)
              : "memory");
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) w[0][r + (k >> 1)][2 * i + (k & 1)] = v[i][k];
        } else if constexpr (GS == 1) {
          u32x4 v[4];
          asm volatile(
              "ds_read_b128 %0, %4\n\tds_read_b128 %1, %5\n\tds_read_b128 %2, %4 offset:2048\n\t"
              "ds_read_b128 %3, %5 offset:2048\n\ts_waitcnt lgkmcnt(0)"
              : "=&v"(v[0]), "=&v"(v[1]), "=&v"(v[2]), "=&v"(v[3])
              : "v"(row + (kg ^ swz) * 16), "v"(row + ((4 + kg) ^ swz) * 16)
              : "memory");
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) w[i & 1][r + (i >> 1)][k] = v[i][k];
        } else {
          // slice i of step h: word kg of piece 4 h + i
          const uint32_t word = row + kg * 4;
          uint2 v[8];
          asm volatile(
              "ds_read2st64_b32 %0, %8 offset0:0 offset1:8\n\tds_read2st64_b32 %1, %9 offset0:0 offset1:8\n\t"
              "ds_read2st64_b32 %2, %10 offset0:0 offset1:8\n\tds_read2st64_b32 %3, %11 offset0:0 offset1:8\n\t"
              "ds_read2st64_b32 %4, %12 offset0:0 offset1:8\n\tds_read2st64_b32 %5, %13 offset0:0 offset1:8\n\t"
              "ds_read2st64_b32 %6, %14 offset0:0 offset1:8\n\tds_read2st64_b32 %7, %15 offset0:0 offset1:8\n\t"
              "s_waitcnt lgkmcnt(0)"
              : "=&v"(v[0]), "=&v"(v[1]), "=&v"(v[2]), "=&v"(v[3]), "=&v"(v[4]), "=&v"(v[5]), "=&v"(v[6]), "=&v"(v[7])
              : "v"(word + (0 ^ swz) * 16), "v"(word + (1 ^ swz) * 16), "v"(word + (2 ^ swz) * 16),
                "v"(word + (3 ^ swz) * 16), "v"(word + (4 ^ swz) * 16), "v"(word + (5 ^ swz) * 16),
                "v"(word + (6 ^ swz) * 16), "v"(word + (7 ^ swz) * 16)
              : "memory");
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            w[i >> 2][r][i & 3] = v[i].x;
            w[i >> 2][r + 1][i & 3] = v[i].y;
          }
        }
      }
    }
  };
  struct ScaleZero {
    Eight sc[GS], z[BITS == 8 && GS == 4 ? 2 : 1];  // eight bytes: the scales of a group of all four steps
  };
  auto load_scales = [&](ScaleZero& q) AWQ_INLINE {
    int s = step_of(ld.part, 0);
    s = s < nsteps ? s : 0;
    const int64_t n = expert_row + first(ld.chunk) + my_row;
    const int64_t as = (n * Gs + s * GS) * 2, az = n * zbw + (BITS == 8 ? s * GS : s * GS / 2);
#pragma unroll
    for (int i = 0; i < GS; ++i) q.sc[i] = load8(g.scales, as + 8 * i, sbytes);
    q.z[0] = load8(g.zeros, az, zbytes);
    if constexpr (BITS == 8 && GS == 4) q.z[1] = load8(g.zeros, az + 8, zbytes);
  };

  half8w a[L][4];  // this wave's part of the tile's rows of X
  auto load_x = [&](const StreamItem& it) AWQ_INLINE {
    const int r = c16;  // rows past the last read the last one, never stored
    int xr = it.rows > 0 ? source(it.row0 + (r < it.rows ? r : it.rows - 1)) : 0;
    if (MODE != kLora && g.order) xr = (int)((unsigned)xr / (unsigned)g.fan);
    constexpr int kOwn = GS == 1 ? 32 : 8, kSlice = GS == 1 ? 8 : 32;  // channels between lanes, between slices
    const uint16_t* const x = g.X + (int64_t)xr * K + kg * kOwn;
#pragma unroll
    for (int j = 0; j < L; ++j) {
      const int s = step_of(it.part, j);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a[j][i] = *reinterpret_cast<const half8w*>(x + (s < nsteps ? s : nsteps - 1) * kGroup + i * kSlice);
        if (s >= nsteps) a[j][i] = half8w{};  // steps past the last add nothing
      }
    }
  };

  f32x4w acc[R];
  auto clear = [&]() AWQ_INLINE {
#pragma unroll
    for (int r = 0; r < R; ++r) acc[r] = f32x4w{0.0f, 0.0f, 0.0f, 0.0f};
  };
  // The scales and zeros of the wave's steps as this lane loaded them, and their 32-bit words for
  // this lane's weight row of tile r, from the lane that loaded that: all at once where they are few
  // (128-channel groups), else when they are used (all of them would take the registers of a tile).
  constexpr int kScaleWords = L * GS / 2, kZeroWords = BITS == 8 ? L * GS / 4 : (L * GS + 7) / 8;
  struct Steps {
    uint64_t sc[(kScaleWords + 1) / 2], z[(kZeroWords + 1) / 2];
    uint32_t sc_of[GS == 1 ? R : 1][kScaleWords], z_of[GS == 1 ? R : 1][kZeroWords];
  };
  auto fetch = [&](const uint64_t* e, int word, int r) AWQ_INLINE -> uint32_t {
    return (uint32_t)__builtin_amdgcn_ds_bpermute((r * 16 + c16) * 4, (int)(uint32_t)(e[word / 2] >> (32 * (word & 1))));
  };
  auto take_scales = [&](Steps& f, const ScaleZero& q) AWQ_INLINE {
#pragma unroll
    for (int i = 0; i < (kScaleWords + 1) / 2; ++i) f.sc[i] = q.sc[i].value();
#pragma unroll
    for (int i = 0; i < (kZeroWords + 1) / 2; ++i) f.z[i] = q.z[i].value();
    if constexpr (GS == 1) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
#pragma unroll
        for (int i = 0; i < kScaleWords; ++i) f.sc_of[r][i] = fetch(f.sc, i, r);
#pragma unroll
        for (int i = 0; i < kZeroWords; ++i) f.z_of[r][i] = fetch(f.z, i, r);
      }
    }
  };
  auto scale_word = [&](const Steps& f, int word, int r) AWQ_INLINE -> uint32_t {
    return GS == 1 ? f.sc_of[GS == 1 ? r : 0][word] : fetch(f.sc, word, r);
  };
  auto zero_word = [&](const Steps& f, int word, int r) AWQ_INLINE -> uint32_t {
    return GS == 1 ? f.z_of[GS == 1 ? r : 0][word] : fetch(f.z, word, r);
  };
  // Step j of the wave's part, codes w; on: the step exists. The R weight tiles are independent
  // chains, walked side by side.
  auto multiply = [&](const uint32_t (&w)[R][W], int j, bool on, const Steps& q) AWQ_INLINE {
#pragma unroll
    for (int gi = 0; gi < GS; ++gi) {
      const int at = j * GS + gi;  // the group among those of the wave's steps
      f32x4w d[R];
      float f[R];
      ZeroPair zp[R];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const uint32_t sc = scale_word(q, at / 2, r) >> (16 * (at & 1));
        f[r] = on ? h2f((uint16_t)sc) : 0.0f;
        zp[r] = zero_pair(BITS == 8 ? (zero_word(q, at / 4, r) >> (8 * (at & 3))) & 0xFF : (zero_word(q, at / 8, r) >> (4 * (at & 7))) & 0xF);
        d[r] = f32x4w{0.0f, 0.0f, 0.0f, 0.0f};
      }
#pragma unroll
      for (int s = gi * 4 / GS; s < (gi + 1) * 4 / GS; ++s)
#pragma unroll
        for (int r = 0; r < R; ++r)
          d[r] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a[j][s], centered<BITS>(w[r], s, zp[r], magic), d[r], 0, 0, 0);
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[r][i] = __builtin_fmaf(f[r], d[r][i], acc[r][i]);
    }
    if constexpr (GS > 1) {  // (left to itself the compiler takes the sums a step later and spills the partial tiles)
#pragma unroll
      for (int r = 0; r < R; ++r) asm volatile("" : "+v"(acc[r]));
    }
  };
  // Adapters among the tile's rows in order of their first row, shared by the waves: their
  // terms start the accumulators, while the item's codes are on their way.
  auto adapters = [&](const StreamItem& it) AWQ_INLINE {
    int src, id;
    bool open;
    const int r = c16;
    src = source(it.row0 + (r < it.rows ? r : it.rows - 1));
    id = r < it.rows ? g.ids[src] : -1;
    open = (unsigned)id < (unsigned)g.groups;
    const int blocks = (g.rank + kLoraBlock - 1) / kLoraBlock;
    // the next adapter whose turn is this wave's, -1 after the last
    int turn = 0;
    auto pick = [&]() AWQ_INLINE -> int {
      while (true) {
        const uint64_t m = __ballot(open);
        if (!m) return -1;
        const int ad = __builtin_amdgcn_readlane(id, __ffsll((unsigned long long)m) - 1);
        open = open && id != ad;
        const bool hit = turn == wave;
        turn = turn + 1 < S ? turn + 1 : 0;
        if (hit) return ad;
      }
    };
    struct Term {
      half8w b[R], hi, lo;
      float f;
    };
    auto load_term = [&](Term& u, int ad, int k) AWQ_INLINE {
      const uint16_t* const B = g.B + ((int64_t)ad * N + first(it.chunk)) * g.rank;
      const int at = k * kLoraBlock + kg * 8;
#pragma unroll
      for (int r = 0; r < R; ++r)
        u.b[r] = at < g.rank ? *reinterpret_cast<const half8w*>(B + (int64_t)weight_row(r * 16 + c16) * g.rank + at)
                             : half8w{};
      const LoraRow* const h = g.H + (int64_t)src * blocks + k;
      const bool mine = id == ad;
      u.hi = mine ? *reinterpret_cast<const half8w*>(h->hi + kg * 8) : half8w{};
      u.lo = mine ? *reinterpret_cast<const half8w*>(h->lo + kg * 8) : half8w{};
      u.f = mine ? h->f : 0.0f;
    };
    int ad = pick(), k = 0;
    if (ad < 0) return;
    Term u;
    load_term(u, ad, k);
    while (ad >= 0) {
      int ad2 = ad, k2 = k + 1;
      if (k2 == blocks) {
        k2 = 0;
        ad2 = pick();
      }
      Term v;
      if (ad2 >= 0) load_term(v, ad2, k2);
      const uint64_t rows_of = __ballot(id == ad);
      float fr[4];
      bool on[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        fr[i] = __shfl(u.f, 4 * kg + i);
        on[i] = (rows_of >> (4 * kg + i)) & 1;
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        f32x4w d{0.0f, 0.0f, 0.0f, 0.0f};
        d = __builtin_amdgcn_mfma_f32_16x16x32_f16(u.hi, u.b[r], d, 0, 0, 0);
        d = __builtin_amdgcn_mfma_f32_16x16x32_f16(u.lo, u.b[r], d, 0, 0, 0);
        // only the adapter's own rows: an Inf or NaN of its B stays out of the others
#pragma unroll
        for (int i = 0; i < 4; ++i)
          acc[r][i] = on[i] ? __builtin_fmaf(fr[i], d[i], acc[r][i]) : acc[r][i];
      }
      u = v;
      ad = ad2;
      k = k2;
    }
  };
  // A barrier for LDS data alone: the DMAs in flight stay in flight.
  auto meet = [&]() AWQ_INLINE { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); };
  // The waves' partial tiles summed in a fixed order and stored. Accumulator layout: element i
  // of lane l is (row 4 (l / 16) + i, column l % 16).
  auto finish = [&](const StreamItem& it) AWQ_INLINE {
    constexpr int RO = MODE == kGated ? R / 2 : R;  // output tiles
    const int col0 = first(it.chunk) + c16;
    auto sum = [&](int tile) AWQ_INLINE {
      f32x4w v = red[tile * 64 + lane];
#pragma unroll
      for (int i = 1; i < S; ++i) v += red[(i * R + tile) * 64 + lane];
      return v;
    };
#pragma unroll
    for (int r = 0; r < R; ++r) red[(wave * R + r) * 64 + lane] = acc[r];
    meet();
    for (int r = wave; r < RO; r += S) {
      f32x4w v = sum(r);
      if constexpr (MODE == kGated) {
        const f32x4w up = sum(r + RO);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = silu_f32(v[i]) * up[i];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = 4 * kg + i;
        if (row < it.rows && r * 16 + c16 < outs) {
          const int64_t yr = MODE == kLora ? source(it.row0 + row) : it.row0 + row;
          g.Y[yr * outs + col0 + r * 16] = f2h_bits(v[i]);
        }
      }
    }
    meet();  // before the next partial tiles
    clear();
  };

  clear();
  open_tile();
  StreamItem it = ld;
  ScaleZero q;
  load_scales(q);
#pragma unroll
  for (int i = 0; i < L / H; ++i) load_codes(i, i);
  load_x(it);
  while (true) {
    const bool more = todo > 1;
    Steps f;
    take_scales(f, q);
    if (more) {
      next();  // ld is a position ahead of it
      load_scales(q);
    }
    if (MODE == kLora && it.part == 0) adapters(it);
#pragma unroll
    for (int i = 0; i < L / H; ++i) {
      uint32_t w[H][R][W];
      take_codes(i, more, w);
      if (more) load_codes(i, i);
#pragma unroll
      for (int h = 0; h < H; ++h) {
        const int s = step_of(it.part, H * i + h);
        if constexpr (H > 1) {
          // an odd last step lies in the second half of its buffer, loaded from one step earlier
          if (h == 0 && s + 1 == nsteps && nsteps > 1) {
            asm volatile("");  // a branch: not a select per word on every step
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
              for (int k = 0; k < W; ++k) w[0][r][k] = w[H - 1][r][k];
          }
        }
        multiply(w[h], H * i + h, s < nsteps, f);
      }
    }
    if (it.part == parts - 1) finish(it);
    if (--todo == 0) break;
    const int tile = it.tile;
    it = ld;
    if (parts > 1 || it.tile != tile) load_x(it);
  }
}

// The variants that the launcher picks from: s waves.
template <int MODE, int BITS, int GS, int R>
void launch_stream_r(const GroupedArgs& g, int s, dim3 grid, hipStream_t stream) {
  constexpr int L = kStreamSteps;
  if (s == 2)
    hipLaunchKernelGGL((k_stream<MODE, BITS, GS, R, L, 2>), grid, dim3(128), 0, stream, g);
  else if (s == 4)
    hipLaunchKernelGGL((k_stream<MODE, BITS, GS, R, L, 4>), grid, dim3(256), 0, stream, g);
  else
    hipLaunchKernelGGL((k_stream<MODE, BITS, GS, R, L, 8>), grid, dim3(512), 0, stream, g);
}

template <int MODE, int BITS, int GS>
void launch_stream_g(const GroupedArgs& g, bool narrow, int s, dim3 grid, hipStream_t stream) {
  constexpr int R = stream_cols(BITS, false) / 16, kNarrow = stream_cols(BITS, true) / 16;
  if (narrow) launch_stream_r<MODE, BITS, GS, kNarrow>(g, s, grid, stream);
  else launch_stream_r<MODE, BITS, GS, R>(g, s, grid, stream);
}

template <int MODE, int BITS>
void launch_stream_t(const GroupedArgs& g, bool narrow, int s, dim3 grid, hipStream_t stream) {
  if (g.group == 128) launch_stream_g<MODE, BITS, 1>(g, narrow, s, grid, stream);
  else if (g.group == 64) launch_stream_g<MODE, BITS, 2>(g, narrow, s, grid, stream);
  else launch_stream_g<MODE, BITS, 4>(g, narrow, s, grid, stream);
}

}  // namespace awq
