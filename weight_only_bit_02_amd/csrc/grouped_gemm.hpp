// MFMA dequant-GEMM on ragged rows: the products of a batch in group order with one packed
// weight per group (experts), or with one shared weight and a low-rank term per row
// (adapters). One template; each instantiation is compiled in its own grouped_*.hip.
//
// Experts: Y[p] = X[x(p)] deq(W_e)^T for offsets[e] <= p < offsets[e + 1]; x(p) = p, or
// order[p] / fan when the rows are gathered (fan = choices per token). The host knows only
// the number of rows: the grid covers the most tiles they can need, every block counts the
// tiles there are from the offsets (one wave scan per 64 groups) and takes its own, or ends.
//
// Tile RTM x 32 rows x 256 columns, K step 128, four waves side by side along the columns,
// each owning all rows x 64 columns (v_mfma_f32_32x32x16_f16), so a column is widened once
// per tile. Both operands go global -> LDS by 16-byte DMA, up to NS - 1 steps ahead in a ring
// of NS buffers that fills LDS (a step of a 64-row tile is multiplied in a quarter of the time
// that its operands take to arrive: with two buffers 256 x 4096 x 4096 took 64 us, a step each
// memory latency; with five 46). A's DMA takes a row address per lane, so gathering costs
// nothing. A row's 16 chunks are stored in slots c ^ (row % 16) and codes quarter-major: both
// are read without bank conflicts. A tile with fewer rows runs a body with fewer row tiles (a
// power of two), so a group's last tile costs the matrix work of the rows it has.
//
// A step is eight slices of 16 channels. While a slice is multiplied, the next one is read and
// widened between the products, across the barrier too: it stands before the last slice.
//
// One barrier per step, with a wait of its own for the DMAs of the step that begins
// (__syncthreads would wait for those of all steps). The DMAs are written as instructions: of
// the builtin's the compiler waits for every one in flight before each read of LDS.
//
// RTM = 8 (not with 8-bit codes: LDS holds no more) serves large groups, 4 middling ones or
// grids that would leave CUs idle, 2 small ones. KW = 4: 64 columns, K steps dealt to the four
// waves, each with a ring of its own and no barrier, sums joined in LDS in the waves' order: four
// times the blocks for batches whose tiles would leave the chip idle, at four times A's traffic
// (64 rows x 4096 x 4096 with adapters 61 us -> 24). grouped_gemm.hip picks.
//
// What bounds it: large groups, the issue of one wave per SIMD (matrix cores 44% busy, vector
// instructions 23%) and the chip's power: 8 experts x 22016 x 4096 gated, 8192 rows, 1586 us in a
// row of them, 932 TFLOP/s (a library fp16 product of 8192^3 reaches 1323). Middling
// groups, the widening, whose cost does not depend on the rows. K of few steps, a tile's start:
// offsets, row indices, first operands, 4 to 5 us before the first product.
//
// Operand values ((q - z) sc rounded to fp16 once) and, for KW = 1, their order along K are those
// of the 256-row GEMM, so an expert's rows equal the plain linear's bit for bit where that runs
// its GEMM. The rounding costs 2^-11 relative per weight at most, some 1.8e-4 of a sum of many
// random terms, beside 2.1e-4 of the output's own rounding (2.7 to 2.9e-4 together); the gated
// form, which has it in both factors, comes to 3.3e-4 where exact weights give 2.1e-4. (Scaling the
// sums in fp32 instead, as grouped_stream.hpp does, takes a second set of sums: 256 rows have no
// registers for it.)
//
// Adapters (MODE kLora): the rows of one batch, optionally through `order` (then Y is
// scattered back through it). After the K loop the rows' adapters are walked one by one, H B_a^T
// (H = scale X A_a^T from the first product's kernel, as fp16 hi + lo under a power of two) is
// added to their own rows, and the next adapter's B is on its way meanwhile.
#pragma once

#include <type_traits>

#include "common.hpp"
#include "groups.hpp"
#include "launch.hpp"
#include "widen.hpp"

namespace awq {


constexpr int kGN = 256, kGK = 128;   // columns of a tile, channels of a K step
constexpr int kGroupedTiles = 4;      // row tiles that share a column panel in the tile order

// G32: 32-channel groups (else 128 or 64). KW: waves along K (1: four along the columns; 4).
template <int MODE, int RTM, int BITS, bool G32, int KW>
__global__ void __launch_bounds__(256) k_grouped(GroupedArgs g) {
  constexpr int BM = RTM * 32, BN = kGN / KW;
  constexpr int kQ = BITS;   // 16-byte quarters of a column's codes per step
  constexpr int kBT = kQ;    // B transfers per wave and step
  constexpr int kBuf = BM * 16 + BN * kQ;  // 16-byte slots of a buffer: A, then codes
  constexpr int kFit = 160 * 1024 / 16 / KW / kBuf, NS = kFit < 5 ? kFit : 5;
  static_assert(NS >= 2, "two buffers fit LDS");
  __shared__ __attribute__((aligned(16))) uint4 lds[KW * NS * kBuf];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int m32 = lane & 31, kh = lane >> 5;
  const int64_t N = g.N, K = g.K, nh = N / 2;
  // this wave among those that share its ring, among those along the columns and along K
  const int part = KW == 1 ? wave : 0, kw = KW == 1 ? 0 : wave;
  uint4* const ring = lds + kw * (NS * kBuf);
  const uint32_t ring_at = lds_address(lds) + kw * (NS * kBuf * 16);

  // ---- this block's tile: XCD blockIdx % 8 takes a contiguous run of the tiles there are
  const int mt = MODE == kLora ? (g.n + BM - 1) / BM : __builtin_amdgcn_readfirstlane(count_tiles<BM>(g.offsets, g.groups, g.n, lane));
  const int64_t tiles = (int64_t)mt * g.nt, per_xcd = (tiles + 7) / 8;
  const int64_t slot = blockIdx.x / 8, t = (int64_t)(blockIdx.x % 8) * per_xcd + slot;
  if (slot >= per_xcd || t >= tiles) return;
  const int first_m = (int)(t / ((int64_t)kGroupedTiles * g.nt)) * kGroupedTiles;
  const int gsz = mt - first_m < kGroupedTiles ? mt - first_m : kGroupedTiles;
  const int within = (int)(t - (int64_t)first_m * g.nt);
  const int64_t n0 = (int64_t)(within / gsz) * (MODE == kGated ? BN / 2 : BN);
  const int at = first_m + within % gsz;
  const RowTile rt = MODE == kLora ? RowTile{0, at * BM, g.n - at * BM < BM ? g.n - at * BM : BM}
                                   : find_tile<BM>(g.offsets, g.groups, g.n, at, lane);
  const int row0 = __builtin_amdgcn_readfirstlane(rt.row0), rows = __builtin_amdgcn_readfirstlane(rt.rows);
  const int64_t e = MODE == kLora ? 0 : __builtin_amdgcn_readfirstlane(rt.e);
  if (rows <= 0) return;

  const int g64 = g.group == 64;
  const int64_t Gs = K / g.group, zbw = BITS == 8 ? Gs : (Gs + 1) / 2, words = K * BITS / 32;
  const int ksteps = (int)(K / kGK), nsteps = (ksteps - kw + KW - 1) / KW;  // all, this wave's
  const uint32_t* const qweight = g.qweight + e * N * words;
  const uint16_t* const scales = g.scales + e * N * Gs;
  const uint8_t* const zeros = g.zeros + e * N * zbw;
  const uint32_t magic = wide_magic();
  uint32_t magic8 = 0;
  if constexpr (BITS == 8) asm volatile("v_mov_b32 %0, 0x64646464" : "=v"(magic8));

  // the row that order names for position p of the batch (anything out of range: row 0)
  auto source = [&](int p) -> int {
    if (!g.order) return p;
    const int o = g.order[p];
    return (unsigned)o < (unsigned)g.n ? o : 0;
  };

  // B DMA map, quarter-major: slot (part * kBT + i) * 64 + lane = 16-byte quarter slot / BN
  // of tile column slot % BN. Gated: tile columns [64 w, 64 w + 32) hold the gate rows and
  // [64 w + 32, 64 w + 64) the up rows of outputs n0 + 32 w ... Columns past the end read the
  // last one (never stored).
  uint32_t boff[kBT];
  const u32x4 W = buffer_words(qweight);
#pragma unroll
  for (int i = 0; i < kBT; ++i) {
    const int s = (part * kBT + i) * 64 + lane;
    const int c = s % BN, q = s / BN;
    int64_t n;
    if constexpr (MODE == kGated) {
      int64_t o = n0 + (c >> 6) * 32 + (c & 31);
      o = o < nh ? o : nh - 1;
      n = (c & 63) >= 32 ? o + nh : o;
    } else {
      n = n0 + c < N ? n0 + c : N - 1;
    }
    boff[i] = (uint32_t)(n * words + q * 4) * 4;
  }
  // this lane's weight rows (gated: gate row and up row): scales and zeros
  int64_t bcol[2];
  if constexpr (MODE == kGated) {
    const int64_t o = n0 + part * 32 + m32;
    bcol[0] = o < nh ? o : nh - 1;
    bcol[1] = bcol[0] + nh;
  } else {
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int64_t n = n0 + part * 64 + b * 32 + m32;
      bcol[b] = n < N ? n : N - 1;
    }
  }
  // per column, the zero(s) and scale(s) of the lane half's 64 channels of a step: one group
  // of 128 (step) or 64 (2 step + kh), or two of 32 (4 step + 2 kh and the next)
  constexpr int kZ = G32 ? 2 : 1;
  struct ScaleZero {
    uint32_t zb[2][BITS == 8 ? kZ : 1], sc[2][kZ];
  };
  auto load_sz = [&](ScaleZero& st, int own) {
    const int64_t step = own * KW + kw < ksteps ? own * KW + kw : ksteps - 1;
    const int64_t g0 = G32 ? 4 * step + 2 * kh : g64 ? 2 * step + kh : step;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
#pragma unroll
      for (int i = 0; i < (BITS == 8 ? kZ : 1); ++i)
        st.zb[b][i] = zeros[bcol[b] * zbw + (BITS == 8 ? g0 + i : g0 >> 1)];
#pragma unroll
      for (int i = 0; i < kZ; ++i) st.sc[b][i] = scales[bcol[b] * Gs + g0 + i];
    }
  };

  // Adapters: adds the adapters' terms of T tiles of 32 rows from r0 on to their accumulators,
  // one adapter after the other by first row (waves along K share them), the next one's B on its
  // way meanwhile.
  auto add_adapters = [&](int r0, auto tc, auto acc_of) __attribute__((always_inline)) {
    constexpr int T = decltype(tc)::value;
    int src[T], id[T];
#pragma unroll
    for (int a = 0; a < T; ++a) {
      const int r = r0 + a * 32 + m32;
      src[a] = source(row0 + (r < rows ? r : rows - 1));
    }
#pragma unroll
    for (int a = 0; a < T; ++a) id[a] = g.ids[src[a]];
    const int blocks = (g.rank + kLoraBlock - 1) / kLoraBlock;
    for (int k = 0; k < blocks; ++k) {
      half8w hi[T][2], lo[T][2];
      float f[T];
      bool todo[T];
#pragma unroll
      for (int a = 0; a < T; ++a) {
        const LoraRow* const h = g.H + (int64_t)src[a] * blocks + k;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          hi[a][s] = *reinterpret_cast<const half8w*>(h->hi + s * 16 + kh * 8);
          lo[a][s] = *reinterpret_cast<const half8w*>(h->lo + s * 16 + kh * 8);
        }
        f[a] = h->f;
        if (k == 0 && r0 + a * 32 + m32 >= rows) id[a] = -1;
        todo[a] = (unsigned)id[a] < (unsigned)g.groups;
      }
      int turn = 0;
      auto pick = [&]() __attribute__((always_inline)) -> int {  // the next adapter, -1 after the last
        while (true) {
          int ad = -1;
#pragma unroll
          for (int a = 0; a < T; ++a) {
            const uint64_t m = __ballot(todo[a]);
            if (ad < 0 && m) ad = __builtin_amdgcn_readlane(id[a], __ffsll((unsigned long long)m) - 1);
          }
          if (ad < 0) return -1;
#pragma unroll
          for (int a = 0; a < T; ++a) todo[a] = todo[a] && id[a] != ad;
          const bool hit = turn == kw;
          turn = turn + 1 < KW ? turn + 1 : 0;
          if (hit) return ad;
        }
      };
      struct Weights {
        half8w w[2][2];
      };
      auto load_b = [&](Weights& v, int ad) __attribute__((always_inline)) {
        const uint16_t* const B = g.B + (int64_t)ad * N * g.rank + k * kLoraBlock + kh * 8;
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int b = 0; b < 2; ++b)
            v.w[s][b] = k * kLoraBlock + s * 16 + kh * 8 < g.rank
                            ? *reinterpret_cast<const half8w*>(B + bcol[b] * g.rank + s * 16)
                            : half8w{};
      };
      int ad = pick();
      if (ad < 0) return;
      Weights now;
      load_b(now, ad);
      while (ad >= 0) {
        const int ad2 = pick();
        Weights then;
        if (ad2 >= 0) load_b(then, ad2);
#pragma unroll
        for (int a = 0; a < T; ++a) {
          const bool mine = id[a] == ad;
          const uint32_t rows_of = (uint32_t)__ballot(mine);
          if (!rows_of) continue;
          f32x16w d[2] = {f32x16w{}, f32x16w{}};
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            const half8w h = mine ? hi[a][s] : half8w{}, l = mine ? lo[a][s] : half8w{};
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              d[b] = __builtin_amdgcn_mfma_f32_32x32x16_f16(h, now.w[s][b], d[b], 0, 0, 0);
              d[b] = __builtin_amdgcn_mfma_f32_32x32x16_f16(l, now.w[s][b], d[b], 0, 0, 0);
            }
          }
          f32x16w* const acc = acc_of(a);
          const uint32_t rows_kh = rows_of >> (4 * kh);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            // only the adapter's own rows: an Inf or NaN of its B stays out of the others
            const int ri = 8 * (i >> 2) + (i & 3);
            const float fr = __shfl(f[a], ri + 4 * kh);
            const bool on = (rows_kh >> ri) & 1;
#pragma unroll
            for (int b = 0; b < 2; ++b) acc[b][i] = on ? __builtin_fmaf(fr, d[b][i], acc[b][i]) : acc[b][i];
          }
        }
        now = then;
        ad = ad2;
      }
    }
  };

  // RT row tiles of 32 rows cover this tile's rows.
  auto run = [&](auto rtc) {
    constexpr int RT = decltype(rtc)::value;
    constexpr int kAT = 2 * RT * KW;  // A transfers per wave and step
    // A DMA map: wave transfer i fills slots (part * kAT + i) * 64 + lane: row r = (part * kAT
    // + i) * 4 + lane / 16, slot lane % 16 <- chunk (lane % 16) ^ (r % 16), as offsets in X (the
    // host admits X below 2^32 bytes). Rows past the last read the last one.
    uint32_t aoff[kAT];
#pragma unroll
    for (int i = 0; i < kAT; ++i) {
      const int r = (part * kAT + i) * 4 + (lane >> 4);
      int x = source(row0 + (r < rows ? r : rows - 1));
      if (MODE != kLora && g.order) x = (int)((unsigned)x / (unsigned)g.fan);
      aoff[i] = (uint32_t)x * (uint32_t)(K * 2) + ((lane & 15) ^ (r & 15)) * 16;
    }
    const u32x4 X = buffer_words(g.X);

    f32x16w acc[RT][2];
#pragma unroll
    for (int a = 0; a < RT; ++a)
#pragma unroll
      for (int b = 0; b < 2; ++b) acc[a][b] = f32x16w{};

    // A slice's products go in kGroups groups of four (RT > 1). Share i of kShares of this wave's
    // DMAs of step `step` into buffer c, if there is such a step, at every kEvery-th group. 256
    // rows send one or two per group (more at once fill the address units' queue, and the products
    // behind them wait: 256 rows x 4096 x 4096 with adapters 136 us in two shares, 122 so); fewer
    // rows are shorter of time than of issue slots and send two halves early (128 rows 73 and 76).
    constexpr int kGroups = RT >= 4 ? RT / 2 : 1, kSends = kAT + kBT;
    constexpr int kShares = RT == 8 ? 6 * kGroups : 2, kEvery = RT == 8 ? 1 : 2 * kGroups;
    auto send = [&](auto c, int step, int i) __attribute__((always_inline)) {
      if (step >= nsteps) return;
      const uint32_t at = (uint32_t)(step * KW + kw);
      const uint32_t to = ring_at + decltype(c)::value * (kBuf * 16);
#pragma unroll
      for (int k = i * kSends / kShares; k < (i + 1) * kSends / kShares; ++k) {
        if (k < kAT)
          dma16_own(X, to + (part * kAT + k) * 1024, aoff[k], at * 256);
        else
          dma16_own(W, to + BM * 256 + (part * kBT + k - kAT) * 1024, boff[k - kAT], at * (kQ * 16));
      }
    };
    // Step `step`'s data has landed: all but the DMAs of the NS - 2 steps after it (other loads in
    // between only make the wait longer), in every wave of the ring, and the reads so far are done.
    auto arrive = [&](int step) __attribute__((always_inline)) {
      if (step + NS - 2 < nsteps)
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"((NS - 2) * kSends) : "memory");
      else
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
      if constexpr (KW == 1) asm volatile("s_barrier" ::: "memory");
    };

    // State of a step: zeros and scales of the lane's columns, widened to pairs; its code words, per
    // column: 4- and 8-bit, the quarters kQ / 2 kh ..; 3-bit, low-plane words 4 kh .. (quarter kh)
    // and high-plane words 8 + 2 kh, 9 + 2 kh
    constexpr int kQL = BITS == 3 ? 1 : kQ / 2;
    half2w zz[2][kZ], zz64[2][kZ], s2[2][kZ];
    uint4 bq[2][kQL];
    uint2 bh[2];
    auto open_step = [&](const ScaleZero& cur, const uint4* bb, int step) __attribute__((always_inline)) {
      const int hi = g64 ? kh : (step * KW + kw) & 1;  // zero nibble: group of 128 (step) or 64 (2 step + kh)
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int i = 0; i < kZ; ++i) {
          uint32_t z;
          if constexpr (BITS == 8)
            z = cur.zb[b][i];
          else
            z = (cur.zb[b][0] >> (4 * (G32 ? i : hi))) & 0xF;
          const uint32_t z1024 = 0x6400u + z, z64 = 0x5400u + (z << 4);
          zz[b][i] = -__builtin_bit_cast(half2w, z1024 | (z1024 << 16));
          zz64[b][i] = -__builtin_bit_cast(half2w, z64 | (z64 << 16));
          s2[b][i] = __builtin_bit_cast(half2w, cur.sc[b][i] | (cur.sc[b][i] << 16));
        }
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int col = part * 64 + b * 32 + m32;
        if constexpr (BITS == 3) {
          bq[b][0] = bb[kh * BN + col];
          const uint4 h4 = bb[2 * BN + col];
          bh[b] = kh ? make_uint2(h4.z, h4.w) : make_uint2(h4.x, h4.y);
        } else {
#pragma unroll
          for (int h = 0; h < kQL; ++h) bq[b][h] = bb[(kQL * kh + h) * BN + col];
        }
      }
    };
    auto rows_of = [&](const uint4* ab, int s, int a) __attribute__((always_inline)) -> half8w {
      const int r = a * 32 + m32;
      return __builtin_bit_cast(half8w, ab[r * 16 + ((kh * 8 + s) ^ (r & 15))]);
    };
    auto columns_of = [&](int s, int b) __attribute__((always_inline)) -> half8w {
      const int zi = G32 ? s >> 2 : 0;  // slices 0-3 lie in the half's first 32 channels
      if constexpr (BITS == 8) {
        const uint4 q = bq[b][s >> 1];  // slice s: words 2 s, 2 s + 1 of the lane half's 16
        return (s & 1) ? widen_word8(q.z, q.w, zz[b][zi], s2[b][zi], magic8)
                       : widen_word8(q.x, q.y, zz[b][zi], s2[b][zi], magic8);
      } else if constexpr (BITS == 3) {
        // slice s = channel pairs 4 s .. 4 s + 3 of the half: low word s / 2 (fields
        // 4 (s % 2) ..), high word s / 4 (bits 4 (s % 4) ..)
        const uint4 q = bq[b][0];
        const uint32_t lo = (s >> 1) == 0 ? q.x : (s >> 1) == 1 ? q.y : (s >> 1) == 2 ? q.z : q.w;
        const uint32_t hiw = (s >> 2) ? bh[b].y : bh[b].x;
        return widen_word3(lo, hiw, 4 * (s & 1), 4 * (s & 3), zz[b][zi], s2[b][zi], magic);
      } else {
        const uint4 q = bq[b][s >> 2];
        const uint32_t w = (s & 3) == 0 ? q.x : (s & 3) == 1 ? q.y : (s & 3) == 2 ? q.z : q.w;
        return widen_word(w, zz[b][zi], zz64[b][zi], s2[b][zi], magic);
      }
    };
    // One slice, from group `at` of the step on: the products of A and B, and between them slice ns
    // of the step at ab into nA and nB, and the shares of the DMAs of step `step` into buffer c. (Left to itself the compiler
    // widens in one piece while the matrix cores wait.)
    auto slice = [&](const half8w (&A)[RT], const half8w (&B)[2], half8w (&nA)[RT], half8w (&nB)[2],
                     const uint4* ab, int ns, auto c, int step, int at) __attribute__((always_inline)) {
      constexpr int kR = RT / kGroups, kV = BITS == 3 ? 9 : 6;
#pragma unroll
      for (int q = 0; q < kGroups; ++q) {
        if ((at + q) % kEvery == 0 && (at + q) / kEvery < kShares) send(c, step, (at + q) / kEvery);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int a = q * kR; a < (q + 1) * kR; ++a) nA[a] = rows_of(ab, ns, a);
        if (q == 0) nB[0] = columns_of(ns, 0);
        if (q == kGroups / 2) nB[1] = columns_of(ns, 1);
#pragma unroll
        for (int a = q * kR; a < (q + 1) * kR; ++a)
#pragma unroll
          for (int b = 0; b < 2; ++b)
            acc[a][b] = __builtin_amdgcn_mfma_f32_32x32x16_f16(A[a], B[b], acc[a][b], 0, 0, 0);
#pragma unroll
        for (int i = 0; i < 2 * kR; ++i) {
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                  // MFMA
          if (i % 2 == 0) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);  // LDS read
          __builtin_amdgcn_sched_group_barrier(0x002, kGroups > 1 ? kV : 2 * kV, 0);  // VALU
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    };

    ScaleZero sz[NS];
    half8w A0[RT], B0[2], A1[RT], B1[2];
    auto prologue = [&](auto c) __attribute__((always_inline)) {
      constexpr int b = decltype(c)::value;
      if constexpr (b < NS) load_sz(sz[b], b);
      if constexpr (b < NS - 1) {
#pragma unroll
        for (int i = 0; i < kShares; ++i) send(c, b, i);
      }
    };
    prologue(std::integral_constant<int, 0>{});
    prologue(std::integral_constant<int, 1>{});
    prologue(std::integral_constant<int, 2>{});
    prologue(std::integral_constant<int, 3>{});
    prologue(std::integral_constant<int, 4>{});
    arrive(0);
    open_step(sz[0], ring + BM * 16, 0);
#pragma unroll
    for (int a = 0; a < RT; ++a) A0[a] = rows_of(ring, 0, a);
#pragma unroll
    for (int b = 0; b < 2; ++b) B0[b] = columns_of(0, b);

    // One K step from buffer C, whose first slice is in registers; the step NS - 1 ahead goes into
    // the buffer of the step before. Before the last slice's products the next step is opened.
    auto body = [&](auto bufc, int step) __attribute__((always_inline)) {
      constexpr int C = decltype(bufc)::value, F = (C + NS - 1) % NS, N1 = (C + 1) % NS;
      const uint4* const ab = ring + C * kBuf;
      constexpr std::integral_constant<int, F> free;
#pragma unroll
      for (int s = 0; s < kGK / 16 - 2; s += 2) {
        slice(A0, B0, A1, B1, ab, s + 1, free, step + NS - 1, s * kGroups);
        slice(A1, B1, A0, B0, ab, s + 2, free, step + NS - 1, (s + 1) * kGroups);
      }
      slice(A0, B0, A1, B1, ab, kGK / 16 - 1, free, step + NS - 1, 6 * kGroups);
      arrive(step + 1);  // (past the last: nothing is in flight, and what is opened is not used)
      load_sz(sz[C], step + NS);
      open_step(sz[N1], ring + N1 * kBuf + BM * 16, step + 1);
      slice(A1, B1, A0, B0, ring + N1 * kBuf, 0, free, nsteps, 7 * kGroups);
    };
    int step = 0;
    auto at = [&](auto c) __attribute__((always_inline)) {
      if constexpr (decltype(c)::value < NS) body(c, step + decltype(c)::value);
    };
    for (; step + NS <= nsteps; step += NS) {
      at(std::integral_constant<int, 0>{});
      at(std::integral_constant<int, 1>{});
      at(std::integral_constant<int, 2>{});
      at(std::integral_constant<int, 3>{});
      at(std::integral_constant<int, 4>{});
    }
    if (step < nsteps) at(std::integral_constant<int, 0>{});
    if (step + 1 < nsteps) at(std::integral_constant<int, 1>{});
    if (step + 2 < nsteps) at(std::integral_constant<int, 2>{});
    if (step + 3 < nsteps) at(std::integral_constant<int, 3>{});

    if constexpr (MODE == kLora) {
      constexpr int T = RT == 8 ? 2 : RT;  // (the sums of 256 rows leave registers for two)
#pragma unroll
      for (int a0 = 0; a0 < RT; a0 += T)
        add_adapters(a0 * 32, std::integral_constant<int, T>{},
                     [&](int a) __attribute__((always_inline)) { return acc[a0 + a]; });
    }
    // 32x32 accumulator layout: element e of lane l is (row 8(e/4) + 4(l/32) + e%4, col l%32).
    const int64_t ldy = MODE == kGated ? nh : N;
    auto store = [&](int r, float v0, float v1) {
      if (r >= rows) return;
      const int64_t yr = MODE == kLora ? source(row0 + r) : row0 + r;
      if constexpr (MODE == kGated) {
        const int64_t col = n0 + part * 32 + m32;
        if (col < nh) g.Y[yr * ldy + col] = f2h_bits(silu_f32(v0) * v1);
      } else {
        const int64_t col = n0 + part * 64 + m32;
        if (col < N) g.Y[yr * ldy + col] = f2h_bits(v0);
        if (col + 32 < N) g.Y[yr * ldy + col + 32] = f2h_bits(v1);
      }
    };
    if constexpr (KW == 1) {
#pragma unroll
      for (int a = 0; a < RT; ++a)
#pragma unroll
        for (int i = 0; i < 16; ++i) store(a * 32 + 8 * (i >> 2) + 4 * kh + (i & 3), acc[a][0][i], acc[a][1][i]);
    } else {
      // the waves' sums meet in LDS, in the waves' order; wave w stores rows 8 w .. of every tile
      static_assert(KW * RT * 8 * 64 <= KW * NS * kBuf, "the sums fit LDS");
      f32x4w* const sums = reinterpret_cast<f32x4w*>(lds);
      __syncthreads();  // no ring is read or filled any more
#pragma unroll
      for (int a = 0; a < RT; ++a)
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            sums[(wave * RT * 8 + (a * 2 + b) * 4 + q) * 64 + lane] =
                f32x4w{acc[a][b][4 * q], acc[a][b][4 * q + 1], acc[a][b][4 * q + 2], acc[a][b][4 * q + 3]};
      __syncthreads();
#pragma unroll
      for (int a = 0; a < RT; ++a) {
        f32x4w v[2];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          v[b] = sums[((a * 2 + b) * 4 + wave) * 64 + lane];
#pragma unroll
          for (int w = 1; w < KW; ++w) v[b] += sums[(w * RT * 8 + (a * 2 + b) * 4 + wave) * 64 + lane];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) store(a * 32 + 8 * wave + 4 * kh + i, v[0][i], v[1][i]);
      }
    }
  };
  if constexpr (RTM == 8) {
    if (rows > 128) return run(std::integral_constant<int, 8>{});
  }
  if constexpr (RTM >= 4) {
    if (rows > 64) return run(std::integral_constant<int, 4>{});
  }
  if constexpr (RTM >= 2) {
    if (rows > 32) return run(std::integral_constant<int, 2>{});
  }
  run(std::integral_constant<int, 1>{});
}

// The variants that the launcher picks from (row tiles of 32, waves along K).
template <int MODE, int BITS, bool G32>
void launch_grouped_g(const GroupedArgs& g, int row_tiles, int k_waves, dim3 grid, hipStream_t stream) {
  constexpr int kSplit = BITS == 8 ? 1 : 2;  // 8-bit: two 64-row steps of four waves would not fit LDS
  if (k_waves > 1)
    hipLaunchKernelGGL((k_grouped<MODE, kSplit, BITS, G32, 4>), grid, dim3(256), 0, stream, g);
  else if (row_tiles == 2)
    hipLaunchKernelGGL((k_grouped<MODE, 2, BITS, G32, 1>), grid, dim3(256), 0, stream, g);
  else if (row_tiles == 4 || BITS == 8)
    hipLaunchKernelGGL((k_grouped<MODE, 4, BITS, G32, 1>), grid, dim3(256), 0, stream, g);
  else
    hipLaunchKernelGGL((k_grouped<MODE, BITS == 8 ? 4 : 8, BITS, G32, 1>), grid, dim3(256), 0, stream, g);
}

template <int MODE, int BITS>
void launch_grouped_t(const GroupedArgs& g, int row_tiles, int k_waves, dim3 grid, hipStream_t stream) {
  if (g.group == 32)
    launch_grouped_g<MODE, BITS, true>(g, row_tiles, k_waves, grid, stream);
  else
    launch_grouped_g<MODE, BITS, false>(g, row_tiles, k_waves, grid, stream);
}

}  // namespace awq
