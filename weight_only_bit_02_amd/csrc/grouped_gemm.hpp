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
// per tile. Both operands go global -> LDS by 16-byte DMA into the other of two buffers
// while a step is multiplied; A's DMA takes a row address per lane, so gathering costs
// nothing. A row's 16 chunks are stored in slots c ^ (row % 16) and codes quarter-major:
// both are read without bank conflicts. A tile with fewer rows runs a body with fewer row
// tiles (a power of two), so a group's last tile costs the matrix work of the rows it has.
//
// RTM = 8 (8-bit codes: 4, LDS holds no more) serves large groups, one wave per SIMD;
// RTM = 2 small ones, two blocks per CU.
//
// Operand values and their order along K are those of the 256-row GEMM, so an expert's rows
// equal the plain linear's bit for bit where that runs its GEMM.
//
// Adapters (MODE kLora): the rows of one batch, optionally through `order` (then Y is
// scattered back through it). Before the K loop each 32-row tile starts, for every adapter
// among its rows, from H B_a^T (H = scale X A_a^T from the first product's kernel, as fp16 hi
// + lo under a power of two), rows of other adapters masked.
#pragma once

#include <type_traits>

#include "common.hpp"
#include "groups.hpp"
#include "launch.hpp"
#include "widen.hpp"

namespace awq {


constexpr int kGN = 256, kGK = 128;   // columns of a tile, channels of a K step
constexpr int kGroupedTiles = 4;      // row tiles that share a column panel in the tile order

template <int MODE, int RTM, int BITS>
__global__ void __launch_bounds__(256, RTM == 2 && BITS != 8 ? 2 : 1) k_grouped(GroupedArgs g) {
  constexpr int BM = RTM * 32;
  constexpr int kQ = BITS;             // 16-byte quarters of a column's codes per step
  constexpr int kBT = kGN * kQ / 256;  // B transfers per wave and step
  __shared__ __attribute__((aligned(16))) uint4 a0s[BM * 16];
  __shared__ __attribute__((aligned(16))) uint4 a1s[BM * 16];
  __shared__ __attribute__((aligned(16))) uint4 b0s[kGN * kQ];
  __shared__ __attribute__((aligned(16))) uint4 b1s[kGN * kQ];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int m32 = lane & 31, kh = lane >> 5;
  const int64_t N = g.N, K = g.K, nh = N / 2;

  // ---- this block's tile: XCD blockIdx % 8 takes a contiguous run of the tiles there are
  const int mt = MODE == kLora ? (g.n + BM - 1) / BM : count_tiles<BM>(g.offsets, g.groups, g.n, lane);
  const int64_t tiles = (int64_t)mt * g.nt, per_xcd = (tiles + 7) / 8;
  const int64_t slot = blockIdx.x / 8, t = (int64_t)(blockIdx.x % 8) * per_xcd + slot;
  if (slot >= per_xcd || t >= tiles) return;
  const int first_m = (int)(t / ((int64_t)kGroupedTiles * g.nt)) * kGroupedTiles;
  const int gsz = mt - first_m < kGroupedTiles ? mt - first_m : kGroupedTiles;
  const int within = (int)(t - (int64_t)first_m * g.nt);
  const int64_t n0 = (int64_t)(within / gsz) * (MODE == kGated ? kGN / 2 : kGN);
  const int at = first_m + within % gsz;
  const RowTile rt = MODE == kLora ? RowTile{0, at * BM, g.n - at * BM < BM ? g.n - at * BM : BM}
                                   : find_tile<BM>(g.offsets, g.groups, g.n, at, lane);
  const int row0 = __builtin_amdgcn_readfirstlane(rt.row0), rows = __builtin_amdgcn_readfirstlane(rt.rows);
  const int64_t e = MODE == kLora ? 0 : __builtin_amdgcn_readfirstlane(rt.e);
  if (rows <= 0) return;

  const int g64 = g.group == 64, g32 = g.group == 32;
  const int64_t Gs = K / g.group, zbw = BITS == 8 ? Gs : (Gs + 1) / 2, words = K * BITS / 32;
  const int64_t nsteps = K / kGK;
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

  // B DMA map, quarter-major: slot (wave * kBT + i) * 64 + lane = 16-byte quarter slot / 256
  // of tile column slot % 256. Gated: tile columns [64 w, 64 w + 32) hold the gate rows and
  // [64 w + 32, 64 w + 64) the up rows of outputs n0 + 32 w ... Columns past the end read the
  // last one (never stored).
  const uint32_t* bptr[kBT];
#pragma unroll
  for (int i = 0; i < kBT; ++i) {
    const int s = (wave * kBT + i) * 64 + lane;
    const int c = s % kGN, q = s / kGN;
    int64_t n;
    if constexpr (MODE == kGated) {
      int64_t o = n0 + (c >> 6) * 32 + (c & 31);
      o = o < nh ? o : nh - 1;
      n = (c & 63) >= 32 ? o + nh : o;
    } else {
      n = n0 + c < N ? n0 + c : N - 1;
    }
    bptr[i] = qweight + n * words + q * 4;
  }
  // this lane's weight rows (gated: gate row and up row): scales and zeros
  int64_t bcol[2];
  if constexpr (MODE == kGated) {
    const int64_t o = n0 + wave * 32 + m32;
    bcol[0] = o < nh ? o : nh - 1;
    bcol[1] = bcol[0] + nh;
  } else {
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int64_t n = n0 + wave * 64 + b * 32 + m32;
      bcol[b] = n < N ? n : N - 1;
    }
  }
  // per column, the zero(s) and scale(s) of the lane half's 64 channels of a step: one group
  // of 128 (step) or 64 (2 step + kh), or two of 32 (4 step + 2 kh and the next)
  struct ScaleZero {
    uint32_t zb[2], sc[2][2];
  };
  auto load_sz = [&](ScaleZero& st, int64_t step) {
    const int64_t g0 = g32 ? 4 * step + 2 * kh : g64 ? 2 * step + kh : step;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      st.zb[b] = zeros[bcol[b] * zbw + (BITS == 8 ? g0 : g0 >> 1)];
      st.sc[b][0] = scales[bcol[b] * Gs + g0];
      if (g32) {
        if constexpr (BITS == 8) st.zb[b] |= (uint32_t)zeros[bcol[b] * zbw + g0 + 1] << 8;
        st.sc[b][1] = scales[bcol[b] * Gs + g0 + 1];
      } else {
        st.sc[b][1] = st.sc[b][0];
      }
    }
  };

  // Adapters: the 32 rows from r0 on, times the adapters' B, into acc (zero at the start): the
  // accumulators begin with the low-rank term, and the K loop adds the linear to it.
  auto lora_tile = [&](int r0, f32x16w (&acc)[2]) {
    const int r = r0 + m32;
    const int src = source(row0 + (r < rows ? r : rows - 1));
    const int id = r < rows ? g.ids[src] : -1;
    const int blocks = (g.rank + kLoraBlock - 1) / kLoraBlock;
    const LoraRow* const h = g.H + (int64_t)src * blocks;
    uint64_t rest = __ballot((unsigned)id < (unsigned)g.groups);
    while (rest) {  // one adapter after the other, by its first row
      const int ad = __builtin_amdgcn_readlane(id, __ffsll((unsigned long long)rest) - 1);
      const bool mine = id == ad;
      const uint64_t rows_of = __ballot(mine);
      rest &= ~rows_of;
      const uint16_t* const B = g.B + (int64_t)ad * N * g.rank;
      for (int k = 0; k < blocks; ++k) {
        f32x16w d[2] = {f32x16w{}, f32x16w{}};
        const float f = h[k].f;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const int at = s * 16 + kh * 8;
          const half8w hi = mine ? *reinterpret_cast<const half8w*>(h[k].hi + at) : half8w{};
          const half8w lo = mine ? *reinterpret_cast<const half8w*>(h[k].lo + at) : half8w{};
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            const half8w bw = k * kLoraBlock + at < g.rank
                                  ? *reinterpret_cast<const half8w*>(B + bcol[b] * g.rank + k * kLoraBlock + at)
                                  : half8w{};
            d[b] = __builtin_amdgcn_mfma_f32_32x32x16_f16(hi, bw, d[b], 0, 0, 0);
            d[b] = __builtin_amdgcn_mfma_f32_32x32x16_f16(lo, bw, d[b], 0, 0, 0);
          }
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          // only the adapter's own rows: an Inf or NaN of its B stays out of the others
          const int ri = 8 * (i >> 2) + 4 * kh + (i & 3);
          const float fr = __shfl(f, ri);
          const bool on = (rows_of >> ri) & 1;
#pragma unroll
          for (int b = 0; b < 2; ++b) acc[b][i] = on ? __builtin_fmaf(fr, d[b][i], acc[b][i]) : acc[b][i];
        }
      }
    }
  };

  // RT row tiles of 32 rows cover this tile's rows.
  auto run = [&](auto rtc) {
    constexpr int RT = decltype(rtc)::value;
    constexpr int kAT = 2 * RT;  // A transfers per wave and step
    // A DMA map: wave transfer i fills slots (wave * kAT + i) * 64 + lane: row r = (wave * kAT
    // + i) * 4 + lane / 16, slot lane % 16 <- chunk (lane % 16) ^ (r % 16), as 16-byte units of
    // X (the host admits X up to 2^32 of them). Rows past the last read the last one.
    uint32_t aoff[kAT];
#pragma unroll
    for (int i = 0; i < kAT; ++i) {
      const int r = (wave * kAT + i) * 4 + (lane >> 4);
      int x = source(row0 + (r < rows ? r : rows - 1));
      if (MODE != kLora && g.order) x = (int)((unsigned)x / (unsigned)g.fan);
      aoff[i] = (uint32_t)x * (uint32_t)(K / 8) + ((lane & 15) ^ (r & 15));
    }
    const uint4* const X = reinterpret_cast<const uint4*>(g.X);

    f32x16w acc[RT][2];
#pragma unroll
    for (int a = 0; a < RT; ++a)
#pragma unroll
      for (int b = 0; b < 2; ++b) acc[a][b] = f32x16w{};

    ScaleZero s0, s1;
#pragma unroll
    for (int i = 0; i < kAT; ++i)
      __builtin_amdgcn_global_load_lds((const void*)(X + aoff[i]), (lds_void*)&a0s[(wave * kAT + i) * 64],
                                       16, 0, 0);
#pragma unroll
    for (int i = 0; i < kBT; ++i)
      __builtin_amdgcn_global_load_lds((const void*)(bptr[i]), (lds_void*)&b0s[(wave * kBT + i) * 64],
                                       16, 0, 0);
    load_sz(s0, 0);
    if constexpr (MODE == kLora) {
#pragma unroll
      for (int a = 0; a < RT; ++a) lora_tile(a * 32, acc[a]);
    }
    __syncthreads();

    // One K step on buffer BUF (a compile-time constant, so each LDS access names one object).
    auto body = [&](auto bufc, ScaleZero& cur, ScaleZero& nxt, int64_t step) {
      constexpr int BUF = decltype(bufc)::value;
      const uint4* ab = BUF ? a1s : a0s;
      const uint4* bb = BUF ? b1s : b0s;
      // the next step's operands (clamped: the last step reloads itself into the idle buffer)
      const int64_t sn = step + 1 < nsteps ? step + 1 : nsteps - 1;
      load_sz(nxt, sn);
      __builtin_amdgcn_sched_barrier(0);  // keep the scale loads at the top of the step
      uint4* const adn = BUF ? a0s : a1s;
      uint4* const bdn = BUF ? b0s : b1s;
      auto dma_a = [&](int i) {
        __builtin_amdgcn_global_load_lds((const void*)(X + (uint64_t)aoff[i] + sn * 16),
                                         (lds_void*)&adn[(wave * kAT + i) * 64], 16, 0, 0);
      };
      auto dma_b = [&](int i) {
        __builtin_amdgcn_global_load_lds((const void*)(bptr[i] + sn * (kQ * 4)),
                                         (lds_void*)&bdn[(wave * kBT + i) * 64], 16, 0, 0);
      };
      half2w zz[2][2], zz64[2][2], s2[2][2];
      const int hi = g64 ? kh : (int)(step & 1);  // zero nibble: group of 128 (step) or 64 (2 step + kh)
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t z;
          if constexpr (BITS == 8)
            z = g32 ? (cur.zb[b] >> (8 * i)) & 0xFF : cur.zb[b];
          else
            z = (cur.zb[b] >> (4 * (g32 ? i : hi))) & 0xF;
          const uint32_t z1024 = 0x6400u + z, z64 = 0x5400u + (z << 4);
          zz[b][i] = -__builtin_bit_cast(half2w, z1024 | (z1024 << 16));
          zz64[b][i] = -__builtin_bit_cast(half2w, z64 | (z64 << 16));
          s2[b][i] = __builtin_bit_cast(half2w, cur.sc[b][i] | (cur.sc[b][i] << 16));
        }
      // this lane's code words of the step, per column: 4- and 8-bit, the quarters kQ / 2 kh ..;
      // 3-bit, low-plane words 4 kh .. (quarter kh) and high-plane words 8 + 2 kh, 9 + 2 kh
      constexpr int kQL = BITS == 3 ? 1 : kQ / 2;
      uint4 bq[2][kQL];
      uint2 bh[2];
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int col = wave * 64 + b * 32 + m32;
        if constexpr (BITS == 3) {
          bq[b][0] = bb[kh * kGN + col];
          const uint4 h4 = bb[2 * kGN + col];
          bh[b] = kh ? make_uint2(h4.z, h4.w) : make_uint2(h4.x, h4.y);
        } else {
#pragma unroll
          for (int h = 0; h < kQL; ++h) bq[b][h] = bb[(kQL * kh + h) * kGN + col];
        }
      }
      auto frags = [&](int s, half8w (&A)[RT], half8w (&B)[2]) {
        const int c = kh * 8 + s;
        const int zi = s >> 2;  // slices 0-3 lie in the half's first 32 channels
#pragma unroll
        for (int a = 0; a < RT; ++a) {
          const int r = a * 32 + m32;
          A[a] = __builtin_bit_cast(half8w, ab[r * 16 + (c ^ (r & 15))]);
        }
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          if constexpr (BITS == 8) {
            const uint4 q = bq[b][s >> 1];  // slice s: words 2 s, 2 s + 1 of the lane half's 16
            B[b] = (s & 1) ? widen_word8(q.z, q.w, zz[b][zi], s2[b][zi], magic8)
                           : widen_word8(q.x, q.y, zz[b][zi], s2[b][zi], magic8);
          } else if constexpr (BITS == 3) {
            // slice s = channel pairs 4 s .. 4 s + 3 of the half: low word s / 2 (fields
            // 4 (s % 2) ..), high word s / 4 (bits 4 (s % 4) ..)
            const uint4 q = bq[b][0];
            const uint32_t lo = (s >> 1) == 0 ? q.x : (s >> 1) == 1 ? q.y : (s >> 1) == 2 ? q.z : q.w;
            const uint32_t hiw = (s >> 2) ? bh[b].y : bh[b].x;
            B[b] = widen_word3(lo, hiw, 4 * (s & 1), 4 * (s & 3), zz[b][zi], s2[b][zi], magic);
          } else {
            const uint4 q = bq[b][s >> 2];
            const uint32_t w = (s & 3) == 0 ? q.x : (s & 3) == 1 ? q.y : (s & 3) == 2 ? q.z : q.w;
            B[b] = widen_word(w, zz[b][zi], zz64[b][zi], s2[b][zi], magic);
          }
        }
      };
      half8w A0[RT], B0[2], A1[RT], B1[2];
      frags(0, A0, B0);
#pragma unroll
      for (int s = 0; s < kGK / 16; s += 2) {
        {  // a quarter of the next step's transfers
          __builtin_amdgcn_sched_barrier(0);
          constexpr int kA4 = (kAT + 3) / 4, kB4 = (kBT + 3) / 4;
#pragma unroll
          for (int i = 0; i < kA4; ++i)
            if ((s >> 1) * kA4 + i < kAT) dma_a((s >> 1) * kA4 + i);
#pragma unroll
          for (int i = 0; i < kB4; ++i)
            if ((s >> 1) * kB4 + i < kBT) dma_b((s >> 1) * kB4 + i);
          __builtin_amdgcn_sched_barrier(0);
        }
        frags(s + 1, A1, B1);
#pragma unroll
        for (int a = 0; a < RT; ++a)
#pragma unroll
          for (int b = 0; b < 2; ++b)
            acc[a][b] = __builtin_amdgcn_mfma_f32_32x32x16_f16(A0[a], B0[b], acc[a][b], 0, 0, 0);
        if (s + 2 < kGK / 16) frags(s + 2, A0, B0);
#pragma unroll
        for (int a = 0; a < RT; ++a)
#pragma unroll
          for (int b = 0; b < 2; ++b)
            acc[a][b] = __builtin_amdgcn_mfma_f32_32x32x16_f16(A1[a], B1[b], acc[a][b], 0, 0, 0);
      }
      __syncthreads();  // the next step's DMA has landed; this step's buffer is free
    };
    int64_t step = 0;
    for (; step + 2 <= nsteps; step += 2) {
      body(std::integral_constant<int, 0>{}, s0, s1, step);
      body(std::integral_constant<int, 1>{}, s1, s0, step + 1);
    }
    if (step < nsteps) body(std::integral_constant<int, 0>{}, s0, s1, step);

    // 32x32 accumulator layout: element e of lane l is (row 8(e/4) + 4(l/32) + e%4, col l%32).
    const int64_t ldy = MODE == kGated ? nh : N;
#pragma unroll
    for (int a = 0; a < RT; ++a)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int r = a * 32 + 8 * (i >> 2) + 4 * kh + (i & 3);
        if (r < rows) {
          const int64_t yr = MODE == kLora ? source(row0 + r) : row0 + r;
          if constexpr (MODE == kGated) {
            const int64_t col = n0 + wave * 32 + m32;
            if (col < nh) g.Y[yr * ldy + col] = f2h_bits(silu_f32(acc[a][0][i]) * acc[a][1][i]);
          } else {
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              const int64_t col = n0 + wave * 64 + b * 32 + m32;
              if (col < N) g.Y[yr * ldy + col] = f2h_bits(acc[a][b][i]);
            }
          }
        }
      }
  };
  if constexpr (RTM == 8) {
    if (rows > 128) return run(std::integral_constant<int, 8>{});
  }
  if constexpr (RTM >= 4) {
    if (rows > 64) return run(std::integral_constant<int, 4>{});
  }
  if (rows > 32) return run(std::integral_constant<int, 2>{});
  run(std::integral_constant<int, 1>{});
}

}  // namespace awq
