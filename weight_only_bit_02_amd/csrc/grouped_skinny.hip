// Ragged-row linear for few rows per group (decoding): the products of grouped_gemm.hpp for
// tiles of up to 32 rows x 32 weight rows, K split over the eight waves of a block.
//
// Decoding streams every active weight once, so what counts is bytes in flight: a tile has
// one block per 32 weight rows, its waves each take an eighth of K and meet in LDS in a fixed
// order. Lane l works on weight row l % 32 and, h = l / 32, on channels [32 h, 32 h + 32) and
// [64 + 32 h, 96 + 32 h) of a 128-channel step, widens 8 channels at a time to exact q - z
// in fp16 and multiplies them with 32 rows of X by v_mfma_f32_32x32x16_f16; the group's scale
// multiplies the partial tile in fp32. With 32-channel groups the lane halves of a slice lie
// in different groups, so there the operand carries the scale ((q - z) sc, one rounding).
// A tile keeps 4, 8 or 16 accumulators per lane by its rows (8, 16, 32). The next step's
// loads are in flight while a step is multiplied.
//
// Gated: 16 gate rows and their 16 up rows. Adapters: see grouped_gemm.hpp; the waves share
// the adapters of a tile.
#include <type_traits>

#include "common.hpp"
#include "groups.hpp"
#include "launch.hpp"
#include "widen.hpp"

namespace awq {

namespace {

constexpr int kS = 8;

// One lane's codes of a 128-channel step: two sets of 32 channels.
template <int BITS>
struct Codes {
  uint32_t w[2][BITS];  // 3-bit: two low-plane words, one high-plane word
};

template <int BITS>
__device__ __forceinline__ void load_codes(Codes<BITS>& c, const uint32_t* step, int h) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if constexpr (BITS == 3) {
      const uint2 lo = *reinterpret_cast<const uint2*>(step + 4 * i + 2 * h);
      c.w[i][0] = lo.x;
      c.w[i][1] = lo.y;
      c.w[i][2] = step[8 + 2 * i + h];
    } else {
#pragma unroll
      for (int q = 0; q < BITS / 4; ++q) {
        const uint4 v = *reinterpret_cast<const uint4*>(step + (2 * i + h) * BITS + 4 * q);
        c.w[i][4 * q] = v.x;
        c.w[i][4 * q + 1] = v.y;
        c.w[i][4 * q + 2] = v.z;
        c.w[i][4 * q + 3] = v.w;
      }
    }
  }
}

// Slice s (8 channels; set s / 4) as exact q - z; zz holds -(1024 + z) in both halves.
template <int BITS>
__device__ __forceinline__ half8w centered(const Codes<BITS>& c, int s, half2w zz, uint32_t magic) {
  half2w d[4];
  const int i = s >> 2, t = s & 3;
  if constexpr (BITS == 4) {
#pragma unroll
    for (int p = 0; p < 4; ++p)
      d[p] = __builtin_bit_cast(half2w, ((c.w[i][t] >> (4 * p)) & 0x000F000Fu) | magic) + zz;
  } else if constexpr (BITS == 8) {
    const uint32_t m8 = 0x64646464u, w0 = c.w[i][2 * t], w1 = c.w[i][2 * t + 1];
    d[0] = __builtin_bit_cast(half2w, __builtin_amdgcn_perm(m8, w0, 0x04010400u)) + zz;
    d[1] = __builtin_bit_cast(half2w, __builtin_amdgcn_perm(m8, w0, 0x04030402u)) + zz;
    d[2] = __builtin_bit_cast(half2w, __builtin_amdgcn_perm(m8, w1, 0x04010400u)) + zz;
    d[3] = __builtin_bit_cast(half2w, __builtin_amdgcn_perm(m8, w1, 0x04030402u)) + zz;
  } else {
#pragma unroll
    for (int p = 0; p < 4; ++p)
      d[p] = __builtin_bit_cast(half2w, widen3_pair(c.w[i][t >> 1], c.w[i][2], 4 * (t & 1) + p, 4 * t + p, magic)) + zz;
  }
  return half8w{d[0][0], d[0][1], d[1][0], d[1][1], d[2][0], d[2][1], d[3][0], d[3][1]};
}

template <int BITS>
struct Stage {
  Codes<BITS> b;
  half8w a[8];
  uint32_t z[2], sc[2];  // per set of 32 channels
};

template <int MODE, int BITS>
__global__ void __launch_bounds__(kS * 64) k_skinny(GroupedArgs g) {
  __shared__ float red[kS][16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int j = lane & 31, h = lane >> 5;
  const int64_t N = g.N, K = g.K, nh = N / 2;
  const int at = blockIdx.y;
  const RowTile rt = MODE == kLora ? RowTile{0, at * 32, g.n - at * 32 < 32 ? g.n - at * 32 : 32}
                                   : find_tile<32>(g.offsets, g.groups, g.n, at, lane);
  const int row0 = __builtin_amdgcn_readfirstlane(rt.row0), rows = __builtin_amdgcn_readfirstlane(rt.rows);
  const int64_t e = MODE == kLora ? 0 : __builtin_amdgcn_readfirstlane(rt.e);
  if (rows <= 0) return;
  const bool g64 = g.group == 64, g32 = g.group == 32;
  const int64_t G = K / kGroup, Gs = K / g.group, zbw = BITS == 8 ? Gs : (Gs + 1) / 2, words = K * BITS / 32;
  int64_t n;
  if constexpr (MODE == kGated) {
    const int64_t o = (int64_t)blockIdx.x * 16 + (j & 15);
    n = (o < nh ? o : nh - 1) + (j >> 4) * nh;
  } else {
    const int64_t o = (int64_t)blockIdx.x * 32 + j;
    n = o < N ? o : N - 1;
  }
  const uint32_t* const qw = g.qweight + (e * N + n) * words;
  const uint16_t* const scales = g.scales + (e * N + n) * Gs;
  const uint8_t* const zeros = g.zeros + (e * N + n) * zbw;
  // this lane's row of X (rows past the last read the last one, never stored)
  int src = row0 + (j < rows ? j : rows - 1);
  if (g.order) {
    const int o = g.order[src];
    src = (unsigned)o < (unsigned)g.n ? o : 0;
  }
  const int64_t xr = MODE != kLora && g.order ? (int)((unsigned)src / (unsigned)g.fan) : src;
  const uint16_t* const X = g.X + xr * K + h * 32;
  const int64_t g0 = G * wave / kS, g1 = G * (wave + 1) / kS;
  const uint32_t magic = wide_magic();

  auto load = [&](Stage<BITS>& st, int64_t step) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      // set i's group: 128, the step; 64, 2 step + i; 32, 4 step + 2 i + h
      const int64_t q = g32 ? 4 * step + 2 * i + h : g64 ? 2 * step + i : step;
      if constexpr (BITS == 8)
        st.z[i] = zeros[q];
      else
        st.z[i] = (zeros[q >> 1] >> (4 * (q & 1))) & 0xF;
      st.sc[i] = scales[q];
    }
    load_codes<BITS>(st.b, qw + step * (4 * BITS), h);
#pragma unroll
    for (int s = 0; s < 8; ++s)
      st.a[s] = *reinterpret_cast<const half8w*>(X + step * kGroup + (s & 3) * 8 + (s >> 2) * 64);
  };

  // E accumulators per lane hold the tile's rows
  auto run = [&](auto ec) {
    constexpr int E = decltype(ec)::value;
    float acc[E];
#pragma unroll
    for (int i = 0; i < E; ++i) acc[i] = 0.0f;
    auto body = [&](const Stage<BITS>& st) {
      half2w zz[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t z = 0x6400u + st.z[i];
        zz[i] = -__builtin_bit_cast(half2w, z | (z << 16));
      }
      f32x16w d{};
      if (g32) {
#pragma unroll
        for (int s = 0; s < 8; ++s) {
          const half8w q = centered<BITS>(st.b, s, zz[s >> 2], magic);
          const _Float16 c = __builtin_bit_cast(_Float16, (uint16_t)st.sc[s >> 2]);
          d = __builtin_amdgcn_mfma_f32_32x32x16_f16(st.a[s], q * half8w{c, c, c, c, c, c, c, c}, d, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < E; ++i) acc[i] += d[i];
      } else {
#pragma unroll
        for (int s = 0; s < 8; ++s) {
          d = __builtin_amdgcn_mfma_f32_32x32x16_f16(st.a[s], centered<BITS>(st.b, s, zz[s >> 2], magic), d, 0, 0, 0);
          if (s == 3 && g64) {
            const float c = h2f((uint16_t)st.sc[0]);
#pragma unroll
            for (int i = 0; i < E; ++i) acc[i] = __builtin_fmaf(c, d[i], acc[i]);
            d = f32x16w{};
          }
        }
        const float c = h2f((uint16_t)st.sc[1]);
#pragma unroll
        for (int i = 0; i < E; ++i) acc[i] = __builtin_fmaf(c, d[i], acc[i]);
      }
    };
    if (g1 > g0) {
      Stage<BITS> s0, s1;
      load(s0, g0);
      int64_t step = g0;
      for (; step + 2 <= g1; step += 2) {
        load(s1, step + 1);
        body(s0);
        load(s0, step + 2 < g1 ? step + 2 : g1 - 1);  // always issued: exact waits on every path
        body(s1);
      }
      if (step < g1) body(s0);
    }
    if constexpr (MODE == kLora) {
      const int id = j < rows ? g.ids[src] : -1;
      const float* const hr = g.H + (int64_t)src * g.rank;
      float mx = 0.0f;  // the row's power of two: its largest |h| goes to [1, 2)
      for (int k = h * 8; k < g.rank; k += 16)
#pragma unroll
        for (int i = 0; i < 8; ++i) mx = fmaxf(mx, __builtin_fabsf(hr[k + i]));
      mx = fmaxf(mx, __shfl_xor(mx, 32));
      const uint32_t ex = __builtin_bit_cast(uint32_t, mx) >> 23;
      const bool fit = ex >= 1 && ex < 253;  // zero, tiny or not finite: as it is
      const float up = fit ? __builtin_bit_cast(float, (254u - ex) << 23) : 1.0f;
      const float down = fit ? __builtin_bit_cast(float, ex << 23) : 1.0f;
      uint64_t rest = __ballot((unsigned)id < (unsigned)g.groups);
      for (int turn = 0; rest; ++turn) {  // one adapter after the other, by its first row
        const int ad = __builtin_amdgcn_readlane(id, __ffsll((unsigned long long)rest) - 1);
        const bool mine = id == ad;
        const uint64_t rows_of = __ballot(mine);
        rest &= ~rows_of;
        if (turn % kS != wave) continue;
        const uint16_t* const B = g.B + ((int64_t)ad * N + n) * g.rank;
        f32x16w d{};
        for (int k = 0; k < g.rank; k += 16) {
          half8w hi{}, lo{}, bw{};
          if (k + h * 8 < g.rank) {
            bw = *reinterpret_cast<const half8w*>(B + k + h * 8);
            if (mine) {
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float v = hr[k + h * 8 + i] * up;
                hi[i] = (_Float16)v;
                lo[i] = (_Float16)(v - (float)hi[i]);
              }
            }
          }
          d = __builtin_amdgcn_mfma_f32_32x32x16_f16(hi, bw, d, 0, 0, 0);
          d = __builtin_amdgcn_mfma_f32_32x32x16_f16(lo, bw, d, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < E; ++i) {
          // only the adapter's own rows: an Inf or NaN of its B stays out of the others
          const int ri = 8 * (i >> 2) + 4 * h + (i & 3);
          const float f = __shfl(down, ri);
          acc[i] = (rows_of >> ri) & 1 ? __builtin_fmaf(f, d[i], acc[i]) : acc[i];
        }
      }
    }
#pragma unroll
    for (int i = 0; i < E; ++i) red[wave][i][lane] = acc[i];
    __syncthreads();
    // 32x32 accumulator layout: element i of lane l is (row 8(i/4) + 4(l/32) + i%4, col l%32);
    // the waves share the elements, each summed over the S partial tiles in a fixed order
    for (int i = wave; i < E; i += kS) {
      float v = red[0][i][lane];
#pragma unroll
      for (int w = 1; w < kS; ++w) v += red[w][i][lane];
      const int r = 8 * (i >> 2) + 4 * h + (i & 3);
      const int yr = MODE == kLora ? __shfl(src, r) : row0 + r;
      if constexpr (MODE == kGated) {
        const float u = __shfl_down(v, 16, 32);  // the up row of column j is held by lane + 16
        const int64_t o = (int64_t)blockIdx.x * 16 + j;
        if (j < 16 && o < nh && r < rows) g.Y[yr * nh + o] = f2h_bits(silu_f32(v) * u);
      } else {
        const int64_t o = (int64_t)blockIdx.x * 32 + j;
        if (o < N && r < rows) g.Y[yr * N + o] = f2h_bits(v);
      }
    }
  };
  if (rows <= 8) return run(std::integral_constant<int, 4>{});
  if (rows <= 16) return run(std::integral_constant<int, 8>{});
  run(std::integral_constant<int, 16>{});
}

template <int BITS>
void launch_bits(const GroupedArgs& g, int mode, dim3 grid, hipStream_t stream) {
  if (mode == kPlain)
    hipLaunchKernelGGL((k_skinny<kPlain, BITS>), grid, dim3(kS * 64), 0, stream, g);
  else if (mode == kGated)
    hipLaunchKernelGGL((k_skinny<kGated, BITS>), grid, dim3(kS * 64), 0, stream, g);
  else
    hipLaunchKernelGGL((k_skinny<kLora, BITS>), grid, dim3(kS * 64), 0, stream, g);
}

}  // namespace

hipError_t launch_grouped_skinny(GroupedArgs g, int mode, int w_bit, hipStream_t stream) {
  const int64_t outs = mode == kGated ? g.N / 2 : g.N, per = mode == kGated ? 16 : 32;
  const int64_t parts = mode == kLora ? 1 : g.groups < g.n ? g.groups : g.n;
  const dim3 grid((unsigned)((outs + per - 1) / per), (unsigned)((g.n + 31 * parts) / 32));
  if (w_bit == 8) launch_bits<8>(g, mode, grid, stream);
  else if (w_bit == 3) launch_bits<3>(g, mode, grid, stream);
  else launch_bits<4>(g, mode, grid, stream);
  return hipGetLastError();
}

}  // namespace awq
