// Rows of a batch by group (experts, adapters): helpers of the kernels that read the
// offsets and the order that awq_group_rows / awq_moe_route write. The host never sees
// them, so every kernel clamps what it reads to the sizes the host passed: wrong contents
// give wrong results, never an access out of range.
#pragma once

#include "common.hpp"

namespace awq {

constexpr int kMaxGroups = 512;

// Inclusive sum over the wave.
__device__ __forceinline__ int wave_scan(int v, int lane) {
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) {
    const int o = __shfl_up(v, d);
    v += lane >= d ? o : 0;
  }
  return v;
}

// Rows [lo, hi) of group e.
__device__ __forceinline__ void group_range(const int32_t* offsets, int e, int n, int& lo, int& hi) {
  const int a = offsets[e], b = offsets[e + 1];
  lo = a < 0 ? 0 : a > n ? n : a;
  hi = b < lo ? lo : b > n ? n : b;
}

// One tile of at most BM rows of one group.
struct RowTile {
  int e;     // the group
  int row0;  // its first row (position in group order)
  int rows;  // 1 .. BM; 0: no such tile
};

// Tiles of BM rows that the groups need together (uniform over the wave).
template <int BM>
__device__ __forceinline__ int count_tiles(const int32_t* offsets, int groups, int n, int lane) {
  int sum = 0;
  for (int c = 0; c < groups; c += kWave) {
    int t = 0;
    if (c + lane < groups) {
      int lo, hi;
      group_range(offsets, c + lane, n, lo, hi);
      t = (hi - lo + BM - 1) / BM;
    }
    sum += __shfl(wave_scan(t, lane), kWave - 1);
  }
  return sum;
}

// Tile `at` of them, in group order (uniform over the wave).
template <int BM>
__device__ __forceinline__ RowTile find_tile(const int32_t* offsets, int groups, int n, int at,
                                             int lane) {
  int before = 0;
  for (int c = 0; c < groups; c += kWave) {
    int lo = 0, hi = 0;
    if (c + lane < groups) group_range(offsets, c + lane, n, lo, hi);
    const int t = (hi - lo + BM - 1) / BM;
    const int incl = before + wave_scan(t, lane);
    const uint64_t m = __ballot(incl > at);
    if (m) {
      const int src = __ffsll((unsigned long long)m) - 1;
      const int k = at - (__shfl(incl, src) - __shfl(t, src));  // tile k of that group
      lo = __shfl(lo, src);
      hi = __shfl(hi, src);
      if ((unsigned)k >= (unsigned)((hi - lo + BM - 1) / BM)) break;  // sums that wrapped (wrong offsets)
      const int row0 = lo + k * BM;
      return RowTile{c + src, row0, hi - row0 < BM ? hi - row0 : BM};
    }
    before = __shfl(incl, kWave - 1);
  }
  return RowTile{0, 0, 0};
}

}  // namespace awq
