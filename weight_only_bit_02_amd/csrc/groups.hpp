// Rows of a batch by group (experts, adapters): helpers of the kernels that read the
// offsets and the order that awq_group_rows / awq_moe_route write. The host never sees
// them, so every kernel clamps what it reads to the sizes the host passed: wrong contents
// give wrong results, never an access out of range.
#pragma once

#include "common.hpp"

namespace awq {

constexpr int kMaxGroups = 512;

// Inclusive sum over the wave: DPP row shifts, then the row broadcasts.
__device__ __forceinline__ int wave_scan(int v) {
#define AWQ_STEP(CTRL, ROWS) v += __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xF, false)
  AWQ_STEP(0x111, 0xF);  // row_shr:1
  AWQ_STEP(0x112, 0xF);
  AWQ_STEP(0x114, 0xF);
  AWQ_STEP(0x118, 0xF);
  AWQ_STEP(0x142, 0xA);  // row_bcast:15 into rows 1 and 3
  AWQ_STEP(0x143, 0xC);  // row_bcast:31 into rows 2 and 3
#undef AWQ_STEP
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
    sum += __builtin_amdgcn_readlane(wave_scan(t), kWave - 1);
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
    const int incl = before + wave_scan(t);
    const uint64_t m = __ballot(incl > at);
    if (m) {
      const int src = __ffsll((unsigned long long)m) - 1;
      // tile k of that group
      const int k = at - (__builtin_amdgcn_readlane(incl, src) - __builtin_amdgcn_readlane(t, src));
      lo = __builtin_amdgcn_readlane(lo, src);
      hi = __builtin_amdgcn_readlane(hi, src);
      if ((unsigned)k >= (unsigned)((hi - lo + BM - 1) / BM)) break;  // sums that wrapped (wrong offsets)
      const int row0 = lo + k * BM;
      return RowTile{c + src, row0, hi - row0 < BM ? hi - row0 : BM};
    }
    before = __builtin_amdgcn_readlane(incl, kWave - 1);
  }
  return RowTile{0, 0, 0};
}

}  // namespace awq
