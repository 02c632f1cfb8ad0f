// Rows of a batch by group (experts, adapters): helpers of the kernels that read the
// offsets and the order that awq_group_rows / awq_moe_route write. The host never sees
// them, so every kernel clamps what it reads to the sizes the host passed: wrong contents
// give wrong results, never an access out of range.
#pragma once

#include "common.hpp"
#include "widen.hpp"

namespace awq {

typedef float f32x4w __attribute__((ext_vector_type(4)));

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

// Descriptor of the memory from p on (uniform): raw, bytes up to 2^32 - 1 (a dword
// that holds the last one reads as zero).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_at(const void* p) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, -1, 0x00020000);
}

// 16 bytes per lane from offset `lane_at` + `at` of b to consecutive slots from lds on. (The
// global_load_lds form counts as a flat access, after which the compiler waits for everything.)
__device__ __forceinline__ void dma16(__amdgpu_buffer_rsrc_t b, uint4* lds, uint32_t lane_at, uint32_t at) {
#if defined(__HIP_DEVICE_COMPILE__)  // the host pass does not know the 16-byte form
  __builtin_amdgcn_raw_ptr_buffer_load_lds(b, (lds_void*)lds, 16, lane_at, at, 0, 0);
#endif
}

// The same as an instruction that the compiler neither counts nor waits for, to the LDS address
// `to` (uniform): the caller waits (vmcnt) before the data is read and before the wave ends, and
// lets no read of LDS that must come before or after pass it. It has no output register. The wait
// states are those that the assembler leaves to the writer: one after m0, five after a vector
// instruction that wrote b or at (1% of a GEMM's time, were they left out).
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ u32x4 buffer_words(const void* p) {
  const uint64_t a = (uint64_t)p;
  return u32x4{(uint32_t)a, (uint32_t)(a >> 32) & 0xFFFF, 0xFFFFFFFFu, 0x00020000u};
}

__device__ __forceinline__ uint32_t lds_address(uint4* p) {
  return __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_void*)p);
}

__device__ __forceinline__ void dma16_own(u32x4 b, uint32_t to, uint32_t lane_at, uint32_t at) {
#if defined(__HIP_DEVICE_COMPILE__)
  asm volatile("s_nop 4\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds" ::"v"(lane_at), "s"(b), "s"(at), "{m0}"(to)
               : "memory");
#endif
}

}  // namespace awq
