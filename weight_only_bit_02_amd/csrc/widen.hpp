// Packed codes -> fp16 MFMA operands, shared by the GEMMs that widen their codes in
// registers (gemm_wide.hip, grouped_gemm.hpp, grouped_stream.hpp).
#pragma once

#include "common.hpp"

namespace awq {

typedef _Float16 half8w __attribute__((ext_vector_type(8)));
typedef _Float16 half2w __attribute__((ext_vector_type(2)));
typedef float f32x16w __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) void lds_void;

__device__ __forceinline__ uint32_t wide_magic() {
  uint32_t m;
  asm volatile("v_mov_b32 %0, 0x64006400" : "=v"(m));
  return m;
}

// One packed word -> its 8 dequantized fp16 channels (q - z) sc, in channel order. zz holds
// -(1024 + z) and zz64 -(64 + z) in both halves, s2 the scale in both halves.
__device__ __forceinline__ half8w widen_word(uint32_t w, half2w zz, half2w zz64, half2w s2,
                                             uint32_t magic) {
  const uint32_t w8 = w >> 8;
  const uint32_t u0 = (w & 0x000F000Fu) | magic, u1 = (w & 0x00F000F0u) | 0x54005400u;
  const uint32_t u2 = (w8 & 0x000F000Fu) | magic, u3 = (w8 & 0x00F000F0u) | 0x54005400u;
  const half2w d0 = (__builtin_bit_cast(half2w, u0) + zz) * s2;
  const half2w d1 = (__builtin_bit_cast(half2w, u1) + zz64) * s2;
  const half2w d2 = (__builtin_bit_cast(half2w, u2) + zz) * s2;
  const half2w d3 = (__builtin_bit_cast(half2w, u3) + zz64) * s2;
  return half8w{d0[0], d0[1], d1[0], d1[1], d2[0], d2[1], d3[0], d3[1]};
}

// Two packed 8-bit words -> their 8 channels (q - z) sc, in channel order: v_perm_b32 against
// 0x64646464 puts byte pairs under the 0x64 exponent byte, (1024 + a, 1024 + b) exactly; zz holds
// -(1024 + z) in both halves.
__device__ __forceinline__ half8w widen_word8(uint32_t w0, uint32_t w1, half2w zz, half2w s2,
                                              uint32_t magic8) {
  const half2w d0 = (__builtin_bit_cast(half2w, __builtin_amdgcn_perm(magic8, w0, 0x04010400u)) + zz) * s2;
  const half2w d1 = (__builtin_bit_cast(half2w, __builtin_amdgcn_perm(magic8, w0, 0x04030402u)) + zz) * s2;
  const half2w d2 = (__builtin_bit_cast(half2w, __builtin_amdgcn_perm(magic8, w1, 0x04010400u)) + zz) * s2;
  const half2w d3 = (__builtin_bit_cast(half2w, __builtin_amdgcn_perm(magic8, w1, 0x04030402u)) + zz) * s2;
  return half8w{d0[0], d0[1], d1[0], d1[1], d2[0], d2[1], d3[0], d3[1]};
}

// Four channel pairs of 3-bit codes -> 8 channels (q - z) sc: pair t takes its low bits from
// field f + t of the low-plane word and bit 2 from bit p + t of the high-plane word (both in
// each 16-bit half), under the 0x6400 exponent: exactly (1024 + q, 1024 + q').
__device__ __forceinline__ half8w widen_word3(uint32_t lo, uint32_t hi, int f, int p, half2w zz,
                                              half2w s2, uint32_t magic) {
  half2w d[4];
#pragma unroll
  for (int t = 0; t < 4; ++t)
    d[t] = (__builtin_bit_cast(half2w, widen3_pair(lo, hi, f + t, p + t, magic)) + zz) * s2;
  return half8w{d[0][0], d[0][1], d[1][0], d[1][1], d[2][0], d[2][1], d[3][0], d[3][1]};
}

}  // namespace awq
