// Adapters, first product: scale[a] X[i] A_a^T for the row's adapter a = ids[i]. The second
// product rides on the linear itself (grouped_gemm.hpp, grouped_stream.hpp).
//
// A block takes 16 rows, 32 ranks and one of the adapters among its rows (slot i of the grid:
// the i-th in order of first appearance), so an adapter's A is read once per 16 rows that
// share it. Sixteen waves split K, each with all the loads of a 128-channel step in flight
// (v_mfma_f32_16x16x32_f16: lane l holds 64 contiguous bytes of X row l % 16 and of A rows
// l % 16 and 16 + l % 16), and meet in LDS in a fixed order. The sums are fp32; a row's 32
// values then leave as fp16 hi + lo under one power of two: 22 significant bits of the
// largest, for the matrix cores of the second product.
#include "common.hpp"
#include "launch.hpp"
#include "widen.hpp"

namespace awq {

namespace {

typedef float f32x4s __attribute__((ext_vector_type(4)));

constexpr int kS = 16;

__global__ void __launch_bounds__(kS * 64)
    k_shrink(const uint16_t* X, int n, int64_t K, const uint16_t* A, const float* scale, int adapters,
             int rank, const int32_t* ids, const int32_t* order, LoraRow* H) {
  __shared__ float red[kS][8][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c16 = lane & 15, kg = lane >> 4;
  const int p = blockIdx.x * 16 + c16;
  int src = p < n ? p : n - 1;
  if (order) {
    const int o = order[src];
    src = (unsigned)o < (unsigned)n ? o : 0;
  }
  const int id = p < n ? ids[src] : -1;
  uint64_t rest = __ballot((unsigned)id < (unsigned)adapters);
  int ad = -1;
  for (int i = 0; i <= (int)blockIdx.y; ++i) {
    if (!rest) return;  // fewer adapters than slots (uniform over the block)
    ad = __builtin_amdgcn_readlane(id, __ffsll((unsigned long long)rest) - 1);
    rest &= ~__ballot(id == ad);
  }
  const int j0 = blockIdx.z * kLoraBlock + c16, j1 = j0 + 16;  // this lane's ranks (past the last: the last)
  const uint16_t* const a0 = A + ((int64_t)ad * rank + (j0 < rank ? j0 : rank - 1)) * K + kg * 32;
  const uint16_t* const a1 = A + ((int64_t)ad * rank + (j1 < rank ? j1 : rank - 1)) * K + kg * 32;
  const uint16_t* const xp = X + (int64_t)src * K + kg * 32;
  const int64_t C = K / 128, c0 = C * wave / kS, c1 = C * (wave + 1) / kS;
  f32x4s acc0{}, acc1{};
#pragma unroll 2
  for (int64_t c = c0; c < c1; ++c) {
    half8w x[4], u[4], v[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      x[s] = *reinterpret_cast<const half8w*>(xp + c * 128 + s * 8);
      u[s] = *reinterpret_cast<const half8w*>(a0 + c * 128 + s * 8);
      v[s] = *reinterpret_cast<const half8w*>(a1 + c * 128 + s * 8);
    }
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      acc0 = __builtin_amdgcn_mfma_f32_16x16x32_f16(x[s], u[s], acc0, 0, 0, 0);
      acc1 = __builtin_amdgcn_mfma_f32_16x16x32_f16(x[s], v[s], acc1, 0, 0, 0);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    red[wave][i][lane] = acc0[i];
    red[wave][4 + i][lane] = acc1[i];
  }
  __syncthreads();
  if (wave >= 4) return;
  // element i of lane l: row 4 (l / 16) + i, rank l % 16 (of either half); wave i takes element i
  const int row = 4 * kg + wave;
  float v0 = red[0][wave][lane], v1 = red[0][4 + wave][lane];
#pragma unroll
  for (int w = 1; w < kS; ++w) {
    v0 += red[w][wave][lane];
    v1 += red[w][4 + wave][lane];
  }
  const float sc = scale[ad];
  v0 = j0 < rank ? sc * v0 : 0.0f;
  v1 = j1 < rank ? sc * v1 : 0.0f;
  float mx = fmaxf(__builtin_fabsf(v0), __builtin_fabsf(v1));
#pragma unroll
  for (int d = 1; d < 16; d <<= 1) mx = fmaxf(mx, __shfl_xor(mx, d));
  const uint32_t ex = __builtin_bit_cast(uint32_t, mx) >> 23;
  const bool fit = ex >= 1 && ex < 253;  // zero, tiny or not finite: as it is
  const float up = fit ? __builtin_bit_cast(float, (254u - ex) << 23) : 1.0f;
  const int to = __shfl(src, row), of = __shfl(id, row);
  if (of != ad) return;
  LoraRow* const h = H + (int64_t)to * gridDim.z + blockIdx.z;
  const _Float16 h0 = (_Float16)(v0 * up), h1 = (_Float16)(v1 * up);
  h->hi[c16] = __builtin_bit_cast(uint16_t, h0);
  h->hi[16 + c16] = __builtin_bit_cast(uint16_t, h1);
  h->lo[c16] = f2h_bits(v0 * up - (float)h0);
  h->lo[16 + c16] = f2h_bits(v1 * up - (float)h1);
  if (c16 == 0) h->f = fit ? __builtin_bit_cast(float, ex << 23) : 1.0f;
}

}  // namespace

hipError_t launch_lora_shrink(const uint16_t* X, int n, int64_t K, const uint16_t* A, const float* scale,
                              int adapters, int rank, const int32_t* ids, const int32_t* order,
                              LoraRow* H, hipStream_t stream) {
  const dim3 grid((unsigned)((n + 15) / 16), (unsigned)(adapters < 16 ? adapters : 16),
                  (unsigned)((rank + kLoraBlock - 1) / kLoraBlock));
  hipLaunchKernelGGL(k_shrink, grid, dim3(kS * 64), 0, stream, X, n, K, A, scale, adapters, rank, ids,
                     order, H);
  return hipGetLastError();
}

}  // namespace awq
