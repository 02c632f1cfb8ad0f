// Adapters, first product: H[i] = scale[a] X[i] A_a^T (fp32 [n][rank]) for the row's adapter
// a = ids[i]. The second product rides on the linear itself (grouped_gemm.hpp,
// grouped_skinny.hip).
//
// A block takes 32 rows, 32 ranks and one of the adapters among its rows (slot i of the grid:
// the i-th in order of first appearance), so an adapter's A is read once per 32 rows that
// share it. Eight waves split K and meet in LDS in a fixed order. Within 64 channels lane
// half h covers [32 h, 32 h + 32) of a row of X and of A: 64 contiguous bytes per lane.
#include "common.hpp"
#include "launch.hpp"
#include "widen.hpp"

namespace awq {

namespace {

constexpr int kS = 8;

__global__ void __launch_bounds__(kS * 64)
    k_shrink(const uint16_t* X, int n, int64_t K, const uint16_t* A, const float* scale, int adapters,
             int rank, const int32_t* ids, const int32_t* order, float* H) {
  __shared__ float red[kS][16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, m32 = lane & 31, kh = lane >> 5;
  const int p = blockIdx.x * 32 + m32;
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
  const int j = blockIdx.z * 32 + m32;  // this lane's rank (past the last: the last, not stored)
  const uint16_t* const ap = A + ((int64_t)ad * rank + (j < rank ? j : rank - 1)) * K + kh * 32;
  const uint16_t* const xp = X + (int64_t)src * K + kh * 32;
  const int64_t C = K / 64, c0 = C * wave / kS, c1 = C * (wave + 1) / kS;
  f32x16w acc{};
#pragma unroll 4
  for (int64_t c = c0; c < c1; ++c) {
    half8w x[4], a[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      x[s] = *reinterpret_cast<const half8w*>(xp + c * 64 + s * 8);
      a[s] = *reinterpret_cast<const half8w*>(ap + c * 64 + s * 8);
    }
#pragma unroll
    for (int s = 0; s < 4; ++s) acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(x[s], a[s], acc, 0, 0, 0);
  }
#pragma unroll
  for (int e = 0; e < 16; ++e) red[wave][e][lane] = acc[e];
  __syncthreads();
  const float sc = scale[ad];
  // 32x32 accumulator layout: element e of lane l is (row 8(e/4) + 4(l/32) + e%4, col l%32)
#pragma unroll
  for (int i = 0; i < 16 / kS; ++i) {
    const int e = wave * (16 / kS) + i;
    float v = red[0][e][lane];
#pragma unroll
    for (int w = 1; w < kS; ++w) v += red[w][e][lane];
    const int r = 8 * (e >> 2) + 4 * kh + (e & 3);
    const int row = __shfl(src, r), of = __shfl(id, r);
    if (of == ad && j < rank) H[(int64_t)row * rank + j] = sc * v;
  }
}

}  // namespace

hipError_t launch_lora_shrink(const uint16_t* X, int n, int64_t K, const uint16_t* A, const float* scale,
                              int adapters, int rank, const int32_t* ids, const int32_t* order, float* H,
                              hipStream_t stream) {
  const dim3 grid((unsigned)((n + 31) / 32), (unsigned)(adapters < 32 ? adapters : 32),
                  (unsigned)((rank + 31) / 32));
  hipLaunchKernelGGL(k_shrink, grid, dim3(kS * 64), 0, stream, X, n, K, A, scale, adapters, rank, ids,
                     order, H);
  return hipGetLastError();
}

}  // namespace awq
