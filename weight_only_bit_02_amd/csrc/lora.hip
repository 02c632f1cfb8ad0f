// Adapters, first product: scale[a] X[i] A_a^T for the row's adapter a = ids[i]. The second
// product rides on the linear itself (grouped_gemm.hpp, grouped_stream.hpp).
//
// A block takes 16 rows, 32 ranks (16 if there are no more) and one of the adapters among its
// rows (slot i of the grid: the i-th in order of first appearance), so an adapter's A is read
// once per 16 rows that share it. Eight waves split K, 64 channels at a time, each with a ring
// of its own in LDS that runs 3 or 4 steps ahead (no barrier), and meet in LDS in a fixed
// order. v_mfma_f32_16x16x32_f16 wants neighbouring lanes on neighbouring rows, an L1 access
// per lane when loaded in that order (it bounded a kernel that did so: 48 rows of 16 adapters x
// 4096 took 15.5 us); the DMA's neighbouring lanes take 128 contiguous bytes of a row instead,
// stored so that the reads have no bank conflicts. The sums are fp32; a row's 32 values then
// leave as fp16 hi + lo under one power of two: 22 significant bits of the largest, for the
// matrix cores of the second product. Bound by latency (ids, first step, sums): one row x 4096,
// rank 16: 4.5 us; 48 rows of 32 adapters, rank 32: 7.1; 2048 rows in runs, rank 16: 8.3.
#include "common.hpp"
#include "groups.hpp"
#include "launch.hpp"
#include "widen.hpp"

namespace awq {

namespace {

typedef float f32x4s __attribute__((ext_vector_type(4)));

constexpr int kS = 8;    // waves
constexpr int kC = 64;   // channels of a step: 8 slots of 16 bytes a row

// NR: ranks of the block, 16 or 32.
template <int NR>
__global__ void __launch_bounds__(kS * 64)
    k_shrink(const uint16_t* X, int n, int64_t K, const uint16_t* A, const float* scale, int adapters,
             int rank, const int32_t* ids, const int32_t* order, LoraRow* H) {
  constexpr int kRows = 16 + NR, kStep = kRows * 8, kSends = kRows / 8, NS = NR == 16 ? 4 : 3;
  __shared__ __attribute__((aligned(16))) uint4 lds[kS * NS * kStep];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c16 = lane & 15, kg = lane >> 4;
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
  const int j0 = blockIdx.z * kLoraBlock + c16, j1 = j0 + 16;  // this lane's ranks

  // DMA i of a step: rows 8 i .. 8 i + 7 (of X, then of A), row r's piece p in slot p ^ (r % 8);
  // ranks past the last read the last one
  uint32_t at[kSends];
#pragma unroll
  for (int i = 0; i < kSends; ++i) {
    const int r = i * 8 + (lane >> 3), piece = (lane & 7) ^ (r & 7);
    int row = __shfl(src, r & 15);
    if (i >= 2) {
      row = blockIdx.z * kLoraBlock + r - 16;
      row = row < rank ? row : rank - 1;
    }
    at[i] = (uint32_t)row * (uint32_t)(K * 2) + piece * 16;
  }
  const u32x4 xs = buffer_words(X), as = buffer_words(A + (int64_t)ad * rank * K);
  uint4* const ring = lds + wave * (NS * kStep);
  const uint32_t ring_at = lds_address(lds) + wave * (NS * kStep * 16);
  const int steps = ((int)(K / kC) - wave + kS - 1) / kS;  // this wave's: wave, wave + kS, ...
  auto send = [&](int step, int buf) __attribute__((always_inline)) {
    const uint32_t k = (uint32_t)(step * kS + wave) * (kC * 2);
#pragma unroll
    for (int i = 0; i < kSends; ++i) dma16_own(i < 2 ? xs : as, ring_at + (buf * kStep + i * 64) * 16, at[i], k);
  };
  for (int i = 0; i < NS && i < steps; ++i) send(i, i);
  f32x4s acc0{}, acc1{};
  int buf = 0;
  for (int step = 0; step < steps; ++step) {
    if (step + NS <= steps)
      asm volatile("s_waitcnt vmcnt(%0)" ::"n"((NS - 1) * kSends) : "memory");
    else
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    const uint4* const b = ring + buf * kStep;
    half8w x[2], u[2], v[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int slot = c16 * 8 + ((s * 4 + kg) ^ (c16 & 7));
      x[s] = __builtin_bit_cast(half8w, b[slot]);
      u[s] = __builtin_bit_cast(half8w, b[128 + slot]);
      if constexpr (NR == 32) v[s] = __builtin_bit_cast(half8w, b[256 + slot]);
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // read: the buffer is free
    if (step + NS < steps) send(step + NS, buf);
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      acc0 = __builtin_amdgcn_mfma_f32_16x16x32_f16(x[s], u[s], acc0, 0, 0, 0);
      if constexpr (NR == 32) acc1 = __builtin_amdgcn_mfma_f32_16x16x32_f16(x[s], v[s], acc1, 0, 0, 0);
    }
    buf = buf + 1 < NS ? buf + 1 : 0;
  }
  __syncthreads();  // no ring is in use any more
  float(*const red)[8][64] = reinterpret_cast<float(*)[8][64]>(lds);
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
  const bool finite0 = __builtin_isfinite(v0), finite1 = __builtin_isfinite(v1);
  float mx = fmaxf(finite0 ? __builtin_fabsf(v0) : 0.0f, finite1 ? __builtin_fabsf(v1) : 0.0f);
#pragma unroll
  for (int d = 1; d < 16; d <<= 1) mx = fmaxf(mx, __shfl_xor(mx, d));
  // the row's power of two, by its largest finite value (2^126 at most: its inverse is normal)
  const uint32_t of_mx = __builtin_bit_cast(uint32_t, mx) >> 23, ex = of_mx < 253 ? of_mx : 253;
  const bool fit = ex >= 1;  // zero or tiny: as it is
  const float up = fit ? __builtin_bit_cast(float, (254u - ex) << 23) : 1.0f;
  const int to = __shfl(src, row), of = __shfl(id, row);
  if (of != ad) return;
  LoraRow* const h = H + (int64_t)to * gridDim.z + blockIdx.z;
  const _Float16 h0 = (_Float16)(v0 * up), h1 = (_Float16)(v1 * up);
  h->hi[c16] = __builtin_bit_cast(uint16_t, h0);
  h->hi[16 + c16] = __builtin_bit_cast(uint16_t, h1);
  h->lo[c16] = finite0 ? f2h_bits(v0 * up - (float)h0) : 0;  // (Inf - Inf)
  h->lo[16 + c16] = finite1 ? f2h_bits(v1 * up - (float)h1) : 0;
  if (c16 == 0) h->f = fit ? __builtin_bit_cast(float, ex << 23) : 1.0f;
}

}  // namespace

hipError_t launch_lora_shrink(const uint16_t* X, int n, int64_t K, const uint16_t* A, const float* scale,
                              int adapters, int rank, const int32_t* ids, const int32_t* order,
                              LoraRow* H, hipStream_t stream) {
  const dim3 grid((unsigned)((n + 15) / 16), (unsigned)(adapters < 16 ? adapters : 16),
                  (unsigned)((rank + kLoraBlock - 1) / kLoraBlock));
  hipLaunchKernelGGL((rank <= 16 ? k_shrink<16> : k_shrink<32>), grid, dim3(kS * 64), 0, stream, X, n, K, A,
                     scale, adapters, rank, ids, order, H);
  return hipGetLastError();
}

}  // namespace awq
