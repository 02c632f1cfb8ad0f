// Expert outputs back to token order: Y[t] = fp16(add[t] + sum_j w[t][j] P[pos[t][j]]).
//
// A memory-bound gather: every row of P is read once, in 16-byte pieces, and a thread keeps
// the top_k pieces of its 8 columns in flight (eight at a time) before it adds them. The sum
// runs in fp32 in the order of the choices and is rounded to fp16 once. Pairs whose position
// lies past the last group (no expert) add nothing and are not read. 4096 tokens x 8 x 4096: 58
// us, 5.1 TB/s read and written, what a copy reaches; 16 tokens: 3.4 us.
#include "common.hpp"
#include "launch.hpp"

namespace awq {

namespace {

constexpr int kThreads = 128;

typedef _Float16 half8c __attribute__((ext_vector_type(8)));

// Columns [8 c, 8 c + 8) of token t; N % 8 == 0, so every piece is 16-byte aligned. KB: pieces
// in flight. UNI: the rows' pieces are whole waves, so a wave has one token (scalar loads).
template <int KB, bool UNI>
__global__ void __launch_bounds__(kThreads)
    k_combine8(const uint16_t* P, const float* weights, const int32_t* pos, const int32_t* valid,
               int64_t T, int top_k, int64_t N, const uint16_t* add, uint16_t* Y, int per_row) {
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (i >= T * per_row) return;
  int t, c;  // (T < 2^31)
  if constexpr (UNI) {
    const int wave = __builtin_amdgcn_readfirstlane((int)(i >> 6)), waves = per_row >> 6;
    t = wave / waves;
    c = (wave - t * waves) * 64 + (threadIdx.x & 63);
  } else {
    t = (int)(i / per_row);
    c = (int)(i - (int64_t)t * per_row);
  }
  const int64_t pairs = T * top_k, pt = (int64_t)t * top_k;
  const int last = (int64_t)*valid < pairs ? *valid : (int)pairs;
  float acc[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) acc[j] = 0.0f;
  half8c a{};
  if (add) a = *reinterpret_cast<const half8c*>(add + (int64_t)t * N + c * 8);
  for (int k0 = 0; k0 < top_k; k0 += KB) {
    half8c v[KB];
    float w[KB];
    bool on[KB];
#pragma unroll
    for (int k = 0; k < KB; ++k) {
      const int kk = k0 + k < top_k ? k0 + k : top_k - 1;
      const int p = pos[pt + kk];
      on[k] = k0 + k < top_k && (unsigned)p < (unsigned)(last < 0 ? 0 : last);
      w[k] = weights[pt + kk];
      v[k] = on[k] ? *reinterpret_cast<const half8c*>(P + (int64_t)p * N + c * 8) : half8c{};
    }
    if (k0 == 0) {
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[j] = (float)a[j];
    }
#pragma unroll
    for (int k = 0; k < KB; ++k)
      if (on[k]) {
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] = __builtin_fmaf(w[k], (float)v[k][j], acc[j]);
      }
  }
  half8c y;
#pragma unroll
  for (int j = 0; j < 8; ++j) y[j] = (_Float16)acc[j];
  *reinterpret_cast<half8c*>(Y + (int64_t)t * N + c * 8) = y;
}

// Any N: one column per thread.
__global__ void __launch_bounds__(kThreads)
    k_combine1(const uint16_t* P, const float* weights, const int32_t* pos, const int32_t* valid,
               int64_t T, int top_k, int64_t N, const uint16_t* add, uint16_t* Y) {
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (i >= T * N) return;
  const int64_t t = i / N, c = i % N;
  const int64_t pairs = T * top_k;
  const int last = (int64_t)*valid < pairs ? *valid : (int)pairs;
  float acc = add ? h2f(add[i]) : 0.0f;
  for (int k = 0; k < top_k; ++k) {
    const int p = pos[t * top_k + k];
    if ((unsigned)p < (unsigned)(last < 0 ? 0 : last))
      acc = __builtin_fmaf(weights[t * top_k + k], h2f(P[(int64_t)p * N + c]), acc);
  }
  Y[i] = f2h_bits(acc);
}

}  // namespace

hipError_t launch_combine(const uint16_t* P, const float* weights, const int32_t* pos,
                          const int32_t* valid, int64_t T, int top_k, int64_t N, const uint16_t* add,
                          uint16_t* Y, hipStream_t stream) {
  if (N % 8 == 0) {
    const int64_t n = T * (N / 8);
    const bool uni = N % 512 == 0 && n >> 6 < 0x7FFFFFFF;
    auto* const f = top_k <= 2   ? (uni ? k_combine8<2, true> : k_combine8<2, false>)
                    : top_k <= 4 ? (uni ? k_combine8<4, true> : k_combine8<4, false>)
                                 : (uni ? k_combine8<8, true> : k_combine8<8, false>);
    hipLaunchKernelGGL(f, dim3((unsigned)((n + kThreads - 1) / kThreads)), dim3(kThreads), 0, stream, P,
                       weights, pos, valid, T, top_k, N, add, Y, (int)(N / 8));
  } else {
    const int64_t n = T * N;
    hipLaunchKernelGGL(k_combine1, dim3((unsigned)((n + kThreads - 1) / kThreads)), dim3(kThreads), 0,
                       stream, P, weights, pos, valid, T, top_k, N, add, Y);
  }
  return hipGetLastError();
}

}  // namespace awq
