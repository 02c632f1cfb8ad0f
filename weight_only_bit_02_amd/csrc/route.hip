// Router of a mixture of experts and the grouping of rows.
//
// Route: per token the top_k largest of E logits (ties to the lowest expert, -inf never
// chosen) and their softmax weights; the T top_k (token, choice) pairs are then put in
// expert order by a stable counting sort: offsets[e] = pairs of the experts before e,
// order[p] = the pair at position p, pos = its inverse. Pairs without an expert (id -1)
// come last. Grouping alone (adapters of a batch's rows) is the same sort on given ids.
//
//   choose: a wave per token. A lane holds E / 64 logits; a choice is one wave maximum
//     (DPP row shifts and broadcasts, no LDS) and a ballot per held value, which gives the
//     lowest index among equals. fp32 throughout; expf and the division are the accurate
//     ones: they run once per chosen expert and per logit, beside top_k reductions.
//   sort: a block takes a contiguous run of pairs, each of its 16 waves a contiguous part of
//     it. Within 64 pairs, a pair's rank among equals comes from one ballot per id bit
//     (the lanes whose ids agree in every bit), so the order never depends on scheduling.
//
// Batches of up to kOneBlockPairs pairs run in one block and one launch. Larger ones take
// two: the first writes each block's count per group, the second sums the counts of the
// blocks before it (at most kMaxBlocks rows of E + 1 integers, from L2) and places its run.
#include <hip/hip_runtime.h>

#include "common.hpp"
#include "groups.hpp"
#include "launch.hpp"

namespace awq {

namespace {

constexpr int kThreads = 1024, kWaves = kThreads / kWave;
constexpr int64_t kOneBlockTokens = 64;   // route: tokens that one block serves alone
constexpr int64_t kOneBlockPairs = 8192;  // grouping: pairs that one block serves alone
constexpr int64_t kMaxBlocks = 256;

// Maximum over the wave (a scalar): row shifts, then the row broadcasts, then lane 63.
__device__ __forceinline__ float wave_max(float v) {
  constexpr float lowest = -__builtin_huge_valf();
#define AWQ_STEP(CTRL, ROWS)                                                                      \
  v = fmaxf(v, __builtin_bit_cast(                                                                \
                   float, __builtin_amdgcn_update_dpp(__builtin_bit_cast(int, lowest),            \
                                                      __builtin_bit_cast(int, v), CTRL, ROWS, 0xF, \
                                                      false)));
  AWQ_STEP(0x111, 0xF)  // row_shr:1
  AWQ_STEP(0x112, 0xF)
  AWQ_STEP(0x114, 0xF)
  AWQ_STEP(0x118, 0xF)
  AWQ_STEP(0x142, 0xA)  // row_bcast:15 into rows 1 and 3
  AWQ_STEP(0x143, 0xC)  // row_bcast:31 into rows 2 and 3
#undef AWQ_STEP
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
}

// A logit as the router takes it: NaN as -inf (no expert), +inf as the largest finite value.
template <typename LT>
__device__ __forceinline__ float logit(LT raw, bool& bad) {
  float v, top;
  if constexpr (sizeof(LT) == 2) {
    v = h2f(raw);
    top = 65504.0f;
  } else {
    v = raw;
    top = 3.40282346638528859812e38f;
  }
  const bool nan = !(v == v), inf = v > top;
  bad |= nan | inf;
  return nan ? -__builtin_huge_valf() : inf ? top : v;
}

// Token t: lane j < top_k leaves with choice j's expert (or -1); weights and ids are written.
template <typename LT, int V>
__device__ __forceinline__ void choose(const LT* logits, int64_t ld, int64_t t, int E, int top_k,
                                       bool renorm, float* weights, int32_t* ids, bool& bad,
                                       int lane) {
  constexpr float lowest = -__builtin_huge_valf();
  float v[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = i * kWave + lane;
    v[i] = e < E ? logit<LT>(logits[t * ld + e], bad) : lowest;
  }
  float left[V], mine = lowest, first = lowest;
  int id = -1;
#pragma unroll
  for (int i = 0; i < V; ++i) left[i] = v[i];
  for (int j = 0; j < top_k; ++j) {
    float m = left[0];
#pragma unroll
    for (int i = 1; i < V; ++i) m = fmaxf(m, left[i]);
    m = wave_max(m);
    if (m == lowest) break;  // nothing but -inf is left (uniform)
    if (j == 0) first = m;
    int found = -1;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const uint64_t same = __ballot(left[i] == m);
      if (found < 0 && same) {
        const int src = __ffsll((unsigned long long)same) - 1;
        found = i * kWave + src;
        if (lane == src) left[i] = lowest;
      }
    }
    if (lane == j) {
      mine = m;
      id = found;
    }
  }
  float sum = 0.0f, w = 0.0f;
  if (first != lowest) {
    w = mine == lowest ? 0.0f : expf(mine - first);
    if (renorm) {
      sum = w;
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) sum += v[i] == lowest ? 0.0f : expf(v[i] - first);
    }
    w /= wave_sum(sum);
  }
  if (lane < top_k) {
    weights[t * top_k + lane] = w;
    ids[t * top_k + lane] = id;
  }
}

// A group id as a key: itself, or `groups` for anything outside [0, groups).
__device__ __forceinline__ int key_of(int id, int groups) { return (unsigned)id < (unsigned)groups ? id : groups; }

// Lanes of the wave (among `live`) whose key equals this lane's.
__device__ __forceinline__ uint64_t same_key(int key, int bits, uint64_t live) {
  uint64_t m = live;
  for (int b = 0; b < bits; ++b) {
    const uint64_t set = __ballot((key >> b) & 1);
    m &= ((key >> b) & 1) ? set : ~set;
  }
  return m;
}

// Exclusive sums of `count` [n] in LDS, in place, by the whole block; ends with a barrier.
__device__ __forceinline__ void block_exclusive(int* count, int n, int* part, int tid) {
  const int lane = tid & 63, wave = tid >> 6;
  int base = 0;
  for (int c = 0; c < n; c += kThreads) {
    const int v = c + tid < n ? count[c + tid] : 0;
    const int incl = wave_scan(v);
    __syncthreads();  // part[] of the pass before has been read
    if (lane == 63) part[wave] = incl;
    __syncthreads();
    int before = base, all = 0;
    for (int w = 0; w < kWaves; ++w) {
      before += w < wave ? part[w] : 0;
      all += part[w];
    }
    if (c + tid < n) count[c + tid] = before + incl - v;
    base += all;
  }
  __syncthreads();
}

// Places pairs [p0, p1): next[w][key] (LDS) is the position of wave w's next pair of a key.
// Counting, the sums over the waves and the placement all walk the pairs in order.
// start[key] (LDS): the position of this block's first pair of the key.
__device__ __forceinline__ void place(const int32_t* ids, int64_t p0, int64_t p1, int groups, int bits,
                                      int* next, const int* start, int32_t* order, int32_t* pos,
                                      int tid) {
  const int lane = tid & 63, wave = tid >> 6, keys = groups + 1;
  const int64_t part = ((p1 - p0 + kWaves - 1) / kWaves + kWave - 1) / kWave * kWave;
  const int64_t w0 = p0 + wave * part < p1 ? p0 + wave * part : p1;
  const int64_t w1 = w0 + part < p1 ? w0 + part : p1;
  for (int i = tid; i < kWaves * keys; i += kThreads) next[i] = 0;
  __syncthreads();
  int* const mine = next + wave * keys;
  const uint64_t below = ((uint64_t)1 << lane) - 1;
  for (int64_t p = w0; p < w1; p += kWave) {
    const bool in = p + lane < w1;
    const int key = in ? key_of(ids[p + lane], groups) : 0;
    const uint64_t same = same_key(key, bits, __ballot(in));
    if (in && (same & below) == 0) mine[key] += __popcll(same);  // the first of its equals
    __builtin_amdgcn_wave_barrier();
  }
  __syncthreads();
  for (int k = tid; k < keys; k += kThreads) {
    int at = start[k];
    for (int w = 0; w < kWaves; ++w) {
      const int c = next[w * keys + k];
      next[w * keys + k] = at;
      at += c;
    }
  }
  __syncthreads();
  for (int64_t p = w0; p < w1; p += kWave) {
    const bool in = p + lane < w1;
    const int key = in ? key_of(ids[p + lane], groups) : 0;
    const uint64_t same = same_key(key, bits, __ballot(in));
    const int at = in ? mine[key] + __popcll(same & below) : 0;
    __builtin_amdgcn_wave_barrier();
    if (in) {
      if ((same & below) == 0) mine[key] += __popcll(same);
      order[at] = (int32_t)(p + lane);
      if (pos) pos[p + lane] = at;
    }
    __builtin_amdgcn_wave_barrier();
  }
}

// The block's pairs [p0, p1) counted per key into count[] (LDS, cleared here).
__device__ __forceinline__ void count_keys(const int32_t* ids, int64_t p0, int64_t p1, int groups,
                                           int* count, int tid) {
  for (int k = tid; k <= groups; k += kThreads) count[k] = 0;
  __syncthreads();
  for (int64_t p = p0 + tid; p < p1; p += kThreads) atomicAdd(&count[key_of(ids[p], groups)], 1);
  __syncthreads();
}

// LDS: [count: groups + 1][part: waves][next: waves (groups + 1)]
__device__ __forceinline__ void sort_alone(const int32_t* ids, int64_t n, int groups, int bits, int* lds,
                                           int32_t* offsets, int32_t* order, int32_t* pos, int tid) {
  int* const count = lds;
  int* const part = count + groups + 1;
  int* const next = part + kWaves;
  count_keys(ids, 0, n, groups, count, tid);
  block_exclusive(count, groups + 1, part, tid);
  for (int k = tid; k <= groups; k += kThreads) offsets[k] = count[k];
  place(ids, 0, n, groups, bits, next, count, order, pos, tid);
}

template <typename LT, int V, bool ALONE>
__global__ void __launch_bounds__(kThreads)
    k_route(const LT* logits, int64_t ld, int64_t T, int64_t per_block, int E, int top_k, int renorm,
            int bits, float* weights, int32_t* ids, int32_t* offsets, int32_t* order, int32_t* pos,
            int* counts, uint32_t* flags) {
  extern __shared__ int lds[];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t t0 = blockIdx.x * per_block;
  const int64_t t1 = t0 + per_block < T ? t0 + per_block : T;
  bool bad = false;
  for (int64_t t = t0 + wave; t < t1; t += kWaves)
    choose<LT, V>(logits, ld, t, E, top_k, renorm, weights, ids, bad, lane);
  if (flags && __ballot(bad) && lane == 0) atomicOr(flags, AWQ_FLAG_NONFINITE_INPUT);
  __syncthreads();  // the block's ids are written
  if constexpr (ALONE) {
    sort_alone(ids, T * top_k, E, bits, lds, offsets, order, pos, tid);
  } else {
    count_keys(ids, t0 * top_k, t1 * top_k, E, lds, tid);
    for (int k = tid; k <= E; k += kThreads) counts[(int64_t)blockIdx.x * (E + 1) + k] = lds[k];
  }
}

__global__ void __launch_bounds__(kThreads)
    k_group_alone(const int32_t* ids, int64_t n, int groups, int bits, int32_t* offsets, int32_t* order,
                  int32_t* pos) {
  extern __shared__ int lds[];
  sort_alone(ids, n, groups, bits, lds, offsets, order, pos, threadIdx.x);
}

__global__ void __launch_bounds__(kThreads)
    k_group_count(const int32_t* ids, int64_t n, int64_t per_block, int groups, int* counts) {
  extern __shared__ int lds[];
  const int64_t p0 = blockIdx.x * per_block, p1 = p0 + per_block < n ? p0 + per_block : n;
  count_keys(ids, p0, p1, groups, lds, threadIdx.x);
  for (int k = threadIdx.x; k <= groups; k += kThreads)
    counts[(int64_t)blockIdx.x * (groups + 1) + k] = lds[k];
}

// Second launch: every block sums the counts of all blocks (total) and of those before it.
// LDS: [total: groups + 1][start: groups + 1][part: waves][next: waves (groups + 1)]
__global__ void __launch_bounds__(kThreads)
    k_group_place(const int32_t* ids, int64_t n, int64_t per_block, int groups, int bits,
                  const int* counts, int32_t* offsets, int32_t* order, int32_t* pos) {
  extern __shared__ int lds[];
  const int keys = groups + 1, tid = threadIdx.x;
  int* const total = lds;
  int* const start = total + keys;
  int* const part = start + keys;
  int* const next = part + kWaves;
  const int blocks = gridDim.x, me = blockIdx.x;
  for (int i = tid; i < 2 * keys; i += kThreads) lds[i] = 0;
  __syncthreads();
  // threads as [slices][keys rounded up to a power of two]: integer sums, any order
  int wide = 1;
  while (wide < keys && wide < kThreads) wide <<= 1;
  for (int k = tid & (wide - 1); k < keys; k += wide) {
    int all = 0, before = 0;
    for (int b = tid / wide; b < blocks; b += kThreads / wide) {
      const int c = counts[(int64_t)b * keys + k];
      all += c;
      before += b < me ? c : 0;
    }
    atomicAdd(&total[k], all);
    atomicAdd(&start[k], before);
  }
  __syncthreads();
  block_exclusive(total, keys, part, tid);
  for (int k = tid; k < keys; k += kThreads) {
    start[k] += total[k];
    if (me == 0) offsets[k] = total[k];
  }
  __syncthreads();
  const int64_t p0 = me * per_block, p1 = p0 + per_block < n ? p0 + per_block : n;
  place(ids, p0, p1, groups, bits, next, start, order, pos, tid);
}

int key_bits(int groups) {  // bits of the keys 0 .. groups
  int b = 1;
  while (groups >> b) ++b;
  return b;
}

size_t alone_lds(int groups) { return ((size_t)(groups + 1) * (kWaves + 1) + kWaves) * 4; }
size_t place_lds(int groups) { return ((size_t)(groups + 1) * (kWaves + 2) + kWaves) * 4; }

int64_t group_run(int64_t n) {  // pairs per block of a grouping in two launches
  const int64_t r = (n + kMaxBlocks - 1) / kMaxBlocks;
  return r < 2048 ? 2048 : r;
}
int64_t route_run(int64_t T) {  // tokens per block of a routing in two launches
  const int64_t r = (T + kMaxBlocks - 1) / kMaxBlocks;
  return r < kWaves ? kWaves : r;
}

hipError_t launch_place(const int32_t* ids, int64_t n, int64_t run, int groups, const int* counts,
                        int32_t* offsets, int32_t* order, int32_t* pos, hipStream_t stream) {
  hipLaunchKernelGGL(k_group_place, dim3((unsigned)((n + run - 1) / run)), dim3(kThreads),
                     place_lds(groups), stream, ids, n, run, groups, key_bits(groups), counts, offsets,
                     order, pos);
  return hipGetLastError();
}

template <typename LT, int V>
hipError_t launch_route_v(const void* logits, int64_t ld, int64_t T, int E, int top_k, bool renorm,
                          float* weights, int32_t* ids, int32_t* offsets, int32_t* order, int32_t* pos,
                          int* counts, uint32_t* flags, hipStream_t stream) {
  const int bits = key_bits(E);
  if (T <= kOneBlockTokens) {
    hipLaunchKernelGGL((k_route<LT, V, true>), dim3(1), dim3(kThreads), alone_lds(E), stream,
                       (const LT*)logits, ld, T, T, E, top_k, renorm, bits, weights, ids, offsets, order,
                       pos, counts, flags);
    return hipGetLastError();
  }
  const int64_t run = route_run(T);
  hipLaunchKernelGGL((k_route<LT, V, false>), dim3((unsigned)((T + run - 1) / run)), dim3(kThreads),
                     (size_t)(E + 1) * 4, stream, (const LT*)logits, ld, T, run, E, top_k, renorm, bits,
                     weights, ids, offsets, order, pos, counts, flags);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  return launch_place(ids, T * top_k, run * top_k, E, counts, offsets, order, pos, stream);
}

template <typename LT>
hipError_t launch_route_t(const void* logits, int64_t ld, int64_t T, int E, int top_k, bool renorm,
                          float* weights, int32_t* ids, int32_t* offsets, int32_t* order, int32_t* pos,
                          int* counts, uint32_t* flags, hipStream_t stream) {
  auto* f = E <= 64    ? launch_route_v<LT, 1>
            : E <= 128 ? launch_route_v<LT, 2>
            : E <= 256 ? launch_route_v<LT, 4>
                       : launch_route_v<LT, 8>;
  return f(logits, ld, T, E, top_k, renorm, weights, ids, offsets, order, pos, counts, flags, stream);
}

}  // namespace

size_t group_rows_workspace(int64_t n, int groups) {
  if (n <= kOneBlockPairs) return 0;
  const int64_t run = group_run(n);
  return (size_t)((n + run - 1) / run) * (groups + 1) * 4;
}

hipError_t launch_group_rows(const int32_t* ids, int64_t n, int groups, int32_t* offsets,
                             int32_t* order, int32_t* pos, int* counts, hipStream_t stream) {
  if (n <= kOneBlockPairs) {
    hipLaunchKernelGGL(k_group_alone, dim3(1), dim3(kThreads), alone_lds(groups), stream, ids, n, groups,
                       key_bits(groups), offsets, order, pos);
    return hipGetLastError();
  }
  const int64_t run = group_run(n);
  hipLaunchKernelGGL(k_group_count, dim3((unsigned)((n + run - 1) / run)), dim3(kThreads),
                     (size_t)(groups + 1) * 4, stream, ids, n, run, groups, counts);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  return launch_place(ids, n, run, groups, counts, offsets, order, pos, stream);
}

size_t moe_route_workspace(int64_t T, int E) {
  if (T <= kOneBlockTokens) return 0;
  const int64_t run = route_run(T);
  return (size_t)((T + run - 1) / run) * (E + 1) * 4;
}

hipError_t launch_moe_route(const void* logits, bool half, int64_t ld, int64_t T, int E, int top_k,
                            bool renorm, float* weights, int32_t* ids, int32_t* offsets, int32_t* order,
                            int32_t* pos, int* counts, uint32_t* flags, hipStream_t stream) {
  return half ? launch_route_t<uint16_t>(logits, ld, T, E, top_k, renorm, weights, ids, offsets, order,
                                         pos, counts, flags, stream)
              : launch_route_t<float>(logits, ld, T, E, top_k, renorm, weights, ids, offsets, order, pos,
                                      counts, flags, stream);
}

}  // namespace awq
