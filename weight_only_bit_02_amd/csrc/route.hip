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
// two: the first writes each block's count per group, key by key, the second sums the counts of
// the blocks before it (at most kMaxBlocks per key, from L2) and places its run.
//
// Bound by latency: one token, 8 of 64 experts: 5.3 us; 2048 rows by 32 adapters: 4.8 us. 8191
// tokens, 8 of 128: 10.1 us for the choice, by its 423 instructions a token (eight maxima in turn),
// and 8.6 for the placement (every block sums the counts of all 256).
#include <hip/hip_runtime.h>

#include "common.hpp"
#include "groups.hpp"
#include "launch.hpp"

namespace awq {

namespace {

constexpr int kThreads = 1024, kWaves = kThreads / kWave;
constexpr int64_t kOneBlockTokens = 64;   // route: tokens that one block serves alone
constexpr int64_t kOneBlockPairs = 8192;  // grouping: pairs that one block serves alone
constexpr int64_t kMaxBlocks = 256;       // a multiple of a wave

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
__device__ __forceinline__ int choose(const LT* logits, int64_t ld, int64_t t, int E, int top_k,
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
  return id;
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

// Runs of up to kThreads kHeld pairs: every thread holds its pairs' keys, so that they are read
// once, and each wave counts its contiguous part of the run in order, in next[w][key] (LDS). A
// pair's rank among its wave's pairs of the same key comes with the count: placing it takes the
// positions of the waves' first pairs alone.
constexpr int kHeld = 8;
struct Held {
  int key[kHeld], rank[kHeld];
};
__device__ __forceinline__ int64_t wave_part(int64_t n) {
  return ((n + kWaves - 1) / kWaves + kWave - 1) / kWave * kWave;
}
// from: ids of the run, in global memory or LDS
__device__ __forceinline__ void hold(Held& h, const int32_t* from, int n, int groups, int tid) {
  const int part = (int)wave_part(n), w0 = (tid >> 6) * part;
#pragma unroll
  for (int c = 0; c < kHeld; ++c) {
    const int i = w0 + c * kWave + (tid & 63);
    h.key[c] = c * kWave < part && i < n ? key_of(from[i], groups) : -1;
  }
}
// next: cleared; ends with a barrier
__device__ __forceinline__ void rank_held(Held& h, int n, int groups, int bits, int* next, int tid) {
  const int part = (int)wave_part(n), lane = tid & 63;
  int* const mine = next + (tid >> 6) * (groups + 1);
  const uint64_t below = ((uint64_t)1 << lane) - 1;
#pragma unroll
  for (int c = 0; c < kHeld; ++c) {
    const bool in = h.key[c] >= 0;
    const uint64_t live = __ballot(in);
    if (c * kWave < part && live) {
      const uint64_t same = same_key(h.key[c], bits, live);
      const int before = in ? mine[h.key[c]] : 0;
      h.rank[c] = before + __popcll(same & below);
      __builtin_amdgcn_wave_barrier();
      if (in && (same & below) == 0) mine[h.key[c]] = before + __popcll(same);  // the first of its equals
      __builtin_amdgcn_wave_barrier();
    }
  }
  __syncthreads();
}
// next[w][key]: from the counts of the waves to the positions of their first pairs, given the
// run's first positions; ends with a barrier
__device__ __forceinline__ void wave_starts(int* next, const int* start, int keys, int tid) {
  for (int k = tid; k < keys; k += kThreads) {
    int at = start[k];
    for (int w = 0; w < kWaves; ++w) {
      const int c = next[w * keys + k];
      next[w * keys + k] = at;
      at += c;
    }
  }
  __syncthreads();
}
__device__ __forceinline__ void place_held(const Held& h, int64_t p0, int n, int groups, const int* next,
                                           int32_t* order, int32_t* pos, int tid) {
  const int part = (int)wave_part(n), w0 = (tid >> 6) * part;
  const int* const mine = next + (tid >> 6) * (groups + 1);
#pragma unroll
  for (int c = 0; c < kHeld; ++c)
    if (h.key[c] >= 0) {
      const int64_t p = p0 + w0 + c * kWave + (tid & 63);
      const int at = mine[h.key[c]] + h.rank[c];
      order[at] = (int32_t)p;
      if (pos) pos[p] = at;
    }
}

// The same for runs of any length, walked twice. Places pairs [p0, p1): next[w][key] (LDS) is the position of wave w's next pair of a key.
// Counting, the sums over the waves and the placement all walk the pairs in order.
// start[key] (LDS): the position of this block's first pair of the key.
__device__ __forceinline__ void place(const int32_t* ids, int64_t p0, int64_t p1, int groups, int bits,
                                      int* next, const int* start, int32_t* order, int32_t* pos,
                                      int tid) {
  const int lane = tid & 63, wave = tid >> 6, keys = groups + 1;
  const int64_t part = wave_part(p1 - p0);
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
  wave_starts(next, start, keys, tid);
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
constexpr int alone_ints(int groups) { return (groups + 1) * (kWaves + 1) + kWaves; }
__device__ __forceinline__ void sort_alone(const int32_t* from, int n, int groups, int bits, int* lds,
                                           int32_t* offsets, int32_t* order, int32_t* pos, int tid) {
  const int keys = groups + 1;
  int* const count = lds;
  int* const part = count + keys;
  int* const next = part + kWaves;
  Held h;
  hold(h, from, n, groups, tid);
  for (int i = tid; i < kWaves * keys; i += kThreads) next[i] = 0;
  __syncthreads();
  rank_held(h, n, groups, bits, next, tid);
  for (int k = tid; k < keys; k += kThreads) {
    int all = 0;
    for (int w = 0; w < kWaves; ++w) all += next[w * keys + k];
    count[k] = all;
  }
  __syncthreads();
  block_exclusive(count, keys, part, tid);
  for (int k = tid; k < keys; k += kThreads) offsets[k] = count[k];
  wave_starts(next, count, keys, tid);
  place_held(h, 0, n, groups, next, order, pos, tid);
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
  if constexpr (ALONE) {
    int* const held = lds + alone_ints(E);  // the ids
    for (int64_t t = wave; t < T; t += kWaves) {
      const int id = choose<LT, V>(logits, ld, t, E, top_k, renorm, weights, ids, bad, lane);
      if (lane < top_k) held[t * top_k + lane] = id;
    }
    __syncthreads();
    sort_alone(held, (int)T * top_k, E, bits, lds, offsets, order, pos, tid);
  } else {
    for (int k = tid; k <= E; k += kThreads) lds[k] = 0;
    __syncthreads();
    for (int64_t t = t0 + wave; t < t1; t += kWaves) {
      const int id = choose<LT, V>(logits, ld, t, E, top_k, renorm, weights, ids, bad, lane);
      if (lane < top_k) atomicAdd(&lds[key_of(id, E)], 1);
    }
    __syncthreads();
    for (int k = tid; k <= E; k += kThreads) counts[(int64_t)k * gridDim.x + blockIdx.x] = lds[k];
  }
  if (flags && __ballot(bad) && lane == 0) atomicOr(flags, AWQ_FLAG_NONFINITE_INPUT);
}

__global__ void __launch_bounds__(kThreads)
    k_group_alone(const int32_t* ids, int64_t n, int groups, int bits, int32_t* offsets, int32_t* order,
                  int32_t* pos) {
  extern __shared__ int lds[];
  sort_alone(ids, (int)n, groups, bits, lds, offsets, order, pos, threadIdx.x);
}

__global__ void __launch_bounds__(kThreads)
    k_group_count(const int32_t* ids, int64_t n, int64_t per_block, int groups, int* counts) {
  extern __shared__ int lds[];
  const int64_t p0 = blockIdx.x * per_block, p1 = p0 + per_block < n ? p0 + per_block : n;
  count_keys(ids, p0, p1, groups, lds, threadIdx.x);
  for (int k = threadIdx.x; k <= groups; k += kThreads)
    counts[(int64_t)k * gridDim.x + blockIdx.x] = lds[k];
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
  const int64_t p0 = me * per_block, p1 = p0 + per_block < n ? p0 + per_block : n;
  const bool held = per_block <= kThreads * kHeld;
  Held h;
  if (held) {
    hold(h, ids + p0, (int)(p1 - p0), groups, tid);
    for (int i = tid; i < kWaves * keys; i += kThreads) next[i] = 0;
  }
  // a wave sums a key's counts of all blocks and of those before this one
  const int lane = tid & 63;
  for (int k = __builtin_amdgcn_readfirstlane(tid >> 6); k < keys; k += kWaves) {
    int all = 0, before = 0;
#pragma unroll
    for (int i = 0; i < kMaxBlocks / kWave; ++i) {
      const int b = i * kWave + lane;
      const int c = b < blocks ? counts[(int64_t)k * blocks + b] : 0;
      all += c;
      before += b < me ? c : 0;
    }
    all = __builtin_amdgcn_readlane(wave_scan(all), 63);
    before = __builtin_amdgcn_readlane(wave_scan(before), 63);
    if (lane == 0) {
      total[k] = all;
      start[k] = before;
    }
  }
  __syncthreads();
  if (held) rank_held(h, (int)(p1 - p0), groups, bits, next, tid);
  block_exclusive(total, keys, part, tid);
  for (int k = tid; k < keys; k += kThreads) {
    start[k] += total[k];
    if (me == 0) offsets[k] = total[k];
  }
  __syncthreads();
  if (held) {
    wave_starts(next, start, keys, tid);
    place_held(h, p0, (int)(p1 - p0), groups, next, order, pos, tid);
  } else {
    place(ids, p0, p1, groups, bits, next, start, order, pos, tid);
  }
}

int key_bits(int groups) {  // bits of the keys 0 .. groups
  int b = 1;
  while (groups >> b) ++b;
  return b;
}

constexpr size_t alone_lds(int groups, int ids) { return (size_t)(alone_ints(groups) + ids) * 4; }
constexpr size_t place_lds(int groups) { return ((size_t)(groups + 1) * (kWaves + 2) + kWaves) * 4; }

// The limits of the entry points that the kernels rely on.
static_assert(AWQ_MAX_GROUPS <= 8 * kWave, "choose() holds at most eight logits a lane");
static_assert(AWQ_MAX_TOP_K <= kWave, "a lane holds one choice");
constexpr size_t kLaunchLds = 64 * 1024;  // dynamic LDS that a launch gets without asking
static_assert(alone_lds(AWQ_MAX_GROUPS, (int)kOneBlockTokens * AWQ_MAX_TOP_K) <= kLaunchLds, "LDS of one block");
static_assert(place_lds(AWQ_MAX_GROUPS) <= kLaunchLds, "LDS of the placement");

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
    hipLaunchKernelGGL((k_route<LT, V, true>), dim3(1), dim3(kThreads), alone_lds(E, (int)T * top_k), stream,
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
    hipLaunchKernelGGL(k_group_alone, dim3(1), dim3(kThreads), alone_lds(groups, 0), stream, ids, n, groups,
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
