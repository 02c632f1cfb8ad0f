// New tokens into the 4-bit cache, and tokens of it back as fp16 (the format: kv_cache.hpp).
//
// Append, per token and head of keys and values, and per group of channels x (keys after their
// rotation, rounded to fp16):
//   lo = min(0, min x), hi = max(0, max x);  sc = (hi - lo) / 15 in fp32, rounded up to 7
//   significant bits, within [2^-14, 4352];  z = clamp(rint(-lo / sc), 0, 15);
//   q = clamp(rint(x / sc) + z, 0, 15).
// The rotation runs in fp64 (its products are exact there), is rounded to fp32 and then to fp16:
// an fp32 rotation would put values of some groups on the other side of a code's border, by the
// order in which it is written.
//
// Both are bound by memory. A wave takes 64 / (D / 8) heads of one row, a lane 8 channels of
// one: 16-byte loads, group extremes by DPP steps, codes as in the weight quantizer.
#include "kv_cache.hpp"
#include "launch.hpp"

namespace awq {

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ void unpack8(uint4 w, uint16_t (&x)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = (uint16_t)(u[i >> 1] >> (16 * (i & 1)));
}
__device__ __forceinline__ uint4 pack8(const uint16_t (&x)[8]) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) u[i] = x[2 * i] | (uint32_t)x[2 * i + 1] << 16;
  return make_uint4(u[0], u[1], u[2], u[3]);
}

__device__ __forceinline__ bool finite16(uint16_t h) { return (h & 0x7C00) != 0x7C00; }

// a cos - b sin (or, with sin negated, the other half of the pair)
__device__ __forceinline__ uint16_t rotated(uint16_t a, uint16_t b, float cos, float sin) {
  const double r = (double)h2f(a) * (double)cos - (double)h2f(b) * (double)sin;
  return f2h_bits((float)r);
}

// The 8 channels from 8 ch on of a head at x, rotated; tab: the position's row, R / 2 cos, then sin.
__device__ __forceinline__ void rotate8(const uint16_t* x, int ch, const float* tab, int R, bool interleaved,
                                        uint16_t (&v)[8]) {
  const int half = R / 2;
  if (interleaved) {  // pairs (2 i, 2 i + 1)
    const float4 c = *reinterpret_cast<const float4*>(tab + 4 * ch);
    const float4 s = *reinterpret_cast<const float4*>(tab + half + 4 * ch);
    const float cs[4] = {c.x, c.y, c.z, c.w}, sn[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint16_t a = v[2 * i], b = v[2 * i + 1];
      v[2 * i] = rotated(a, b, cs[i], sn[i]);
      v[2 * i + 1] = rotated(b, a, cs[i], -sn[i]);
    }
  } else {  // pairs (i, i + R / 2); half is a multiple of 8
    const bool upper = 8 * ch >= half;
    uint16_t o[8];
    unpack8(*reinterpret_cast<const uint4*>(x + 8 * ch + (upper ? -half : half)), o);
    const float* cp = tab + 8 * ch - (upper ? half : 0);
    const float* sp = cp + half;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = rotated(v[i], o[i], cp[i], upper ? -sp[i] : sp[i]);
  }
}

struct Sources {
  const uint16_t *q, *k, *v;  // rows of heads, D channels each
  int64_t q_ld, k_ld, v_ld;
  uint16_t* out;              // rotated queries
  int64_t out_ld;
  const float* table;         // [table_rows][rotary]
  int64_t table_rows;
  int rotary, interleaved;
  int q_heads;                // 0: no queries
};

template <int D>
__global__ void __launch_bounds__(kThreads) k_kv_append(KvView c, Sources a, uint32_t* flags) {
  constexpr int kLanes = D / 8, kHeads = kWave / kLanes;
  const int lane = threadIdx.x & (kWave - 1);
  const int heads = a.q_heads + 2 * c.heads, per_row = (heads + kHeads - 1) / kHeads;
  const int64_t id = (int64_t)blockIdx.x * (kThreads / kWave) + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  if (id >= (int64_t)c.n_rows * per_row) return;
  const int t = (int)(id / per_row);
  const int hd = (int)(id - (int64_t)t * per_row) * kHeads + lane / kLanes, ch = lane % kLanes;
  const int s = kv_find(c, t, lane);
  if (s >= c.seqs) return;  // a row behind the last sequence
  const KvSeq q = kv_sequence(c, s);
  const int64_t pos = (int64_t)q.length - q.rows + (t - q.row0);
  // what the lane's head is: queries, keys, values, or none
  const int kind = hd < a.q_heads ? 0 : hd < a.q_heads + c.heads ? 1 : hd < heads ? 2 : 3;
  const int head = kind == 0 ? hd : kind == 1 ? hd - a.q_heads : hd - a.q_heads - c.heads;
  uint16_t v[8] = {};
  bool bad = false, over = false;
  if (kind < 3) {
    const uint16_t* x = kind == 0 ? a.q + t * a.q_ld : kind == 1 ? a.k + t * a.k_ld : a.v + t * a.v_ld;
    x += (int64_t)head * D;
    unpack8(*reinterpret_cast<const uint4*>(x + 8 * ch), v);
#pragma unroll
    for (int i = 0; i < 8; ++i) bad |= !finite16(v[i]);
    if (kind < 2 && 8 * ch < a.rotary) {
      const int64_t row = pos < 0 ? 0 : pos < a.table_rows ? pos : a.table_rows - 1;
      rotate8(x, ch, a.table + row * a.rotary, a.rotary, a.interleaved != 0, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) over |= !finite16(v[i]);
    }
    if (kind == 0) *reinterpret_cast<uint4*>(a.out + t * a.out_ld + (int64_t)head * D + 8 * ch) = pack8(v);
  }
  // quantize (every lane takes part in the exchanges; queries and idle lanes store nothing)
  float w[8], mn = 0.0f, mx = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    w[i] = h2f(v[i]);
    mn = fminf(mn, w[i]);
    mx = fmaxf(mx, w[i]);
  }
  group_minmax(mn, mx, c.group);
  GroupQ g;
  g.qmax = 15.0f;
  float sc = div_small(mx - mn, 15.0f, 1.0f / 15.0f);
  sc = __builtin_bit_cast(float, (__builtin_bit_cast(uint32_t, sc) + 0x1FFFFu) & ~0x1FFFFu);  // up to 7 bits
  g.clamped = sc > 4352.0f;
  g.scf = fminf(fmaxf(sc, 0x1p-14f), 4352.0f);
  g.sch = f2h_bits(g.scf);  // exact
  g.rcp = __builtin_amdgcn_rcpf(g.scf);
  const float nmn[1] = {-mn};
  float zq[1], codes[8];
  rint_quotients(nmn, g.scf, g.rcp, zq);
  g.z = __builtin_amdgcn_fmed3f(zq[0], 0.0f, 15.0f);
  quant_codes(w, g, codes);
  const int page = kind == 1 || kind == 2 ? c.page_of(s, pos) : -1;
  const int place = (int)(pos & ((1 << c.page_shift) - 1));
  const int64_t at = (int64_t)(page < 0 ? 0 : page) * c.heads + head;  // the head's part of the page
  // natural nibbles, and those of the three lanes that share the lane's cells
  uint32_t word = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) word |= (uint32_t)codes[i] << (4 * i);
  const int j = (ch >> 1) & 3;
  uint32_t cell0 = 0, cell1 = 0;
#pragma unroll
  for (int o = 0; o < 4; ++o) {
    const uint32_t u = __shfl_xor(word, 2 * o) >> (8 * j);
    cell0 |= (u & 15) << (4 * (j ^ o));
    cell1 |= ((u >> 4) & 15) << (4 * (j ^ o));
  }
  if (page >= 0) {
    if (kind == 1) {
      uint32_t* row = reinterpret_cast<uint32_t*>(c.k_codes + at * c.code_bytes() + (int64_t)place * (D / 2));
      row[(ch & 3) * (D / 32) + (ch >> 2)] = pack_codes8(codes);
    } else {
      uint16_t* unit = reinterpret_cast<uint16_t*>(c.v_codes + at * c.code_bytes() + (int64_t)(place >> 4) * (8 * D));
      const int col = 8 * (ch & 1) + 2 * j;  // cells (h, col, w, i) and (h, col + 1, w, i)
      unit += ((((place >> 2) & 3) * 16 + col) * (D / 64) + (ch >> 3)) * 4 + (place & 3);
      unit[0] = (uint16_t)cell0;
      unit[(D / 64) * 4] = (uint16_t)cell1;
    }
    const int per_group = c.group / 8;
    if (ch % per_group == 0) {
      uint16_t* p = (kind == 1 ? c.k_params : c.v_params) + at * c.param_words();
      p[((int64_t)(ch / per_group) << c.page_shift) + place] = (uint16_t)(g.sch | (uint32_t)g.z);
    }
  }
  if (flags) {
    const uint32_t f = (bad ? AWQ_FLAG_NONFINITE_INPUT : 0u) | (over && !bad ? AWQ_FLAG_OVERFLOW : 0u) |
                       (page >= 0 && g.clamped ? AWQ_FLAG_SCALE_CLAMPED : 0u);
    const uint32_t all = (__ballot(f & AWQ_FLAG_NONFINITE_INPUT) ? AWQ_FLAG_NONFINITE_INPUT : 0u) |
                         (__ballot(f & AWQ_FLAG_OVERFLOW) ? AWQ_FLAG_OVERFLOW : 0u) |
                         (__ballot(f & AWQ_FLAG_SCALE_CLAMPED) ? AWQ_FLAG_SCALE_CLAMPED : 0u);
    if (all && lane == 0) atomicOr(flags, all);
  }
}

// Keys and values of the batch's rows out of the cache; a token without a page: zeros.
template <int D>
__global__ void __launch_bounds__(kThreads) k_kv_read(KvView c, uint16_t* k, uint16_t* v) {
  constexpr int kLanes = D / 8, kHeads = kWave / kLanes;
  const int lane = threadIdx.x & (kWave - 1);
  const int per_row = (2 * c.heads + kHeads - 1) / kHeads;
  const int64_t id = (int64_t)blockIdx.x * (kThreads / kWave) + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  if (id >= (int64_t)c.n_rows * per_row) return;
  const int t = (int)(id / per_row);
  const int hd = (int)(id - (int64_t)t * per_row) * kHeads + lane / kLanes, ch = lane % kLanes;
  const int s = kv_find(c, t, lane);
  if (s >= c.seqs) return;
  const KvSeq q = kv_sequence(c, s);
  const int64_t pos = (int64_t)q.length - q.rows + (t - q.row0);
  const bool values = hd >= c.heads, some = hd < 2 * c.heads;
  const int head = values ? hd - c.heads : hd;
  const int page = some ? c.page_of(s, pos) : -1;
  const int place = (int)(pos & ((1 << c.page_shift) - 1));
  const int64_t at = (int64_t)(page < 0 ? 0 : page) * c.heads + head;
  uint32_t par = 0, word = 0, cells = 0;
  const int j = (ch >> 1) & 3;
  if (page >= 0) {
    const uint16_t* p = (values ? c.v_params : c.k_params) + at * c.param_words();
    par = p[((int64_t)(ch / (c.group / 8)) << c.page_shift) + place];
    if (values) {
      const uint16_t* unit =
          reinterpret_cast<const uint16_t*>(c.v_codes + at * c.code_bytes() + (int64_t)(place >> 4) * (8 * D));
      unit += ((((place >> 2) & 3) * 16 + 8 * (ch & 1) + 2 * j) * (D / 64) + (ch >> 3)) * 4 + (place & 3);
      cells = unit[0] | (uint32_t)unit[(D / 64) * 4] << 16;
    } else {
      word = reinterpret_cast<const uint32_t*>(c.k_codes + at * c.code_bytes() + (int64_t)place * (D / 2))[
          (ch & 3) * (D / 32) + (ch >> 2)];
    }
  }
  const float sc = h2f(par & 0xFFF0);
  const int z = par & 15;
  uint16_t y[8] = {};
  uint32_t of[4] = {};  // the cells of columns 8 b + 2 o and 8 b + 2 o + 1
#pragma unroll
  for (int o = 0; o < 4; ++o) {
    const uint32_t u = __shfl_xor(cells, 2 * o);
    const int from = j ^ o;
#pragma unroll
    for (int i = 0; i < 4; ++i) of[i] = from == i ? u : of[i];
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t code = values ? of[i >> 1] >> (16 * (i & 1) + 4 * j) : word >> (4 * kNibbleOf[i]);
    y[i] = f2h_bits((float)((int)(code & 15) - z) * sc);  // exact
  }
  if (some) *reinterpret_cast<uint4*>((values ? v : k) + ((int64_t)t * c.heads + head) * D + 8 * ch) = pack8(y);
}

dim3 grid_of(int64_t rows, int heads, int dim) {
  const int per_wave = kWave / (dim / 8);
  const int64_t waves = rows * ((heads + per_wave - 1) / per_wave);
  return dim3((unsigned)((waves + kThreads / kWave - 1) / (kThreads / kWave)));
}

}  // namespace

hipError_t launch_kv_append(const KvView& c, const uint16_t* q, int64_t q_ld, int q_heads, uint16_t* out,
                            int64_t out_ld, const uint16_t* k, int64_t k_ld, const uint16_t* v, int64_t v_ld,
                            const float* table, int64_t table_rows, int rotary, bool interleaved, uint32_t* flags,
                            hipStream_t stream) {
  const Sources a{q, k, v, q_ld, k_ld, v_ld, out, out_ld, table, table_rows, rotary, interleaved, q_heads};
  auto* const f = c.dim == 64 ? k_kv_append<64> : c.dim == 128 ? k_kv_append<128> : k_kv_append<256>;
  hipLaunchKernelGGL(f, grid_of(c.n_rows, q_heads + 2 * c.heads, c.dim), dim3(kThreads), 0, stream, c, a, flags);
  return hipGetLastError();
}

hipError_t launch_kv_read(const KvView& c, uint16_t* k, uint16_t* v, hipStream_t stream) {
  auto* const f = c.dim == 64 ? k_kv_read<64> : c.dim == 128 ? k_kv_read<128> : k_kv_read<256>;
  hipLaunchKernelGGL(f, grid_of(c.n_rows, 2 * c.heads, c.dim), dim3(kThreads), 0, stream, c, k, v);
  return hipGetLastError();
}

}  // namespace awq
