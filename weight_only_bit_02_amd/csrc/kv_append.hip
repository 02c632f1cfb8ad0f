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
// Both move few bytes a value, so that the instructions count as much. A wave takes 64 / (D / 8)
// rows, a lane 8 channels of one row; it goes through heads, one after the other, the next one's
// loads under way: the lane's sequence, page, cos and sin are found once for all its heads. Four
// waves take adjacent heads, 1 KB of a row together (rows by waves instead, 256 B of a row at a
// time: 71 us for the call below, not 60). With one row and 512 / D heads a wave, and the weight
// quantizer's quotients, the call took 377 instructions a wave and head step instead of 116, and
// 114 us; reading took 45.
//
// Measured, 6300 rows, 32 heads each of queries, keys and values, D = 128: append 60 us (222 MB,
// 3.7 TB/s; its vector instructions alone are 34 us), read 27 us (130 MB, 4.8 TB/s). Short calls
// are chains of dependent loads: sequence, page, data; 4 to 5 us for up to 64 rows.
// Stores past the caches (nontemporal) take 19 us for that reading and 57 for that append, but the next
// kernel pays for it: reading 8192 rows of 32 heads and copying them, 100 us for 95.
#include "kv_cache.hpp"
#include "launch.hpp"

#include <type_traits>

namespace awq {

namespace {

constexpr int kThreads = 256, kWaves = kThreads / kWave;

template <int D>
struct Lanes {
  static constexpr int kRow = D / 8;          // lanes of a row
  static constexpr int kRows = kWave / kRow;  // rows of a wave, and of its block
};

// A lane's row.
struct RowPlace {
  int t;        // its row, within the tensors
  bool live;    // it belongs to a sequence
  int64_t pos;
  int64_t page;  // -1: none
  int place;     // in the page
};

template <int D>
__device__ __forceinline__ RowPlace place_of(const KvView& c, int block, int lane) {
  constexpr int kRow = Lanes<D>::kRow;
  const int t = block * Lanes<D>::kRows + lane / kRow;
  RowPlace r;
  r.t = t < c.n_rows ? t : c.n_rows - 1;
  const int s = kv_find<kRow>(c, r.t, lane);
  r.live = t < c.n_rows && s < c.seqs;
  const KvSeq q = kv_sequence(c, r.live ? s : 0);
  r.pos = (int64_t)q.length - q.rows + (r.t - q.row0);
  r.page = r.live ? c.page_of(s, r.pos) : -1;
  r.place = (int)(r.pos & ((1 << c.page_shift) - 1));
  return r;
}

// What a block takes: rows, and heads [h0, h1) of queries, keys and values, its waves one after the
// other.
struct Work {
  int block, h0, h1, wave;
};
__device__ __forceinline__ Work work_of(int heads, int per_block) {
  const int steps = (heads + per_block - 1) / per_block;
  Work w;
  w.block = __builtin_amdgcn_readfirstlane(blockIdx.x / steps);
  w.h0 = (blockIdx.x - w.block * steps) * per_block;
  w.h1 = w.h0 + per_block < heads ? w.h0 + per_block : heads;
  w.wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  return w;
}

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

// An Inf or NaN among 8 values: 0 x is then NaN.
__device__ __forceinline__ bool nonfinite8(uint4 w) {
  const half2w zero = {0, 0};
  half2w n = __builtin_bit_cast(half2w, w.x) * zero;
  n = __builtin_elementwise_fma(__builtin_bit_cast(half2w, w.y), zero, n);
  n = __builtin_elementwise_fma(__builtin_bit_cast(half2w, w.z), zero, n);
  n = __builtin_elementwise_fma(__builtin_bit_cast(half2w, w.w), zero, n);
  return (__builtin_bit_cast(uint32_t, n) & 0x7FFF7FFFu) != 0;
}

// Nibbles 0..7 to the order (0, 2, 4, 6, 1, 3, 5, 7), and back.
__device__ __forceinline__ uint32_t unzip(uint32_t x) {
  x = (x & 0xF00FF00Fu) | ((x >> 4) & 0x00F000F0u) | ((x << 4) & 0x0F000F00u);
  return __builtin_amdgcn_perm(0, x, 0x03010200);
}
__device__ __forceinline__ uint32_t zip(uint32_t x) {
  x = __builtin_amdgcn_perm(0, x, 0x03010200);
  return (x & 0xF00FF00Fu) | ((x >> 4) & 0x00F000F0u) | ((x << 4) & 0x0F000F00u);
}

// Byte o of lane j to byte j of lane o, over the four lanes 2 j apart (j = lane / 2 % 4).
__device__ __forceinline__ uint32_t across(uint32_t x, int lane) {
  const auto moved = [](uint32_t v, auto ctrl) {
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, decltype(ctrl)::value, 0xF, 0xF, true);
  };
  uint32_t p = moved(x, std::integral_constant<int, 0x4E>());  // the lane 2 away
  x = __builtin_amdgcn_perm(p, x, lane & 2 ? 0x03070105 : 0x06020400);
  p = moved(x, std::integral_constant<int, 0x141>());          // 4 away: 7 away ...
  p = moved(p, std::integral_constant<int, 0x1B>());           // ... then 3
  return __builtin_amdgcn_perm(p, x, lane & 4 ? 0x03020706 : 0x05040100);
}

// a cos - b sin (or, with sin negated, the other half of the pair): the products are exact in fp64,
// so the fused form is the rounded difference.
__device__ __forceinline__ uint16_t rotated(uint16_t a, uint16_t b, float cos, float sin) {
  const double r = __builtin_fma((double)h2f(a), (double)cos, -((double)h2f(b) * (double)sin));
  return f2h_bits((float)r);
}

struct Sources {
  const uint16_t *q, *k, *v;  // rows of heads, D channels each
  int64_t q_ld, k_ld, v_ld;
  uint16_t* out;              // rotated queries
  int64_t out_ld;
  const float* table;         // [table_rows][rotary]
  int64_t table_rows;
  int rotary;
  int q_heads;                // 0: no queries
  int per_block;              // heads
};

// Quotients of fp16 values by a scale of 7 bits, |x / sc| < 32, rounded to whole numbers as fp32
// does it, kept as 1.5 2^23 + the number. Near a half, x and the half's multiple of sc are both
// multiples of 2^-11 of sc's power of two: x / sc is a half exactly or off by more than 2^-12. So
// x rcp (off by less than 2^-17) is rounded to steps of 2^-13 first, which puts a half where it is
// and nothing on its other side, then to whole numbers, halves to even.
__device__ __forceinline__ float whole(float x, float rcp) {
  return __builtin_fmaf(x, rcp, 1536.0f) + (12582912.0f - 1536.0f);
}

struct Codes {
  uint32_t low;   // bits of 1.5 2^23 - z
  float u[8];     // 1.5 2^23 - z + code
  uint16_t param;
  bool clamped;
};

__device__ __forceinline__ Codes quantize8(const uint16_t (&v)[8], int group) {
  Codes q;
  float w[8], mn = 0.0f, mx = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    w[i] = h2f(v[i]);
    mn = fminf(mn, w[i]);
    mx = fmaxf(mx, w[i]);
  }
  group_minmax(mn, mx, group);
  float sc = div_small(mx - mn, 15.0f, 1.0f / 15.0f);
  sc = __builtin_bit_cast(float, (__builtin_bit_cast(uint32_t, sc) + 0x1FFFFu) & ~0x1FFFFu);  // up to 7 bits
  q.clamped = sc > 4352.0f;
  sc = __builtin_amdgcn_fmed3f(sc, 0x1p-14f, 4352.0f);
  const float rcp = __builtin_amdgcn_rcpf(sc);
  const float z = __builtin_amdgcn_fmed3f(whole(-mn, rcp), 12582912.0f, 12582927.0f) - 12582912.0f;
  q.param = (uint16_t)(f2h_bits(sc) | (uint32_t)z);  // the scale: exact
  const float lo = 12582912.0f - z, hi = 12582927.0f - z;
  q.low = __builtin_bit_cast(uint32_t, lo);
#pragma unroll
  for (int i = 0; i < 8; ++i) q.u[i] = __builtin_amdgcn_fmed3f(whole(w[i], rcp), lo, hi);
  return q;
}

// The codes as a word, channel i in nibble i (kNatural) or in nibble order 0, 2, 4, 6, 1, 3, 5, 7.
template <bool kNatural>
__device__ __forceinline__ uint32_t pack_word(const Codes& q) {
  uint32_t word = 0;
#pragma unroll
  for (int i = 7; i >= 0; --i) {
    const int of = kNatural ? i : i < 4 ? 2 * i : 2 * i - 7;
    word = (word << 4) + __builtin_bit_cast(uint32_t, q.u[of]);
  }
  return word - q.low * 0x11111111u;
}

// A lane's part in its row.
template <bool kPairs>
struct Turn {
  bool on, upper;  // its channels turn; they are the pairs' second
  int half;        // rotary / 2
  float cos[kPairs ? 4 : 8], sin[kPairs ? 4 : 8];
};

// What a lane met: an Inf or NaN in its input, one that the rotation made, a clamped scale.
struct Met {
  bool odd, over, clamped;
};

enum Kind { kQueries, kKeys, kValues };

// A wave's of heads [lo, hi) of queries, keys or values: x are the lane's channels of head 0, to(head, word or
// values, parameter) takes what comes out.
template <int D, Kind kKind, bool kPairs, class To>
__device__ __forceinline__ void put_heads(const uint16_t* x, int lo, int hi, int wave, const Turn<kPairs>& turn, int group,
                                          int lane, bool checks, Met& met, To&& to) {
  lo += wave;
  if (lo >= hi) return;
  const int partner = turn.upper ? -turn.half : turn.half;
  const bool two = kKind != kValues && !kPairs && turn.on;  // pairs of channels far apart: both are loaded
  int h = lo;
  uint4 next = *reinterpret_cast<const uint4*>(x + (int64_t)h * D), next_o = next;
  if (two) next_o = *reinterpret_cast<const uint4*>(x + (int64_t)h * D + partner);
  for (; h < hi; h += kWaves) {
    const uint4 own = next, other = next_o;
    const int64_t at = (int64_t)(h + kWaves < hi ? h + kWaves : h) * D;
    next = *reinterpret_cast<const uint4*>(x + at);
    if (two) next_o = *reinterpret_cast<const uint4*>(x + at + partner);
    const bool odd = checks && nonfinite8(own);
    met.odd |= odd;
    uint16_t v[8];
    unpack8(own, v);
    if (kKind != kValues && turn.on) {
      uint16_t o[8], y[8];
      unpack8(other, o);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        y[i] = !kPairs ? rotated(v[i], o[i], turn.cos[i], turn.sin[i])
                       : rotated(v[i], v[i ^ 1], turn.cos[i / 2], i & 1 ? -turn.sin[i / 2] : turn.sin[i / 2]);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = y[i];
      // (of finite pairs: an Inf in the other half is no overflow)
      met.over |= checks && !odd && !(two && nonfinite8(other)) && nonfinite8(pack8(v));
    }
    if constexpr (kKind == kQueries) {
      to(h, pack8(v), (uint16_t)0);
    } else {
      const Codes q = quantize8(v, group);
      met.clamped |= q.clamped;
      if constexpr (kKind == kKeys) to(h, pack_word<false>(q), q.param);
      else to(h, unzip(across(pack_word<true>(q), lane)), q.param);
    }
  }
}

// kPairs: channels 2 i and 2 i + 1 turn together, else i and i + R / 2 (a multiple of 8).
template <int D, bool kPairs>
__global__ void __launch_bounds__(kThreads) k_kv_append(KvView c, Sources a, uint32_t* flags) {
  constexpr int kRow = Lanes<D>::kRow;
  const int lane = threadIdx.x & (kWave - 1), ch = lane % kRow;
  const Work w = work_of(a.q_heads + 2 * c.heads, a.per_block);
  const RowPlace r = place_of<D>(c, w.block, lane);
  if (!__ballot(r.live)) return;
  Turn<kPairs> turn;
  turn.half = a.rotary / 2;
  turn.on = 8 * ch < a.rotary;
  turn.upper = 8 * ch >= turn.half;
  if (turn.on) {
    const int64_t row = r.pos < 0 ? 0 : r.pos < a.table_rows ? r.pos : a.table_rows - 1;
    const float* tab = a.table + row * a.rotary + (kPairs ? 4 * ch : 8 * ch - (turn.upper ? turn.half : 0));
#pragma unroll
    for (int i = 0; i < (kPairs ? 4 : 8); ++i) {
      turn.cos[i] = tab[i];
      turn.sin[i] = !kPairs && turn.upper ? -tab[turn.half + i] : tab[turn.half + i];
    }
  }
  const int64_t at = (r.page < 0 ? 0 : r.page) * c.heads;
  const int per_group = c.group / 8;
  const int64_t par = at * c.param_words() + ((int64_t)(ch / per_group) << c.page_shift) + r.place;
  const bool stores = r.page >= 0, stores_par = stores && ch % per_group == 0, checks = flags != nullptr;
  Met met{};
  const auto within = [&](int h, int n) { return h < 0 ? 0 : h < n ? h : n; };
  {
    uint16_t* const out = a.out + r.t * a.out_ld + 8 * ch;
    put_heads<D, kQueries>(a.q + r.t * a.q_ld + 8 * ch, w.h0, within(w.h1, a.q_heads), w.wave, turn, c.group, lane,
                           checks, met, [&](int h, uint4 y, uint16_t) {
                             if (r.live) *reinterpret_cast<uint4*>(out + (int64_t)h * D) = y;
                           });
  }
  {
    uint8_t* const row = c.k_codes + at * c.code_bytes() + (int64_t)r.place * (D / 2) +
                         4 * ((ch & 3) * (D / 32) + (ch >> 2));
    const int before = a.q_heads;
    put_heads<D, kKeys>(a.k + r.t * a.k_ld + 8 * ch, within(w.h0 - before, c.heads), within(w.h1 - before, c.heads),
                        w.wave, turn, c.group, lane, checks, met, [&](int h, uint32_t word, uint16_t param) {
                          if (stores) *reinterpret_cast<uint32_t*>(row + h * c.code_bytes()) = word;
                          if (stores_par) c.k_params[par + h * c.param_words()] = param;
                        });
  }
  {
    // cells (h, col, w, i) and (h, col + 1, w, i)
    const int col = 8 * (ch & 1) + 2 * ((ch >> 1) & 3);
    uint8_t* const row = c.v_codes + at * c.code_bytes() + (int64_t)(r.place >> 4) * (8 * D) +
                         2 * (((((r.place >> 2) & 3) * 16 + col) * (D / 64) + (ch >> 3)) * 4 + (r.place & 3));
    const int before = a.q_heads + c.heads;
    put_heads<D, kValues>(a.v + r.t * a.v_ld + 8 * ch, within(w.h0 - before, c.heads), within(w.h1 - before, c.heads),
                          w.wave, turn, c.group, lane, checks, met, [&](int h, uint32_t cells, uint16_t param) {
                            if (stores) {
                              uint16_t* cell = reinterpret_cast<uint16_t*>(row + h * c.code_bytes());
                              cell[0] = (uint16_t)cells;
                              cell[(D / 64) * 4] = (uint16_t)(cells >> 16);
                            }
                            if (stores_par) c.v_params[par + h * c.param_words()] = param;
                          });
  }
  if (checks) {
    const uint32_t all = (__ballot(r.live && met.odd) ? AWQ_FLAG_NONFINITE_INPUT : 0u) |
                         (__ballot(r.live && met.over) ? AWQ_FLAG_OVERFLOW : 0u) |
                         (__ballot(stores && met.clamped) ? AWQ_FLAG_SCALE_CLAMPED : 0u);
    if (all && lane == 0) atomicOr(flags, all);
  }
}

// Keys and values of the batch's rows out of the cache; a token without a page: zeros.
template <int D>
__global__ void __launch_bounds__(kThreads) k_kv_read(KvView c, uint16_t* k, uint16_t* v, int per_block) {
  constexpr int kRow = Lanes<D>::kRow;
  constexpr int kAtOnce = 4;
  const int lane = threadIdx.x & (kWave - 1), ch = lane % kRow;
  const Work w = work_of(2 * c.heads, per_block);
  const RowPlace r = place_of<D>(c, w.block, lane);
  if (!__ballot(r.live)) return;
  const int64_t at = (r.page < 0 ? 0 : r.page) * c.heads;
  const int col = 8 * (ch & 1) + 2 * ((ch >> 1) & 3);
  const uint8_t* const k_row = c.k_codes + at * c.code_bytes() + (int64_t)r.place * (D / 2) +
                               4 * ((ch & 3) * (D / 32) + (ch >> 2));
  const uint8_t* const v_row = c.v_codes + at * c.code_bytes() + (int64_t)(r.place >> 4) * (8 * D) +
                               2 * (((((r.place >> 2) & 3) * 16 + col) * (D / 64) + (ch >> 3)) * 4 + (r.place & 3));
  const int64_t par_at = at * c.param_words() + ((int64_t)(ch / (c.group / 8)) << c.page_shift) + r.place;
  const int64_t out = (int64_t)r.t * c.heads * D + 8 * ch;
  const uint32_t magic = wide_magic();
  for (int h0 = w.h0 + w.wave; h0 < w.h1; h0 += kAtOnce * kWaves) {
    uint32_t word[kAtOnce], par[kAtOnce];
#pragma unroll
    for (int n = 0; n < kAtOnce; ++n) {
      const int h = h0 + n * kWaves < w.h1 ? h0 + n * kWaves : h0;
      const bool values = h >= c.heads;
      const int head = values ? h - c.heads : h;
      word[n] = par[n] = 0;
      if (r.page >= 0) {
        par[n] = (values ? c.v_params : c.k_params)[par_at + head * c.param_words()];
        if (values) {
          const uint16_t* cell = reinterpret_cast<const uint16_t*>(v_row + head * c.code_bytes());
          word[n] = cell[0] | (uint32_t)cell[(D / 64) * 4] << 16;
        } else {
          word[n] = *reinterpret_cast<const uint32_t*>(k_row + head * c.code_bytes());
        }
      }
    }
#pragma unroll
    for (int n = 0; n < kAtOnce; ++n) {
      const int h = h0 + n * kWaves;
      if (h >= w.h1) break;
      const bool values = h >= c.heads;
      const int head = values ? h - c.heads : h;
      uint32_t x = word[n];
      if (values) x = unzip(across(zip(x), lane));
      // code - zero and its product with the scale are exact in fp16; widen_word wants zeros negated
      const uint32_t z = par[n] & 15, zz = 0xE400u | z, zz64 = 0xD400u | z << 4, sc = par[n] & 0xFFF0u;
      const half8w y = widen_word(x, __builtin_bit_cast(half2w, zz | zz << 16),
                                  __builtin_bit_cast(half2w, zz64 | zz64 << 16),
                                  __builtin_bit_cast(half2w, sc | sc << 16), magic);
      if (r.live) *reinterpret_cast<half8w*>((values ? v : k) + out + (int64_t)head * D) = y;
    }
  }
}

// Heads of a block: as many as leave one wave to every place on the card, 8192. Half or twice as
// many waves: 3 % slower appends, 30 % slower reads (14.6 us, not 11.1, for 43 MB).
constexpr int64_t kFill = 8192;
struct Grid {
  dim3 blocks;
  int per_block;
};
Grid grid_of(int64_t rows, int heads, int dim) {
  const int per_wave = kWave / (dim / 8);
  const int64_t blocks = (rows + per_wave - 1) / per_wave;
  const int64_t per_step = (blocks * heads + kFill - 1) / kFill;  // heads of a wave
  const int64_t steps = (heads + kWaves * per_step - 1) / (kWaves * per_step);
  const int per_block = (int)(((heads + steps - 1) / steps + kWaves - 1) / kWaves * kWaves);
  return {dim3((unsigned)(blocks * ((heads + per_block - 1) / per_block))), per_block};
}

}  // namespace

hipError_t launch_kv_append(const KvView& c, const uint16_t* q, int64_t q_ld, int q_heads, uint16_t* out,
                            int64_t out_ld, const uint16_t* k, int64_t k_ld, const uint16_t* v, int64_t v_ld,
                            const float* table, int64_t table_rows, int rotary, bool interleaved, uint32_t* flags,
                            hipStream_t stream) {
  const Grid g = grid_of(c.n_rows, q_heads + 2 * c.heads, c.dim);
  const Sources a{q,     k,          v,      q_ld,        k_ld,    v_ld,      out, out_ld,
                  table, table_rows, rotary, q_heads, g.per_block};
  auto* const f = interleaved ? (c.dim == 64    ? k_kv_append<64, true>
                                 : c.dim == 128 ? k_kv_append<128, true>
                                                : k_kv_append<256, true>)
                              : (c.dim == 64    ? k_kv_append<64, false>
                                 : c.dim == 128 ? k_kv_append<128, false>
                                                : k_kv_append<256, false>);
  hipLaunchKernelGGL(f, g.blocks, dim3(kThreads), 0, stream, c, a, flags);
  return hipGetLastError();
}

hipError_t launch_kv_read(const KvView& c, uint16_t* k, uint16_t* v, hipStream_t stream) {
  const Grid g = grid_of(c.n_rows, 2 * c.heads, c.dim);
  auto* const f = c.dim == 64 ? k_kv_read<64> : c.dim == 128 ? k_kv_read<128> : k_kv_read<256>;
  hipLaunchKernelGGL(f, g.blocks, dim3(kThreads), 0, stream, c, k, v, g.per_block);
  return hipGetLastError();
}

}  // namespace awq
