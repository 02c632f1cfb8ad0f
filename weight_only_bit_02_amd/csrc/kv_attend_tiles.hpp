// Attention over the 4-bit cache, tile form: many query rows per sequence and head of keys
// (prompts and pieces of them).
//
// A block takes 32 rows a wave of one head of keys, so that the codes are widened once for all
// of them: keys as fp16 [token][channel], values transposed, [channel][token], in LDS.
// v_mfma_f32_32x32x16_f16: S^T = K Q^T leaves lane (h, c) = (lane / 32, lane % 32) row c's scores of
// tokens 8 i + 4 h + 0..3, which are the second operand of O^T = V^T P^T for values whose tokens lie
// in that order: LDS holds them so. Probabilities go to the second product rounded to fp16 (an
// error of the output's own size; hi + lo would be half as much matrix work again), below 2^-21 of the row's
// largest in steps of 2^-31 of it (kLift).
//
// A step: scores and softmax, widening of a later step's codes, the second product. The block's
// second four waves, which share the SIMDs with the first four, run half a step behind, so that one
// wave's products meet the other's vector work (in step, the two add up); there is one barrier a
// step, after the first waves' second product and the second waves' softmax. A step's codes are
// widened by each wave its share, one step ahead into one of three buffers, from registers loaded
// a step before that.
//
// Measured, D = 128, groups of 128: a prompt of 4096 tokens, 32 heads, 155-161 us by card, 853-888
// TFLOP/s; pieces of 257-1024 rows behind 2000-12345 tokens, 64 heads on 8 of keys, groups of 64:
// 893-925 us, 822-851 TFLOP/s (a large product of the library: 1211). Matrix cores are busy for 37% of
// the cycles and vector instructions for 50%, softmax 131 and widening some 100 a wave and step beside
// 2048 cycles of products: the SIMD issues them in turn, and its two waves overlap what they can.
// Operands read eight products ahead, all waves in step, widening between the products, two running
// sums, or addresses in scalar registers: no gain or a loss.
//
// 16-byte pieces of an LDS row are exchanged by the row's number, so that the 16 rows that a
// read touches at a time lie in different banks.
#pragma once

#include "kv_attend.hpp"

namespace awq {

template <int D>
struct TileShape {
  static constexpr int kWaves = D == 256 ? 4 : 8;  // D = 256: a wave's sums take the registers of two
  static constexpr int kRows = 32 * kWaves;
  static constexpr int kThreads = kWaves * kWave;
  static constexpr int kTokens = 8192 / D;         // of a step: 4 KB of codes of each kind
  static constexpr int kWords = 1024 / kThreads;   // of codes of each kind per thread and step
  static constexpr int kUnitThreads = 16 * kThreads / kTokens;  // threads of 16 tokens
};

// 16-byte slot of piece `c` of row r, rows of N pieces: 16 rows at the same c lie in different
// banks (16 slots of them).
template <int N>
__device__ __forceinline__ int swizzled(int r, int c) {
  constexpr int kMix = N < 16 ? N : 16;
  return r * N + (c ^ (r / (16 / kMix) % kMix));
}

// A thread's codes and parameters of one step.
template <int D, int G>
struct TileCodes {
  static constexpr int kWords = TileShape<D>::kWords, kPerGroup = D / 32 / G;
  static constexpr int kGroups = kWords > kPerGroup ? kWords / kPerGroup : 1;  // that the thread's words have
  uint32_t k[kWords], v[kWords];
  uint32_t kp[kGroups];  // of the token and its neighbour (a 16-bit load would be waited for to be widened)
  uint2 vp[kGroups];
  int page;
};

// N products with an operand from LDS each, four at a time with the next four's reads under way
// (left to itself the compiler reads and waits just before each product). read(i) gives operand
// i, multiply(i, operand) takes it; the first four have been read.
template <int N, class Read, class Multiply>
__device__ __forceinline__ void products(half8w (&first)[4], const Read& read, const Multiply& multiply) {
  static_assert(N % 4 == 0, "");
  half8w b[2][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) b[0][i] = first[i];
#pragma unroll
  for (int k = 0; k < N; k += 4) {
    __builtin_amdgcn_sched_barrier(0);
    if (k + 4 < N) {
#pragma unroll
      for (int i = 0; i < 4; ++i) b[k / 4 + 1 & 1][i] = read(k + 4 + i);
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < 4; ++i) multiply(k + i, b[k / 4 & 1][i]);
  }
  __builtin_amdgcn_sched_barrier(0);
}

template <int D, int G>
__global__ void __launch_bounds__(TileShape<D>::kThreads) k_attend_tiles(KvView v, AttendArgs a, AttendList list) {
  using T = TileShape<D>;
  using Codes = TileCodes<D, G>;
  constexpr int kTokens = T::kTokens, kWords = T::kWords, kSlices = D / 16, kParts = kTokens / 32;
  __shared__ uint4 keys[3][kTokens * D / 8];    // [token][D / 8]
  __shared__ uint4 vals[3][kTokens * D / 8];    // [channel][kTokens / 8]
  __shared__ int there[3][kTokens / 16];        // whether 16 tokens have a page

  const int tid = threadIdx.x, lane = tid & (kWave - 1), h = lane >> 5, c = lane & 31;
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const Magic magic = magics();
  AttendSeqs seqs(v, a, list, lane);
  int unit, to, s, before, tiles_before;
  AttendSeq w;
  AttendSplit split{};
  AttendCut cut(1, 1);
  if (a.direct) {  // one item a block, the heads of a tile together, a sequence's last tiles first
    const int tile = blockIdx.x / v.heads;
    s = seqs.find(tile, true, before, tiles_before);
    if (s >= v.seqs) return;
    w = seqs.get(s);
    const int j = w.tiles - 1 - (tile - tiles_before);
    unit = before;
    for (int i = 0; i < j; ++i) unit += attend_chunks(a, list, w, i) * v.heads;
    const int n = attend_chunks(a, list, w, j);
    unit += (int)(blockIdx.x - tile * v.heads) * n;
    to = unit + n;
  } else {
    const int total = seqs.units();
    const int blocks = (int)gridDim.x < total ? (int)gridDim.x : total;
    if ((int)blockIdx.x >= blocks) {
      attend_split(a, split);
      return;
    }
    cut = AttendCut(total, blocks);
    unit = cut.start(blockIdx.x);
    to = cut.start(blockIdx.x + 1);
    s = seqs.find(unit, false, before, tiles_before);
    if (s >= v.seqs) {  // (wrong rows)
      attend_split(a, split);
      return;
    }
    w = seqs.get(s);
  }

  // The thread's part of a step's codes: `kWords` words of 16 tokens' keys, and of their values. The
  // order of the threads lets 16 lanes' 16-byte pieces of keys, and 32 lanes' 8-byte pieces of
  // values, lie in different banks.
  const int sub = tid / T::kUnitThreads, in = tid % T::kUnitThreads;
  const int k_h = in & 3;
  const int k_token = D == 64 ? (in >> 2 & 1) | (in >> 3 & 1) << 3 | (in >> 4) << 1 : (in >> 2 & 3) << 2 | in >> 5;
  const int k_s = D == 64 ? 0 : (in >> 4 & 1) * kWords;            // words (k_h, k_s), (k_h, k_s + 1) ...
  const int v_c = in & 15, v_h = (in >> 4 & 1) << 1 | (in >> 5 & 1);
  const int v_w = D == 64 ? 0 : (in >> 6) * (kWords / 2);          // cells (v_h, v_c, v_w), ...
  const uint32_t code_page = v.heads * (uint32_t)v.code_bytes(), par_page = v.heads * (uint32_t)v.param_words();

  while (unit < to) {
    const int at = unit - before;
    if (at < 0) break;  // sums that wrapped (wrong rows)
    if (at >= w.units) {
      before += w.units;
      if (++s >= v.seqs) break;
      w = attend_seq(v, a, list, s);
      continue;
    }
    const AttendItem x = attend_item(v, a, list, w, at);
    const int u0 = x.chunk, u1 = x.chunks - u0 < to - unit ? x.chunks : u0 + (to - unit);

    const int r0 = x.tile * T::kRows, r1 = (r0 + T::kRows < w.flat ? r0 + T::kRows : w.flat) - 1;
    const int p0 = w.q.length - w.q.rows, last = w.q.tokens - 1;
    // the wave's rows
    const int wr0 = r0 + 32 * wave, wr1 = wr0 + 31 < r1 ? wr0 + 31 : r1;
    const int row = wr0 + c, rin = row <= r1 ? row : r1;
    const int token = rin / a.share, q_head = x.head * a.share + rin - token * a.share;
    const int p = p0 + token;
    const int hi = attend_last(a, p, last), lo = a.window > 0 ? p - a.window + 1 : 0;
    half8w q[kSlices];
    {
      const uint16_t* qr = a.q + (w.q.row0 + token) * a.q_ld + (int64_t)q_head * D;
#pragma unroll
      for (int t = 0; t < kSlices; ++t) {
        const uint4 b = row <= r1 ? *reinterpret_cast<const uint4*>(qr + 16 * t + 8 * h) : make_uint4(0, 0, 0, 0);
        q[t] = __builtin_bit_cast(half8w, b);
      }
    }
    // tokens that all of the wave's rows see, that any does, and that any of the block's does
    const int pa = p0 + wr0 / a.share, pb = p0 + wr1 / a.share, pe = p0 + r1 / a.share;
    const int all_hi = attend_last(a, pa, last), any_hi = attend_last(a, pb, last);
    const int all_lo = a.window > 0 ? pb - a.window + 1 : 0, any_lo = a.window > 0 ? pa - a.window + 1 : 0;
    const int end = attend_last(a, pe, last) + 1;
    const int t0 = w.first + u0 * kAttendChunk;
    const int t1 = w.first + u1 * kAttendChunk < end ? w.first + u1 * kAttendChunk : end;
    const bool rows = wr0 <= r1;

    f32x16w o[D / 32];
    float m = -__builtin_inff(), l = 0.0f;
#pragma unroll
    for (int n = 0; n < D / 32; ++n) o[n] = f32x16w{};

    // The page table's entry of the thread's 16 tokens of a step; looked at when it is used.
    const int32_t* const table = v.table + (int64_t)s * v.max_pages;
    const auto entry_of = [&](int tb) AWQ_INLINE {
      const int at = (tb + 16 * sub) >> v.page_shift;
      return table[at < v.max_pages ? at : v.max_pages - 1];
    };
    const uint8_t* const kb0 =
        v.k_codes + x.head * v.code_bytes() + k_token * (D / 2) + 4 * (k_h * (D / 32) + k_s);
    const uint8_t* const vb0 =
        v.v_codes + x.head * v.code_bytes() + 4 * ((v_h * 16 + v_c) * (D / 32) + 2 * v_w);
    const uint16_t* const kq0 =
        v.k_params + x.head * v.param_words() + (k_token & ~1) + ((k_s / Codes::kPerGroup) << v.page_shift);
    const uint16_t* const vq0 =
        v.v_params + x.head * v.param_words() + 4 * v_h + ((2 * v_w / Codes::kPerGroup) << v.page_shift);
    const auto load = [&](Codes& d, int entry, int tb) AWQ_INLINE {
      d.page = tb + 16 * sub < t1 ? v.page(entry) : -1;
      const uint32_t page = d.page < 0 ? 0 : d.page;  // (page 0 for none: not looked at)
      const uint32_t place = (uint32_t)(tb + 16 * sub) & ((1u << v.page_shift) - 1);
      const uint64_t code = (uint64_t)page * code_page + place * (D / 2), par = (uint64_t)page * par_page + place;
      if constexpr (kWords == 2) {
        const uint2 y = *reinterpret_cast<const uint2*>(kb0 + code), z = *reinterpret_cast<const uint2*>(vb0 + code);
        d.k[0] = y.x, d.k[1] = y.y, d.v[0] = z.x, d.v[1] = z.y;
      } else {
        const uint4 y = *reinterpret_cast<const uint4*>(kb0 + code), z = *reinterpret_cast<const uint4*>(vb0 + code);
        d.k[0] = y.x, d.k[1] = y.y, d.k[2] = y.z, d.k[3] = y.w;
        d.v[0] = z.x, d.v[1] = z.y, d.v[2] = z.z, d.v[3] = z.w;
      }
#pragma unroll
      for (int i = 0; i < Codes::kGroups; ++i) {
        d.kp[i] = *reinterpret_cast<const uint32_t*>(kq0 + par + (i << v.page_shift));
        d.vp[i] = *reinterpret_cast<const uint2*>(vq0 + par + (i << v.page_shift));
      }
    };
    const auto widen = [&](const Codes& d, int buf) AWQ_INLINE {
      if (in == 0) there[buf][sub] = d.page >= 0;
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        const uint32_t kp = d.kp[i / Codes::kPerGroup];
        const Params2 y = params2(__builtin_amdgcn_perm(kp, kp, k_token & 1 ? 0x03020302u : 0x01000100u));
        half2w e[4];
        widen4(d.k[i], y.zz, y.zz64, y.s2, magic, e);
        const half8w b{e[0][0], e[0][1], e[1][0], e[1][1], e[2][0], e[2][1], e[3][0], e[3][1]};
        keys[buf][swizzled<D / 8>(16 * sub + k_token, 4 * (k_s + i) + k_h)] = __builtin_bit_cast(uint4, b);
      }
      uint2 vp[Codes::kGroups];
#pragma unroll
      for (int i = 0; i < Codes::kGroups; ++i) vp[i] = make_uint2(attend_finite(d.vp[i].x), attend_finite(d.vp[i].y));
#pragma unroll
      for (int i = 0; i < kWords / 2; ++i) {  // channels v_c + 16 (4 (v_w + i) + j)
#pragma unroll
        for (int g = 0; g < 2; ++g) {         // j = 2 g, 2 g + 1: one group
          const uint2 p = vp[(2 * i + g) / Codes::kPerGroup];
          const Params2 y = params2(p.x), z = params2(p.y);
          half2w e[4], f[4];
          widen4(d.v[2 * i], y.zz, y.zz64, y.s2, magic, e);
          widen4(d.v[2 * i + 1], z.zz, z.zz64, z.s2, magic, f);
#pragma unroll
          for (int j = 2 * g; j < 2 * g + 2; ++j) {
            const int ch = v_c + 16 * (4 * (v_w + i) + j);
            uint2* slot = reinterpret_cast<uint2*>(vals[buf] + swizzled<kTokens / 8>(ch, 2 * sub + (v_h & 1)));
            slot[v_h >> 1] = make_uint2(__builtin_bit_cast(uint32_t, e[j]), __builtin_bit_cast(uint32_t, f[j]));
          }
        }
      }
    };
    half8w pr[kParts][2], first[4];
    const auto read_key = [&](int buf, int i) AWQ_INLINE {  // operand i of the scores
      return __builtin_bit_cast(half8w, keys[buf][swizzled<D / 8>(32 * (i % kParts) + c, 2 * (i / kParts) + h)]);
    };
    const auto read_value = [&](int buf, int i) AWQ_INLINE {  // of the second product
      constexpr int kN = D / 32;
      return __builtin_bit_cast(half8w, vals[buf][swizzled<kTokens / 8>(32 * (i % kN) + c, 2 * (i / kN) + h)]);
    };
    const auto seen = [&](int tb) { return rows && tb <= any_hi && tb + kTokens > any_lo; };
    // scores and probabilities of a step
    const auto score = [&](int tb, int buf) AWQ_INLINE {
      if (!seen(tb)) return;
      const int paged = there[buf][lane % (kTokens / 16)];
      f32x16w sc[kParts];
#pragma unroll
      for (int t = 0; t < kParts; ++t) sc[t] = f32x16w{};
      __builtin_amdgcn_s_setprio(1);  // products first: 2% over equal waves
      products<kParts * kSlices>(
          first, [&](int i) AWQ_INLINE { return read_key(buf, i); },
          [&](int i, half8w b) AWQ_INLINE {
            sc[i % kParts] = __builtin_amdgcn_mfma_f32_32x32x16_f16(b, q[i / kParts], sc[i % kParts], 0, 0, 0);
          });
      __builtin_amdgcn_s_setprio(0);
      // (empty asm: nothing of a branch ahead of it)
      const float none = -__builtin_inff();
      if (tb + kTokens > all_hi + 1) {
        asm volatile("");
        const int most = hi - tb - 4 * h;
#pragma unroll
        for (int t = 0; t < kParts; ++t)
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (32 * t + 8 * (i >> 2) + (i & 3) > most) sc[t][i] = none;
      }
      if (tb < all_lo) {
        asm volatile("");
        const int least = lo - tb - 4 * h;
#pragma unroll
        for (int t = 0; t < kParts; ++t)
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (32 * t + 8 * (i >> 2) + (i & 3) < least) sc[t][i] = none;
      }
      const uint64_t gone = __ballot(paged == 0);  // 16 tokens without a page, by bits
      if (gone) {
        asm volatile("");
#pragma unroll
        for (int t = 0; t < kParts; ++t)
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (gone >> (2 * t + (i >> 3)) & 1) sc[t][i] = none;
      }
      float top = sc[0][0];
#pragma unroll
      for (int t = 0; t < kParts; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) top = fmaxf(top, sc[t][i]);
      top *= a.scale_log2;
      if (__ballot(top > m + kLazy)) {
        asm volatile("");
        top = fmaxf(fmaxf(top, __shfl_xor(top, 32)), m);
        const float f = top > m ? __builtin_amdgcn_exp2f(m - top) : 1.0f;
        m = top;
        l *= f;
#pragma unroll
        for (int n = 0; n < D / 32; ++n) o[n] *= f;
      }
      float base = m == -__builtin_inff() ? 0.0f : m - kLift;
      if (__ballot(__builtin_fabsf(base) > kFar)) {
        asm volatile("");
        if (__builtin_fabsf(base) > kFar) {
#pragma unroll
          for (int t = 0; t < kParts; ++t)
#pragma unroll
            for (int i = 0; i < 16; ++i) sc[t][i] = attend_far(sc[t][i], m, a.scale_log2);
          base = -kLift;
        }
      }
#pragma unroll
      for (int t = 0; t < kParts; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[t][i], a.scale_log2, -base));
          l += e;
          pr[t][i >> 3][i & 7] = (_Float16)e;
        }
    };
    const auto add = [&](int tb, int buf) AWQ_INLINE {
      if (!seen(tb)) return;
      __builtin_amdgcn_s_setprio(1);
      products<2 * kParts * (D / 32)>(
          first, [&](int i) AWQ_INLINE { return read_value(buf, i); },
          [&](int i, half8w b) AWQ_INLINE {
            const int n = i % (D / 32), k = i / (D / 32);
            o[n] = __builtin_amdgcn_mfma_f32_32x32x16_f16(b, pr[k >> 1][k & 1], o[n], 0, 0, 0);
          });
      __builtin_amdgcn_s_setprio(0);
    };
    // LDS alone is waited for: loads stay in flight
    const auto meet = [&]() AWQ_INLINE { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); };

    const bool behind = wave >= T::kWaves / 2;
    const auto advance = [&](Codes& d, int& entry, int tb, int buf) AWQ_INLINE {  // widens step tb, loads the next
      widen(d, buf);
      load(d, entry, tb + kTokens);
      entry = entry_of(tb + 2 * kTokens);
    };
    Codes next;
    load(next, entry_of(t0), t0);
    int entry = entry_of(t0 + kTokens);
    meet();  // the item before is done with the buffers
    advance(next, entry, t0, 0);
    meet();
    if (behind) advance(next, entry, t0 + kTokens, 1);
    int buf = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) first[i] = read_key(0, i);
    for (int tb = t0; tb < t1; tb += kTokens) {
      const int after = buf == 2 ? 0 : buf + 1;
      score(tb, buf);
#pragma unroll
      for (int i = 0; i < 4; ++i) first[i] = read_value(buf, i);
      if (behind) meet();
      // (buf + 1 + behind) % 3
      advance(next, entry, tb + (behind ? 2 : 1) * kTokens, behind ? (after == 2 ? 0 : after + 1) : after);
      add(tb, buf);
      if (!behind) meet();
#pragma unroll
      for (int i = 0; i < 4; ++i) first[i] = read_key(after, i);
      buf = after;
    }

    const bool alone = u0 == 0 && u1 == x.chunks;
    if (u1 < x.chunks) {
      const int b0 = cut.block(unit - u0), b1 = cut.block(unit - u0 + x.chunks - 1);
      split = AttendSplit{w.q.row0, r0, r1, x.head, b1 - b0 + 1, (int)blockIdx.x - b0};
    }
    l += __shfl_xor(l, 32);
    if (rows && row <= r1) {
      if (alone) {
        const float d = l == 0.0f ? 0.0f : 1.0f / l;  // no token: zeros
        uint16_t* y = a.out + (w.q.row0 + token) * a.out_ld + (int64_t)q_head * D;
#pragma unroll
        for (int n = 0; n < D / 32; ++n)
#pragma unroll
          for (int i = 0; i < 16; i += 4) {
            half4a b;
#pragma unroll
            for (int k = 0; k < 4; ++k) b[k] = (_Float16)(o[n][i + k] * d);
            *reinterpret_cast<half4a*>(y + 32 * n + 2 * i + 4 * h) = b;
          }
        if (a.lse && h == 0)
          a.lse[(int64_t)(w.q.row0 + token) * a.q_heads + q_head] = attend_lse(m, l * kDrop);
      } else {
        const int64_t slot = ((int64_t)2 * blockIdx.x + (u0 == 0 ? 1 : 0)) * T::kRows + (row - r0);
        float* y = a.part + slot * D;
#pragma unroll
        for (int n = 0; n < D / 32; ++n)
#pragma unroll
          for (int i = 0; i < 16; i += 4)
            *reinterpret_cast<f32x4w*>(y + 32 * n + 2 * i + 4 * h) =
                f32x4w{o[n][i], o[n][i + 1], o[n][i + 2], o[n][i + 3]} * kDrop;
        if (h == 0) a.part_ml[slot] = make_float2(m, l * kDrop);
      }
    }
    unit += u1 - u0;
  }
  attend_split(a, split);
}

template <int D, int G>
hipError_t attend_tiles(const KvView& v, const AttendArgs& a, const AttendList& list, hipStream_t stream) {
  hipLaunchKernelGGL((k_attend_tiles<D, G>), dim3(a.blocks), dim3(TileShape<D>::kThreads), 0, stream, v, a, list);
  return hipGetLastError();
}

}  // namespace awq
