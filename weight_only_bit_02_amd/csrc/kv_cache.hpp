// The paged key / value cache held in 4 bits: its format, and helpers of the kernels that write
// and read it (kv_append.hip, kv_attend.hpp).
//
// One 16-bit word per (token, head, group of channels) holds a scale of 7 significant bits (the
// upper 12 bits of its fp16 form; the sign and the low mantissa bits are zero) and the zero in
// the low four bits. A value is (code - zero) scale: 4 bits times 7 bits, so it is exact in fp16
// and the matrix cores' operands carry no rounding, wherever scale and zero are applied.
//
// Codes lie as the matrix cores take them (v_mfma_f32_16x16x32_f16; lane = 16 h + c):
//   keys    a token's row of D / 8 words; word h (D / 32) + s holds channels 32 s + 8 h + i: a lane
//           loads its operands of all D / 32 slices at once, 16 tokens are one contiguous piece
//   values  16 tokens are one contiguous piece of 16-bit cells [4 h][16 c][D / 64 w][4 i]: cell
//           (h, c, w, i) holds token 4 h + i's channels c + 16 (4 w + j) in nibble j: a lane loads
//           four tokens of its D / 16 channels at once, two tokens to a 32-bit word
#pragma once

#include "common.hpp"
#include "widen.hpp"

namespace awq {

// What the host passes of awq_kv_cache and awq_kv_batch. The kernels read rows, lengths and
// page_table from the device and clamp what they find: wrong contents give wrong results, never
// an access out of range.
struct KvView {
  uint8_t *k_codes, *v_codes;
  uint16_t *k_params, *v_params;
  const int32_t *rows, *lengths, *table;
  int64_t pages;
  int page_shift;  // log2 of the page's tokens, 4 or more
  int heads;       // of keys and values
  int dim, group;
  int seqs, max_pages;
  int n_rows;

  // Bytes of one head's codes (keys or values) of a page, and 16-bit words of its parameters.
  __device__ __forceinline__ int64_t code_bytes() const { return ((int64_t)dim / 2) << page_shift; }
  __device__ __forceinline__ int64_t param_words() const { return ((int64_t)(dim / group)) << page_shift; }

  // The page table's entry for token `pos` of sequence s (-1 beyond it); the page, -1 if there is none.
  __device__ __forceinline__ int entry(int s, int64_t pos) const {
    const int64_t at = pos >> page_shift;
    return pos < 0 || at >= max_pages ? -1 : table[(int64_t)s * max_pages + at];
  }
  __device__ __forceinline__ int page(int entry) const { return entry >= 0 && entry < pages ? entry : -1; }
  __device__ __forceinline__ int page_of(int s, int64_t pos) const { return page(entry(s, pos)); }
};

// One sequence of the batch: its first row, its rows and its tokens in the cache.
struct KvSeq {
  int row0, rows;
  int length;  // as passed (a row's position goes by it)
  int tokens;  // of them that the page table can hold
};

__device__ __forceinline__ KvSeq kv_sequence(const KvView& v, int s) {
  const int a = v.rows[s], b = v.rows[s + 1];
  KvSeq q;
  q.row0 = a < 0 ? 0 : a > v.n_rows ? v.n_rows : a;
  const int end = b < q.row0 ? q.row0 : b > v.n_rows ? v.n_rows : b;
  q.rows = end - q.row0;
  const int most = v.max_pages << v.page_shift;  // < 2^30
  q.length = v.lengths[s];
  q.length = q.length < 0 ? 0 : q.length > (1 << 30) ? 1 << 30 : q.length;
  q.tokens = q.length > most ? most : q.length;
  return q;
}

// The sequence of row t: how many rows[s + 1] are at most t; seqs: none. W adjacent lanes have one
// t, and search for it with W probes a step.
template <int W>
__device__ __forceinline__ int kv_find(const KvView& v, int t, int lane) {
  const int first = v.rows[0];
  int lo = 0, n = v.seqs;
  while (n > 0) {
    const int step = (n + W - 1) / W;
    const int at = (lane % W + 1) * step;
    const bool before = at <= n && v.rows[lo + (at <= n ? at : 0)] <= t;
    const uint64_t found = __ballot(before) >> (lane / W * W);
    const int c = __popcll(found & (~0ull >> (64 - W)));
    lo += c * step;
    n = n - c * step < step - 1 ? n - c * step : step - 1;
  }
  return t < first ? v.seqs : lo;
}

// An item (rows of one sequence and head of keys) that several blocks took, one after the other.
struct AttendSplit {
  int row0;    // the sequence's first row
  int r0, r1;  // the item's rows x heads of the sequence
  int head;    // of keys
  int blocks;  // 0: none
  int index;   // which of them this is
};

// Queries of one attention call, beside the batch.
struct AttendArgs {
  const uint16_t* q;  // rows of q_heads heads, q_ld apart
  uint16_t* out;
  float* lse;         // [n_rows][q_heads] or NULL
  int64_t q_ld, out_ld;
  int q_heads, share;  // share = q_heads / heads of keys
  float scale_log2;    // scale / ln 2
  int causal, window;  // window 0: none
  // of one kernel: its blocks; their sums, unnormalised [2 blocks][rows of a tile][dim], with (maximum
  // of log2, sum) [2 blocks][rows]: item that went on from the block before, item that goes on
  int blocks, direct;
  float* part;
  float2* part_ml;
  AttendSplit* split;  // [blocks], NULL: nothing is split
};

hipError_t launch_kv_append(const KvView& c, const uint16_t* q, int64_t q_ld, int q_heads, uint16_t* out,
                            int64_t out_ld, const uint16_t* k, int64_t k_ld, const uint16_t* v, int64_t v_ld,
                            const float* table, int64_t table_rows, int rotary, bool interleaved, uint32_t* flags,
                            hipStream_t stream);
hipError_t launch_kv_read(const KvView& c, uint16_t* k, uint16_t* v, hipStream_t stream);

// Attention (kv_attend.hip). The plan goes by what the host knows: sizes, not lengths.
struct AttendPart {  // one kernel's share
  int tile;          // rows of a tile; 0: the kernel does not run
  int blocks;
  bool direct, join; // one item a block; items may be split over blocks
  size_t part, part_ml, split;  // offsets in the workspace
};
struct AttendPlan {
  AttendPart stream, tiles;
  int few;       // rows x share up to which a sequence is streamed
  size_t bytes;  // of the workspace
};
AttendPlan attend_plan(int64_t n_rows, int seqs, int max_rows, int64_t max_tokens, int share, int heads, int dim,
                       int group);
hipError_t launch_attend(const KvView& c, AttendArgs a, const AttendPlan& p, void* workspace, hipStream_t stream);

}  // namespace awq
