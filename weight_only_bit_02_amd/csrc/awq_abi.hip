// C ABI of libawq_mi355x: argument validation, workspace layout, kernel dispatch.
// The operations and their sources are documented in include/awq.h.
#include <stdlib.h>
#include <string.h>

#include <mutex>

#include "awq.h"
#include "kv_cache.hpp"
#include "launch.hpp"

// Workspace of awq_search_scales_noalloc: a static device array, one copy per GPU for as
// long as the process lives. Host code never passes `scratch` itself to a kernel (on the
// host it is only a stand-in for the symbol): its device address is looked up once per
// device with hipGetSymbolAddress and kept in g_scratch_ptr.
static __device__ __attribute__((aligned(256))) unsigned char scratch[AWQ_NOALLOC_SCRATCH_BYTES];
namespace {
constexpr int kMaxDevices = 64;
std::mutex g_scratch_mu;
void* g_scratch_ptr[kMaxDevices];
}  // namespace

namespace {

constexpr int64_t kMaxDim = (int64_t)1 << 31;

awq_config resolve(const awq_config* cfg) {
  if (cfg) return *cfg;
  return awq_config{4, 128, 1, 20};
}

bool supported(const awq_config& c) {
  return (c.w_bit == 3 || c.w_bit == 4 || c.w_bit == 8) &&
         (c.group_size == 128 || c.group_size == 64 || c.group_size == 32) &&
         (c.zero_point == 0 || c.zero_point == 1) && c.n_grid >= 1 && c.n_grid <= 64;
}

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
bool aligned4(const void* p) { return ((uintptr_t)p & 3u) == 0; }

bool good_nk(int64_t N, int64_t K) {
  return N >= 1 && K >= 128 && K % 128 == 0 && N < kMaxDim && K < kMaxDim;
}

awq_status hip_status(hipError_t e) { return e == hipSuccess ? AWQ_OK : AWQ_ERR_HIP; }

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

// Search workspace: [u: int64 K][act: fp64 K][s_grid: fp16 n_grid K]
// [partials: fp64 n_grid x row tiles x token chunks][errf: fp64 n_grid][cand: n_grid bytes]
// [xp: X in MFMA operand order, T rounded up to 64 tokens]
struct SearchLayout {
  size_t u, act, sgrid, partials, errf, cand, xp, total;
  int64_t n_partials;  // per grid point
};

SearchLayout search_layout(int64_t T, int64_t N, int64_t K, int n_grid) {
  SearchLayout L;
  const int64_t ntiles = (N + awq::search_row_tile() - 1) / awq::search_row_tile();
  const int64_t chunk = awq::search_token_chunk(T);
  L.n_partials = ntiles * ((T + chunk - 1) / chunk);
  L.u = 0;
  L.act = align256(L.u + (size_t)K * 8);
  L.sgrid = align256(L.act + (size_t)K * 8);
  L.partials = align256(L.sgrid + (size_t)n_grid * K * 2);
  L.errf = align256(L.partials + (size_t)n_grid * L.n_partials * 8);
  L.cand = align256(L.errf + (size_t)n_grid * 8);
  L.xp = align256(L.cand + (size_t)n_grid);
  L.total = align256(L.xp + awq::packed_x_bytes(T, K));
  return L;
}

// Clip-search workspace: [err: fp64 n_shrink x N x G]
// [xp: X in MFMA operand order, T rounded up to 64 tokens; or, in the Gram form, the
//  per-group G' and the channel scales]
struct ClipLayout {
  size_t err, xp, total;
};

ClipLayout clip_layout(int64_t T, int64_t N, int64_t K, int n_shrink, int group) {
  ClipLayout L;
  L.err = 0;
  L.xp = align256(L.err + awq::clip_err_bytes(T, N, K, n_shrink, group));
  L.total = align256(L.xp + awq::clip_scratch_bytes(T, K, group));
  return L;
}

// Limits of the expert and adapter calls.
constexpr int64_t kMaxRows = (int64_t)1 << 30;      // positions and rows are kept in 32 bits
constexpr int64_t kMaxElements = ((int64_t)1 << 31) - 1;  // of X and of an adapter's A: their bytes end
                                                          // below 2^32 - 1, the most a descriptor covers
constexpr int64_t kMaxKvRows = (int64_t)1 << 22;    // rows of a batch of the cache's calls
constexpr int64_t kSkinnyMaxRows = 65536;           // its grid: one row of blocks per row tile

// One weight's codes are addressed with 32-bit offsets too.
bool good_weight(int64_t N, int64_t K, int w_bit) { return N < ((int64_t)1 << 32) / (K * w_bit / 8); }

bool good_groups(int32_t g) { return g >= 1 && g <= AWQ_MAX_GROUPS; }
bool good_rank(int32_t r) { return r >= 8 && r <= AWQ_MAX_LORA_RANK && r % 8 == 0; }
bool good_workspace(const void* p, size_t have, size_t need) {
  return need == 0 || (p && have >= need && aligned16(p));
}
// A launch has fewer than 2^32 threads: fewer than 2^24 blocks of 256. The narrowest tiles are 64
// rows x 128 outputs, of GEMM64K 32 x 32 (which AUTO takes for few blocks only).
bool grouped_grid_ok(int64_t n, int64_t N, int64_t groups, int kernel) {
  const int64_t rows = kernel == AWQ_GROUPED_GEMM64K ? 32 : 64, outs = kernel == AWQ_GROUPED_GEMM64K ? 32 : 128;
  return n / rows + groups + 1 < ((int64_t)1 << 24) / (N / outs + 1);
}

// Largest M that AWQ_LINEAR_AUTO serves with a GEMV-class kernel (above it, the MFMA
// GEMM); AWQ_GEMV_MAX_M overrides it (0 .. 64) to measure the crossover.
int gemv_max_m_from_env() {
  const char* e = getenv("AWQ_GEMV_MAX_M");
  if (!e) return awq::kSkinnyMaxM;
  int v = atoi(e);
  if (v < 0) v = 0;
  if (v > awq::kSkinnyMaxM) v = awq::kSkinnyMaxM;
  return v;
}
const int g_gemv_max_m = gemv_max_m_from_env();

}  // namespace

extern "C" {

const char* awq_status_string(awq_status s) {
  // callers may pass any integer: read it as one (a value outside the enumerators is not a
  // valid awq_status in C++, so it must not be switched on as one)
  int v = 0;
  static_assert(sizeof(s) == sizeof(v), "awq_status is an int-sized enum");
  memcpy(&v, &s, sizeof v);
  switch (v) {
    case AWQ_OK: return "ok";
    case AWQ_ERR_NULL_POINTER: return "a required pointer is NULL";
    case AWQ_ERR_BAD_SHAPE: return "bad shape (sizes must be >= 1, K a multiple of 128, T <= 8192)";
    case AWQ_ERR_UNSUPPORTED: return "unsupported config (w_bit 3, 4 or 8, group_size 128, 64 or 32, zero_point 0 or 1, 1 <= n_grid <= 64)";
    case AWQ_ERR_MISALIGNED: return "a base pointer is not 16-byte aligned";
    case AWQ_ERR_WORKSPACE: return "workspace missing or too small";
    case AWQ_ERR_HIP: return "HIP launch error";
    case AWQ_ERR_SCRATCH_LIMIT:
      return "the call needs more scratch than the static AWQ_NOALLOC_SCRATCH_BYTES array";
  }
  return "unknown status";
}

int32_t awq_gemv_max_m(void) { return g_gemv_max_m; }

awq_status awq_quantize_pack(const void* W, int64_t N, int64_t K, const void* s,
                             const awq_config* cfg, uint32_t* qweight, void* scales,
                             uint8_t* zeros, uint32_t* flags, void* stream) {
  return awq_quantize_pack_clipped(W, N, K, s, nullptr, 0, cfg, qweight, scales, zeros, flags,
                                   stream);
}

awq_status awq_quantize_pack_clipped(const void* W, int64_t N, int64_t K, const void* s,
                                     const uint8_t* clip_idx, int32_t clip_steps,
                                     const awq_config* cfg, uint32_t* qweight, void* scales,
                                     uint8_t* zeros, uint32_t* flags, void* stream) {
  const awq_config c = resolve(cfg);
  if (!W || !qweight || !scales || !zeros) return AWQ_ERR_NULL_POINTER;
  if (!supported(c)) return AWQ_ERR_UNSUPPORTED;
  if (!good_nk(N, K)) return AWQ_ERR_BAD_SHAPE;
  if (clip_idx && (clip_steps < 1 || clip_steps > 65535)) return AWQ_ERR_BAD_SHAPE;
  if (!aligned16(W) || !aligned16(qweight) || !aligned16(scales) || !aligned16(zeros) ||
      (s && !aligned16(s)) || (flags && !aligned4(flags)))
    return AWQ_ERR_MISALIGNED;
  return hip_status(awq::launch_quant_pack((const uint16_t*)W, N, K, (const uint16_t*)s, qweight,
                                           (uint16_t*)scales, zeros, clip_idx, clip_steps,
                                           c.zero_point == 0, c.group_size, c.w_bit, flags,
                                           (hipStream_t)stream));
}

size_t awq_activation_stats_workspace_size(int64_t T, int64_t K) {
  (void)T;
  return K > 0 ? align256((size_t)K * 8) : 0;
}

awq_status awq_activation_stats(const void* X, int64_t T, int64_t K, double* act_mean,
                                void* workspace, size_t workspace_bytes, uint32_t* flags,
                                void* stream) {
  if (!X || !act_mean) return AWQ_ERR_NULL_POINTER;
  if (T < 1 || T > AWQ_MAX_CALIB_TOKENS || !good_nk(1, K)) return AWQ_ERR_BAD_SHAPE;
  if (!workspace || workspace_bytes < awq_activation_stats_workspace_size(T, K))
    return AWQ_ERR_WORKSPACE;
  if (!aligned16(X) || !aligned16(act_mean) || !aligned16(workspace) ||
      (flags && !aligned4(flags)))
    return AWQ_ERR_MISALIGNED;
  hipStream_t st = (hipStream_t)stream;
  auto* u = (unsigned long long*)workspace;
  hipError_t e = awq::launch_zero_u64(u, K, st);
  if (e == hipSuccess) e = awq::launch_act_sums((const uint16_t*)X, T, K, u, flags, st);
  if (e == hipSuccess) e = awq::launch_act_finalize(u, T, K, act_mean, st);
  return hip_status(e);
}

awq_status awq_candidate_scales(const double* act_mean, int64_t K, const awq_config* cfg,
                                void* s_grid, void* stream) {
  const awq_config c = resolve(cfg);
  if (!act_mean || !s_grid) return AWQ_ERR_NULL_POINTER;
  if (!supported(c)) return AWQ_ERR_UNSUPPORTED;
  if (!good_nk(1, K)) return AWQ_ERR_BAD_SHAPE;
  if (!aligned16(act_mean) || !aligned16(s_grid)) return AWQ_ERR_MISALIGNED;
  return hip_status(
      awq::launch_scalegen(act_mean, K, c.n_grid, (uint16_t*)s_grid, (hipStream_t)stream));
}

size_t awq_search_workspace_size(int64_t T, int64_t N, int64_t K, const awq_config* cfg) {
  const awq_config c = resolve(cfg);
  if (!supported(c) || T < 1 || T > AWQ_MAX_CALIB_TOKENS || !good_nk(N, K)) return 0;
  return search_layout(T, N, K, c.n_grid).total;
}

awq_status awq_search_scales(const void* X, int64_t T, const void* W, int64_t N, int64_t K,
                             const awq_config* cfg, void* s_best, int32_t* best_idx,
                             double* err, void* s_grid, void* workspace,
                             size_t workspace_bytes, uint32_t* flags, void* stream) {
  const awq_config c = resolve(cfg);
  if (!X || !W || !s_best || !best_idx) return AWQ_ERR_NULL_POINTER;
  if (!supported(c)) return AWQ_ERR_UNSUPPORTED;
  if (T < 1 || T > AWQ_MAX_CALIB_TOKENS || !good_nk(N, K)) return AWQ_ERR_BAD_SHAPE;
  const SearchLayout L = search_layout(T, N, K, c.n_grid);
  if (!workspace || workspace_bytes < L.total) return AWQ_ERR_WORKSPACE;
  if (!aligned16(X) || !aligned16(W) || !aligned16(s_best) || !aligned4(best_idx) ||
      (err && !aligned16(err)) || (s_grid && !aligned16(s_grid)) || !aligned16(workspace) ||
      (flags && !aligned4(flags)))
    return AWQ_ERR_MISALIGNED;
  hipStream_t st = (hipStream_t)stream;
  char* ws = (char*)workspace;
  auto* u = (unsigned long long*)(ws + L.u);
  auto* act = (double*)(ws + L.act);
  auto* sg = s_grid ? (uint16_t*)s_grid : (uint16_t*)(ws + L.sgrid);
  auto* partials = (double*)(ws + L.partials);
  const auto* Xh = (const uint16_t*)X;
  hipError_t e = awq::launch_zero_u64(u, K, st);
  if (e == hipSuccess) e = awq::launch_act_sums(Xh, T, K, u, flags, st);
  if (e == hipSuccess) e = awq::launch_act_finalize(u, T, K, act, st);
  if (e == hipSuccess) e = awq::launch_scalegen(act, K, c.n_grid, sg, st);
  const bool one_term = awq::search_one_term(T, N, K);
  auto* errf = (double*)(ws + L.errf);
  auto* cand = (uint8_t*)(ws + L.cand);
  if (e == hipSuccess)
    e = awq::launch_search_err(Xh, T, (const uint16_t*)W, N, K, sg, c.n_grid, c.zero_point == 0,
                               c.group_size, c.w_bit, (uint4*)(ws + L.xp), partials, errf, cand,
                               one_term, flags, st);
  if (e == hipSuccess)
    e = awq::launch_search_reduce(partials, c.n_grid, L.n_partials, one_term ? cand : nullptr,
                                  errf, sg, K, (uint16_t*)s_best, best_idx, err, flags, st);
  return hip_status(e);
}

awq_status awq_search_scales_noalloc(const void* X, int64_t T, const void* W, int64_t N,
                                     int64_t K, const awq_config* cfg, void* s_best,
                                     int32_t* best_idx, double* err, void* s_grid,
                                     uint32_t* flags, void* stream) {
  const awq_config c = resolve(cfg);
  if (!X || !W || !s_best || !best_idx) return AWQ_ERR_NULL_POINTER;
  if (!supported(c)) return AWQ_ERR_UNSUPPORTED;
  if (T < 1 || T > AWQ_MAX_CALIB_TOKENS || !good_nk(N, K)) return AWQ_ERR_BAD_SHAPE;
  if (search_layout(T, N, K, c.n_grid).total > (size_t)AWQ_NOALLOC_SCRATCH_BYTES)
    return AWQ_ERR_SCRATCH_LIMIT;
  // the current device's copy of the array (looked up on the first call on each device)
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return AWQ_ERR_HIP;
  void* ws = nullptr;
  {
    std::lock_guard<std::mutex> lock(g_scratch_mu);
    if (!g_scratch_ptr[dev]) {
      void* p = nullptr;
      if (hipGetSymbolAddress(&p, HIP_SYMBOL(scratch)) != hipSuccess || !p) return AWQ_ERR_HIP;
      g_scratch_ptr[dev] = p;
    }
    ws = g_scratch_ptr[dev];
  }
  return awq_search_scales(X, T, W, N, K, cfg, s_best, best_idx, err, s_grid, ws,
                           (size_t)AWQ_NOALLOC_SCRATCH_BYTES, flags, stream);
}

static awq_status linear_common(const void* X, int64_t M, const uint32_t* qweight,
                                const void* scales, const uint8_t* zeros, int64_t N, int64_t K,
                                const awq_config* cfg, void* Y, uint32_t* flags,
                                awq_linear_kernel kernel_arg, bool gated, void* stream) {
  // the caller may pass any integer: validate it as one before it is used as the enum
  int kv = 0;
  static_assert(sizeof(kernel_arg) == sizeof(kv), "awq_linear_kernel is an int-sized enum");
  memcpy(&kv, &kernel_arg, sizeof kv);
  const awq_config c = resolve(cfg);
  if (!X || !qweight || !scales || !zeros || !Y) return AWQ_ERR_NULL_POINTER;
  if (!supported(c)) return AWQ_ERR_UNSUPPORTED;
  if (M < 1 || M >= kMaxDim || !good_nk(N, K)) return AWQ_ERR_BAD_SHAPE;
  if (gated && (N < 2 || N % 2 != 0)) return AWQ_ERR_BAD_SHAPE;
  if (kv < AWQ_LINEAR_AUTO || kv > AWQ_LINEAR_GEMM_WIDE) return AWQ_ERR_UNSUPPORTED;
  awq_linear_kernel kernel = (awq_linear_kernel)kv;
  if (kernel == AWQ_LINEAR_GEMM_WIDE && !awq::gemm_wide_supported(K, c.group_size, c.w_bit, gated))
    return AWQ_ERR_UNSUPPORTED;
  if (kernel == AWQ_LINEAR_GEMV && M > awq::kGemvMaxM) return AWQ_ERR_BAD_SHAPE;
  if (kernel == AWQ_LINEAR_SKINNY && M > awq::kSkinnyMaxM) return AWQ_ERR_BAD_SHAPE;
  if (!aligned16(X) || !aligned16(qweight) || !aligned16(scales) || !aligned16(zeros) ||
      !aligned16(Y) || (flags && !aligned4(flags)))
    return AWQ_ERR_MISALIGNED;
  hipStream_t st = (hipStream_t)stream;
  if (flags) {
    // data conditions: a scan of X and the group scales ahead of the linear kernel
    const hipError_t e = awq::launch_nonfinite_scan((const uint16_t*)X, M * K,
                                                    (const uint16_t*)scales,
                                                    N * (K / c.group_size), flags, st);
    if (e != hipSuccess) return AWQ_ERR_HIP;
  }
  // AUTO, measured on the Llama-2-7B layer: the vector-ALU GEMV up to M = 3 (its dot cost
  // grows with M), the MFMA skinny GEMV up to g_gemv_max_m, the MFMA GEMM above.
  if (kernel == AWQ_LINEAR_AUTO && c.w_bit != 4) {
    kernel = M <= awq::kGemvMaxM ? AWQ_LINEAR_GEMV
             : M <= awq::kSkinnyMaxM ? AWQ_LINEAR_SKINNY : AWQ_LINEAR_GEMM;
    // the 256-row GEMM where it takes the format (8-bit: plain outputs on 128-column tiles;
    // 3-bit: 256-column tiles), by the 4-bit rule below
    if (kernel == AWQ_LINEAR_GEMM && awq::gemm_wide_supported(K, c.group_size, c.w_bit, gated) &&
        (gated ? awq::gemm_wide_tiles(M, N, true, c.w_bit) >= awq::kWideMinTilesGated
               : M >= awq::kWideMinM))
      kernel = AWQ_LINEAR_GEMM_WIDE;
  }
  if (kernel == AWQ_LINEAR_AUTO) {
    kernel = M <= awq::kVgemvAutoMaxM && M <= g_gemv_max_m ? AWQ_LINEAR_GEMV
             : M <= g_gemv_max_m                            ? AWQ_LINEAR_SKINNY
                                                            : AWQ_LINEAR_GEMM;
    // the 256-row tiling (measured on the Llama-2-7B shapes at M = 128..2048): plain outputs
    // from 128 rows, where its 128-column tiles already beat the 128-row GEMM on every shape;
    // fused gate|up (256-column tiles only) once it has 160 tiles (ahead from 172, behind at
    // 86 and below, where the 128-row tiles give twice as many CUs work)
    if (kernel == AWQ_LINEAR_GEMM && awq::gemm_wide_supported(K, c.group_size, c.w_bit, gated) &&
        (gated ? awq::gemm_wide_tiles(M, N, true, c.w_bit) >= awq::kWideMinTilesGated
               : M >= awq::kWideMinM))
      kernel = AWQ_LINEAR_GEMM_WIDE;
  }
  const auto* Xh = (const uint16_t*)X;
  const auto* sc = (const uint16_t*)scales;
  auto* Yh = (uint16_t*)Y;
  if (c.w_bit == 8) {
    // 8-bit codes: the vector GEMV (M <= 8), the skinny MFMA GEMV (M <= 64), the GEMMs
    if (kernel == AWQ_LINEAR_GEMM_WIDE)
      return hip_status(awq::launch_gemm_wide(Xh, M, qweight, sc, zeros, N, K, c.group_size, 8, Yh,
                                              gated, st));
    if (kernel == AWQ_LINEAR_GEMV)
      return hip_status(
          awq::launch_gemv8(Xh, M, qweight, sc, zeros, N, K, c.group_size, Yh, gated, st));
    if (kernel == AWQ_LINEAR_SKINNY)
      return hip_status(
          awq::launch_gemv_mfma8(Xh, M, qweight, sc, zeros, N, K, c.group_size, Yh, gated, st));
    return hip_status(
        awq::launch_gemm(Xh, M, qweight, sc, zeros, N, K, c.group_size, 8, Yh, gated, st));
  }
  if (c.w_bit == 3) {
    // 3-bit codes: the same kernels' 3-bit forms, with the same thresholds
    if (kernel == AWQ_LINEAR_GEMM_WIDE)
      return hip_status(awq::launch_gemm_wide(Xh, M, qweight, sc, zeros, N, K, c.group_size, 3, Yh,
                                              gated, st));
    if (kernel == AWQ_LINEAR_GEMV)
      return hip_status(
          awq::launch_gemv3(Xh, M, qweight, sc, zeros, N, K, c.group_size, Yh, gated, st));
    if (kernel == AWQ_LINEAR_SKINNY)
      return hip_status(
          awq::launch_gemv_mfma3(Xh, M, qweight, sc, zeros, N, K, c.group_size, Yh, gated, st));
    return hip_status(
        awq::launch_gemm(Xh, M, qweight, sc, zeros, N, K, c.group_size, 3, Yh, gated, st));
  }
  switch (kernel) {
    case AWQ_LINEAR_GEMM_WIDE:
      return hip_status(
          awq::launch_gemm_wide(Xh, M, qweight, sc, zeros, N, K, c.group_size, 4, Yh, gated, st));
    case AWQ_LINEAR_GEMV:
      return hip_status(
          awq::launch_gemv(Xh, M, qweight, sc, zeros, N, K, c.group_size, Yh, gated, st));
    case AWQ_LINEAR_SKINNY:
      return hip_status(
          awq::launch_gemv_mfma(Xh, M, qweight, sc, zeros, N, K, c.group_size, Yh, gated, st));
    default:
      return hip_status(
          awq::launch_gemm(Xh, M, qweight, sc, zeros, N, K, c.group_size, 4, Yh, gated, st));
  }
}

awq_status awq_linear_w4a16_ex(const void* X, int64_t M, const uint32_t* qweight,
                               const void* scales, const uint8_t* zeros, int64_t N, int64_t K,
                               const awq_config* cfg, void* Y, uint32_t* flags,
                               awq_linear_kernel kernel, void* stream) {
  return linear_common(X, M, qweight, scales, zeros, N, K, cfg, Y, flags, kernel, false, stream);
}

awq_status awq_linear_w4a16(const void* X, int64_t M, const uint32_t* qweight,
                            const void* scales, const uint8_t* zeros, int64_t N, int64_t K,
                            const awq_config* cfg, void* Y, uint32_t* flags, void* stream) {
  return awq_linear_w4a16_ex(X, M, qweight, scales, zeros, N, K, cfg, Y, flags, AWQ_LINEAR_AUTO,
                             stream);
}

awq_status awq_linear_w4a16_gated_silu_ex(const void* X, int64_t M, const uint32_t* qweight,
                                          const void* scales, const uint8_t* zeros, int64_t N,
                                          int64_t K, const awq_config* cfg, void* Y,
                                          uint32_t* flags, awq_linear_kernel kernel,
                                          void* stream) {
  return linear_common(X, M, qweight, scales, zeros, N, K, cfg, Y, flags, kernel, true, stream);
}

awq_status awq_linear_w4a16_gated_silu(const void* X, int64_t M, const uint32_t* qweight,
                                       const void* scales, const uint8_t* zeros, int64_t N,
                                       int64_t K, const awq_config* cfg, void* Y,
                                       uint32_t* flags, void* stream) {
  return awq_linear_w4a16_gated_silu_ex(X, M, qweight, scales, zeros, N, K, cfg, Y, flags,
                                        AWQ_LINEAR_AUTO, stream);
}

size_t awq_clip_search_workspace_size(int64_t T, int64_t N, int64_t K, int32_t n_shrink,
                                      const awq_config* cfg) {
  const awq_config c = resolve(cfg);
  if (!supported(c) || !good_nk(N, K) || n_shrink < 1) return 0;
  if (T < 1 || T > awq::kClipMaxTokens) return 0;
  return clip_layout(T, N, K, n_shrink, c.group_size).total;
}

awq_status awq_clip_search(const void* X, int64_t T, const void* W, int64_t N, int64_t K,
                           const void* s, int32_t clip_steps, int32_t n_shrink,
                           const awq_config* cfg, uint8_t* clip_idx, double* err,
                           void* workspace, size_t workspace_bytes, uint32_t* flags,
                           void* stream) {
  const awq_config c = resolve(cfg);
  if (!X || !W || !clip_idx) return AWQ_ERR_NULL_POINTER;
  if (!supported(c)) return AWQ_ERR_UNSUPPORTED;
  if (T < 1 || T > awq::kClipMaxTokens || !good_nk(N, K)) return AWQ_ERR_BAD_SHAPE;
  if (clip_steps < 1 || clip_steps > 65535 || n_shrink < 1 || n_shrink > clip_steps ||
      n_shrink > awq::kClipMaxShrink)
    return AWQ_ERR_BAD_SHAPE;
  if (!aligned16(X) || !aligned16(W) || (s && !aligned16(s)) || (err && !aligned16(err)) ||
      (flags && !aligned4(flags)))
    return AWQ_ERR_MISALIGNED;
  const ClipLayout L = clip_layout(T, N, K, n_shrink, c.group_size);
  if (!workspace || workspace_bytes < L.total || !aligned16(workspace)) return AWQ_ERR_WORKSPACE;
  char* ws = (char*)workspace;
  hipStream_t st = (hipStream_t)stream;
  void* errs = ws + L.err;
  hipError_t e = awq::launch_clip_err((const uint16_t*)X, T, (const uint16_t*)W, N, K,
                                      (const uint16_t*)s, clip_steps, n_shrink, c.zero_point == 0,
                                      c.group_size, c.w_bit, (uint4*)(ws + L.xp), errs, flags, st);
  if (e == hipSuccess)
    e = awq::launch_clip_reduce(errs, T, n_shrink, N, K, c.group_size, clip_idx, err, flags, st);
  return hip_status(e);
}

awq_status awq_apply_inverse_scale(const void* A, int64_t rows, int64_t cols, const void* s,
                                   int32_t axis, void* out, uint32_t* flags, void* stream) {
  if (!A || !s || !out) return AWQ_ERR_NULL_POINTER;
  if (axis != 0 && axis != 1) return AWQ_ERR_UNSUPPORTED;
  if (rows < 1 || cols < 8 || cols % 8 != 0 || rows >= kMaxDim || cols >= kMaxDim)
    return AWQ_ERR_BAD_SHAPE;
  if (!aligned16(A) || !aligned16(s) || !aligned16(out) || (flags && !aligned4(flags)))
    return AWQ_ERR_MISALIGNED;
  return hip_status(awq::launch_inverse_scale((const uint16_t*)A, rows, cols, (const uint16_t*)s,
                                              axis, (uint16_t*)out, flags, (hipStream_t)stream));
}

size_t awq_group_rows_workspace_size(int64_t n, int32_t groups) {
  if (n < 1 || n >= kMaxRows || !good_groups(groups)) return 0;
  return align256(awq::group_rows_workspace(n, groups));
}

awq_status awq_group_rows(const int32_t* ids, int64_t n, int32_t groups, int32_t* offsets,
                          int32_t* order, int32_t* pos, void* workspace, size_t workspace_bytes,
                          void* stream) {
  if (!ids || !offsets || !order) return AWQ_ERR_NULL_POINTER;
  if (n < 1 || n >= kMaxRows || !good_groups(groups)) return AWQ_ERR_BAD_SHAPE;
  if (!good_workspace(workspace, workspace_bytes, awq_group_rows_workspace_size(n, groups)))
    return AWQ_ERR_WORKSPACE;
  if (!aligned16(ids) || !aligned16(offsets) || !aligned16(order) || (pos && !aligned16(pos)))
    return AWQ_ERR_MISALIGNED;
  return hip_status(awq::launch_group_rows(ids, n, groups, offsets, order, pos, (int*)workspace,
                                           (hipStream_t)stream));
}

size_t awq_moe_route_workspace_size(int64_t T, int32_t E) {
  if (T < 1 || T >= kMaxRows || !good_groups(E)) return 0;
  return align256(awq::moe_route_workspace(T, E));
}

awq_status awq_moe_route(const void* logits, awq_logits_type type, int64_t T, int32_t E,
                         int64_t ld, int32_t top_k, int32_t renormalize, float* weights,
                         int32_t* ids, int32_t* offsets, int32_t* order, int32_t* pos,
                         void* workspace, size_t workspace_bytes, uint32_t* flags, void* stream) {
  int tv = 0;  // any integer may arrive: read it as one
  static_assert(sizeof(type) == sizeof(tv), "awq_logits_type is an int-sized enum");
  memcpy(&tv, &type, sizeof tv);
  if (!logits || !weights || !ids || !offsets || !order || !pos) return AWQ_ERR_NULL_POINTER;
  if ((tv != AWQ_LOGITS_FP16 && tv != AWQ_LOGITS_FP32) || (renormalize != 0 && renormalize != 1))
    return AWQ_ERR_UNSUPPORTED;
  if (T < 1 || !good_groups(E) || ld < E || ld >= kMaxDim || top_k < 1 || top_k > E ||
      top_k > AWQ_MAX_TOP_K || T >= kMaxRows / top_k)
    return AWQ_ERR_BAD_SHAPE;
  if (!good_workspace(workspace, workspace_bytes, awq_moe_route_workspace_size(T, E)))
    return AWQ_ERR_WORKSPACE;
  if (((uintptr_t)logits & (tv == AWQ_LOGITS_FP16 ? 1u : 3u)) != 0 || !aligned16(weights) ||
      !aligned16(ids) || !aligned16(offsets) || !aligned16(order) || !aligned16(pos) ||
      (flags && !aligned4(flags)))
    return AWQ_ERR_MISALIGNED;
  return hip_status(awq::launch_moe_route(logits, tv == AWQ_LOGITS_FP16, ld, T, E, top_k,
                                          renormalize != 0, weights, ids, offsets, order, pos,
                                          (int*)workspace, flags, (hipStream_t)stream));
}

static awq_status grouped_common(const void* X, int64_t x_rows, const int32_t* offsets,
                                 const int32_t* order, int64_t n_rows, int32_t fan, int32_t groups,
                                 const uint32_t* qweight, const void* scales, const uint8_t* zeros,
                                 int64_t N, int64_t K, const awq_config* cfg, void* Y, uint32_t* flags,
                                 awq_grouped_kernel kernel_arg, bool gated, void* stream) {
  int kv = 0;
  static_assert(sizeof(kernel_arg) == sizeof(kv), "awq_grouped_kernel is an int-sized enum");
  memcpy(&kv, &kernel_arg, sizeof kv);
  const awq_config c = resolve(cfg);
  if (!X || !offsets || !qweight || !scales || !zeros || !Y) return AWQ_ERR_NULL_POINTER;
  if (!supported(c) || kv < AWQ_GROUPED_AUTO || kv > AWQ_GROUPED_GEMM64K) return AWQ_ERR_UNSUPPORTED;
  if (n_rows < 1 || n_rows >= kMaxRows || x_rows < 1 || x_rows >= kMaxRows || !good_nk(N, K) ||
      !good_groups(groups) || (gated && N % 2 != 0))
    return AWQ_ERR_BAD_SHAPE;
  if (order ? fan < 1 || x_rows < (n_rows + fan - 1) / fan : x_rows < n_rows) return AWQ_ERR_BAD_SHAPE;
  if (x_rows > kMaxElements / K || !good_weight(N, K, c.w_bit) || !grouped_grid_ok(n_rows, N, groups, kv))
    return AWQ_ERR_BAD_SHAPE;
  if (kv == AWQ_GROUPED_SKINNY && n_rows > kSkinnyMaxRows) return AWQ_ERR_BAD_SHAPE;
  if (!aligned16(X) || !aligned16(offsets) || (order && !aligned16(order)) || !aligned16(qweight) ||
      !aligned16(scales) || !aligned16(zeros) || !aligned16(Y) || (flags && !aligned4(flags)))
    return AWQ_ERR_MISALIGNED;
  hipStream_t st = (hipStream_t)stream;
  if (flags) {
    // X in group order: rows behind the last group's are no input (a linear before this one leaves
    // them as they were); how many there are stands on the device
    const hipError_t e = awq::launch_nonfinite_scan((const uint16_t*)X, (order ? x_rows : n_rows) * K,
                                                    (const uint16_t*)scales, groups * N * (K / c.group_size),
                                                    flags, st, order ? nullptr : offsets + groups, K);
    if (e != hipSuccess) return AWQ_ERR_HIP;
  }
  awq::GroupedArgs g{};
  g.X = (const uint16_t*)X;
  g.offsets = offsets;
  g.order = order;
  g.qweight = qweight;
  g.scales = (const uint16_t*)scales;
  g.zeros = zeros;
  g.Y = (uint16_t*)Y;
  g.N = N;
  g.K = K;
  g.n = (int)n_rows;
  g.fan = fan;
  g.groups = groups;
  g.group = c.group_size;
  const int mode = gated ? awq::kGated : awq::kPlain;
  const bool streams = awq::grouped_stream_supported(groups, N, K, c.group_size, c.w_bit);
  if (kv == AWQ_GROUPED_AUTO)
    kv = streams && n_rows <= kSkinnyMaxRows && n_rows <= (int64_t)awq::skinny_mean_rows(c.w_bit) * groups
             ? AWQ_GROUPED_SKINNY
             : awq::choose_grouped_gemm(g, mode, c.w_bit);
  if (kv == AWQ_GROUPED_SKINNY && streams) return hip_status(awq::launch_grouped_stream(g, mode, c.w_bit, st));
  if (kv == AWQ_GROUPED_SKINNY) kv = AWQ_GROUPED_GEMM64;
  return hip_status(awq::launch_grouped_gemm(g, mode, c.w_bit, kv, st));
}

awq_status awq_linear_w4a16_grouped(const void* X, int64_t x_rows, const int32_t* offsets,
                                    const int32_t* order, int64_t n_rows, int32_t fan,
                                    int32_t groups, const uint32_t* qweight, const void* scales,
                                    const uint8_t* zeros, int64_t N, int64_t K,
                                    const awq_config* cfg, void* Y, uint32_t* flags,
                                    awq_grouped_kernel kernel, void* stream) {
  return grouped_common(X, x_rows, offsets, order, n_rows, fan, groups, qweight, scales, zeros, N, K,
                        cfg, Y, flags, kernel, false, stream);
}

awq_status awq_linear_w4a16_grouped_gated_silu(const void* X, int64_t x_rows,
                                               const int32_t* offsets, const int32_t* order,
                                               int64_t n_rows, int32_t fan, int32_t groups,
                                               const uint32_t* qweight, const void* scales,
                                               const uint8_t* zeros, int64_t N, int64_t K,
                                               const awq_config* cfg, void* Y, uint32_t* flags,
                                               awq_grouped_kernel kernel, void* stream) {
  return grouped_common(X, x_rows, offsets, order, n_rows, fan, groups, qweight, scales, zeros, N, K,
                        cfg, Y, flags, kernel, true, stream);
}

awq_status awq_moe_combine(const void* P, const float* weights, const int32_t* pos,
                           const int32_t* offsets, int32_t groups, int64_t T, int32_t top_k,
                           int64_t N, const void* add, void* Y, void* stream) {
  if (!P || !weights || !pos || !offsets || !Y) return AWQ_ERR_NULL_POINTER;
  // a launch has fewer than 2^32 threads, whole blocks of 128: of 8 values each, or of one
  const int64_t most = (((int64_t)1 << 32) - 128) * (N % 8 == 0 ? 8 : 1);
  if (!good_groups(groups) || T < 1 || top_k < 1 || top_k > AWQ_MAX_TOP_K || T >= kMaxRows / top_k ||
      N < 1 || N >= kMaxDim || T > most / N)
    return AWQ_ERR_BAD_SHAPE;
  if (!aligned16(P) || !aligned16(weights) || !aligned16(pos) || !aligned16(offsets) ||
      (add && !aligned16(add)) || !aligned16(Y))
    return AWQ_ERR_MISALIGNED;
  return hip_status(awq::launch_combine((const uint16_t*)P, weights, pos, offsets + groups, T, top_k, N,
                                        (const uint16_t*)add, (uint16_t*)Y, (hipStream_t)stream));
}

size_t awq_linear_w4a16_lora_workspace_size(int64_t M, int32_t rank) {
  if (M < 1 || M >= kMaxRows || !good_rank(rank)) return 0;
  return align256((size_t)M * ((rank + awq::kLoraBlock - 1) / awq::kLoraBlock) * sizeof(awq::LoraRow));
}

awq_status awq_linear_w4a16_lora(const void* X, int64_t M, const uint32_t* qweight,
                                 const void* scales, const uint8_t* zeros, int64_t N, int64_t K,
                                 const awq_config* cfg, const void* A, const void* B,
                                 const float* lora_scale, int32_t adapters, int32_t rank,
                                 const int32_t* ids, const int32_t* order, void* Y,
                                 void* workspace, size_t workspace_bytes, uint32_t* flags,
                                 awq_grouped_kernel kernel_arg, void* stream) {
  int kv = 0;
  memcpy(&kv, &kernel_arg, sizeof kv);
  const awq_config c = resolve(cfg);
  if (!X || !qweight || !scales || !zeros || !A || !B || !lora_scale || !ids || !Y)
    return AWQ_ERR_NULL_POINTER;
  if (!supported(c) || kv < AWQ_GROUPED_AUTO || kv > AWQ_GROUPED_GEMM64K) return AWQ_ERR_UNSUPPORTED;
  if (M < 1 || M >= kMaxRows || !good_nk(N, K) || !good_groups(adapters) || !good_rank(rank) ||
      M > kMaxElements / K || rank > kMaxElements / K || !good_weight(N, K, c.w_bit) ||
      !grouped_grid_ok(M, N, 1, kv))
    return AWQ_ERR_BAD_SHAPE;
  if (kv == AWQ_GROUPED_SKINNY && M > AWQ_LORA_SKINNY_MAX_M) return AWQ_ERR_BAD_SHAPE;
  if (!good_workspace(workspace, workspace_bytes, awq_linear_w4a16_lora_workspace_size(M, rank)))
    return AWQ_ERR_WORKSPACE;
  if (!aligned16(X) || !aligned16(qweight) || !aligned16(scales) || !aligned16(zeros) ||
      !aligned16(A) || !aligned16(B) || !aligned16(lora_scale) || !aligned16(ids) ||
      (order && !aligned16(order)) || !aligned16(Y) || (flags && !aligned4(flags)))
    return AWQ_ERR_MISALIGNED;
  hipStream_t st = (hipStream_t)stream;
  hipError_t e = hipSuccess;
  if (flags) {
    e = awq::launch_nonfinite_scan((const uint16_t*)X, M * K, (const uint16_t*)scales,
                                   N * (K / c.group_size), flags, st);
    if (e == hipSuccess)
      e = awq::launch_nonfinite_scan((const uint16_t*)A, (int64_t)adapters * rank * K, (const uint16_t*)B,
                                     (int64_t)adapters * rank * N, flags, st, nullptr, 0, lora_scale, adapters);
    if (e != hipSuccess) return AWQ_ERR_HIP;
  }
  e = awq::launch_lora_shrink((const uint16_t*)X, (int)M, K, (const uint16_t*)A, lora_scale, adapters,
                              rank, ids, order, (awq::LoraRow*)workspace, st);
  if (e != hipSuccess) return AWQ_ERR_HIP;
  awq::GroupedArgs g{};
  g.X = (const uint16_t*)X;
  g.order = order;
  g.qweight = qweight;
  g.scales = (const uint16_t*)scales;
  g.zeros = zeros;
  g.Y = (uint16_t*)Y;
  g.ids = ids;
  g.H = (const awq::LoraRow*)workspace;
  g.B = (const uint16_t*)B;
  g.N = N;
  g.K = K;
  g.n = (int)M;
  g.fan = 1;
  g.groups = adapters;
  g.group = c.group_size;
  g.rank = rank;
  const bool streams = awq::grouped_stream_supported(1, N, K, c.group_size, c.w_bit);
  if (kv == AWQ_GROUPED_AUTO)
    kv = streams && M <= awq::kLoraSkinnyRows ? AWQ_GROUPED_SKINNY : awq::choose_grouped_gemm(g, awq::kLora, c.w_bit);
  if (kv == AWQ_GROUPED_SKINNY && streams) return hip_status(awq::launch_grouped_stream(g, awq::kLora, c.w_bit, st));
  if (kv == AWQ_GROUPED_SKINNY) kv = AWQ_GROUPED_GEMM64;
  return hip_status(awq::launch_grouped_gemm(g, awq::kLora, c.w_bit, kv, st));
}

// ------------------------------------------------------------------ the 4-bit key / value cache

static awq_status kv_view(const awq_kv_cache* cache, const awq_kv_batch* batch, awq::KvView& v) {
  if (!cache || !batch || !cache->k_codes || !cache->k_params || !cache->v_codes || !cache->v_params ||
      !batch->rows || !batch->lengths || !batch->page_table)
    return AWQ_ERR_NULL_POINTER;
  if ((cache->head_dim != 64 && cache->head_dim != 128 && cache->head_dim != 256) ||
      (cache->group_size != 32 && cache->group_size != 64 && cache->group_size != 128) ||
      cache->group_size > cache->head_dim || cache->page_size < 16 || cache->page_size > 4096 ||
      (cache->page_size & (cache->page_size - 1)) != 0)
    return AWQ_ERR_UNSUPPORTED;
  if (cache->pages < 1 || cache->pages >= kMaxDim || cache->kv_heads < 1 || cache->kv_heads > AWQ_MAX_HEADS ||
      batch->n_rows < 1 || batch->n_rows >= kMaxKvRows || batch->seqs < 1 || batch->seqs > AWQ_MAX_SEQUENCES ||
      batch->max_pages < 1 || batch->max_pages >= kMaxRows / cache->page_size || batch->max_rows < 1 ||
      batch->max_rows > batch->n_rows)
    return AWQ_ERR_BAD_SHAPE;
  if (!aligned16(cache->k_codes) || !aligned16(cache->k_params) || !aligned16(cache->v_codes) ||
      !aligned16(cache->v_params) || !aligned16(batch->rows) || !aligned16(batch->lengths) ||
      !aligned16(batch->page_table))
    return AWQ_ERR_MISALIGNED;
  v = awq::KvView{};
  v.k_codes = (uint8_t*)cache->k_codes;
  v.v_codes = (uint8_t*)cache->v_codes;
  v.k_params = (uint16_t*)cache->k_params;
  v.v_params = (uint16_t*)cache->v_params;
  v.rows = batch->rows;
  v.lengths = batch->lengths;
  v.table = batch->page_table;
  v.pages = cache->pages;
  for (int p = cache->page_size; p > 1; p >>= 1) ++v.page_shift;
  v.heads = cache->kv_heads;
  v.dim = cache->head_dim;
  v.group = cache->group_size;
  v.seqs = batch->seqs;
  v.max_pages = batch->max_pages;
  v.n_rows = (int)batch->n_rows;
  return AWQ_OK;
}

// A launch has fewer than 2^32 threads: 8 channels each.
static bool kv_grid_ok(int64_t n_rows, int64_t heads, int dim) {
  return n_rows <= (((int64_t)1 << 26) - 4) / ((heads * dim + 511) / 512);
}

// Rows `ld` values apart hold `heads` heads: 16-byte pieces.
static bool good_ld(int64_t ld, int64_t heads, int dim) { return ld >= heads * dim && ld % 8 == 0 && ld < kMaxDim; }

awq_status awq_kv_append(const awq_kv_cache* cache, const awq_kv_batch* batch, const void* k, int64_t k_ld,
                         const void* v, int64_t v_ld, const void* q, int64_t q_ld, int32_t q_heads, void* q_out,
                         int64_t q_out_ld, const float* cos_sin, int64_t positions, int32_t rotary_dim,
                         int32_t interleaved, uint32_t* flags, void* stream) {
  awq::KvView c;
  if (!k || !v || (q != nullptr) != (q_out != nullptr) || (q && !cos_sin)) return AWQ_ERR_NULL_POINTER;
  const awq_status s = kv_view(cache, batch, c);
  if (s != AWQ_OK) return s;
  if (interleaved != 0 && interleaved != 1) return AWQ_ERR_UNSUPPORTED;
  if (!good_ld(k_ld, c.heads, c.dim) || !good_ld(v_ld, c.heads, c.dim)) return AWQ_ERR_BAD_SHAPE;
  if (q && (q_heads < 1 || q_heads > AWQ_MAX_HEADS || !good_ld(q_ld, q_heads, c.dim) ||
            !good_ld(q_out_ld, q_heads, c.dim)))
    return AWQ_ERR_BAD_SHAPE;
  if (!kv_grid_ok(c.n_rows, (q ? q_heads : 0) + 2 * (int64_t)c.heads, c.dim)) return AWQ_ERR_BAD_SHAPE;
  if (cos_sin && (positions < 1 || positions >= kMaxDim || rotary_dim < 16 || rotary_dim > c.dim || rotary_dim % 16 != 0))
    return AWQ_ERR_BAD_SHAPE;
  if (!aligned16(k) || !aligned16(v) || (q && (!aligned16(q) || !aligned16(q_out))) ||
      (cos_sin && !aligned16(cos_sin)) || (flags && !aligned4(flags)))
    return AWQ_ERR_MISALIGNED;
  return hip_status(awq::launch_kv_append(c, (const uint16_t*)q, q_ld, q ? q_heads : 0, (uint16_t*)q_out, q_out_ld,
                                          (const uint16_t*)k, k_ld, (const uint16_t*)v, v_ld, cos_sin, positions,
                                          cos_sin ? rotary_dim : 0, interleaved != 0, flags, (hipStream_t)stream));
}

awq_status awq_kv_read(const awq_kv_cache* cache, const awq_kv_batch* batch, void* k, void* v, void* stream) {
  awq::KvView c;
  if (!k || !v) return AWQ_ERR_NULL_POINTER;
  const awq_status s = kv_view(cache, batch, c);
  if (s != AWQ_OK) return s;
  if (!kv_grid_ok(c.n_rows, 2 * (int64_t)c.heads, c.dim)) return AWQ_ERR_BAD_SHAPE;
  if (!aligned16(k) || !aligned16(v)) return AWQ_ERR_MISALIGNED;
  return hip_status(awq::launch_kv_read(c, (uint16_t*)k, (uint16_t*)v, (hipStream_t)stream));
}

// Rows of 64 lanes and of blocks, and units of the work list, stay below 2^31.
static bool attend_sizes_ok(int64_t n_rows, int32_t seqs, int32_t max_rows, int64_t max_tokens, int32_t q_heads,
                            int32_t kv_heads, int32_t head_dim) {
  if (n_rows < 1 || n_rows >= kMaxKvRows || seqs < 1 || seqs > AWQ_MAX_SEQUENCES || max_rows < 1 ||
      max_rows > n_rows || max_tokens < 1 || max_tokens >= kMaxRows || kv_heads < 1 || q_heads < kv_heads ||
      q_heads > AWQ_MAX_HEADS || q_heads % kv_heads != 0 ||
      (head_dim != 64 && head_dim != 128 && head_dim != 256) || n_rows >= ((int64_t)1 << 24) / q_heads)
    return false;
  const int64_t tiles = n_rows * (q_heads / kv_heads) / 16 + seqs;
  return tiles * kv_heads < kMaxDim / (max_tokens / 256 + 1);
}

size_t awq_attention_kv4_workspace_size(int64_t n_rows, int32_t seqs, int32_t max_rows, int64_t max_tokens,
                                        int32_t q_heads, int32_t kv_heads, int32_t head_dim) {
  if (!attend_sizes_ok(n_rows, seqs, max_rows, max_tokens, q_heads, kv_heads, head_dim)) return 0;
  return awq::attend_plan(n_rows, seqs, max_rows, max_tokens, q_heads / kv_heads, kv_heads, head_dim, 32)
      .bytes;
}

awq_status awq_attention_kv4(const void* q, int64_t q_ld, int32_t q_heads, const awq_kv_cache* cache,
                             const awq_kv_batch* batch, float scale, int32_t causal, int64_t window, void* out,
                             int64_t out_ld, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  awq::KvView c;
  if (!q || !out) return AWQ_ERR_NULL_POINTER;
  const awq_status s = kv_view(cache, batch, c);
  if (s != AWQ_OK) return s;
  if ((causal != 0 && causal != 1) || !(scale > 0.0f && scale < 1e20f)) return AWQ_ERR_UNSUPPORTED;
  const int64_t max_tokens = (int64_t)batch->max_pages * cache->page_size;
  if (!attend_sizes_ok(batch->n_rows, batch->seqs, batch->max_rows, max_tokens, q_heads, c.heads, c.dim) ||
      !good_ld(q_ld, q_heads, c.dim) || !good_ld(out_ld, q_heads, c.dim) || window < 0)
    return AWQ_ERR_BAD_SHAPE;
  const awq::AttendPlan p = awq::attend_plan(batch->n_rows, batch->seqs, batch->max_rows, max_tokens,
                                             q_heads / c.heads, c.heads, c.dim, c.group);
  if (!good_workspace(workspace, workspace_bytes, p.bytes)) return AWQ_ERR_WORKSPACE;
  if (!aligned16(q) || !aligned16(out) || (lse && !aligned4(lse))) return AWQ_ERR_MISALIGNED;
  awq::AttendArgs a{};
  a.q = (const uint16_t*)q;
  a.out = (uint16_t*)out;
  a.lse = lse;
  a.q_ld = q_ld;
  a.out_ld = out_ld;
  a.q_heads = q_heads;
  a.share = q_heads / c.heads;
  a.scale_log2 = scale * 1.44269504088896341f;
  a.causal = causal;
  a.window = window >= kMaxRows ? 0 : (int)window;  // positions stay below
  return hip_status(awq::launch_attend(c, a, p, workspace, (hipStream_t)stream));
}

}  // extern "C"
