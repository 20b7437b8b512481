// C ABI of the norms around a block and of the adapters beside a projection (declared in include/fp8w8a8.h): argument
// validation, launches.

#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "api_common.h"
#include "device_cache.h"
#include "lora.h"
#include "moe_plan.h"
#include "norm.cuh"

namespace {

using namespace fp8k;

fp8_status check_row_vector(const void* p) { return aligned(p, 2) ? FP8_OK : FP8_ERR_MISALIGNED; }

// Whether all rows of bf16 start on boundaries of `bytes`.
bool rows_start_on(int bytes, const void* p, int64_t rows, int64_t ld) {
  return aligned(p, uintptr_t(bytes)) && (rows <= 1 || ld * 2 % bytes == 0);
}

PerDeviceCache<const void*, int> g_norm_ctas;

template <int kThreads, int kUnits, bool kPost, bool kGate, bool kVec>
fp8_status launch_norm_of(const norm::Params& p, int sms, cudaStream_t st) {
  auto kernel = norm::residual_norm_kernel<kThreads, kUnits, kPost, kGate, kVec>;
  int dev = 0, per_sm = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return FP8_ERR_CUDA;
  if (p.rows > sms &&  // (fewer: one CTA each)
      !g_norm_ctas.get(dev, reinterpret_cast<const void*>(kernel), &per_sm, [&](int* v) {
        return report_cuda(cudaOccupancyMaxActiveBlocksPerMultiprocessor(v, kernel, kThreads, 0), "norm occupancy") ==
                   cudaSuccess &&
               *v > 0;
      }))
    return FP8_ERR_CUDA;
  const int64_t grid = std::min<int64_t>(p.rows, int64_t(sms) * std::max(per_sm, 1));
  return launch(kernel, dim3(unsigned(grid)), dim3(kThreads), 0, st, true, dim3(1, 1, 1), p);
}
template <int kThreads, int kUnits, bool kVec>
fp8_status launch_norm(const norm::Params& p, int sms, cudaStream_t st) {
  if (p.post_w)
    return p.gate ? launch_norm_of<kThreads, kUnits, true, true, kVec>(p, sms, st)
                  : launch_norm_of<kThreads, kUnits, true, false, kVec>(p, sms, st);
  return p.gate ? launch_norm_of<kThreads, kUnits, false, true, kVec>(p, sms, st)
                : launch_norm_of<kThreads, kUnits, false, false, kVec>(p, sms, st);
}

// Threads of a row, as few as hold it at a unit each: two units a thread for rows of 8192 took 64 us against 56 (4096 rows with
// both norms, a gate and codes).
fp8_status launch_norm_any(const norm::Params& p, int sms, cudaStream_t st) {
  const int units = (p.cols + norm::kUnit - 1) / norm::kUnit;
  if (!p.vec) {
    if (units <= 32) return launch_norm<32, 1, false>(p, sms, st);
    if (units <= 128) return launch_norm<128, 1, false>(p, sms, st);
    if (units <= 256) return launch_norm<256, 1, false>(p, sms, st);
    if (units <= 512) return launch_norm<512, 1, false>(p, sms, st);
    if (units <= 1024) return launch_norm<1024, 1, false>(p, sms, st);
    return launch_norm<1024, 2, false>(p, sms, st);
  }
  if (units <= 32) return launch_norm<32, 1, true>(p, sms, st);
  if (units <= 64) return launch_norm<64, 1, true>(p, sms, st);
  if (units <= 128) return launch_norm<128, 1, true>(p, sms, st);
  if (units <= 256) return launch_norm<256, 1, true>(p, sms, st);
  if (units <= 512) return launch_norm<512, 1, true>(p, sms, st);
  if (units <= 1024) return launch_norm<1024, 1, true>(p, sms, st);
  return launch_norm<1024, 2, true>(p, sms, st);
}

// What both calls share, up to r.
fp8_status fill_norm(norm::Params& p, const void* y, int64_t M, int64_t H, int64_t ldy, const void* post_w,
                     const void* gate, int64_t ldg, float scale, const void* residual, int64_t ldr, const void* w,
                     float eps, int plus_one, void* r, int64_t ldro) {
  FP8_TRY(check_bf16_mat(y, M, H, ldy));
  if (H > norm::kMaxCols) return FP8_ERR_INVALID_ARG;
  if (!(eps > 0.0f) || !std::isfinite(eps) || !std::isfinite(scale)) return FP8_ERR_INVALID_ARG;
  if (plus_one != 0 && plus_one != 1) return FP8_ERR_INVALID_ARG;
  if (gate != nullptr && ldg != 0) FP8_TRY(check_bf16_mat(gate, M, H, ldg));
  if (residual != nullptr) FP8_TRY(check_bf16_mat(residual, M, H, ldr));
  if (r != nullptr) FP8_TRY(check_bf16_mat(r, M, H, ldro));
  if (crosses(r, ldro, y, ldy, M) || crosses(r, ldro, residual, ldr, M)) return FP8_ERR_INVALID_ARG;
  FP8_TRY(check_row_vector(post_w));
  FP8_TRY(check_row_vector(gate));
  FP8_TRY(check_row_vector(w));
  p.rows = M;
  p.cols = int(H);
  p.y = static_cast<const uint16_t*>(y);
  p.ldy = ldy;
  p.post_w = static_cast<const uint16_t*>(post_w);
  p.gate = static_cast<const uint16_t*>(gate);
  p.ldg = ldg;
  p.residual = static_cast<const uint16_t*>(residual);
  p.ldr = ldr;
  p.w = static_cast<const uint16_t*>(w);
  p.scale = scale;
  p.eps = eps;
  p.w_offset = plus_one ? 1.0f : 0.0f;
  p.inv_cols = H > 0 ? 1.0f / float(H) : 0.0f;
  p.r = static_cast<uint16_t*>(r);
  p.ldro = ldro;
  auto rows_on = [&](int bytes) {
    return H * 2 % bytes == 0 && rows_start_on(bytes, y, M, ldy) && rows_start_on(bytes, gate, M, ldg) &&
           rows_start_on(bytes, residual, M, ldr) && rows_start_on(bytes, r, M, ldro);
  };
  p.vec = rows_on(16) && aligned(post_w, 16) && aligned(w, 16);
  p.wide = p.vec && rows_on(32);
  return FP8_OK;
}

// ---- adapters ----

constexpr int kMaxAdapters = 511;                // one more class of the sort stands for none
constexpr int64_t kMaxLoraDim = int64_t(1) << 30;  // columns past a tile's last keep 32-bit indexes

bool lora_sizes_ok(int64_t M, int64_t K, int64_t N, int64_t L, int64_t r) {
  return M >= 0 && M <= kMaxDim - block::kRowTile && K >= 0 && K <= kMaxLoraDim && N >= 0 && N <= kMaxLoraDim && L >= 0 &&
         L <= kMaxAdapters && r >= 1 && r <= lora::kMaxRank;
}

// A cluster a token, or rows sorted by adapter: by the estimated time in us. A token takes 0.06 and its adapter's w MB at
// 8.5 MB/us; the sorted form 16 and its adapters (between one and min(L, M): half) at 2.2. Measured, by token and sorted
// (tokens of 32 adapters drawn at random; of one): K 4096 N 4096 r 64, 64 tokens 10 and 25; 17, 128 tokens 18 and 27; 18, 256
// tokens 33 and 27; 19. r 16: 128 tokens 9 and 29; 17, 256 tokens 17 and 29; 17. N 14336 r 64: 64 tokens 22 and 44; 18, 128
// tokens 38 and 46; 19. K 8192 N 8192 r 128: 64 tokens 35 and 54; 27, 128 tokens 65 and 60; 27. Rows that start off 16-byte
// boundaries take both longer: K 4098 N 4096 r 64: 64 tokens 22 and 28; 20, K 6014 N 1280 r 105: 64 tokens 36 and 35; 33.
// (By sizes alone, since they decide on the workspace, which is asked for before there is an address: views of whole rows
// that start off a boundary go by the rule of those on one.)
bool lora_by_token(int64_t M, int64_t K, int64_t N, int64_t L, int64_t r) {
  const double w = 2e-6 * double(r) * double(K + N);
  const double sorted = 16.0 + double(std::min(L, M)) * w / 4.4;
  if (K % 8 != 0 || r % 8 != 0) return M <= 512 && double(M) * (0.058 + w / 3.3) <= 1.4 * sorted;
  return M <= 512 && double(M) * (0.058 + w / 8.5) <= sorted;
}

struct LoraWs {
  size_t n_tiles, tiles, counts, pos, order, v, total;
  int64_t max_tiles;
  int splits;
};
LoraWs lora_ws(int64_t M, int64_t K, int64_t N, int64_t L, int64_t r) {
  Carver c;
  LoraWs w = {};
  if (lora_by_token(M, K, N, L, r)) return w;
  w.max_tiles = M / block::kRowTile + std::min(L + 1, M);
  w.splits = lora::splits_of(M, K, L, r);
  w.n_tiles = c.take(4);
  w.tiles = c.take(size_t(w.max_tiles) * sizeof(block::RowTile));
  w.counts = c.take(moe::plan_counts_bytes(M, L + 1));
  w.pos = c.take(size_t(M) * 4);
  w.order = c.take(size_t(M) * 4);
  w.v = c.take(size_t(w.splits) * size_t(M) * size_t(lora::padded_rank(r)) * 4);
  w.total = c.at;
  return w;
}

}  // namespace

FP8_API fp8_status fp8_residual_norm(const void* y_bf16, int64_t M, int64_t H, int64_t ldy, const void* post_w_bf16,
                                     const void* gate_bf16, int64_t ldg, float scale, const void* residual_bf16,
                                     int64_t ldr, const void* w_bf16, float eps, int plus_one, void* r_bf16,
                                     int64_t ldro, void* n_bf16, int64_t ldn, fp8_stream_t stream) {
  norm::Params p = {};
  FP8_TRY(fill_norm(p, y_bf16, M, H, ldy, post_w_bf16, gate_bf16, ldg, scale, residual_bf16, ldr, w_bf16, eps,
                    plus_one, r_bf16, ldro));
  if (n_bf16 != nullptr) FP8_TRY(check_bf16_mat(n_bf16, M, H, ldn));
  if (crosses(n_bf16, ldn, y_bf16, ldy, M) || crosses(n_bf16, ldn, residual_bf16, ldr, M)) return FP8_ERR_INVALID_ARG;
  if (M == 0 || H == 0) return FP8_OK;
  if ((w_bf16 == nullptr) != (n_bf16 == nullptr)) return FP8_ERR_INVALID_ARG;
  if (n_bf16 == r_bf16) return FP8_ERR_INVALID_ARG;  // nothing to write, or one over the other
  p.pre = n_bf16 != nullptr;
  p.n = static_cast<uint16_t*>(n_bf16);
  p.ldn = ldn;
  p.vec = p.vec && rows_start_on(16, n_bf16, M, ldn);
  p.wide = p.wide && rows_start_on(32, n_bf16, M, ldn);
  int sms = 0;
  FP8_TRY(current_device(&sms));
  return launch_norm_any(p, sms, reinterpret_cast<cudaStream_t>(stream));
}

FP8_API fp8_status fp8_residual_norm_quantize(const void* y_bf16, int64_t M, int64_t H, int64_t ldy,
                                              const void* post_w_bf16, const void* gate_bf16, int64_t ldg,
                                              float scale, const void* residual_bf16, int64_t ldr,
                                              const void* w_bf16, float eps, int plus_one, void* r_bf16,
                                              int64_t ldro, uint8_t* qn, int64_t ldq, float* s_n, int64_t lds,
                                              fp8_stream_t stream) {
  norm::Params p = {};
  FP8_TRY(fill_norm(p, y_bf16, M, H, ldy, post_w_bf16, gate_bf16, ldg, scale, residual_bf16, ldr, w_bf16, eps,
                    plus_one, r_bf16, ldro));
  FP8_TRY(check_fp8_mat(qn, M, H, ldq));
  FP8_TRY(check_row_scales(s_n, M, H, lds));
  if (M == 0) return FP8_OK;
  if (H > 0 && w_bf16 == nullptr) return FP8_ERR_INVALID_ARG;
  p.pre = 1;
  p.q = qn;
  p.ldq = ldq;
  p.s = s_n;
  p.lds = lds;
  int sms = 0;
  FP8_TRY(current_device(&sms));
  return launch_norm_any(p, sms, reinterpret_cast<cudaStream_t>(stream));
}

FP8_API size_t fp8_lora_workspace_bytes(int64_t M, int64_t K, int64_t N, int64_t L, int64_t r) {
  if (!lora_sizes_ok(M, K, N, L, r) || M == 0 || K == 0 || N == 0 || L == 0) return 0;
  return lora_ws(M, K, N, L, r).total;
}

static fp8_status lora_call(const void* y_bf16, int64_t M, int64_t N, int64_t ldy, const void* x_bf16, int64_t K,
                            int64_t ldx, const void* a_bf16, const void* b_bf16, int64_t L, int64_t r, const int32_t* ids,
                            const float* scales, void* out_bf16, int64_t ldo, void* ws, size_t ws_bytes,
                            fp8_stream_t stream, lora::Withhold withhold) {
  if (!lora_sizes_ok(M, K, N, L, r)) return FP8_ERR_INVALID_ARG;
  FP8_TRY(check_bf16_mat(y_bf16, M, N, ldy));
  FP8_TRY(check_bf16_mat(x_bf16, M, K, ldx));
  FP8_TRY(check_bf16_mat(out_bf16, M, N, ldo));
  if (!aligned(a_bf16, 2) || !aligned(b_bf16, 2) || !aligned(ids, 4) || !aligned(scales, 4)) return FP8_ERR_MISALIGNED;
  if (M == 0 || N == 0) return FP8_OK;
  if (crosses(out_bf16, ldo, y_bf16, ldy, M)) return FP8_ERR_INVALID_ARG;
  const bool none = K == 0 || L == 0;
  if (!none && out_bf16 == x_bf16) return FP8_ERR_INVALID_ARG;
  if (!none && (a_bf16 == nullptr || b_bf16 == nullptr || ids == nullptr)) return FP8_ERR_INVALID_ARG;
  FP8_TRY(check_ws(ws, ws_bytes, fp8_lora_workspace_bytes(M, K, N, L, r)));
  int sms = 0;
  FP8_TRY(current_device(&sms));
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (none) {  // every product is empty
    if (out_bf16 == y_bf16) return FP8_OK;
    return report_cuda(cudaMemcpy2DAsync(out_bf16, size_t(ldo) * 2, y_bf16, size_t(ldy) * 2, size_t(N) * 2, size_t(M),
                                         cudaMemcpyDeviceToDevice, st),
                       "lora copy") == cudaSuccess
               ? FP8_OK
               : FP8_ERR_CUDA;
  }
  lora::Args p = {};
  p.y = static_cast<const uint16_t*>(y_bf16);
  p.M = M;
  p.N = N;
  p.ldy = ldy;
  p.x = static_cast<const uint16_t*>(x_bf16);
  p.K = K;
  p.ldx = ldx;
  p.a = static_cast<const uint16_t*>(a_bf16);
  p.b = static_cast<const uint16_t*>(b_bf16);
  p.adapters = int(L);
  p.rank = int(r);
  p.ids = ids;
  p.scales = scales;
  p.out = static_cast<uint16_t*>(out_bf16);
  p.ldo = ldo;
  if (lora_by_token(M, K, N, L, r)) return lora::launch_tokens(p, sms, st) ? FP8_OK : FP8_ERR_CUDA;
  const LoraWs w = lora_ws(M, K, N, L, r);
  uint8_t* base = static_cast<uint8_t*>(ws);
  lora::Sorted s = {};
  block::RowTile* tiles = reinterpret_cast<block::RowTile*>(base + w.tiles);
  int* n_tiles = reinterpret_cast<int*>(base + w.n_tiles);
  int* order = reinterpret_cast<int*>(base + w.order);
  // rows sorted by adapter, those without one last, as adapter L
  FP8_TRY(moe::launch_plan({ids, M, int(L) + 1, int(L), reinterpret_cast<int*>(base + w.counts),
                            reinterpret_cast<int*>(base + w.pos), order, tiles, n_tiles, nullptr},
                           st));
  s.tiles = tiles;
  s.n_tiles = n_tiles;
  s.max_tiles = w.max_tiles;
  s.order = order;
  s.v = reinterpret_cast<float*>(base + w.v);
  s.splits = w.splits;
  return lora::launch_sorted(p, s, sms, st, withhold) ? FP8_OK : FP8_ERR_CUDA;
}

FP8_API fp8_status fp8_lora_add(const void* y_bf16, int64_t M, int64_t N, int64_t ldy, const void* x_bf16, int64_t K,
                                int64_t ldx, const void* a_bf16, const void* b_bf16, int64_t L, int64_t r,
                                const int32_t* ids, const float* scales, void* out_bf16, int64_t ldo, void* ws,
                                size_t ws_bytes, fp8_stream_t stream) {
  return lora_call(y_bf16, M, N, ldy, x_bf16, K, ldx, a_bf16, b_bf16, L, r, ids, scales, out_bf16, ldo, ws, ws_bytes, stream,
                   lora::Withhold::kNone);
}

FP8_API fp8_status fp8_lora_selftest_timeout(int form, const void* y_bf16, int64_t M, int64_t N, int64_t ldy,
                                             const void* x_bf16, int64_t K, int64_t ldx, const void* a_bf16,
                                             const void* b_bf16, int64_t L, int64_t r, const int32_t* ids,
                                             const float* scales, void* out_bf16, int64_t ldo, void* ws, size_t ws_bytes,
                                             fp8_stream_t stream) {
  if (form < 0 || form > 2 || !lora_sizes_ok(M, K, N, L, r) || M < 1 || K < 1 || N < 1 || L < 1) return FP8_ERR_INVALID_ARG;
  if (lora_by_token(M, K, N, L, r)) return FP8_ERR_INVALID_ARG;  // a token at a time has nothing to wait for
  if (form == 0 && (K % 8 != 0 || ldx % 8 != 0 || !aligned(x_bf16, 16) || !aligned(a_bf16, 16))) return FP8_ERR_INVALID_ARG;
  if (form == 1 && (r > 64 || r % 8 != 0 || N % 8 != 0 || ldy % 8 != 0 || ldo % 8 != 0 || !aligned(b_bf16, 16) ||
                    !aligned(y_bf16, 16) || !aligned(out_bf16, 16)))
    return FP8_ERR_INVALID_ARG;
  if (form == 2 && r > 192) return FP8_ERR_INVALID_ARG;
  return lora_call(y_bf16, M, N, ldy, x_bf16, K, ldx, a_bf16, b_bf16, L, r, ids, scales, out_bf16, ldo, ws, ws_bytes, stream,
                   lora::Withhold(form));
}
