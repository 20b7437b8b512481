// C ABI of the block-scaled FP8 linear and the mixture of experts (declared in
// include/fp8w8a8.h): argument validation, workspace layout, launches.

#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "api_common.h"
#include "block_gemm.h"
#include "block_gemv.h"
#include "block_quant.cuh"
#include "device_cache.h"
#include "moe.cuh"

namespace {

using namespace fp8k;
using block::blocks_of;

// Largest row count: a row tile may reach kRowTile past the last row with 32-bit coordinates.
constexpr int64_t kMaxRows = kMaxDim - block::kRowTile;

int elementwise_grid(int64_t items, int per_cta, int sms, int ctas_per_sm) {
  const int64_t g = (items + per_cta - 1) / per_cta;
  return int(std::max<int64_t>(1, std::min<int64_t>(g, int64_t(sms) * ctas_per_sm)));
}

// A -> codes and scales; pos / copies: see the kernel.
fp8_status launch_quantize_rows(const BF16Mat& a, uint8_t* q, int64_t ldq, float* s, int64_t lds, const int* pos,
                                int copies, int sms, cudaStream_t st) {
  const int64_t units = a.rows * blocks_of(ldq) * 8;
  const int grid = elementwise_grid(units, block::kQThreads, sms, 8);
  auto go = [&](auto kernel) {
    return launch(kernel, dim3(grid), dim3(block::kQThreads), 0, st, true, dim3(1, 1, 1), a.p, a.rows, a.cols, a.ld,
                  a.vec(), q, ldq, s, lds, pos, copies);
  };
  // the loop index passes `units` by up to a grid stride
  return units < (int64_t(1) << 31) ? go(block::quantize_rows_1x128_kernel<uint32_t>)
                                    : go(block::quantize_rows_1x128_kernel<uint64_t>);
}

// Scales of rows: fp32 [K blocks][lds], lds >= rows.
fp8_status check_row_scales(const float* s, int64_t rows, int64_t K, int64_t lds) {
  if (lds < std::max<int64_t>(rows, 1)) return FP8_ERR_INVALID_ARG;
  if (rows > 0 && K > 0 && s == nullptr) return FP8_ERR_INVALID_ARG;
  return aligned(s, 4) ? FP8_OK : FP8_ERR_MISALIGNED;
}

struct Carver {
  size_t at = 0;
  size_t take(size_t bytes) {
    const size_t p = at;
    at = round_up_256(at + bytes);
    return p;
  }
};

// Whether the GEMV takes a dense product. Its CTAs each bring in their K slices of A, so its time grows
// with M * K and the GEMM's does not (both stream the weights, so N decides nothing). Graphs over weights
// that together pass L2, in us, GEMV and GEMM: K 4096 N 6144 M 8 11.0 and 13.0, M 12 14.5 and 13.0; K 4096
// N 28672 M 8 24.3 and 26.6, M 12 29.1 and 26.6; K 2048 N 14336 M 12 12.4 and 12.7, M 16 13.2 and 12.7; K
// 14336 N 4096 M 4 17.3 and 20.6, M 8 24.1 and 19.8; K 1000 N 1027 M 16 6.0 and 9.7. Of 64 shapes with K
// from 1024 to 14336, N from 4096 to 28672 and up to 16 rows, the side not taken is 5 percent or more faster in
// four: K 8192 N 8192 M 6 (GEMV 18.2, GEMM 21.1) and M 8 (19.3, 21.1), K 8192 N 28672 M 6 (43.1, 45.3), K 1024
// N 28672 M 16 (13.4, 11.6).
bool uses_gemv(int64_t M, int64_t K) {
  return block::gemv_fits(M, K, 1) && (M <= 4 || M * K <= 40 * 1024);
}
// One kernel quantizes A and streams the weights.
bool linear_fused(int64_t M, int64_t K) { return uses_gemv(M, K) && block::gemv_quantizes(M, K); }

// Workspace of fp8_block_linear: codes of A, then its scales; none when one kernel does both.
struct LinearWs {
  size_t qa, s_a, total;
  int64_t lds;  // M rounded up to 4: the GEMM copies whole 16-byte pieces of a block's scales
};
LinearWs linear_ws(int64_t M, int64_t K) {
  Carver c;
  LinearWs w = {};
  if (linear_fused(M, K)) return w;
  const int64_t rows = uses_gemv(M, K) ? M : block::gemm_held_rows(M, round_up16(K));
  w.qa = c.take(size_t(rows) * size_t(round_up16(K)));
  w.lds = (M + 3) / 4 * 4;
  w.s_a = c.take(size_t(blocks_of(K)) * size_t(w.lds) * 4);
  w.total = c.at;
  return w;
}

fp8_status block_mm(const uint8_t* qa, int64_t M, int64_t K, int64_t ldqa, const float* s_a, int64_t lds_a,
                    const uint8_t* qw, int64_t N, int64_t ldqw, const float* s_w, const void* bias, void* y,
                    int64_t ldy, int64_t held_rows, int sms, cudaStream_t st) {
  if (uses_gemv(M, K)) {
    block::GemvArgs v = {};
    v.src = block::kSrcCodes;
    v.a = qa;
    v.lda = ldqa;
    v.s_a = s_a;
    v.lds_a = lds_a;
    v.M = M;
    v.qw = qw;
    v.ldw = ldqw;
    v.s_w = s_w;
    v.N = N;
    v.K = K;
    v.bias = static_cast<const uint16_t*>(bias);
    v.y = static_cast<uint16_t*>(y);
    v.ldy = ldy;
    return block::gemv_launch(v, block::kGemvBf16, sms, st) ? FP8_OK : FP8_ERR_CUDA;
  }
  block::GemmArgs g = {};
  g.qa = qa;
  g.rows = M;
  g.held_rows = held_rows;
  g.lda = ldqa;
  g.s_a = s_a;
  g.lds_a = lds_a;
  g.qw = qw;
  g.mats = 1;
  g.ldw = ldqw;
  g.s_w = s_w;
  g.N = N;
  g.K = K;
  g.bias = static_cast<const uint16_t*>(bias);
  g.y = static_cast<uint16_t*>(y);
  g.ldy = ldy;
  return block::gemm_launch(g, block::kOutBf16, sms, st) ? FP8_OK : FP8_ERR_CUDA;
}

// y[m, :] = bias (or 0): the product over no K.
__global__ void rows_of_bias_kernel(const uint16_t* __restrict__ bias, uint16_t* __restrict__ y, int64_t M, int64_t N,
                                    int64_t ldy) {
  pdl_trigger();
  pdl_wait();
  for (int64_t i = int64_t(blockIdx.x) * blockDim.x + threadIdx.x; i < M * N; i += int64_t(gridDim.x) * blockDim.x) {
    const int64_t m = i / N, n = i - m * N;
    y[m * ldy + n] = bias ? bias[n] : uint16_t(0);
  }
}

fp8_status launch_rows_of_bias(const void* bias, void* y, int64_t M, int64_t N, int64_t ldy, int sms,
                               cudaStream_t st) {
  return launch(rows_of_bias_kernel, dim3(elementwise_grid(M * N, 256, sms, 8)), dim3(256), 0, st, true,
                dim3(1, 1, 1), static_cast<const uint16_t*>(bias), static_cast<uint16_t*>(y), M, N, ldy);
}

fp8_status check_product(int64_t M, int64_t K, const uint8_t* qw, int64_t N, int64_t ldqw, const float* s_w,
                         const void* bias, const void* y, int64_t ldy) {
  FP8_TRY(check_fp8_mat(qw, N, K, ldqw));
  FP8_TRY(check_bf16_mat(y, M, N, ldy));
  if (M > kMaxRows) return FP8_ERR_INVALID_ARG;
  if (N > 0 && K > 0 && s_w == nullptr) return FP8_ERR_INVALID_ARG;
  if (!aligned(bias, 2) || !aligned(s_w, 4)) return FP8_ERR_MISALIGNED;
  return FP8_OK;
}

// How the experts run. One token: a GEMV over its pairs for h, one over all of their h for y (two
// launches). More: sort the pairs, quantize, two tensor-core products, weighted sum (five). Experts of
// 2048 x 1408, 8 of 64 a token: one token 29 us (36 as sorted pairs), 16 tokens 97 us (104 as GEMVs
// over sorted pairs, which are not kept).
bool one_token(int64_t T, int64_t k, int64_t H, int64_t I) {
  return T == 1 && block::gemv_fits(1, H, 2) && block::gemv_fits(1, k * blocks_of(I) * block::kBlock, 1);
}

// CTAs that sort the pairs; more than one need their counts first (the whole layer, experts of 2048 x
// 1408, in us: 4096 pairs 131.7, by one CTA 134.5; 8192 pairs 161.1 and 170.8).
int plan_ctas(int64_t pairs) {
  if (pairs <= 2 * moe::kPlanPairs) return 1;  // a second launch costs more than it saves
  return int(std::min<int64_t>(moe::kPlanMaxCtas, (pairs + moe::kPlanPairs - 1) / moe::kPlanPairs));
}

struct MoeWs {
  size_t n_tiles, tiles, counts, pos, qx, s_x, h, s_h, y, total;
  int64_t pairs, max_tiles, ldx, ldh, ldy, lds;
};
MoeWs moe_ws(int64_t T, int64_t k, int64_t E, int64_t H, int64_t I) {
  Carver c;
  MoeWs w = {};
  w.pairs = T * k;
  w.ldh = round_up16(I);
  const size_t pairs = size_t(w.pairs);
  if (one_token(T, k, H, I)) {
    w.h = c.take(pairs * size_t(w.ldh) * 4);  // fp32; the second GEMV quantizes it
  } else {
    w.max_tiles = w.pairs / block::kRowTile + std::min(E, w.pairs);
    w.ldx = round_up16(H);
    w.ldy = (H + 7) / 8 * 8;
    w.lds = (w.pairs + 3) / 4 * 4;
    w.n_tiles = c.take(4);
    w.tiles = c.take(size_t(w.max_tiles) * sizeof(block::RowTile));
    w.counts = c.take(plan_ctas(w.pairs) > 1 ? size_t(plan_ctas(w.pairs)) * size_t(E) * 4 : 0);
    w.pos = c.take(pairs * 4);
    w.y = c.take(pairs * size_t(w.ldy) * 4);
    w.qx = c.take(size_t(block::gemm_held_rows(w.pairs, w.ldx)) * size_t(w.ldx));
    w.s_x = c.take(size_t(w.lds) * size_t(blocks_of(H)) * 4);
    w.h = c.take(size_t(block::gemm_held_rows(w.pairs, w.ldh)) * size_t(w.ldh));
    w.s_h = c.take(size_t(w.lds) * size_t(blocks_of(I)) * 4);
  }
  w.total = c.at;
  return w;
}

// (the last: sizes of the workspace stay far below 2^64)
bool moe_sizes_ok(int64_t T, int64_t k, int64_t E, int64_t H, int64_t I) {
  return T >= 0 && k >= 1 && k <= moe::kMaxChosen && E >= 1 && E <= moe::kMaxExperts && H >= 0 && H <= kMaxDim &&
         I >= 1 && I <= kMaxDim / 2 && T <= kMaxRows / k && T * k <= (int64_t(1) << 56) / (H + I);
}

PerDeviceCache<const void*, int> g_attr_cache;

fp8_status launch_plan(const int32_t* ids, int64_t pairs, int E, int* counts, int* pos, block::RowTile* tiles,
                       int* n_tiles, cudaStream_t st) {
  const size_t smem = size_t(moe::kPlanWarps + 1) * E * sizeof(int);
  int dev = 0, set = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return FP8_ERR_CUDA;
  if (!g_attr_cache.get(dev, reinterpret_cast<const void*>(moe::plan_kernel), &set, [&](int* v) {
        *v = 1;
        return report_cuda(cudaFuncSetAttribute(moe::plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                (moe::kPlanWarps + 1) * moe::kMaxExperts * int(sizeof(int))),
                           "plan smem attribute") == cudaSuccess;
      }))
    return FP8_ERR_CUDA;
  const int ctas = plan_ctas(pairs);
  if (ctas > 1)
    FP8_TRY(launch(moe::plan_count_kernel, dim3(ctas), dim3(moe::kPlanThreads), 0, st, true, dim3(1, 1, 1), ids, pairs,
                   E, counts));
  return launch(moe::plan_kernel, dim3(ctas), dim3(moe::kPlanThreads), smem, st, true, dim3(1, 1, 1), ids, pairs, E,
                ctas > 1 ? static_cast<const int*>(counts) : nullptr, pos, tiles, n_tiles);
}

template <typename T>
fp8_status launch_route(const T* logits, const moe::RouteParams& p, int sms, cudaStream_t st) {
  auto go = [&](auto kernel) {
    const int grid = int((p.tokens + moe::kRouteThreads / 32 - 1) / (moe::kRouteThreads / 32));
    return launch(kernel, dim3(grid), dim3(moe::kRouteThreads), 0, st, true, dim3(1, 1, 1), logits, p);
  };
  if (p.experts <= 32) return go(moe::route_kernel<T, 1>);
  if (p.experts <= 64) return go(moe::route_kernel<T, 2>);
  if (p.experts <= 128) return go(moe::route_kernel<T, 4>);
  if (p.experts <= 256) return go(moe::route_kernel<T, 8>);
  return go(moe::route_kernel<T, 16>);
}

}  // namespace

// ---------------------------------------------------------------------------
// block-scaled linear
// ---------------------------------------------------------------------------

FP8_API fp8_status fp8_block_quantize_weight(const void* w_bf16, int64_t B, int64_t N, int64_t K, int64_t ldw,
                                             int64_t mat_stride, uint8_t* qw, int64_t ldq, float* s_w,
                                             fp8_stream_t stream) {
  FP8_TRY(check_bf16_mat(w_bf16, N, K, ldw));
  FP8_TRY(check_fp8_mat(qw, N, K, ldq));
  if (B < 0 || B > kMaxDim || (B > 1 && mat_stride < 0)) return FP8_ERR_INVALID_ARG;
  if (!aligned(s_w, 4)) return FP8_ERR_MISALIGNED;
  if (B == 0 || N == 0) return FP8_OK;
  if (K > 0 && s_w == nullptr) return FP8_ERR_INVALID_ARG;
  int sms = 0;
  FP8_TRY(current_device(&sms));
  const BF16Mat W{static_cast<const uint16_t*>(w_bf16), N, K, ldw};
  const int vec = W.vec() && (B == 1 || mat_stride % 8 == 0);
  const int64_t blocks = B * blocks_of(N) * blocks_of(ldq);
  // no early programmatic trigger: a following product may read qW before its own wait
  return launch(block::quantize_128x128_kernel, dim3(elementwise_grid(blocks, 1, sms, 64)), dim3(block::kQThreads), 0,
                reinterpret_cast<cudaStream_t>(stream), false, dim3(1, 1, 1), W.p, B, N, K, ldw, mat_stride, vec, qw,
                ldq, s_w);
}

FP8_API fp8_status fp8_block_quantize_act(const void* a_bf16, int64_t M, int64_t K, int64_t lda, uint8_t* qa,
                                          int64_t ldq, float* s_a, int64_t lds, fp8_stream_t stream) {
  FP8_TRY(check_bf16_mat(a_bf16, M, K, lda));
  FP8_TRY(check_fp8_mat(qa, M, K, ldq));
  FP8_TRY(check_row_scales(s_a, M, K, lds));
  if (M == 0) return FP8_OK;
  int sms = 0;
  FP8_TRY(current_device(&sms));
  const BF16Mat A{static_cast<const uint16_t*>(a_bf16), M, K, lda};
  return launch_quantize_rows(A, qa, ldq, s_a, lds, nullptr, 0, sms, reinterpret_cast<cudaStream_t>(stream));
}

FP8_API fp8_status fp8_block_scaled_mm(const uint8_t* qa, int64_t M, int64_t K, int64_t ldqa, const float* s_a,
                                       int64_t lds, const uint8_t* qw, int64_t N, int64_t ldqw, const float* s_w,
                                       const void* bias_bf16, void* y_bf16, int64_t ldy, fp8_stream_t stream) {
  FP8_TRY(check_fp8_mat(qa, M, K, ldqa));
  FP8_TRY(check_row_scales(s_a, M, K, lds));
  FP8_TRY(check_product(M, K, qw, N, ldqw, s_w, bias_bf16, y_bf16, ldy));
  if (M == 0 || N == 0) return FP8_OK;
  int sms = 0;
  FP8_TRY(current_device(&sms));
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (K == 0) return launch_rows_of_bias(bias_bf16, y_bf16, M, N, ldy, sms, st);
  return block_mm(qa, M, K, ldqa, s_a, lds, qw, N, ldqw, s_w, bias_bf16, y_bf16, ldy, M, sms, st);
}

FP8_API size_t fp8_block_workspace_bytes(int64_t M, int64_t K, int64_t N) {
  if (M <= 0 || K <= 0 || N <= 0) return 0;
  return linear_ws(M, K).total;
}

FP8_API fp8_status fp8_block_linear(const void* a_bf16, int64_t M, int64_t K, int64_t lda, const uint8_t* qw,
                                    int64_t N, int64_t ldqw, const float* s_w, const void* bias_bf16, void* y_bf16,
                                    int64_t ldy, void* ws, size_t ws_bytes, fp8_stream_t stream) {
  FP8_TRY(check_bf16_mat(a_bf16, M, K, lda));
  FP8_TRY(check_product(M, K, qw, N, ldqw, s_w, bias_bf16, y_bf16, ldy));
  if (M == 0 || N == 0) return FP8_OK;
  FP8_TRY(check_ws(ws, ws_bytes, fp8_block_workspace_bytes(M, K, N)));
  int sms = 0;
  FP8_TRY(current_device(&sms));
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (K == 0) return launch_rows_of_bias(bias_bf16, y_bf16, M, N, ldy, sms, st);
  const BF16Mat A{static_cast<const uint16_t*>(a_bf16), M, K, lda};
  if (linear_fused(M, K)) {
    block::GemvArgs v = {};
    v.src = block::kSrcBf16;
    v.a = A.p;
    v.lda = lda;
    v.M = M;
    v.qw = qw;
    v.ldw = ldqw;
    v.s_w = s_w;
    v.N = N;
    v.K = K;
    v.bias = static_cast<const uint16_t*>(bias_bf16);
    v.y = static_cast<uint16_t*>(y_bf16);
    v.ldy = ldy;
    return block::gemv_launch(v, block::kGemvBf16, sms, st) ? FP8_OK : FP8_ERR_CUDA;
  }
  const LinearWs w = linear_ws(M, K);
  uint8_t* qa = static_cast<uint8_t*>(ws) + w.qa;
  float* s_a = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + w.s_a);
  FP8_TRY(launch_quantize_rows(A, qa, round_up16(K), s_a, w.lds, nullptr, 0, sms, st));
  return block_mm(qa, M, K, round_up16(K), s_a, w.lds, qw, N, ldqw, s_w, bias_bf16, y_bf16, ldy,
                  block::gemm_held_rows(M, round_up16(K)), sms, st);
}

FP8_API fp8_status fp8_block_selftest_timeout(int form, const uint8_t* qa, int64_t M, int64_t K, int64_t ldqa,
                                              const float* s_a, int64_t lds, const uint8_t* qw, int64_t N,
                                              int64_t ldqw, const float* s_w, void* y, int64_t ldy, float* s_y,
                                              int64_t lds_y, fp8_stream_t stream) {
  if (form < 0 || form > 2 || M < 1 || N < 1 || K < 1) return FP8_ERR_INVALID_ARG;
  FP8_TRY(check_fp8_mat(qa, M, K, ldqa));
  FP8_TRY(check_row_scales(s_a, M, K, lds));
  if (form == 2) {
    FP8_TRY(check_fp8_mat(qw, N, K, ldqw));
    FP8_TRY(check_fp8_mat(y, M, N, ldy));
    FP8_TRY(check_row_scales(s_y, M, N, lds_y));
    if (M > kMaxRows || s_w == nullptr) return FP8_ERR_INVALID_ARG;
    if (!aligned(s_w, 4)) return FP8_ERR_MISALIGNED;
  } else {
    FP8_TRY(check_product(M, K, qw, N, ldqw, s_w, nullptr, y, ldy));
    if (N % 8 != 0 || ldy % 8 != 0) return FP8_ERR_INVALID_ARG;
    if (!aligned(y, 16)) return FP8_ERR_MISALIGNED;
    if (form == 1 && K <= block::kBlock) return FP8_ERR_INVALID_ARG;
  }
  int sms = 0;
  FP8_TRY(current_device(&sms));
  block::GemmArgs g = {};
  g.qa = qa;
  g.rows = g.held_rows = M;
  g.lda = ldqa;
  g.s_a = s_a;
  g.lds_a = lds;
  g.qw = qw;
  g.mats = form == 2 ? 2 : 1;
  g.ldw = ldqw;
  g.s_w = s_w;
  g.N = N;
  g.K = K;
  g.y = static_cast<uint16_t*>(y);
  g.ldy = ldy;
  g.qh = static_cast<uint8_t*>(y);
  g.ldh = ldy;
  g.s_h = s_y;
  g.lds_h = lds_y;
  return block::gemm_launch_withheld(g, form == 2 ? block::kOutSwiglu : block::kOutBf16, form == 1 ? 2 : 1, sms,
                                     reinterpret_cast<cudaStream_t>(stream))
             ? FP8_OK
             : FP8_ERR_CUDA;
}

// ---------------------------------------------------------------------------
// mixture of experts
// ---------------------------------------------------------------------------

FP8_API fp8_status fp8_moe_route(const void* logits, int logits_bf16, int64_t T, int64_t E, int64_t ld, int sigmoid,
                                 const float* bias, int groups, int keep_groups, int k, int renormalize, float factor,
                                 int32_t* ids, float* weights, fp8_stream_t stream) {
  return fp8_moe_route_ex(logits, logits_bf16, T, E, ld, sigmoid, bias, groups, keep_groups, 0, k, renormalize, factor,
                          ids, weights, stream);
}

FP8_API fp8_status fp8_moe_route_ex(const void* logits, int logits_bf16, int64_t T, int64_t E, int64_t ld, int sigmoid,
                                    const float* bias, int groups, int keep_groups, int group_max, int k,
                                    int renormalize, float factor, int32_t* ids, float* weights,
                                    fp8_stream_t stream) {
  if (T < 0 || T > kMaxDim || E < 1 || E > moe::kMaxExperts || ld < E) return FP8_ERR_INVALID_ARG;
  if ((logits_bf16 != 0 && logits_bf16 != 1) || (sigmoid != 0 && sigmoid != 1) ||
      (renormalize != 0 && renormalize != 1) || (group_max != 0 && group_max != 1))
    return FP8_ERR_INVALID_ARG;
  if (groups < 1 || groups > moe::kMaxGroups || E % groups != 0 || keep_groups < 1 || keep_groups > groups)
    return FP8_ERR_INVALID_ARG;
  if (k < 1 || k > moe::kMaxChosen || k > keep_groups * (E / groups)) return FP8_ERR_INVALID_ARG;
  if (!aligned(logits, logits_bf16 ? 2 : 4) || !aligned(bias, 4) || !aligned(ids, 4) || !aligned(weights, 4))
    return FP8_ERR_MISALIGNED;
  if (T == 0) return FP8_OK;
  if (logits == nullptr || ids == nullptr || weights == nullptr) return FP8_ERR_INVALID_ARG;
  int sms = 0;
  FP8_TRY(current_device(&sms));
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  moe::RouteParams p = {};
  p.tokens = T;
  p.ld = ld;
  p.vec = aligned(logits, 16) && ld * (logits_bf16 ? 2 : 4) % 16 == 0;
  p.experts = int(E);
  p.k = k;
  p.groups = groups;
  p.keep = keep_groups;
  p.sigmoid = sigmoid;
  p.renorm = renormalize;
  p.pair_score = !group_max && (sigmoid || bias != nullptr);
  p.factor = factor;
  p.bias = bias;
  p.ids = ids;
  p.weights = weights;
  return logits_bf16 ? launch_route(static_cast<const uint16_t*>(logits), p, sms, st)
                     : launch_route(static_cast<const float*>(logits), p, sms, st);
}

FP8_API size_t fp8_moe_workspace_bytes(int64_t T, int64_t k, int64_t E, int64_t H, int64_t I) {
  if (!moe_sizes_ok(T, k, E, H, I) || T == 0 || H == 0) return 0;
  return moe_ws(T, k, E, H, I).total;
}

FP8_API fp8_status fp8_moe_experts(const void* x_bf16, int64_t T, int64_t H, int64_t ldx, const int32_t* ids,
                                   const float* weights, int64_t k, const uint8_t* qw13, int64_t ldq13,
                                   const float* s13, const uint8_t* qw2, int64_t ldq2, const float* s2, int64_t E,
                                   int64_t I, void* y_bf16, int64_t ldy, void* ws, size_t ws_bytes,
                                   fp8_stream_t stream) {
  if (!moe_sizes_ok(T, k, E, H, I)) return FP8_ERR_INVALID_ARG;
  FP8_TRY(check_bf16_mat(x_bf16, T, H, ldx));
  FP8_TRY(check_bf16_mat(y_bf16, T, H, ldy));
  FP8_TRY(check_fp8_mat(qw13, I, H, ldq13));
  FP8_TRY(check_fp8_mat(qw2, H, I, ldq2));
  if (!aligned(ids, 4) || !aligned(weights, 4) || !aligned(s13, 4) || !aligned(s2, 4)) return FP8_ERR_MISALIGNED;
  if (T == 0 || H == 0) return FP8_OK;
  if (ids == nullptr || weights == nullptr || s13 == nullptr || s2 == nullptr) return FP8_ERR_INVALID_ARG;
  const MoeWs w = moe_ws(T, k, E, H, I);
  FP8_TRY(check_ws(ws, ws_bytes, w.total));
  int sms = 0;
  FP8_TRY(current_device(&sms));
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  uint8_t* b = static_cast<uint8_t*>(ws);
  const BF16Mat X{static_cast<const uint16_t*>(x_bf16), T, H, ldx};

  if (one_token(T, k, H, I)) {
    block::GemvArgs v = {};
    v.src = block::kSrcBf16;
    v.a = X.p;
    v.lda = ldx;
    v.ids = ids;
    v.weights = weights;
    v.pairs = int(k);
    v.experts = E;
    v.qw = qw13;
    v.ldw = ldq13;
    v.s_w = s13;
    v.N = I;
    v.K = H;
    v.y32 = reinterpret_cast<float*>(b + w.h);
    v.ldy32 = w.ldh;
    if (!block::gemv_launch(v, block::kGemvSwiglu, sms, st)) return FP8_ERR_CUDA;
    v.src = block::kSrcF32;
    v.a = b + w.h;
    v.lda = w.ldh;
    v.qw = qw2;
    v.ldw = ldq2;
    v.s_w = s2;
    v.N = H;
    v.K = I;
    v.y = static_cast<uint16_t*>(y_bf16);
    v.ldy = ldy;
    return block::gemv_launch(v, block::kGemvSum, sms, st) ? FP8_OK : FP8_ERR_CUDA;
  }

  int* n_tiles = reinterpret_cast<int*>(b + w.n_tiles);
  block::RowTile* tiles = reinterpret_cast<block::RowTile*>(b + w.tiles);
  int* pos = reinterpret_cast<int*>(b + w.pos);
  float* y32 = reinterpret_cast<float*>(b + w.y);
  FP8_TRY(launch_plan(ids, w.pairs, int(E), reinterpret_cast<int*>(b + w.counts), pos, tiles, n_tiles, st));
  // quantize each token once into its rows; gate and up products with SwiGLU and the quantization
  // of h in their epilogue; the product back; the weighted sum
  float* s_x = reinterpret_cast<float*>(b + w.s_x);
  float* s_h = reinterpret_cast<float*>(b + w.s_h);
  FP8_TRY(launch_quantize_rows(X, b + w.qx, w.ldx, s_x, w.lds, pos, int(k), sms, st));
  block::GemmArgs g = {};
  g.rows = w.pairs;
  g.tiles = tiles;
  g.n_tiles = n_tiles;
  g.max_tiles = w.max_tiles;
  g.qa = b + w.qx;
  g.lda = w.ldx;
  g.held_rows = block::gemm_held_rows(w.pairs, w.ldx);
  g.s_a = s_x;
  g.lds_a = w.lds;
  g.qw = qw13;
  g.mats = 2 * E;
  g.ldw = ldq13;
  g.s_w = s13;
  g.N = I;
  g.K = H;
  g.qh = b + w.h;
  g.ldh = w.ldh;
  g.s_h = s_h;
  g.lds_h = w.lds;
  if (!block::gemm_launch(g, block::kOutSwiglu, sms, st)) return FP8_ERR_CUDA;
  g.qa = b + w.h;
  g.lda = w.ldh;
  g.held_rows = block::gemm_held_rows(w.pairs, w.ldh);
  g.s_a = s_h;
  g.qw = qw2;
  g.mats = E;
  g.ldw = ldq2;
  g.s_w = s2;
  g.N = H;
  g.K = I;
  g.y32 = y32;
  g.ldy32 = w.ldy;
  if (!block::gemm_launch(g, block::kOutF32, sms, st)) return FP8_ERR_CUDA;
  const int vec = aligned(y_bf16, 8) && ldy % 4 == 0;
  return launch(moe::weighted_sum_kernel, dim3(elementwise_grid(T * ((H + 3) / 4), moe::kSumThreads, sms, 8)),
                dim3(moe::kSumThreads), 0, st, true, dim3(1, 1, 1), static_cast<const float*>(y32), w.ldy,
                static_cast<const int*>(pos), weights, int(k), T, H, static_cast<uint16_t*>(y_bf16), ldy, vec);
}
