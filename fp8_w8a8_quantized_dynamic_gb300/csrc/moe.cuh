// Mixture of experts: choice of experts, the order of the routed rows, and their weighted sum.
#pragma once

#include <cfloat>
#include <cmath>

#include "block_gemm.h"
#include "device_common.cuh"
#include "tcgen05.cuh"

namespace fp8k {
namespace moe {

constexpr int kMaxExperts = 512;
constexpr int kMaxChosen = 32;
constexpr int kMaxGroups = 32;
constexpr int kRouteThreads = 256;  // eight tokens a CTA, one warp each

// Larger key = larger float (-0 and +0 alike); 0 is below every float's key.
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

__device__ __forceinline__ float load_logit(const float* p) { return __ldg(p); }
__device__ __forceinline__ float load_logit(const uint16_t* p) { return bf16_bits_to_float(__ldg(p)); }
// A NaN is never chosen before a number: it counts as -inf.
template <typename T>
__device__ __forceinline__ float clean_logit(const T* p) {
  const float x = load_logit(p);
  return x != x ? -INFINITY : x;
}

struct RouteParams {
  int64_t tokens, ld;
  int experts, k, groups, keep;
  int sigmoid, renorm;
  float factor;
  const float* bias;
  int32_t* ids;
  float* weights;
};

// One warp a token; lane l holds the experts l, l + 32, ... The choice runs on
//   softmax without bias: the logit itself (the order of the probabilities),
//   softmax with bias: p + bias,   sigmoid: 1 / (1 + exp(-x)) (+ bias),
// each in fp32 with the accurate exp and division: equal scores are equal bits and the lowest
// index wins them. The k largest come out one at a time: a lane's best of its own, the warp's
// best key, then the lowest expert that has it. Bound: issue slots (about k rounds of two warp
// reductions a token); the logits are read once.
template <typename T, int kPerLane>
__global__ void __launch_bounds__(kRouteThreads)
route_kernel(const T* __restrict__ logits, const __grid_constant__ RouteParams p) {
  __shared__ float sh_choice[kRouteThreads / 32][kPerLane * 32];
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int E = p.experts;
  const int64_t nwarps = int64_t(gridDim.x) * (kRouteThreads / 32);
  for (int64_t t = int64_t(blockIdx.x) * (kRouteThreads / 32) + warp; t < p.tokens; t += nwarps) {
    const T* row = logits + t * p.ld;
    float c[kPerLane];
    float mx = -INFINITY;
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
      const int e = i * 32 + lane;
      c[i] = e < E ? clean_logit(row + e) : -INFINITY;
      mx = fmaxf(mx, c[i]);
    }
    float inv_arg = 0.0f;  // softmax: the sum of exp(x - max)
    if (!p.sigmoid) {
      mx = warp_max(mx);
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < kPerLane; ++i) {
        // x == max covers max = +inf, whose difference is NaN
        const float e = c[i] == mx ? 1.0f : expf(c[i] - mx);
        sum += (i * 32 + lane < E) ? e : 0.0f;
        if (p.bias) c[i] = e;
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      inv_arg = sum;
      if (p.bias) {
#pragma unroll
        for (int i = 0; i < kPerLane; ++i)
          if (i * 32 + lane < E) c[i] = c[i] / sum + __ldg(p.bias + i * 32 + lane);
      }
    } else {
#pragma unroll
      for (int i = 0; i < kPerLane; ++i) {
        c[i] = 1.0f / (1.0f + expf(-c[i]));
        if (p.bias && i * 32 + lane < E) c[i] += __ldg(p.bias + i * 32 + lane);
      }
    }
    if (p.groups > 1) {
      const int size = E / p.groups;
      float* sh = sh_choice[warp];
      __syncwarp();
#pragma unroll
      for (int i = 0; i < kPerLane; ++i)
        if (i * 32 + lane < E) sh[i * 32 + lane] = c[i];
      __syncwarp();
      // lane g scores group g: its best choice, or the sum of its two best
      float score = -INFINITY;
      if (lane < p.groups) {
        float b1 = -INFINITY, b2 = -INFINITY;
        int j = lane % size;  // staggered start: the groups' first elements share a bank
        for (int n = 0; n < size; ++n) {
          const float v = sh[lane * size + j];
          b2 = fmaxf(b2, fminf(b1, v));
          b1 = fmaxf(b1, v);
          j = j + 1 == size ? 0 : j + 1;
        }
        score = ((p.sigmoid || p.bias) && size > 1) ? b1 + b2 : b1;
      }
      // a group stays when fewer than `keep` groups beat it (ties: the lower index first)
      const uint32_t mine = order_key(score);
      int beaten_by = 0;
      for (int g = 0; g < p.groups; ++g) {
        const uint32_t other = __shfl_sync(0xffffffffu, mine, g);
        beaten_by += other > mine || (other == mine && g < lane);
      }
      const uint32_t stays = __ballot_sync(0xffffffffu, lane < p.groups && beaten_by < p.keep);
#pragma unroll
      for (int i = 0; i < kPerLane; ++i) {
        const int e = i * 32 + lane;
        if (e < E && !((stays >> (e / size)) & 1u)) c[i] = -INFINITY;
      }
    }
    uint32_t key[kPerLane];
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) key[i] = i * 32 + lane < E ? max(order_key(c[i]), 1u) : 0u;  // 0: taken
    int my_id = 0;
    for (int j = 0; j < p.k; ++j) {
      uint32_t best = key[0];
      int at = 0;
#pragma unroll
      for (int i = 1; i < kPerLane; ++i)
        if (key[i] > best) best = key[i], at = i;
      const uint32_t top = __reduce_max_sync(0xffffffffu, best);
      const uint32_t e = __reduce_min_sync(0xffffffffu, best == top ? uint32_t(at * 32 + lane) : 0xFFFFFFFFu);
      if ((e & 31u) == uint32_t(lane)) {
#pragma unroll
        for (int i = 0; i < kPerLane; ++i)
          if (uint32_t(i) == (e >> 5)) key[i] = 0u;
      }
      if (lane == j) my_id = int(e);
    }
    float w = 0.0f;
    if (lane < p.k) {
      const float x = clean_logit(row + my_id);
      if (p.sigmoid)
        w = 1.0f / (1.0f + expf(-x));
      else if (mx != -INFINITY)  // a row with nothing to choose from gets no weight
        w = (x == mx ? 1.0f : expf(x - mx)) / inv_arg;
    }
    if (p.renorm) {
      float sum = w;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      w = w / (sum + 1e-20f);
    }
    if (lane < p.k) {
      p.ids[t * p.k + lane] = my_id;
      p.weights[t * p.k + lane] = w * p.factor;
    }
  }
}

constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;

// Order of the routed pairs: pair i (= token * k + j) with expert ids[i] in [0, experts) gets row
// pos[i], rows sorted by expert and, within one, by pair (stable, so nothing depends on timing);
// any other id gives -1; row_src (may be null) gets the token of each row. Then the row tiles, of
// tile_rows rows each. One CTA: each warp counts its
// contiguous share of the pairs by expert in shared memory (equal ids of a step are found by a
// warp match), the counts are scanned over warps and experts, and the second walk hands out rows.
__global__ void __launch_bounds__(kPlanThreads, 1)
plan_kernel(const int32_t* __restrict__ ids, int64_t pairs, int experts, int k, int tile_rows, int* __restrict__ pos,
            int* __restrict__ row_src, block::RowTile* __restrict__ tiles, int* __restrict__ n_tiles) {
  extern __shared__ int count[];  // [kPlanWarps][experts], then [experts] totals
  int* total = count + kPlanWarps * experts;
  __shared__ int warp_sum[2][kPlanWarps];
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < kPlanWarps * experts; i += kPlanThreads) count[i] = 0;
  __syncthreads();
  const int64_t share = (pairs + kPlanWarps * 32 - 1) / (kPlanWarps * 32) * 32;
  const int64_t begin = min(pairs, share * warp), end = min(pairs, begin + share);
  int* mine = count + warp * experts;
  for (int64_t i = begin; i < end; i += 32) {
    const int id = i + lane < end ? ids[i + lane] : -1;
    const bool in = id >= 0 && id < experts;
    const uint32_t same = __match_any_sync(0xffffffffu, in ? id : -1);
    if (in && lane == __ffs(same) - 1) mine[id] += __popc(same);
    __syncwarp();
  }
  __syncthreads();
  // experts are scanned in order: thread e < experts sums its column over the warps
  int tot = 0;
  if (int(threadIdx.x) < experts) {
    for (int w = 0; w < kPlanWarps; ++w) {
      const int v = count[w * experts + threadIdx.x];
      count[w * experts + threadIdx.x] = tot;
      tot += v;
    }
  }
  const int my_tiles = (tot + tile_rows - 1) / tile_rows;
  int rows_before = tot, tiles_before = my_tiles;  // inclusive scans over the experts
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int a = __shfl_up_sync(0xffffffffu, rows_before, o), b = __shfl_up_sync(0xffffffffu, tiles_before, o);
    if (lane >= o) rows_before += a, tiles_before += b;
  }
  if (lane == 31) warp_sum[0][warp] = rows_before, warp_sum[1][warp] = tiles_before;
  __syncthreads();
  int base_r = 0, base_t = 0, all_t = 0;
  for (int w = 0; w < kPlanWarps; ++w) {
    if (w < warp) base_r += warp_sum[0][w], base_t += warp_sum[1][w];
    all_t += warp_sum[1][w];
  }
  rows_before += base_r - tot;
  tiles_before += base_t - my_tiles;
  if (int(threadIdx.x) < experts) {
    total[threadIdx.x] = rows_before;
    for (int j = 0; j < my_tiles; ++j) {
      const int r0 = rows_before + j * tile_rows;
      tiles[tiles_before + j] = block::RowTile{int(threadIdx.x), r0, rows_before + tot, 0};
    }
  }
  if (threadIdx.x == 0) *n_tiles = all_t;
  __syncthreads();
  for (int64_t i = begin; i < end; i += 32) {
    const int id = i + lane < end ? ids[i + lane] : -1;
    const bool in = id >= 0 && id < experts;
    const uint32_t same = __match_any_sync(0xffffffffu, in ? id : -1);
    int d = -1;
    if (in) d = total[id] + mine[id] + __popc(same & ((1u << lane) - 1));
    __syncwarp();
    if (in && lane == __ffs(same) - 1) mine[id] += __popc(same);
    __syncwarp();
    if (i + lane < end) pos[i + lane] = d;
    if (row_src != nullptr && d >= 0) row_src[d] = int((i + lane) / k);
  }
}

constexpr int kSumThreads = 256;

// out[t] = bf16(sum_j w[t, j] y[pos[t, j]]) over the pairs that have a row, in the order of j, in
// fp32 (a token with none gets zeros). Four columns a thread; HBM bounds it.
__global__ void __launch_bounds__(kSumThreads)
weighted_sum_kernel(const float* __restrict__ y, int64_t ldy32, const int* __restrict__ pos,
                    const float* __restrict__ weights, int k, int64_t tokens, int64_t cols, uint16_t* __restrict__ out,
                    int64_t ldo, int vec) {
  pdl_trigger();
  pdl_wait();
  const int64_t upr = (cols + 3) / 4;
  for (int64_t u = int64_t(blockIdx.x) * kSumThreads + threadIdx.x; u < tokens * upr;
       u += int64_t(gridDim.x) * kSumThreads) {
    const int64_t t = u / upr;
    const int64_t c = (u - t * upr) * 4;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int j0 = 0; j0 < k; j0 += 8) {
      float4 v[8];
      float w[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int d = j0 + j < k ? pos[t * k + j0 + j] : -1;
        w[j] = d >= 0 ? weights[t * k + j0 + j] : 0.0f;
        v[j] = d >= 0 ? __ldcs(reinterpret_cast<const float4*>(y + int64_t(d) * ldy32 + c))
                      : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        acc.x = fmaf(w[j], v[j].x, acc.x);
        acc.y = fmaf(w[j], v[j].y, acc.y);
        acc.z = fmaf(w[j], v[j].z, acc.z);
        acc.w = fmaf(w[j], v[j].w, acc.w);
      }
    }
    uint16_t* dst = out + t * ldo + c;
    if (vec && c + 4 <= cols) {
      *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
    } else {
      const float a[4] = {acc.x, acc.y, acc.z, acc.w};
      for (int e = 0; e < 4; ++e)
        if (c + e < cols) dst[e] = __bfloat16_as_ushort(__float2bfloat16_rn(a[e]));
    }
  }
}

}  // namespace moe
}  // namespace fp8k
