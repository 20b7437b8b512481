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

template <int kN>
struct Count {
  static constexpr int value = kN;
};

struct RouteParams {
  int64_t tokens, ld;
  int experts, k, groups, keep;
  int sigmoid, renorm;
  int pair_score;  // a group's score is the sum of its two best choices, else the best one
  int vec;  // rows start on 16-byte boundaries
  float factor;
  const float* bias;
  int32_t* ids;
  float* weights;
};

// n / d for 0 <= n <= 1024 and inv = 1 / d: the half keeps the product clear of whole numbers.
__device__ __forceinline__ int quotient_of(int n, float inv) { return int((float(n) + 0.5f) * inv); }

// The k largest of the warp's keys, one at a time; key i of lane l has index l * kCount + i, so the
// lowest lane, and in it the lowest i, is the lowest index. Key 0 marks no key. Lane j returns the
// index of the j-th largest. Up to eight keys a lane are sorted first (neighbours exchanged only when
// strictly out of order: equal keys keep their order), so a round is the warp's largest head, the
// first lane that has it, and a shift there; sixteen are searched again in the winner's lane.
template <int kCount>
__device__ __forceinline__ int take_largest(uint32_t (&key)[kCount], int k, int lane) {
  int mine = 0;
  if constexpr (kCount <= 8) {
    int at[kCount];
#pragma unroll
    for (int i = 0; i < kCount; ++i) at[i] = lane * kCount + i;
#pragma unroll
    for (int pass = 0; pass < kCount; ++pass)
#pragma unroll
      for (int i = pass & 1; i + 1 < kCount; i += 2) {
        const bool swap = key[i] < key[i + 1];
        const uint32_t hi = max(key[i], key[i + 1]), lo = min(key[i], key[i + 1]);
        const int a = swap ? at[i + 1] : at[i], b = swap ? at[i] : at[i + 1];
        key[i] = hi, key[i + 1] = lo, at[i] = a, at[i + 1] = b;
      }
    for (int j = 0; j < k; ++j) {
      const uint32_t top = __reduce_max_sync(0xffffffffu, key[0]);
      const int winner = __ffs(__ballot_sync(0xffffffffu, key[0] == top)) - 1;
      const int e = __shfl_sync(0xffffffffu, at[0], winner);
      if (lane == j) mine = e;
      if (lane == winner) {
#pragma unroll
        for (int i = 0; i + 1 < kCount; ++i) key[i] = key[i + 1], at[i] = at[i + 1];
        key[kCount - 1] = 0u;
      }
    }
  } else {
    uint32_t best = 0u;
#pragma unroll
    for (int i = 0; i < kCount; ++i) best = max(best, key[i]);
    for (int j = 0; j < k; ++j) {
      const uint32_t top = __reduce_max_sync(0xffffffffu, best);
      const int winner = __ffs(__ballot_sync(0xffffffffu, best == top)) - 1;
      int first = 0;
      if (lane == winner) {
#pragma unroll
        for (int i = kCount - 1; i >= 0; --i)
          if (key[i] == top) first = i;
        best = 0u;
#pragma unroll
        for (int i = 0; i < kCount; ++i) {
          if (i == first) key[i] = 0u;
          best = max(best, key[i]);
        }
      }
      const int e = __shfl_sync(0xffffffffu, lane * kCount + first, winner);
      if (lane == j) mine = e;
    }
  }
  return mine;
}

// Logits [lane * kPerLane, +kPerLane) of a row of E, -inf past the end; `vec`: rows start on 16 bytes.
template <int kPerLane>
__device__ __forceinline__ void load_logits(const float* row, int lane, int E, int vec, float (&c)[kPerLane]) {
  const int e0 = lane * kPerLane;
  if (kPerLane % 4 == 0 && vec && e0 + kPerLane <= E) {
#pragma unroll
    for (int i = 0; i < kPerLane / 4; ++i) {
      const float4 v = __ldg(reinterpret_cast<const float4*>(row + e0) + i);
      c[4 * i] = v.x, c[4 * i + 1] = v.y, c[4 * i + 2] = v.z, c[4 * i + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) c[i] = e0 + i < E ? __ldg(row + e0 + i) : -INFINITY;
  }
}
template <int kPerLane>
__device__ __forceinline__ void load_logits(const uint16_t* row, int lane, int E, int vec, float (&c)[kPerLane]) {
  const int e0 = lane * kPerLane;
  if (kPerLane % 8 == 0 && vec && e0 + kPerLane <= E) {
#pragma unroll
    for (int i = 0; i < kPerLane / 8; ++i) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(row + e0) + i);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) c[8 * i + 2 * j] = bf16_lo(w[j]), c[8 * i + 2 * j + 1] = bf16_hi(w[j]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) c[i] = e0 + i < E ? bf16_bits_to_float(__ldg(row + e0 + i)) : -INFINITY;
  }
}

// One warp a token; lane l holds the experts l * kPerLane .. The choice runs on
//   softmax without bias: the logit itself (the order of the probabilities),
//   softmax with bias: p + bias,   sigmoid: 1 / (1 + exp(-x)) (+ bias),
// each in fp32 with the accurate exp and division: equal scores are equal bits and the lowest
// index wins them. With groups, 32 / groups lanes (rounded down to a power of two) find a group's
// two best each in its share, and only the experts of the groups that stay are looked at again, in
// their order (without that, and with the keys of a lane unsorted, 24.7 and 22.5 us below). 16384 tokens of
// 256 experts in 8 groups, k = 8, take 19.6 us. Not memory (the logits, read once, are 2.5 us) but
// instructions set that: 1123 a token, 14.7 us if every scheduler issued one a cycle. While they have warps
// the schedulers issue in 76 percent of the cycles; 64 registers a thread allow half of the warps an SM
// holds, and 2048 CTAs are 3.4 waves of them, so that the last one runs part empty.
template <typename T, int kPerLane>
__global__ void __launch_bounds__(kRouteThreads)
route_kernel(const T* __restrict__ logits, const __grid_constant__ RouteParams p) {
  __shared__ __align__(16) float sh_choice[kRouteThreads / 32][kPerLane * 32];
  __shared__ uint8_t sh_kept[kRouteThreads / 32][kMaxGroups];
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int E = p.experts;
  const int size = E / p.groups;
  const int lanes_log2 = 31 - __clz(32 / p.groups);  // lanes that share a group
  const float inv_size = 1.0f / float(size);
  const int64_t nwarps = int64_t(gridDim.x) * (kRouteThreads / 32);
  for (int64_t t = int64_t(blockIdx.x) * (kRouteThreads / 32) + warp; t < p.tokens; t += nwarps) {
    const T* row = logits + t * p.ld;
    float c[kPerLane];
    float mx = -INFINITY, sum = 0.0f;
    load_logits(row, lane, E, p.vec, c);
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
      c[i] = c[i] != c[i] ? -INFINITY : c[i];  // a NaN is never chosen before a number
      mx = fmaxf(mx, c[i]);
    }
    const int e0 = lane * kPerLane;
    if (!p.sigmoid) {
      mx = warp_max(mx);
#pragma unroll
      for (int i = 0; i < kPerLane; ++i) {
        // x == max covers max = +inf, whose difference is NaN
        const float e = c[i] == mx ? 1.0f : expf(c[i] - mx);
        sum += e0 + i < E ? e : 0.0f;
        if (p.bias) c[i] = mx == -INFINITY ? 0.0f : e;  // a row of only -inf: p = 0, the bias alone chooses
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (p.bias) {
#pragma unroll
        for (int i = 0; i < kPerLane; ++i)
          if (e0 + i < E) c[i] = c[i] / sum + __ldg(p.bias + e0 + i);
      }
    } else {
#pragma unroll
      for (int i = 0; i < kPerLane; ++i) {
        c[i] = __frcp_rn(1.0f + expf(-c[i]));  // the rounded 1 / x
        if (p.bias && e0 + i < E) c[i] += __ldg(p.bias + e0 + i);
      }
    }
    int my_id;
    uint32_t key[kPerLane];
    if (p.groups > 1) {
      float* sh = sh_choice[warp];
      __syncwarp();  // the warp has left its last token's choices
      if constexpr (kPerLane % 4 == 0) {
#pragma unroll
        for (int i = 0; i < kPerLane; i += 4)
          *reinterpret_cast<float4*>(sh + e0 + i) = make_float4(c[i], c[i + 1], c[i + 2], c[i + 3]);
      } else {
#pragma unroll
        for (int i = 0; i < kPerLane; ++i) sh[e0 + i] = c[i];
      }
      __syncwarp();
      // a group's score: its best choice, or the sum of its two best
      const int lanes = 1 << lanes_log2, group = lane >> lanes_log2, sub = lane & (lanes - 1);
      float b1 = -INFINITY, b2 = -INFINITY;
      if (group < p.groups) {
        // staggered: groups a multiple of 32 experts apart would meet in one bank
        const int rounds = (size + lanes - 1) >> lanes_log2;
        int n = group % rounds;
        for (int r = 0; r < rounds; ++r) {
          const int j = (n << lanes_log2) + sub;
          n = n + 1 == rounds ? 0 : n + 1;
          const float v = j < size ? sh[group * size + j] : -INFINITY;
          b2 = fmaxf(b2, fminf(b1, v));
          b1 = fmaxf(b1, v);
        }
      }
      for (int o = 1; o < lanes; o <<= 1) {
        const float o1 = __shfl_xor_sync(0xffffffffu, b1, o), o2 = __shfl_xor_sync(0xffffffffu, b2, o);
        b2 = fmaxf(fmaxf(b2, o2), fminf(b1, o1));
        b1 = fmaxf(b1, o1);
      }
      const uint32_t mine = order_key(p.pair_score && size > 1 ? b1 + b2 : b1);
      // a group stays when fewer than `keep` groups beat it (ties: the lower index first)
      int beaten_by = 0;
      for (int g = 0; g < p.groups; ++g) {
        const uint32_t other = __shfl_sync(0xffffffffu, mine, g << lanes_log2);
        beaten_by += other > mine || (other == mine && g < group);
      }
      const bool stays = group < p.groups && sub == 0 && beaten_by < p.keep;
      const uint32_t all = __ballot_sync(0xffffffffu, stays);
      if (stays) sh_kept[warp][__popc(all & ((1u << lane) - 1))] = uint8_t(group);
      __syncwarp();
      const int n = p.keep * size;  // candidates, in the experts' order
      auto expert_of = [&](int q) {
        const int kg = quotient_of(q, inv_size);
        return int(sh_kept[warp][kg]) * size + (q - kg * size);
      };
      auto pick = [&](auto count) {
        constexpr int kCount = decltype(count)::value;
        uint32_t some[kCount];
#pragma unroll
        for (int i = 0; i < kCount; ++i) {
          const int q = lane * kCount + i;
          some[i] = q < n ? max(order_key(sh[expert_of(q)]), 1u) : 0u;
        }
        return take_largest<kCount>(some, p.k, lane);
      };
      constexpr int kFew = kPerLane > 1 ? kPerLane / 2 : 1;
      const int q = n <= kFew * 32 ? pick(Count<kFew>()) : pick(Count<kPerLane>());
      my_id = lane < p.k ? expert_of(q) : 0;
    } else {
#pragma unroll
      for (int i = 0; i < kPerLane; ++i) key[i] = e0 + i < E ? max(order_key(c[i]), 1u) : 0u;  // 0: taken
      my_id = take_largest<kPerLane>(key, p.k, lane);
    }
    float w = 0.0f;
    if (lane < p.k) {
      const float x = clean_logit(row + my_id);
      if (p.sigmoid)
        w = __frcp_rn(1.0f + expf(-x));
      else if (mx != -INFINITY)  // a row with nothing to choose from gets no weight
        w = (x == mx ? 1.0f : expf(x - mx)) / sum;
    }
    if (p.renorm) {
      float total = w;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
      w = w / (total + 1e-20f);
    }
    if (lane < p.k) {
      p.ids[t * p.k + lane] = my_id;
      p.weights[t * p.k + lane] = w * p.factor;
    }
  }
}

constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;

constexpr int kPlanPairs = 1024;  // pairs of one CTA, about (a step of every warp)
constexpr int kPlanMaxCtas = 128;

// The pairs [begin, end) of CTA `part` of `parts`, whole warp steps.
__device__ __forceinline__ void plan_range(int64_t pairs, int part, int parts, int64_t& begin, int64_t& end) {
  const int64_t share = (pairs + int64_t(parts) * 32 - 1) / (int64_t(parts) * 32) * 32;
  begin = min(pairs, share * part);
  end = min(pairs, begin + share);
}

// counts[cta][expert] of the CTA's pairs, for a plan of several CTAs.
__global__ void __launch_bounds__(kPlanThreads, 1)
plan_count_kernel(const int32_t* __restrict__ ids, int64_t pairs, int experts, int* __restrict__ counts) {
  __shared__ int count[kMaxExperts];
  pdl_trigger();
  pdl_wait();
  for (int i = threadIdx.x; i < experts; i += kPlanThreads) count[i] = 0;
  __syncthreads();
  int64_t begin, end;
  plan_range(pairs, blockIdx.x, gridDim.x, begin, end);
  for (int64_t i = begin + threadIdx.x; i < end; i += kPlanThreads) {
    const int id = ids[i];
    if (id >= 0 && id < experts) atomicAdd(&count[id], 1);  // sums of ones: any order
  }
  __syncthreads();
  for (int i = threadIdx.x; i < experts; i += kPlanThreads) counts[blockIdx.x * experts + i] = count[i];
}

// Order of the routed pairs: pair i (= token * k + j) with expert ids[i] in [0, experts) gets row
// pos[i], rows sorted by expert and, within one, by pair (stable, so nothing depends on timing);
// any other id gives -1. Then the row tiles. A CTA's warps count their contiguous shares of the CTA's pairs by expert in
// shared memory (equal ids of a step are found by a warp match), the counts are scanned over warps,
// CTAs (from plan_count_kernel; one CTA needs none) and experts, and a second walk hands out rows.
// One CTA sorts 65536 pairs in 109 us, 64 CTAs in 11 us.
__global__ void __launch_bounds__(kPlanThreads, 1)
plan_kernel(const int32_t* __restrict__ ids, int64_t pairs, int experts, const int* __restrict__ counts,
            int* __restrict__ pos, block::RowTile* __restrict__ tiles, int* __restrict__ n_tiles) {
  extern __shared__ int count[];  // [kPlanWarps][experts], then [experts] first rows
  int* total = count + kPlanWarps * experts;
  __shared__ int warp_sum[2][kPlanWarps];
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < kPlanWarps * experts; i += kPlanThreads) count[i] = 0;
  __syncthreads();
  int64_t cta_begin, cta_end, begin, end;
  plan_range(pairs, blockIdx.x, gridDim.x, cta_begin, cta_end);
  plan_range(cta_end - cta_begin, warp, kPlanWarps, begin, end);
  begin += cta_begin, end += cta_begin;
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
    int before = 0;  // this expert's pairs in the CTAs before this one
    if (counts != nullptr) {
#pragma unroll 8
      for (int c = 0; c < int(gridDim.x); ++c) {
        const int v = counts[c * experts + threadIdx.x];
        before += c < int(blockIdx.x) ? v : 0;
        tot += v;
      }
    }
    for (int w = 0; w < kPlanWarps; ++w) {
      const int v = count[w * experts + threadIdx.x];
      count[w * experts + threadIdx.x] = before;
      before += v;
    }
    if (counts == nullptr) tot = before;
  }
  const int my_tiles = (tot + block::kRowTile - 1) / block::kRowTile;
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
    // the CTAs share out an expert's tiles
    for (int j = blockIdx.x; j < my_tiles; j += gridDim.x) {
      const int r0 = rows_before + j * block::kRowTile;
      tiles[tiles_before + j] = block::RowTile{int(threadIdx.x), r0, rows_before + tot, 0};
    }
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) *n_tiles = all_t;
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
  }
}

constexpr int kSumThreads = 256;

// out[t] = bf16(sum_j w[t, j] y[pos[t, j]]) over the pairs that have a row, in the order of j, in
// fp32 (a token with none gets zeros). Four columns a thread, eight pairs' loads in flight; HBM bounds
// it: 65536 rows of 4096 in 162 us (1.14 GB, 7.0 TB/s).
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
