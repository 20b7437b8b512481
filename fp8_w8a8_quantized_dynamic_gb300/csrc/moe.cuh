// Mixture of experts: choice of experts, the order of the routed rows, and their weighted sum.
#pragma once

#include <cfloat>
#include <cmath>

#include "any_rows.cuh"
#include "block_gemm.h"
#include "device_common.cuh"
#include "moe_plan.h"
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
constexpr int kPlanCluster = 8;  // CTAs that exchange their counts through distributed shared memory
constexpr int kPlanClusterPairs = 8192;  // that they sort, at most

// Where a CTA learns of the other CTAs' pairs: there are none, from its cluster, from plan_count_kernel.
enum class PlanBy : int { kAlone, kCluster, kCounts };

// The pairs [begin, end) of CTA `part` of `parts`, whole warp steps.
__device__ __forceinline__ void plan_range(int64_t pairs, int part, int parts, int64_t& begin, int64_t& end) {
  const int64_t share = (pairs + int64_t(parts) * 32 - 1) / (int64_t(parts) * 32) * 32;
  begin = min(pairs, share * part);
  end = min(pairs, begin + share);
}

// The expert that an id stands for, -1 for none.
__device__ __forceinline__ int expert_of(int id, const Plan& p) { return id >= 0 && id < p.experts ? id : p.spare; }

// counts[cta][expert] of the CTA's pairs, for a plan of several CTAs.
__global__ void __launch_bounds__(kPlanThreads, 1)
plan_count_kernel(const __grid_constant__ Plan p) {
  const int experts = p.experts;
  __shared__ int count[kMaxExperts];
  pdl_trigger();
  pdl_wait();
  for (int i = threadIdx.x; i < experts; i += kPlanThreads) count[i] = 0;
  __syncthreads();
  int64_t begin, end;
  plan_range(p.pairs, blockIdx.x, gridDim.x, begin, end);
  for (int64_t i = begin + threadIdx.x; i < end; i += kPlanThreads) {
    const int id = expert_of(p.ids[i], p);
    if (id >= 0) atomicAdd(&count[id], 1);  // sums of ones: any order
  }
  __syncthreads();
  for (int i = threadIdx.x; i < experts; i += kPlanThreads) p.counts[blockIdx.x * experts + i] = count[i];
}

// Order of the routed pairs: pair i (= token * k + j) with expert ids[i] in [0, experts) gets row
// pos[i], rows sorted by expert and, within one, by pair (stable, so nothing depends on timing);
// any other id gives -1, or counts as expert `spare`. Then the row tiles and the experts' first rows (where wanted). A
// CTA's warps count their contiguous shares of the CTA's pairs by expert in shared memory (equal ids of a step are found by a
// warp match), the counts are scanned over warps, CTAs (PlanBy) and experts, and a second walk hands out rows.
// One CTA sorts 65536 pairs in 109 us, 64 CTAs in 8.4 us after counting in 3.6.
__global__ void __launch_bounds__(kPlanThreads, 1)
plan_kernel(const __grid_constant__ Plan p, PlanBy by) {
  const int experts = p.experts;
  extern __shared__ int count[];  // [kPlanWarps][experts], then [experts] first rows
  int* total = count + kPlanWarps * experts;
  __shared__ int warp_sum[2][kPlanWarps];
  __shared__ int in_cta[kMaxExperts];        // pairs of each expert in this CTA
  __shared__ int elsewhere[2][kMaxExperts];  // in the CTAs before this one, and in all
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < kPlanWarps * experts; i += kPlanThreads) count[i] = 0;
  if (threadIdx.x < kMaxExperts) elsewhere[0][threadIdx.x] = elsewhere[1][threadIdx.x] = 0;
  __syncthreads();
  int64_t cta_begin, cta_end, begin, end;
  plan_range(p.pairs, blockIdx.x, gridDim.x, cta_begin, cta_end);
  plan_range(cta_end - cta_begin, warp, kPlanWarps, begin, end);
  begin += cta_begin, end += cta_begin;
  int* mine = count + warp * experts;
  for (int64_t i = begin; i < end; i += 32) {
    const int id = i + lane < end ? expert_of(p.ids[i + lane], p) : -1;
    const bool in = id >= 0;
    const uint32_t same = __match_any_sync(0xffffffffu, id);
    if (in && lane == __ffs(same) - 1) mine[id] += __popc(same);
    __syncwarp();
  }
  __syncthreads();
  // thread e < experts sums its column over the warps
  int mine_in_cta = 0;
  if (int(threadIdx.x) < experts) {
    for (int w0 = 0; w0 < kPlanWarps; w0 += 8) {
      int v[8];
#pragma unroll
      for (int w = 0; w < 8; ++w) v[w] = count[(w0 + w) * experts + threadIdx.x];
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        count[(w0 + w) * experts + threadIdx.x] = mine_in_cta;
        mine_in_cta += v[w];
      }
    }
    in_cta[threadIdx.x] = mine_in_cta;
  }
  // this CTA's place: every expert's pairs in the CTAs before it, and in all of them
  int before = 0, tot = mine_in_cta;
  if (by == PlanBy::kCluster) {
    pair_sync();  // the whole cluster
    tot = 0;
    if (int(threadIdx.x) < experts)
      for (int c = 0; c < int(gridDim.x); ++c) {
        const int v = int(ld_cluster_u32(map_to_rank(smem_u32(&in_cta[threadIdx.x]), c)));
        before += c < int(blockIdx.x) ? v : 0;
        tot += v;
      }
  } else if (by == PlanBy::kCounts) {  // (by as many threads as there are)
    const int wide = experts <= 32 ? 32 : 1 << (32 - __clz(experts - 1)), e = threadIdx.x & (wide - 1);
    if (e < experts) {
      int b = 0, all = 0;
#pragma unroll 4
      for (int c = threadIdx.x / wide; c < int(gridDim.x); c += kPlanThreads / wide) {
        const int v = p.counts[c * experts + e];
        b += c < int(blockIdx.x) ? v : 0;
        all += v;
      }
      atomicAdd(&elsewhere[0][e], b);  // sums of whole numbers: any order
      atomicAdd(&elsewhere[1][e], all);
    }
    __syncthreads();
    before = threadIdx.x < kMaxExperts ? elsewhere[0][threadIdx.x] : 0;
    tot = int(threadIdx.x) < experts ? elsewhere[1][threadIdx.x] : 0;
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
    total[threadIdx.x] = rows_before + before;
    // the CTAs share out an expert's tiles
    for (int j = blockIdx.x; p.tiles != nullptr && j < my_tiles; j += gridDim.x) {
      const int r0 = rows_before + j * block::kRowTile;
      p.tiles[tiles_before + j] = block::RowTile{int(threadIdx.x), r0, rows_before + tot, 0};
    }
    if (p.offsets != nullptr && blockIdx.x == 0) {
      p.offsets[threadIdx.x] = rows_before;
      if (int(threadIdx.x) == experts - 1) p.offsets[experts] = rows_before + tot;
    }
  }
  if (p.n_tiles != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *p.n_tiles = all_t;
  __syncthreads();
  for (int64_t i = begin; i < end; i += 32) {
    const int id = i + lane < end ? expert_of(p.ids[i + lane], p) : -1;
    const bool in = id >= 0;
    const uint32_t same = __match_any_sync(0xffffffffu, id);
    int d = -1;
    if (in) d = total[id] + mine[id] + __popc(same & ((1u << lane) - 1));
    __syncwarp();
    if (in && lane == __ffs(same) - 1) mine[id] += __popc(same);
    __syncwarp();
    if (i + lane < end) p.pos[i + lane] = d;
    if (d >= 0 && p.order != nullptr) p.order[d] = int(i) + lane;
  }
  if (by == PlanBy::kCluster) pair_sync();  // no CTA leaves while another reads its sums
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

// ---------------------------------------------------------------------------
// tokens sorted by expert and back
// ---------------------------------------------------------------------------

constexpr int kRowThreads = 256;

// u / d; by 32 bits where both allow it, a fraction of the 64-bit division's instructions.
__device__ __forceinline__ int64_t quotient_of_unit(int64_t u, int64_t d) {
  return ((u | d) >> 32) == 0 ? int64_t(uint32_t(u) / uint32_t(d)) : u / d;
}

// Row t of x to the rows pos[t, j] of xs (those in [0, rows)), as U-sized pieces: `pieces` of a row, row strides in pieces.
// A row is read once for all of its copies. Bounds: HBM's writes (8192 rows of 4096 bf16 to eight rows each, 91 us, 6.6 TB/s).
template <typename U>
__global__ void __launch_bounds__(kRowThreads)
rows_out_kernel(const U* __restrict__ x, int64_t ldx, int64_t tokens, int64_t pieces, const int* __restrict__ pos, int k,
                int64_t rows, U* __restrict__ xs, int64_t ldxs) {
  pdl_trigger();
  pdl_wait();
  for (int64_t u = int64_t(blockIdx.x) * kRowThreads + threadIdx.x; u < tokens * pieces;
       u += int64_t(gridDim.x) * kRowThreads) {
    const int64_t t = quotient_of_unit(u, pieces), c = u - t * pieces;
    const U v = x[t * ldx + c];
    for (int j = 0; j < k; ++j) {
      const int d = pos[t * k + j];
      if (d >= 0 && d < rows) xs[int64_t(d) * ldxs + c] = v;
    }
  }
}

// The same where rows start or end off 16-byte boundaries: eight 16-bit values a thread (cols and row strides in them).
__global__ void __launch_bounds__(kRowThreads)
rows_out_any_kernel(const uint16_t* __restrict__ x, int64_t ldx, int64_t tokens, int64_t cols, const int* __restrict__ pos,
                    int k, int64_t rows, uint16_t* __restrict__ xs, int64_t ldxs) {
  pdl_trigger();
  pdl_wait();
  const int64_t upr = (cols + 7) / 8, units = tokens * upr;
  for (int64_t u = int64_t(blockIdx.x) * kRowThreads + threadIdx.x; u - (threadIdx.x & 31) < units;
       u += int64_t(gridDim.x) * kRowThreads) {  // (whole warps)
    const bool live = u < units;
    const int64_t t = live ? quotient_of_unit(u, upr) : 0, c = live ? (u - t * upr) * 8 : 0;
    const uint4 v = live ? load8_any(x + t * ldx, c, cols) : make_uint4(0, 0, 0, 0);
    for (int j = 0; j < k; ++j) {
      const int d = live ? pos[t * k + j] : -1;
      // (lanes of two tokens may meet: one has a row where the other has none)
      store8_any(xs + int64_t(d) * ldxs, c, cols, v, d >= 0 && d < rows);
    }
  }
}

constexpr int kFewPairs = 1024;  // that every CTA of few_rows_out_kernel looks at by itself

// The same with the sort, for few pairs: a CTA a token and kRowThreads pieces of its row. The row of a pair is the number of
// pairs that come before it, which a warp counts over all of them; an expert's first row likewise. (Any id >= experts
// is in no count: e is at most experts.)
template <typename U>
__global__ void __launch_bounds__(kRowThreads)
few_rows_out_kernel(const U* __restrict__ x, int64_t ldx, int64_t pieces, const int32_t* __restrict__ ids, int pairs, int k,
                    int experts, int* __restrict__ pos, int* __restrict__ offsets, U* __restrict__ xs, int64_t ldxs) {
  __shared__ int row_of[kMaxChosen];
  __shared__ int id_of[kFewPairs];
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t t = blockIdx.x, c = int64_t(blockIdx.y) * kRowThreads + threadIdx.x;
  const bool live = pairs > 0 && c < pieces;
  U v = {};
  if (live) v = x[t * ldx + c];  // under way while the rows are counted
  for (int i = threadIdx.x; i < pairs; i += kRowThreads) id_of[i] = ids[i];
  __syncthreads();
  // kept pairs of experts before e, and those of e before pair p, by a warp
  auto before = [&](int e, int p) {
    int n = 0;
    for (int i = lane; i < pairs; i += 32) {
      const int id = id_of[i];
      n += (id >= 0 && id < e) || (id == e && i < p);
    }
    return __reduce_add_sync(0xffffffffu, n);
  };
  for (int j = warp; pairs > 0 && j < k; j += kRowThreads / 32) {
    const int p = int(t) * k + j, e = id_of[p];
    const int n = e >= 0 && e < experts ? before(e, p) : -1;
    if (lane == 0) {
      row_of[j] = n;
      if (blockIdx.y == 0) pos[p] = n;
    }
  }
  const int ctas = int(gridDim.x * gridDim.y), cta = int(blockIdx.y * gridDim.x + blockIdx.x);
  if (pairs <= 64) {  // a thread an expert, the last CTAs first: the first ones' warps count rows
    for (int e = (ctas - 1 - cta) * kRowThreads + int(threadIdx.x); e <= experts; e += ctas * kRowThreads) {
      int n = 0;
      for (int i = 0; i < pairs; ++i) n += id_of[i] >= 0 && id_of[i] < e;
      offsets[e] = n;
    }
  } else {
    for (int e = cta * (kRowThreads / 32) + warp; e <= experts; e += ctas * (kRowThreads / 32)) {
      const int n = before(e, 0);
      if (lane == 0) offsets[e] = n;
    }
  }
  __syncthreads();
  if (!live) return;
  for (int j = 0; j < k; ++j) {
    const int d = row_of[j];
    if (d >= 0) xs[int64_t(d) * ldxs + c] = v;
  }
}

// Rows pass in pieces of kPiece bytes on boundaries of as many: 16, or 4 where the rows do not allow it. bf16 rows that start
// off 4-byte boundaries (kPiece 2) pass in whole 16-byte pieces that are shifted into place, stores by whole warps (store8_any).
template <typename T, int kPiece>
constexpr int kColsOf = (kPiece == 4 ? 4 : 16) / int(sizeof(T));

// The columns of a piece as they are held, as fp32 and back.
__device__ __forceinline__ void values_of(uint4 v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) f[2 * i] = bf16_lo(w[i]), f[2 * i + 1] = bf16_hi(w[i]);
}
__device__ __forceinline__ void values_of(uint4 v, float (&f)[4]) {
  f[0] = __uint_as_float(v.x), f[1] = __uint_as_float(v.y), f[2] = __uint_as_float(v.z), f[3] = __uint_as_float(v.w);
}
__device__ __forceinline__ void values_of(uint32_t v, float (&f)[2]) { f[0] = bf16_lo(v), f[1] = bf16_hi(v); }
__device__ __forceinline__ void values_of(uint32_t v, float (&f)[1]) { f[0] = __uint_as_float(v); }
__device__ __forceinline__ uint4 held(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}
__device__ __forceinline__ uint4 held(const float (&f)[4]) {
  return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}
__device__ __forceinline__ uint32_t held(const float (&f)[2]) { return pack_bf16x2(f[0], f[1]); }
__device__ __forceinline__ uint32_t held(const float (&f)[1]) { return __float_as_uint(f[0]); }

// (kPiece 2: as loaded, shifted into place where they are used: until then more loads go out)
template <int kPiece>
struct HeldAs {
  using type = uint4;
  static __device__ __forceinline__ uint4 zero() { return make_uint4(0, 0, 0, 0); }
};
template <>
struct HeldAs<4> {
  using type = uint32_t;
  static __device__ __forceinline__ uint32_t zero() { return 0u; }
};
template <>
struct HeldAs<2> {
  using type = Raw8;
  static __device__ __forceinline__ Raw8 zero() { return Raw8{make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)}; }
};
// Where the values of a row start in their pieces.
template <int kPiece, typename T>
__device__ __forceinline__ int start_of(const T* row) {
  return kPiece == 2 ? off_piece(reinterpret_cast<const uint16_t*>(row)) : 0;
}
template <int kPiece, typename T>
__device__ __forceinline__ typename HeldAs<kPiece>::type load_cols(const T* row, int64_t c, int64_t cols) {
  if constexpr (kPiece == 2)
    return load8_raw(reinterpret_cast<const uint16_t*>(row), start_of<kPiece>(row), int(c), int(cols));
  else
    return __ldcs(reinterpret_cast<const typename HeldAs<kPiece>::type*>(row + c));
}
template <int kPiece, int kN>
__device__ __forceinline__ void values_at(const typename HeldAs<kPiece>::type& v, int start, int64_t c, int64_t cols, float (&f)[kN]) {
  if constexpr (kPiece == 2)
    values_of(values8(v, start, int(c), int(cols)), f);
  else
    values_of(v, f);
}
template <int kPiece, typename T, typename U>
__device__ __forceinline__ void store_cols(T* row, int64_t c, int64_t cols, U v, bool live) {
  if constexpr (kPiece == 2)
    store8_any(reinterpret_cast<uint16_t*>(row), c, cols, v, live);
  else if (live)
    __stcs(reinterpret_cast<U*>(row + c), v);
}

template <int kPiece>
constexpr int kRowBatch = kPiece == 2 ? 4 : 8;  // rows' pieces that a thread has under way

// y[t] = sum_j w[t, j] ys[pos[t, j]] (weights null: 1) over the pairs that have a row, in the order of j, in fp32, the columns
// of a piece a thread. kB: rows at a time, one to eight; where k <= kB < 8, as many columns more: a thread has eight loads
// under way (one at a time: 251 us for the two gradients below, eight 171, then). Bounds: HBM (8192 tokens of eight rows of 2048
// bf16, 47 us, 6.4 TB/s).
template <typename T, int kPiece, int kB>
__global__ void __launch_bounds__(kRowThreads, kPiece == 2 ? 3 : 4)
rows_back_kernel(const T* __restrict__ ys, int64_t ldys, int64_t rows, const int* __restrict__ pos,
                 const float* __restrict__ weights, int k, int64_t tokens, int64_t cols, T* __restrict__ y, int64_t ldy) {
  constexpr int kN = kColsOf<T, kPiece>, kP = kRowBatch<kPiece> / kB;
  using Held = typename HeldAs<kPiece>::type;
  pdl_trigger();
  pdl_wait();
  const int64_t upr = (cols + kN - 1) / kN, units = tokens * upr;
  for (int64_t u0 = int64_t(blockIdx.x) * kRowThreads * kP + threadIdx.x; u0 - (threadIdx.x & 31) < units;
       u0 += int64_t(gridDim.x) * kRowThreads * kP) {  // (whole warps)
    int64_t t[kP], c[kP];
    bool live[kP];
    Held v[kP][kB];
    int start[kP][kB];
    float w[kP][kB], acc[kN];
    auto load = [&](int p, int j0) {
#pragma unroll
      for (int j = 0; j < kB; ++j) {
        const int d = live[p] && j0 + j < k ? pos[t[p] * k + j0 + j] : -1;
        const bool in = d >= 0 && d < rows;
        w[p][j] = in ? (weights ? weights[t[p] * k + j0 + j] : 1.0f) : 0.0f;
        start[p][j] = start_of<kPiece>(ys + (in ? int64_t(d) * ldys : 0));
        v[p][j] = in ? load_cols<kPiece>(ys + int64_t(d) * ldys, c[p], cols) : HeldAs<kPiece>::zero();
      }
    };
    auto add = [&](int p) {
#pragma unroll
      for (int j = 0; j < kB; ++j) {
        float f[kN];
        values_at<kPiece>(v[p][j], start[p][j], c[p], cols, f);
#pragma unroll
        for (int i = 0; i < kN; ++i) acc[i] = fmaf(w[p][j], f[i], acc[i]);
      }
    };
#pragma unroll
    for (int p = 0; p < kP; ++p) {
      const int64_t u = u0 + p * kRowThreads;
      live[p] = u < units;
      t[p] = live[p] ? quotient_of_unit(u, upr) : 0;
      c[p] = live[p] ? (u - t[p] * upr) * kN : 0;
      load(p, 0);
    }
#pragma unroll
    for (int p = 0; p < kP; ++p) {
#pragma unroll
      for (int i = 0; i < kN; ++i) acc[i] = 0.0f;
      add(p);
      if constexpr (kP == 1)
        for (int j0 = kB; j0 < k; j0 += kB) {
          load(p, j0);
          add(p);
        }
      store_cols<kPiece>(y + t[p] * ldy, c[p], cols, held(acc), live[p]);
    }
  }
}

// The gradient of rows_back: dys[pos[t, j]] = w[t, j] dy[t], dw[t, j] = <dy[t], ys[pos[t, j]]> (0 for a pair without a
// row), fp32 sums in a fixed order. dys may be ys. blockDim.x threads a token (a power of two from 32), blockDim.y tokens a
// CTA. kB: pairs at a time; where there are few, as many columns more. Bounds: HBM's reads and writes in turn (8192 tokens of
// eight rows of 2048 bf16, 90 us, 6.3 TB/s; 101 at four CTAs an SM, with spills). CTAs that stay, with the pairs held by lanes, took
// 197 us for both gradients against 171, then.
template <typename T, int kPiece, int kB>
__global__ void __launch_bounds__(kRowThreads, kB == 8 || kPiece == 2 ? 3 : 4)
rows_back_grad_kernel(const T* __restrict__ dy, int64_t lddy, const T* ys, int64_t ldys, int64_t rows,
                      const int* __restrict__ pos, const float* __restrict__ weights, int k, int64_t tokens, int64_t cols,
                      T* dys, int64_t lddys, float* __restrict__ dw) {
  constexpr int kN = kColsOf<T, kPiece>, kP = kB < 4 ? 4 / kB : 1;
  using Held = typename HeldAs<kPiece>::type;
  __shared__ float part[kRowThreads / 32][kB];
  pdl_trigger();
  pdl_wait();
  const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t step = int64_t(gridDim.x) * blockDim.y, wide = int64_t(blockDim.x) * kN;
  for (int64_t t0 = int64_t(blockIdx.x) * blockDim.y; t0 < tokens; t0 += step) {
    const int64_t t = t0 + threadIdx.y;
    for (int j0 = 0; j0 < k; j0 += kB) {
      float sum[kB] = {};
      if (t < tokens) {
        int d[kB];
        float w[kB];
#pragma unroll
        for (int j = 0; j < kB; ++j) {
          d[j] = j0 + j < k ? pos[t * k + j0 + j] : -1;
          if (d[j] >= rows) d[j] = -1;
          w[j] = d[j] >= 0 ? weights[t * k + j0 + j] : 0.0f;
        }
        for (int64_t c0 = int64_t(threadIdx.x) * kN; c0 - int64_t(lane) * kN < cols; c0 += wide * kP) {  // (whole warps)
          Held g[kP], v[kP][kB];
#pragma unroll
          for (int p = 0; p < kP; ++p) {
            const int64_t c = c0 + p * wide;
            g[p] = c < cols ? load_cols<kPiece>(dy + t * lddy, c, cols) : HeldAs<kPiece>::zero();
#pragma unroll
            for (int j = 0; j < kB; ++j)
              v[p][j] = c < cols && d[j] >= 0 ? load_cols<kPiece>(ys + int64_t(d[j]) * ldys, c, cols) : HeldAs<kPiece>::zero();
          }
#pragma unroll
          for (int p = 0; p < kP; ++p) {
            float h[kN];
            const int64_t c = c0 + p * wide;
            values_at<kPiece>(g[p], start_of<kPiece>(dy + t * lddy), c, cols, h);
#pragma unroll
            for (int j = 0; j < kB; ++j) {
              if (d[j] < 0) continue;  // (of the token: the whole warp)
              float f[kN], o[kN];
              values_at<kPiece>(v[p][j], start_of<kPiece>(ys + int64_t(d[j]) * ldys), c, cols, f);
#pragma unroll
              for (int i = 0; i < kN; ++i) {
                sum[j] = fmaf(h[i], f[i], sum[j]);
                o[i] = w[j] * h[i];
              }
              store_cols<kPiece>(dys + int64_t(d[j]) * lddys, c, cols, held(o), c < cols);
            }
          }
        }
      }
#pragma unroll
      for (int j = 0; j < kB; ++j) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], o);
        if (lane == 0) part[threadIdx.y * warps + warp][j] = sum[j];
      }
      __syncthreads();
      if (t < tokens && threadIdx.x < kB && j0 + int(threadIdx.x) < k) {
        float v = 0.0f;
        for (int i = 0; i < warps; ++i) v += part[threadIdx.y * warps + i][threadIdx.x];
        dw[t * k + j0 + threadIdx.x] = v;
      }
      __syncthreads();
    }
  }
}

}  // namespace moe
}  // namespace fp8k
