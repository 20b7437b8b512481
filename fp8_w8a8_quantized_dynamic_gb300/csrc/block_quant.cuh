// Block quantization for sm_103a: bf16 rows -> e4m3 codes with one scale per row and 128 columns
// (activations), bf16 matrices -> codes with one scale per 128 x 128 block (weights).
//
//   s = fl32(amax / 448) (1 when amax is 0),  q = e4m3(fl32(x / s))
//
// No scale depends on data outside its block, so one pass reads the input and writes the codes (2 bytes
// read and 1 written an element).
#pragma once

#include "block_gemm.h"
#include "device_common.cuh"

namespace fp8k {
namespace block {

constexpr int kQThreads = 256;

// Sixteen columns c .. c + 15 of a row (zero at and beyond cols).
struct Sixteen {
  uint4 a, b;
};
__device__ __forceinline__ Sixteen load16(const uint16_t* __restrict__ row, int64_t c, int64_t cols, int vec) {
  Sixteen v;
  if (vec && c + 16 <= cols) {
    v.a = ld_nc_v4(row + c);
    v.b = ld_nc_v4(row + c + 8);
  } else {
    v.a = load8_bf16(row, int(c), int(cols), 0);
    v.b = load8_bf16(row, int(c) + 8, int(cols), 0);
  }
  return v;
}

// Magnitudes compare as 16-bit integers, a NaN above infinity: a block with a NaN gets a NaN
// scale and so a NaN product, as the formula has it.
__device__ __forceinline__ uint32_t amax16(const Sixteen& v) { return abs_max_v4(abs_max_v4(0u, v.a), v.b); }

__device__ __forceinline__ uint4 codes16(const Sixteen& v, const ExactScale& k, float s) {
  const uint2 lo = quant8_exact<kFmtE4M3>(v.a, k, s, false), hi = quant8_exact<kFmtE4M3>(v.b, k, s, false);
  return make_uint4(lo.x, lo.y, hi.x, hi.y);
}

// Maximum over the eight lanes that hold one 128-column block.
__device__ __forceinline__ uint32_t max_of_eight(uint32_t m2) {
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) m2 = __vmaxu2(m2, __shfl_xor_sync(0xffffffffu, m2, o));
  return m2;
}

// A [rows, cols] -> q [rows or sorted rows, ldq], zero from cols on, s [K blocks][lds]. Eight lanes hold a
// block of a row, sixteen columns each. copies == 0: row r of A goes to row r. copies > 0: it goes to the
// rows pos[r * copies + j], j < copies (a negative one is skipped): the rows of many experts,
// each token quantized once. Bound by HBM: 32 registers a thread let eight CTAs on an SM, whose loads
// cover its latency: 16384 x 4096 back to back in 38.7 us (203 MB, 5.3 TB/s; five CTAs took a sixth more).
// Rows of 4095, which start anywhere, take two-byte loads: 74 us (66 to then 72 in whole words exchanged
// between lanes: not kept).
template <typename Idx>
__global__ void __launch_bounds__(kQThreads, 8)
quantize_rows_1x128_kernel(const uint16_t* __restrict__ a, int64_t rows, int64_t cols, int64_t ld, int vec,
                           uint8_t* __restrict__ q, int64_t ldq, float* __restrict__ s, int64_t lds,
                           const int* __restrict__ pos, int copies) {
  pdl_trigger();
  pdl_wait();
  const Idx upr = static_cast<Idx>((ldq + kBlock - 1) / kBlock) * 8;  // sixteen-column units of a row, whole blocks
  const Idx units = static_cast<Idx>(rows) * upr;
  const Idx stride = static_cast<Idx>(gridDim.x) * kQThreads;
  const Idx rounded = (units + 31) / 32 * 32;  // whole warps take part in the shuffles
  for (Idx u = static_cast<Idx>(blockIdx.x) * kQThreads + threadIdx.x; u < rounded; u += stride) {
    const int64_t r = u / upr;
    const int64_t i = u - static_cast<Idx>(r) * upr;
    const int64_t c = i * 16;
    Sixteen v = {};
    const bool in = u < units && c < cols;
    if (in) v = load16(a + r * ld, c, cols, vec);
    const float sc = scale_from_amax<kFmtE4M3>(u16x2_max_to_float(max_of_eight(amax16(v))));
    const ExactScale k = make_exact_scale(sc);
    const uint4 o = codes16(v, k, sc);
    if (u >= units) continue;
    if (copies == 0) {
      if (c < ldq) *reinterpret_cast<uint4*>(q + r * ldq + c) = o;
      if ((i & 7) == 0 && in) s[(i >> 3) * lds + r] = sc;
    } else {
      for (int j = 0; j < copies; ++j) {
        const int d = pos[r * copies + j];
        if (d < 0) continue;
        if (c < ldq) *reinterpret_cast<uint4*>(q + int64_t(d) * ldq + c) = o;
        if ((i & 7) == 0 && in) s[(i >> 3) * lds + d] = sc;
      }
    }
  }
}

// W [mats][N, K] -> q [mats][N, ldq], zero from K on, s [mats][N blocks][K blocks]. One CTA a 128 x 128
// block (past the last of K, to ldq: of zeros, without a scale): a thread holds half a row of it (64 columns)
// in registers between the maximum and the codes. Runs once, when weights are loaded, at 3.1 TB/s (128 x
// 2048 x 4096 in 1.03 ms, 28672 x 4096 in 113 us): each CTA loads, meets for the maximum and stores one
// block after the other, and nothing overlaps those but the SM's other CTAs.
__global__ void __launch_bounds__(kQThreads)
quantize_128x128_kernel(const uint16_t* __restrict__ w, int64_t mats, int64_t N, int64_t K, int64_t ld,
                        int64_t mat_stride, int vec, uint8_t* __restrict__ q, int64_t ldq, float* __restrict__ s) {
  __shared__ uint32_t red[kQThreads / 32];
  pdl_wait();
  const int64_t nb = (N + kBlock - 1) / kBlock, kb = (K + kBlock - 1) / kBlock, ldb = (ldq + kBlock - 1) / kBlock;
  for (int64_t blk = blockIdx.x; blk < mats * nb * ldb; blk += gridDim.x) {
    const int64_t m = blk / (nb * ldb), in = blk - m * nb * ldb;
    const int64_t j = in / ldb, b = in - j * ldb;
    const int64_t r = j * kBlock + (threadIdx.x >> 1);
    const int64_t c0 = b * kBlock + (threadIdx.x & 1) * 64;
    Sixteen v[4] = {};
    uint32_t m2 = 0;
    if (r < N) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (c0 + i * 16 < K) v[i] = load16(w + m * mat_stride + r * ld, c0 + i * 16, K, vec);
        m2 = __vmaxu2(m2, amax16(v[i]));
      }
    }
    uint32_t mx = max(m2 & 0xFFFFu, m2 >> 16);
    mx = __reduce_max_sync(0xffffffffu, mx);
    __syncthreads();  // the previous block's maxima have been read
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = mx;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kQThreads / 32; ++i) mx = max(mx, red[i]);
    const float sc = scale_from_amax<kFmtE4M3>(__uint_as_float(mx << 16));
    const ExactScale k = make_exact_scale(sc);
    if (threadIdx.x == 0 && b < kb) s[(m * nb + j) * kb + b] = sc;
    if (r < N) {
      uint8_t* dst = q + (m * N + r) * ldq;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (c0 + i * 16 < ldq) *reinterpret_cast<uint4*>(dst + c0 + i * 16) = codes16(v[i], k, sc);
    }
  }
}

}  // namespace block
}  // namespace fp8k
