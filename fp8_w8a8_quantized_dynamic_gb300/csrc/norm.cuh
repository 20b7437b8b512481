// Root-mean-square norms around a block, fused with its gate, residual and the block quantization:
//
//   t = y, or y / sqrt(mean y^2 + eps) * post_w        (the norm after the block)
//   r = residual + scale * gate * t                    (bf16 out)
//   n = r / sqrt(mean r^2 + eps) * w                   (the norm before the next block, of the unrounded r)
//   out: n as bf16, or s = fl32(amax / 448), q = e4m3(fl32(n / s)) per 128 columns
//
// One pass: a CTA holds a row in fp32 registers between the loads, the two sums and the stores.
#pragma once

#include <algorithm>

#include "block_gemm.h"
#include "device_common.cuh"
#include "tcgen05.cuh"

namespace fp8k {
namespace norm {

constexpr int kMaxThreads = 1024;
constexpr int kMaxUnits = 4;                          // eight columns each
constexpr int kMaxCols = kMaxThreads * kMaxUnits * 8;

struct Params {
  int64_t rows;
  int cols;
  const uint16_t* y;
  int64_t ldy;
  const uint16_t* post_w;    // may be null: no norm of y
  const uint16_t* gate;      // may be null; row stride 0: one gate a channel
  int64_t ldg;
  const uint16_t* residual;  // may be null
  int64_t ldr;
  const uint16_t* w;
  int pre;                   // n or the codes are wanted, else r alone
  float scale, eps, w_offset;
  uint16_t* r;               // may be null
  int64_t ldro;
  uint16_t* n;               // may be null
  int64_t ldn;
  uint8_t* q;                // may be null
  int64_t ldq;
  float* s;
  int64_t lds;
  int vec_y, vec_post, vec_gate, vec_res, vec_w, vec_r, vec_n;  // rows start on 16-byte boundaries
};

__device__ __forceinline__ void unpack8(uint4 v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) f[2 * i] = bf16_lo(w[i]), f[2 * i + 1] = bf16_hi(w[i]);
}

// Eight columns from c on (those before cols) as bf16.
__device__ __forceinline__ void store8_bf16(uint16_t* row, int c, int cols, int vec, const float (&f)[8]) {
  if (vec && c + 8 <= cols) {
    *reinterpret_cast<uint4*>(row + c) = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                                    pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < cols) row[c + i] = __bfloat16_as_ushort(__float2bfloat16_rn(f[i]));
  }
}

template <int kThreads>
__device__ __forceinline__ float block_sum(float v, float (&red)[2][kThreads / 32], int& turn) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  // sums take the two halves in turn: one barrier each is enough
  float(&mine)[kThreads / 32] = red[turn & 1];
  ++turn;
  if ((threadIdx.x & 31) == 0) mine[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.0f;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) v += mine[i];
  return v;
}

// 1 / sqrt(mean v^2 + eps) of the CTA's row. Squares of bf16's range may pass fp32's: then once more of v 2^-80.
template <int kThreads, int kUnits>
__device__ __forceinline__ float inverse_rms(const float (&v)[kUnits][8], const Params& p,
                                             float (&red)[2][kThreads / 32], int& turn) {
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < kUnits; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fmaf(v[i][j], v[i][j], ss);
  ss = block_sum<kThreads>(ss, red, turn);
  if (ss <= 0x1.fffffep127f) return __frcp_rn(__fsqrt_rn(__fdiv_rn(ss, float(p.cols)) + p.eps));
  ss = 0.0f;
#pragma unroll
  for (int i = 0; i < kUnits; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float x = v[i][j] * 0x1p-80f;
      ss = fmaf(x, x, ss);
    }
  ss = block_sum<kThreads>(ss, red, turn);
  return __frcp_rn(__fsqrt_rn(__fdiv_rn(ss, float(p.cols)))) * 0x1p-80f;
}

// A thread's raw values of one row.
template <int kUnits, bool kGate>
struct Raw {
  uint4 y[kUnits], res[kUnits], gate[kGate ? kUnits : 1];
};

template <int kThreads, int kUnits, bool kGate>
__device__ __forceinline__ void load_row(Raw<kUnits, kGate>& in, const Params& p, int64_t row) {
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const int c = (i * kThreads + threadIdx.x) * 8;
    in.y[i] = in.res[i] = make_uint4(0, 0, 0, 0);
    if constexpr (kGate) in.gate[i] = make_uint4(0, 0, 0, 0);
    if (c < p.cols) {
      in.y[i] = load8_bf16(p.y + row * p.ldy, c, p.cols, p.vec_y);
      if (p.residual) in.res[i] = load8_bf16(p.residual + row * p.ldr, c, p.cols, p.vec_res);
      if constexpr (kGate) in.gate[i] = load8_bf16(p.gate + row * p.ldg, c, p.cols, p.vec_gate);
    }
  }
}

template <int kThreads, int kUnits>
constexpr bool kAhead = kThreads * kUnits < 4096;  // else a row in fp32 alone takes the registers
// CTAs of an SM, by the registers that a row takes.
constexpr int ctas_of(int threads, int units) {
  return units == 1 ? 1536 / threads : std::max(1, 2048 / (threads * units));
}

// A CTA takes every gridDim.x-th row. The loads of its next row are under way while it sums, joins and stores the one
// in its registers.
template <int kThreads, int kUnits, bool kPost, bool kGate>
__global__ void __launch_bounds__(kThreads, ctas_of(kThreads, kUnits))
residual_norm_kernel(const __grid_constant__ Params p) {
  __shared__ float red[2][kThreads / 32];
  pdl_trigger();
  const int cols = p.cols;
  auto col_of = [&](int i) { return (i * kThreads + int(threadIdx.x)) * 8; };
  auto weights = [&](const uint16_t* w, int vec, int i, float (&f)[8]) {
    const int c = col_of(i);
    unpack8(c < cols ? load8_bf16(w, c, cols, vec) : make_uint4(0, 0, 0, 0), f);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] += p.w_offset;
  };
  pdl_wait();
  int turn = 0;
  Raw<kUnits, kGate> in;
  int64_t row = blockIdx.x;
  if (kAhead<kThreads, kUnits> && row < p.rows) load_row<kThreads>(in, p, row);
  for (; row < p.rows; row += gridDim.x) {
    if (!kAhead<kThreads, kUnits>) load_row<kThreads>(in, p, row);
    float v[kUnits][8];
#pragma unroll
    for (int i = 0; i < kUnits; ++i) unpack8(in.y[i], v[i]);
    if constexpr (kPost) {
      const float inv = inverse_rms<kThreads, kUnits>(v, p, red, turn);
#pragma unroll
      for (int i = 0; i < kUnits; ++i) {
        float f[8];
        weights(p.post_w, p.vec_post, i, f);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = v[i][j] * inv * f[j];
      }
    }
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      float f[8];
      if constexpr (kGate) {
        unpack8(in.gate[i], f);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] *= f[j];
      }
      unpack8(in.res[i], f);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = fmaf(p.scale, v[i][j], f[j]);
    }
    if (kAhead<kThreads, kUnits> && row + gridDim.x < p.rows) load_row<kThreads>(in, p, row + gridDim.x);
    if (p.r) {
#pragma unroll
      for (int i = 0; i < kUnits; ++i)
        if (col_of(i) < cols) store8_bf16(p.r + row * p.ldro, col_of(i), cols, p.vec_r, v[i]);
    }
    if (!p.pre) continue;
    const float inv = inverse_rms<kThreads, kUnits>(v, p, red, turn);
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const int c = col_of(i);
      float f[8];
      weights(p.w, p.vec_w, i, f);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = c + j < cols ? v[i][j] * inv * f[j] : 0.0f;
      if (p.n && c < cols) store8_bf16(p.n + row * p.ldn, c, cols, p.vec_n, v[i]);
      if (p.q) {
        // sixteen lanes hold a block of 128 columns; magnitudes compare as integers, which keeps a NaN
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(fabsf(v[i][j])));
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        const float sc = scale_from_amax<kFmtE4M3>(__uint_as_float(m));
        const ExactScale k = make_exact_scale(sc);
        uint32_t code[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float* x = &v[i][4 * h];
          code[h] = quant4_exact_f32<kFmtE4M3>(pack_f32x2(x[0], x[1]), pack_f32x2(x[2], x[3]), k, sc);
          // the sign of zero is kept
          const uint32_t lo = __byte_perm(__float_as_uint(x[0]), __float_as_uint(x[1]), 0x0073);
          const uint32_t hi = __byte_perm(__float_as_uint(x[2]), __float_as_uint(x[3]), 0x0073);
          code[h] = (code[h] & 0x7F7F7F7Fu) | (((lo & 0xFFFFu) | (hi << 16)) & 0x80808080u);
        }
        if (c < p.ldq) *reinterpret_cast<uint2*>(p.q + row * p.ldq + c) = make_uint2(code[0], code[1]);
        if ((threadIdx.x & 15) == 0 && c < cols) p.s[int64_t(c / block::kBlock) * p.lds + row] = sc;
      }
    }
    if (p.q)  // zeros to the end of a longer row
      for (int64_t c = (int64_t(kUnits) * kThreads + threadIdx.x) * 8; c < p.ldq; c += kThreads * 8)
        *reinterpret_cast<uint2*>(p.q + row * p.ldq + c) = make_uint2(0, 0);
  }
}

}  // namespace norm
}  // namespace fp8k
