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
  int vec;  // all rows start on 16-byte boundaries and are whole eights
};

// Eight fp32 values in four packed pairs: the arithmetic below takes two at a time.
struct Eight {
  uint64_t p[4];
};
__device__ __forceinline__ Eight unpack8(uint4 v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  Eight e;
#pragma unroll
  for (int i = 0; i < 4; ++i) e.p[i] = pack_f32x2(bf16_lo(w[i]), bf16_hi(w[i]));
  return e;
}
__device__ __forceinline__ uint64_t both(float x) { return pack_f32x2(x, x); }
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint32_t cvt_bf16x2(uint64_t p) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi_of(p)), "f"(lo_of(p)));
  return d;
}

// kVec: rows start on 16-byte boundaries and are whole eights. Else single values, zeros from cols on.
template <bool kVec>
__device__ __forceinline__ uint4 load8(const uint16_t* row, int c, int cols) {
  return kVec ? ld_nc_v4(row + c) : load8_bf16(row, c, cols, 0);
}
template <bool kVec>
__device__ __forceinline__ void store8(uint16_t* row, int c, int cols, const Eight& e) {
  if constexpr (kVec) {
    *reinterpret_cast<uint4*>(row + c) =
        make_uint4(cvt_bf16x2(e.p[0]), cvt_bf16x2(e.p[1]), cvt_bf16x2(e.p[2]), cvt_bf16x2(e.p[3]));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w = cvt_bf16x2(e.p[i]);
      if (c + 2 * i < cols) row[c + 2 * i] = uint16_t(w);
      if (c + 2 * i + 1 < cols) row[c + 2 * i + 1] = uint16_t(w >> 16);
    }
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

// Sum of the squares of factor * v over the CTA's row.
template <int kThreads, int kUnits>
__device__ __forceinline__ float squares(const Eight (&v)[kUnits], float factor, float (&red)[2][kThreads / 32], int& turn) {
  uint64_t ss[2] = {0, 0};
  const uint64_t f = both(factor);
#pragma unroll
  for (int i = 0; i < kUnits; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint64_t x = factor == 1.0f ? v[i].p[j] : mul_f32x2(v[i].p[j], f);
      ss[j & 1] = fma_f32x2(x, x, ss[j & 1]);
    }
  const uint64_t s = add_f32x2(ss[0], ss[1]);
  return block_sum<kThreads>(lo_of(s) + hi_of(s), red, turn);
}

// 1 / sqrt(mean v^2 + eps) of the CTA's row. Squares of bf16's range may pass fp32's: then once more of v 2^-80.
template <int kThreads, int kUnits>
__device__ __forceinline__ float inverse_rms(const Eight (&v)[kUnits], const Params& p, float (&red)[2][kThreads / 32],
                                             int& turn) {
  float ss = squares<kThreads, kUnits>(v, 1.0f, red, turn);
  if (ss <= 0x1.fffffep127f) return __frcp_rn(__fsqrt_rn(__fdiv_rn(ss, float(p.cols)) + p.eps));
  ss = squares<kThreads, kUnits>(v, 0x1p-80f, red, turn);
  return __frcp_rn(__fsqrt_rn(__fdiv_rn(ss, float(p.cols)))) * 0x1p-80f;
}

// A thread's raw values of one row.
template <int kUnits, bool kGate>
struct Raw {
  uint4 y[kUnits], res[kUnits], gate[kGate ? kUnits : 1];
};

template <int kThreads, int kUnits, bool kGate, bool kVec>
__device__ __forceinline__ void load_row(Raw<kUnits, kGate>& in, const Params& p, int64_t row) {
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const int c = (i * kThreads + threadIdx.x) * 8;
    in.y[i] = in.res[i] = make_uint4(0, 0, 0, 0);
    if constexpr (kGate) in.gate[i] = make_uint4(0, 0, 0, 0);
    if (c < p.cols) {
      in.y[i] = load8<kVec>(p.y + row * p.ldy, c, p.cols);
      if (p.residual) in.res[i] = load8<kVec>(p.residual + row * p.ldr, c, p.cols);
      if constexpr (kGate) in.gate[i] = load8<kVec>(p.gate + row * p.ldg, c, p.cols);
    }
  }
}

template <int kThreads, int kUnits>
constexpr bool kAhead = kThreads * kUnits < 4096;  // else a row in fp32 alone takes the registers
// CTAs of an SM, by the registers that a row takes.
constexpr int ctas_of(int threads, int units) {
  return units == 1 ? 1536 / threads : std::max(1, 2048 / (threads * units));
}

// Scales and reciprocals of a thread's units, each shared by the sixteen lanes that hold its 128 columns. Magnitudes
// compare as integers, which keeps a NaN. Units are shared out over the lanes as far as they go: in each exchange a lane
// keeps the maxima of half of them, computes the scale of the one it ends with, and all fetch theirs from it.
template <int kUnits>
__device__ __forceinline__ void block_scales(const Eight (&v)[kUnits], float (&s)[kUnits], float (&r)[kUnits]) {
  uint32_t m[kUnits];
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    m[i] = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      m[i] = max(m[i], max(uint32_t(v[i].p[j]) & 0x7FFFFFFFu, uint32_t(v[i].p[j] >> 32) & 0x7FFFFFFFu));
  }
  const int lane = threadIdx.x & 31;
  int left = kUnits;
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) {
    if (left > 1) {
      left >>= 1;
      const bool upper = (lane & o) != 0;
#pragma unroll
      for (int i = 0; i < kUnits / 2; ++i)
        if (i < left) {
          const uint32_t send = upper ? m[i] : m[i + left], keep = upper ? m[i + left] : m[i];
          m[i] = max(keep, __shfl_xor_sync(0xffffffffu, send, o));
        }
    } else {
      m[0] = max(m[0], __shfl_xor_sync(0xffffffffu, m[0], o));
    }
  }
  const float sc = scale_from_amax<kFmtE4M3>(__uint_as_float(m[0]));
  const float rc = __frcp_rn(sc);
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    // unit i's lanes: bit 3 of the lane is its highest index bit, bit 2 the next
    const int from = kUnits == 1 ? lane : (lane & 16) | (kUnits == 2 ? i << 3 : i << 2);
    s[i] = kUnits == 1 ? sc : __shfl_sync(0xffffffffu, sc, from);
    r[i] = kUnits == 1 ? rc : __shfl_sync(0xffffffffu, rc, from);
  }
}

// Codes of eight values under scale s with r = fl32(1 / s); the sign of zero is kept.
__device__ __forceinline__ uint2 codes8(const Eight& e, float s, float r) {
  ExactScale k;
  const float r_lo = fmaf(-s, r, 1.0f) * r;
  k.r2 = both(r);
  k.r_lo2 = both(r_lo);
  k.neg_s2 = both(-s);
  k.fast = s >= 0x1p-80f && s <= 0x1p100f;
  uint32_t code[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint64_t a = e.p[2 * h], b = e.p[2 * h + 1];
    code[h] = quant4_exact_f32<kFmtE4M3>(a, b, k, s);
    const uint32_t lo = __byte_perm(uint32_t(a), uint32_t(a >> 32), 0x0073);
    const uint32_t hi = __byte_perm(uint32_t(b), uint32_t(b >> 32), 0x0073);
    code[h] = (code[h] & 0x7F7F7F7Fu) | (__byte_perm(lo, hi, 0x5410) & 0x80808080u);
  }
  return make_uint2(code[0], code[1]);
}

// A CTA takes every gridDim.x-th row. The loads of its next row are under way while it sums, joins and stores the one
// in its registers.
template <int kThreads, int kUnits, bool kPost, bool kGate, bool kVec>
__global__ void __launch_bounds__(kThreads, ctas_of(kThreads, kUnits))
residual_norm_kernel(const __grid_constant__ Params p) {
  __shared__ float red[2][kThreads / 32];
  pdl_trigger();
  const int cols = p.cols;
  auto col_of = [&](int i) { return (i * kThreads + int(threadIdx.x)) * 8; };
  // v * inv * (w_offset + w)
  auto scaled = [&](const uint16_t* w, int i, Eight& v, float inv) {
    const int c = col_of(i);
    Eight f = unpack8(c < cols ? load8<kVec>(w, c, cols) : make_uint4(0, 0, 0, 0));
    if (p.w_offset != 0.0f) {
#pragma unroll
      for (int j = 0; j < 4; ++j) f.p[j] = add_f32x2(f.p[j], both(p.w_offset));
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) v.p[j] = mul_f32x2(mul_f32x2(v.p[j], both(inv)), f.p[j]);
  };
  pdl_wait();
  int turn = 0;
  Raw<kUnits, kGate> in;
  int64_t row = blockIdx.x;
  if (kAhead<kThreads, kUnits> && row < p.rows) load_row<kThreads, kUnits, kGate, kVec>(in, p, row);
  for (; row < p.rows; row += gridDim.x) {
    if (!kAhead<kThreads, kUnits>) load_row<kThreads, kUnits, kGate, kVec>(in, p, row);
    Eight v[kUnits];
#pragma unroll
    for (int i = 0; i < kUnits; ++i) v[i] = unpack8(in.y[i]);
    if constexpr (kPost) {
      const float inv = inverse_rms<kThreads, kUnits>(v, p, red, turn);
#pragma unroll
      for (int i = 0; i < kUnits; ++i) scaled(p.post_w, i, v[i], inv);
    }
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      if constexpr (kGate) {
        const Eight f = unpack8(in.gate[i]);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[i].p[j] = mul_f32x2(v[i].p[j], f.p[j]);
      }
      const Eight f = unpack8(in.res[i]);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[i].p[j] = fma_f32x2(both(p.scale), v[i].p[j], f.p[j]);
    }
    if (kAhead<kThreads, kUnits> && row + gridDim.x < p.rows)
      load_row<kThreads, kUnits, kGate, kVec>(in, p, row + gridDim.x);
    if (p.r) {
#pragma unroll
      for (int i = 0; i < kUnits; ++i)
        if (col_of(i) < cols) store8<kVec>(p.r + row * p.ldro, col_of(i), cols, v[i]);
    }
    if (!p.pre) continue;
    const float inv = inverse_rms<kThreads, kUnits>(v, p, red, turn);
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const int c = col_of(i);
      scaled(p.w, i, v[i], inv);
      if (c + 8 > cols) {  // nothing past the last column counts
#pragma unroll
        for (int j = 0; j < 4; ++j)
          v[i].p[j] = pack_f32x2(c + 2 * j < cols ? lo_of(v[i].p[j]) : 0.0f, c + 2 * j + 1 < cols ? hi_of(v[i].p[j]) : 0.0f);
      }
      if (p.n && c < cols) store8<kVec>(p.n + row * p.ldn, c, cols, v[i]);
    }
    if (p.q) {
      float s[kUnits], r[kUnits];
      block_scales<kUnits>(v, s, r);
#pragma unroll
      for (int i = 0; i < kUnits; ++i) {
        const int c = col_of(i);
        if (c < p.ldq) *reinterpret_cast<uint2*>(p.q + row * p.ldq + c) = codes8(v[i], s[i], r[i]);
        if ((threadIdx.x & 15) == 0 && c < cols) p.s[int64_t(c / block::kBlock) * p.lds + row] = s[i];
      }
      // zeros to the end of a longer row
      for (int64_t c = (int64_t(kUnits) * kThreads + threadIdx.x) * 8; c < p.ldq; c += kThreads * 8)
        *reinterpret_cast<uint2*>(p.q + row * p.ldq + c) = make_uint2(0, 0);
    }
  }
}

}  // namespace norm
}  // namespace fp8k
