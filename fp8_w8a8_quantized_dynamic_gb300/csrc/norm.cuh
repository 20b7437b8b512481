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

#include "any_rows.cuh"
#include "block_gemm.h"
#include "device_common.cuh"
#include "tcgen05.cuh"

namespace fp8k {
namespace norm {

constexpr int kUnit = 16;       // adjacent columns of a thread: eight lanes hold a block of 128
constexpr int kMaxThreads = 1024;
constexpr int kMaxUnits = 2;
constexpr int kMaxCols = kMaxThreads * kMaxUnits * kUnit;

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
  float scale, eps, w_offset, inv_cols;
  uint16_t* r;               // may be null
  int64_t ldro;
  uint16_t* n;               // may be null
  int64_t ldn;
  uint8_t* q;                // may be null
  int64_t ldq;
  float* s;
  int64_t lds;
  int vec;   // all rows start on 16-byte boundaries and are whole eights
  int wide;  // .. on 32-byte boundaries and are whole sixteens
};

// A unit as it is held, and as fp32 in packed pairs: the arithmetic below takes two values at a time.
struct Held {
  uint32_t w[8];
};
struct Values {
  uint64_t p[8];
};
__device__ __forceinline__ Values values_of(const Held& h) {
  Values v;
#pragma unroll
  for (int i = 0; i < 8; ++i) v.p[i] = pack_f32x2(bf16_lo(h.w[i]), bf16_hi(h.w[i]));
  return v;
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
__device__ __forceinline__ Held zeros() {
  Held h;
#pragma unroll
  for (int i = 0; i < 8; ++i) h.w[i] = 0;
  return h;
}
__device__ __forceinline__ void put8(Held& h, int at, uint4 v) {
  h.w[at] = v.x, h.w[at + 1] = v.y, h.w[at + 2] = v.z, h.w[at + 3] = v.w;
}

// (not through the read-only path: r may be written over y or the residual)
__device__ __forceinline__ uint4 load_16(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

// A unit from column c < cols of a row that starts and ends anywhere, zeros from cols on: the two or three whole 16-byte
// pieces that hold its values (each holds one of the row's, so that all of it may be read), shifted into place. The shift is
// one for the row.
__device__ __forceinline__ Held load_unit_any(const uint16_t* row, int c, int cols) {
  const uint16_t* first = row + c;
  const int shift = int(reinterpret_cast<uintptr_t>(first) >> 1) & 7;
  const uint4* piece = reinterpret_cast<const uint4*>(first - shift);
  const int n = min(kUnit, cols - c);
  uint32_t w[12];
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const uint4 v = 8 * i - shift < n ? load_piece(piece + i) : make_uint4(0, 0, 0, 0);
    w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
  }
  if (shift != 0) {
#pragma unroll
    for (int i = 0; i < 10; ++i) w[i] = shift & 4 ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < 9; ++i) w[i] = shift & 2 ? w[i + 1] : w[i];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], shift & 1 ? 16 : 0);
  }
  if (n < kUnit) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = 2 * i + 1 < n ? w[i] : 2 * i < n ? w[i] & 0xFFFFu : 0u;
  }
  Held h;
#pragma unroll
  for (int i = 0; i < 8; ++i) h.w[i] = w[i];
  return h;
}

// A unit of a row from column c < cols on, zeros from cols on. kVec: see Params::vec.
template <bool kVec>
__device__ __forceinline__ Held load_unit(const uint16_t* row, int c, int cols, int wide) {
  if constexpr (!kVec) return load_unit_any(row, c, cols);
  Held h;
  if (wide) {
    asm volatile("ld.global.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(h.w[0]), "=r"(h.w[1]), "=r"(h.w[2]), "=r"(h.w[3]), "=r"(h.w[4]), "=r"(h.w[5]), "=r"(h.w[6]),
                   "=r"(h.w[7]) : "l"(row + c));
  } else {
    put8(h, 0, load_16(row + c));
    put8(h, 4, c + 8 < cols ? load_16(row + c + 8) : make_uint4(0, 0, 0, 0));
  }
  return h;
}
// The same of a weight, which stays in L1 for the CTA's next rows.
template <bool kVec>
__device__ __forceinline__ Held load_weights(const uint16_t* w, int c, int cols) {
  if constexpr (!kVec) return load_unit_any(w, c, cols);
  Held h;
  put8(h, 0, __ldg(reinterpret_cast<const uint4*>(w + c)));
  put8(h, 4, c + 8 < cols ? __ldg(reinterpret_cast<const uint4*>(w + c + 8)) : make_uint4(0, 0, 0, 0));
  return h;
}
// The units of a warp's lanes as bf16, each from its column c on; rows that start and end anywhere by whole warps.
template <bool kVec>
__device__ __forceinline__ void store_unit(uint16_t* row, int c, int cols, int wide, const Values& v) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = cvt_bf16x2(v.p[i]);
  if constexpr (!kVec) {
    const int lane = threadIdx.x & 31;
    store16_run(row, c, cols, make_uint4(w[0], w[1], w[2], w[3]), make_uint4(w[4], w[5], w[6], w[7]), c < cols, lane > 0,
                lane < 31 && c + kUnit < cols);
  } else if (c >= cols) {
    return;
  } else if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
                 :: "l"(row + c), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    *reinterpret_cast<uint4*>(row + c) = make_uint4(w[0], w[1], w[2], w[3]);
    if (c + 8 < cols) *reinterpret_cast<uint4*>(row + c + 8) = make_uint4(w[4], w[5], w[6], w[7]);
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
  if constexpr (kThreads >= 128) {
#pragma unroll
    for (int i = 0; i < kThreads / 128; ++i) {
      const float4 f = reinterpret_cast<const float4*>(mine)[i];
      v += (f.x + f.y) + (f.z + f.w);
    }
  } else {
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) v += mine[i];
  }
  return v;
}

// Sum of the squares of factor * v over the CTA's row.
template <int kThreads, int kUnits>
__device__ __forceinline__ float squares(const Values (&v)[kUnits], float factor, float (&red)[2][kThreads / 32], int& turn) {
  uint64_t ss[2] = {0, 0};
  const uint64_t f = both(factor);
#pragma unroll
  for (int i = 0; i < kUnits; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint64_t x = factor == 1.0f ? v[i].p[j] : mul_f32x2(v[i].p[j], f);
      ss[j & 1] = fma_f32x2(x, x, ss[j & 1]);
    }
  const uint64_t s = add_f32x2(ss[0], ss[1]);
  return block_sum<kThreads>(lo_of(s) + hi_of(s), red, turn);
}

// 1 / sqrt(mean v^2 + eps) of the CTA's row, the root correctly rounded (the fast one, two units off, takes no less time here).
// Squares of bf16's range may pass fp32's, and where the mean and eps are below 2^-100 they may lose bits that count: then once
// more of v 2^-80 (eps is nothing beside them) or v 2^60.
template <int kThreads, int kUnits>
__device__ __forceinline__ float inverse_rms(const Values (&v)[kUnits], const Params& p, float (&red)[2][kThreads / 32],
                                             int& turn) {
  const float ss = squares<kThreads, kUnits>(v, 1.0f, red, turn);
  const float mean = fmaf(ss, p.inv_cols, p.eps);
  if (mean >= 0x1p-100f && ss <= 0x1.fffffep127f) return __frsqrt_rn(mean);
  const float f = mean < 0x1p-100f ? 0x1p60f : 0x1p-80f, eps = mean < 0x1p-100f ? p.eps * 0x1p120f : 0.0f;
  return __frsqrt_rn(fmaf(squares<kThreads, kUnits>(v, f, red, turn), p.inv_cols, eps)) * f;
}

// A thread's raw values of one row.
template <int kUnits, bool kGate>
struct Raw {
  Held y[kUnits], res[kUnits], gate[kGate ? kUnits : 1];
};

template <int kThreads, int kUnits, bool kGate, bool kVec>
__device__ __forceinline__ void load_row(Raw<kUnits, kGate>& in, const Params& p, int64_t row) {
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const int c = (i * kThreads + threadIdx.x) * kUnit;
    in.y[i] = in.res[i] = zeros();
    if constexpr (kGate) in.gate[i] = zeros();
    if (c < p.cols) {
      in.y[i] = load_unit<kVec>(p.y + row * p.ldy, c, p.cols, p.wide);
      if (p.residual) in.res[i] = load_unit<kVec>(p.residual + row * p.ldr, c, p.cols, p.wide);
      if constexpr (kGate) in.gate[i] = load_unit<kVec>(p.gate + row * p.ldg, c, p.cols, p.wide);
    }
  }
}

template <int kThreads, int kUnits>
constexpr bool kAhead = kThreads * kUnits < 2048;  // else a row in fp32 alone takes the registers
// CTAs of an SM, by the registers that a row takes.
constexpr int ctas_of(int threads, int units) { return std::max(1, 1024 / (threads * units)); }

// The larger magnitude; a NaN stays one.
__device__ __forceinline__ float larger(float a, float b) {
  float d;
  asm("max.NaN.xorsign.abs.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// The scale of the 128 columns that eight lanes hold.
__device__ __forceinline__ float block_scale(const Values& v) {
  float m = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = larger(m, larger(lo_of(v.p[j]), hi_of(v.p[j])));
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) m = larger(m, __shfl_xor_sync(0xffffffffu, m, o));
  return scale_from_amax<kFmtE4M3>(fabsf(m));
}

// Codes of a unit under scale s; the sign of zero is kept.
__device__ __forceinline__ uint4 codes_of(const Values& v, float s) {
  const ExactScale k = make_exact_scale(s);
  uint32_t code[4];
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    const uint64_t a = v.p[2 * h], b = v.p[2 * h + 1];
    code[h] = quant4_exact_f32<kFmtE4M3>(a, b, k, s);
    const uint32_t lo = __byte_perm(uint32_t(a), uint32_t(a >> 32), 0x0073);
    const uint32_t hi = __byte_perm(uint32_t(b), uint32_t(b >> 32), 0x0073);
    code[h] = (code[h] & 0x7F7F7F7Fu) | (__byte_perm(lo, hi, 0x5410) & 0x80808080u);
  }
  return make_uint4(code[0], code[1], code[2], code[3]);
}

// A CTA takes every gridDim.x-th row. The loads of its next row are under way while it sums, joins and stores the one
// in its registers (16384 x 4096: 129 us without, 110 with, then). Sixteen adjacent columns a thread make 32-byte accesses and a
// block's scale one of eight lanes (95 us in 16-byte accesses, 75 so).
// Bounds: HBM for the plain form (16384 x 4096 to r and codes, 75 us, 6.2 TB/s); with both norms and a gate the two sums' barriers
// and the arithmetic beside it (4096 x 8192, 57 us, 5.3 TB/s, 59 percent of the issue slots); a launch and its chain of loads, two
// sums and stores for few rows (one of 4096, 2.3 us). Rows that start anywhere pay for their shifts (5615 x 2997, 53 us, 2.8 TB/s).
template <int kThreads, int kUnits, bool kPost, bool kGate, bool kVec>
__global__ void __launch_bounds__(kThreads, ctas_of(kThreads, kUnits))
residual_norm_kernel(const __grid_constant__ Params p) {
  __shared__ __align__(16) float red[2][kThreads / 32];
  pdl_trigger();
  const int cols = p.cols;
  auto col_of = [&](int i) { return (i * kThreads + int(threadIdx.x)) * kUnit; };
  // v * inv * (w_offset + w)
  auto scaled = [&](const uint16_t* w, int i, Values& v, float inv) {
    Values f = values_of(col_of(i) < cols ? load_weights<kVec>(w, col_of(i), cols) : zeros());
    if (p.w_offset != 0.0f) {
#pragma unroll
      for (int j = 0; j < 8; ++j) f.p[j] = add_f32x2(f.p[j], both(p.w_offset));
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) v.p[j] = mul_f32x2(mul_f32x2(v.p[j], both(inv)), f.p[j]);
  };
  pdl_wait();
  int turn = 0;
  Raw<kUnits, kGate> in;
  int64_t row = blockIdx.x;
  if (kAhead<kThreads, kUnits> && row < p.rows) load_row<kThreads, kUnits, kGate, kVec>(in, p, row);
  for (; row < p.rows; row += gridDim.x) {
    if (!kAhead<kThreads, kUnits>) load_row<kThreads, kUnits, kGate, kVec>(in, p, row);
    Values v[kUnits];
#pragma unroll
    for (int i = 0; i < kUnits; ++i) v[i] = values_of(in.y[i]);
    if constexpr (kPost) {
      const float inv = inverse_rms<kThreads, kUnits>(v, p, red, turn);
#pragma unroll
      for (int i = 0; i < kUnits; ++i) scaled(p.post_w, i, v[i], inv);
    }
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      if constexpr (kGate) {
        const Values f = values_of(in.gate[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i].p[j] = mul_f32x2(v[i].p[j], f.p[j]);
      }
      const Values f = values_of(in.res[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i].p[j] = fma_f32x2(both(p.scale), v[i].p[j], f.p[j]);
    }
    if (kAhead<kThreads, kUnits> && row + gridDim.x < p.rows)
      load_row<kThreads, kUnits, kGate, kVec>(in, p, row + gridDim.x);
    if (p.r) {
#pragma unroll
      for (int i = 0; i < kUnits; ++i)
        store_unit<kVec>(p.r + row * p.ldro, col_of(i), cols, p.wide, v[i]);
    }
    if (!p.pre) continue;
    const float inv = inverse_rms<kThreads, kUnits>(v, p, red, turn);
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const int c = col_of(i);
      scaled(p.w, i, v[i], inv);
      if (c + kUnit > cols) {  // nothing past the last column counts
#pragma unroll
        for (int j = 0; j < 8; ++j)
          v[i].p[j] = pack_f32x2(c + 2 * j < cols ? lo_of(v[i].p[j]) : 0.0f, c + 2 * j + 1 < cols ? hi_of(v[i].p[j]) : 0.0f);
      }
      if (p.n) store_unit<kVec>(p.n + row * p.ldn, c, cols, p.wide, v[i]);
      if (p.q) {
        const float s = block_scale(v[i]);
        const uint4 q = codes_of(v[i], s);
        if (c < p.ldq) *reinterpret_cast<uint4*>(p.q + row * p.ldq + c) = q;
        if ((threadIdx.x & 7) == 0 && c < cols) p.s[int64_t(c / block::kBlock) * p.lds + row] = s;
      }
    }
    if (p.q)  // zeros to the end of a longer row
      for (int64_t c = (int64_t(kUnits) * kThreads + threadIdx.x) * kUnit; c < p.ldq; c += kThreads * kUnit)
        *reinterpret_cast<uint4*>(p.q + row * p.ldq + c) = make_uint4(0, 0, 0, 0);
  }
}

}  // namespace norm
}  // namespace fp8k
