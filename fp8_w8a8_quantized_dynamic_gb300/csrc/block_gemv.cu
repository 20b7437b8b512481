// Block-scaled FP8 GEMV for sm_103a: the product for few rows, bound by streaming the weights.
//
// A CTA of eight warps takes 16 weight rows at a time (kGemvSwiglu: 16 of gate and the same 16
// of up); the warps share out K in whole 128-wide blocks. A lane loads 16 bytes of two weight
// rows straight into the registers that mma.sync m16n8k32 takes as its A operand: its four words
// are the fragments of two MMAs under a permutation of k that the activations follow, so nothing
// passes through shared memory and nothing is rearranged. The loads run kDepth blocks ahead, over
// the ends of row groups, and the first ones are in flight before the kernel waits for its
// activations. Block partials are added, scaled, in fp32; the warps' sums meet in shared memory
// in a fixed order.
//
// Activations: each warp quantizes its own K slice of every row into its own shared memory (no
// barrier), or copies codes that a kernel before it wrote. Rows are 64 modulo 128 bytes apart, so
// a quarter warp's 16-byte reads (two rows of four) touch every bank once.

#include "block_gemv.h"

#include <algorithm>

#include "api_common.h"
#include "device_cache.h"
#include "device_common.cuh"
#include "tcgen05.cuh"

namespace fp8k {
namespace block {

constexpr int kGvWarps = 8;
constexpr int kGvThreads = kGvWarps * 32;
constexpr int kGvRows = 16;

struct GvParams {
  const void* a;
  int64_t lda;
  const float* s_a;
  int64_t lds_a;
  const int* row_src;
  int M;
  const RowTile* tiles;
  const int* n_tiles;
  const int32_t* ids;
  const float* weights;
  int pairs, experts;
  const uint8_t* qw;
  int64_t ldw;
  const float* s_w;
  int N, K, kb, nb;
  int groups;   // row groups of one matrix
  int kbw;      // K blocks of one warp
  int vec;      // activation rows are 16-byte aligned
  const uint16_t* bias;
  uint16_t* y;
  int64_t ldy;
  float* y32;
  int64_t ldy32;
};

__device__ __forceinline__ uint4 ld_stream_v4(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

__device__ __forceinline__ void mma_e4m3(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Sixteen values -> codes, any scale.
__device__ __forceinline__ uint4 codes_of_f32(const float (&x)[16], float s) {
  const ExactScale k = make_exact_scale(s);
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (k.fast) {
      const uint64_t p = pack_f32x2(x[4 * i], x[4 * i + 1]), q = pack_f32x2(x[4 * i + 2], x[4 * i + 3]);
      const uint64_t a = fma_f32x2(p, k.r2, mul_f32x2(p, k.r_lo2)), b = fma_f32x2(q, k.r2, mul_f32x2(q, k.r_lo2));
      w[i] = cvt_fp8x4<kFmtE4M3>(fma_f32x2(fma_f32x2(k.neg_s2, a, p), k.r2, a),
                                 fma_f32x2(fma_f32x2(k.neg_s2, b, q), k.r2, b));
    } else {
      w[i] = quant2_divide<kFmtE4M3>(x[4 * i], x[4 * i + 1], s) |
             (quant2_divide<kFmtE4M3>(x[4 * i + 2], x[4 * i + 3], s) << 16);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// kNT: eight-row activation tiles (1 or 2).
template <int kNT, int kSrc, int kOut>
__global__ void __launch_bounds__(kGvThreads, 2)
block_gemv_kernel(const __grid_constant__ GvParams p) {
  constexpr bool kGated = kOut == kGemvSwiglu;
  constexpr bool kSum = kOut == kGemvSum;
  constexpr int kMats = kGated ? 2 : 1;
  constexpr int kDepth = kGated ? 2 : 4;  // blocks in flight a lane: 256 bytes either way
  extern __shared__ __align__(16) uint8_t act[];
  __shared__ float red[2][kGvWarps][kMats][kNT * 8][kGvRows];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int kbw = p.kbw;
  const int kb0 = warp * kbw;                         // this warp's blocks [kb0, kb0 + kbw)
  const int total_kb = kSum ? p.kb * p.pairs : p.kb;  // kSum: the pairs' K one after the other
  const bool one_token = kGated && p.ids != nullptr;

  // shared memory of this warp: rows of codes, then scales [kbw][8 kNT]
  const int stride = kbw * kBlock + 64;
  const int rows_held = kSum || one_token ? 1 : kNT * 8;
  const int rows_max = min(rows_held, p.M);
  const int warp_bytes = rows_max * stride + kbw * kNT * 8 * 4;
  uint8_t* my_act = act + warp * warp_bytes;
  float* my_scale = reinterpret_cast<float*>(my_act + rows_max * stride);

  auto expert_of_pair = [&](int j) {
    const int e = __ldg(p.ids + j);
    return e >= 0 && e < p.experts ? e : -1;
  };
  // unit -> row tile and row group; tile -> expert and rows
  auto tile_of = [&](int ti, int& expert, int& row0, int& rows) {
    if (kSum) {
      expert = 0, row0 = 0, rows = 1;
    } else if (one_token) {
      expert = expert_of_pair(ti), row0 = ti, rows = 1;
    } else if (p.tiles != nullptr) {
      const int4 v = *reinterpret_cast<const int4*>(p.tiles + ti);
      expert = v.x, row0 = v.y, rows = min(v.z - v.y, kNT * 8);
    } else {
      expert = 0, row0 = 0, rows = p.M;
    }
  };

  // dense weights do not depend on the kernel before; kSum's ids are older than it too (the
  // kernel before starts its dependents after its own wait)
  bool waited = false;
  if (!kSum && (p.tiles != nullptr || one_token)) {
    pdl_wait();
    waited = true;
  }
  pdl_trigger();

  const int n_tiles = kSum ? 1 : one_token ? p.pairs : p.tiles != nullptr ? *p.n_tiles : 1;
  const int units = n_tiles * p.groups;
  // contiguous units, so a CTA sees few tiles
  const int first = int(int64_t(units) * blockIdx.x / gridDim.x);
  const int last = int(int64_t(units) * (blockIdx.x + 1) / gridDim.x);
  if (first >= last) return;

  // the load side of the pipeline walks (unit, block) kDepth steps ahead
  uint4 buf[kDepth][kMats][4];
  int lu = first, lj = 0, l_tile = -1, l_expert = 0;
  const uint8_t* l_row0 = nullptr;
  const uint8_t* l_row1 = nullptr;
  int64_t l_mat = int64_t(p.N) * p.ldw;
  auto place = [&]() {  // pointers of the load side's unit
    const int ti = lu / p.groups, grp = lu - ti * p.groups;
    if (!kSum && ti != l_tile) {
      int r0, rows;
      tile_of(ti, l_expert, r0, rows);
      l_tile = ti;
    }
    const int r = grp * kGvRows + g;
    const uint8_t* base = p.qw + int64_t(kMats) * max(l_expert, 0) * l_mat;
    l_row0 = base + int64_t(min(r, p.N - 1)) * p.ldw + t * 16;
    l_row1 = base + int64_t(min(r + 8, p.N - 1)) * p.ldw + t * 16;
  };
  auto issue = [&](uint4 (&b)[kMats][4]) {
    const int kbi = kb0 + lj;
    int kb = kbi, expert = l_expert;
    int64_t off = 0;
    bool in = lu < last && kbi < total_kb;
    if (kSum) {
      const int j = kbi / p.kb;
      kb = kbi - j * p.kb;
      if (in) {
        expert = expert_of_pair(j);
        off = int64_t(expert) * l_mat;
      }
    }
    in = in && expert >= 0;
    const int64_t c = int64_t(kb) * kBlock;
    const bool in0 = in && c + t * 16 < p.ldw, in1 = in && c + 64 + t * 16 < p.ldw;
#pragma unroll
    for (int m = 0; m < kMats; ++m) {
      const uint8_t* r0 = l_row0 + off + m * l_mat + c;
      const uint8_t* r1 = l_row1 + off + m * l_mat + c;
      b[m][0] = in0 ? ld_stream_v4(r0) : make_uint4(0, 0, 0, 0);
      b[m][1] = in0 ? ld_stream_v4(r1) : make_uint4(0, 0, 0, 0);
      b[m][2] = in1 ? ld_stream_v4(r0 + 64) : make_uint4(0, 0, 0, 0);
      b[m][3] = in1 ? ld_stream_v4(r1 + 64) : make_uint4(0, 0, 0, 0);
    }
    if (++lj == kbw) {
      lj = 0;
      if (++lu < last) place();
    }
  };
  place();
#pragma unroll
  for (int d = 0; d < kDepth; ++d) issue(buf[d]);
  if (!waited) pdl_wait();

  int tile = -1, expert = 0, row0 = 0, rows = 0;
  // codes and scales of this warp's K slice for the rows of the current tile
  auto fill = [&]() {
    __syncwarp();
    if constexpr (kSrc == kSrcCodes) {
      const uint8_t* a = static_cast<const uint8_t*>(p.a);
      for (int i = lane; i < rows * kbw * 8; i += 32) {
        const int r = i / (kbw * 8), c = i - r * kbw * 8;
        const int64_t col = int64_t(kb0) * kBlock + c * 16;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (col < p.lda && kb0 + c / 8 < p.kb) v = *reinterpret_cast<const uint4*>(a + int64_t(row0 + r) * p.lda + col);
        *reinterpret_cast<uint4*>(my_act + r * stride + c * 16) = v;
      }
      for (int i = lane; i < kbw * kNT * 8; i += 32) {
        const int kb = i / (kNT * 8), r = i - kb * kNT * 8;
        my_scale[i] = r < rows && kb0 + kb < p.kb ? p.s_a[int64_t(kb0 + kb) * p.lds_a + row0 + r] : 0.0f;
      }
    } else {
      // eight lanes quantize one block of one row, sixteen values each
      const int items = rows * kbw;
      for (int i0 = 0; i0 < items; i0 += 4) {
        const int i = i0 + (lane >> 3), l8 = lane & 7;
        const int r = i / kbw, j = i - r * kbw;
        int kb = kb0 + j;
        const bool in = i < items && kb < total_kb;
        int64_t src_row = row0 + r;
        float wt = 1.0f;
        bool use = in;
        if (kSum && in) {
          src_row = kb / p.kb;
          use = expert_of_pair(int(src_row)) >= 0;
          if (use) wt = __ldg(p.weights + src_row);
          kb -= int(src_row) * p.kb;
        }
        if (one_token) src_row = 0;
        if (p.row_src != nullptr && in) src_row = __ldg(p.row_src + row0 + r);
        const int c = kb * kBlock + l8 * 16;
        uint4 codes = make_uint4(0, 0, 0, 0);
        float s;
        if constexpr (kSrc == kSrcBf16) {
          uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
          if (use && c < p.K) {
            const uint16_t* row = static_cast<const uint16_t*>(p.a) + src_row * p.lda;
            lo = load8_bf16(row, c, p.K, p.vec);
            hi = load8_bf16(row, c + 8, p.K, p.vec);
          }
          uint32_t m2 = abs_max_v4(abs_max_v4(0u, lo), hi);
#pragma unroll
          for (int o = 4; o > 0; o >>= 1) m2 = __vmaxu2(m2, __shfl_xor_sync(0xffffffffu, m2, o));
          s = scale_from_amax<kFmtE4M3>(u16x2_max_to_float(m2));
          const ExactScale k = make_exact_scale(s);
          const uint2 q0 = quant8_exact<kFmtE4M3>(lo, k, s, false), q1 = quant8_exact<kFmtE4M3>(hi, k, s, false);
          codes = make_uint4(q0.x, q0.y, q1.x, q1.y);
        } else {
          float x[16];
          uint32_t m = 0;
          const float* row = static_cast<const float*>(p.a) + src_row * p.lda + c;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            // rows are padded to whole sixteens with zeros by their producer
            const float4 v = use && c + q * 4 < p.lda ? *reinterpret_cast<const float4*>(row + q * 4)
                                                      : make_float4(0.f, 0.f, 0.f, 0.f);
            x[4 * q] = v.x, x[4 * q + 1] = v.y, x[4 * q + 2] = v.z, x[4 * q + 3] = v.w;
          }
#pragma unroll
          for (int q = 0; q < 16; ++q) m = max(m, __float_as_uint(fabsf(x[q])));
#pragma unroll
          for (int o = 4; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
          s = scale_from_amax<kFmtE4M3>(__uint_as_float(m));
          codes = codes_of_f32(x, s);
        }
        if (i < items) {
          *reinterpret_cast<uint4*>(my_act + r * stride + j * kBlock + l8 * 16) = codes;
          if (l8 == 0) my_scale[j * kNT * 8 + r] = use ? s * wt : 0.0f;
        }
      }
    }
    __syncwarp();
  };

  float acc[kMats][kNT][4];
  auto clear = [&]() {
#pragma unroll
    for (int m = 0; m < kMats; ++m)
#pragma unroll
      for (int n = 0; n < kNT; ++n)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[m][n][c] = 0.0f;
  };
  clear();

  int u = first, j = 0, parity = 0;
  const int64_t steps = int64_t(last - first) * kbw;
  const float* sw = nullptr;
  for (int64_t s0 = 0; s0 < steps; s0 += kDepth) {
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
      if (s0 + d >= steps) break;
      if (j == 0) {
        const int ti = u / p.groups, grp = u - ti * p.groups;
        if (ti != tile) {
          tile = ti;
          tile_of(ti, expert, row0, rows);
          fill();
        }
        sw = p.s_w + (int64_t(kMats) * max(expert, 0) * p.nb + grp * kGvRows / kBlock) * p.kb;
      }
      const int kbi = kb0 + j;
      if (kbi < total_kb && expert >= 0) {
        float w_scale[kMats];
        if (kSum) {
          const int pj = kbi / p.kb;
          const int e = max(expert_of_pair(pj), 0);
          w_scale[0] = __ldg(sw + int64_t(e) * p.nb * p.kb + (kbi - pj * p.kb));
        } else {
#pragma unroll
          for (int m = 0; m < kMats; ++m) w_scale[m] = __ldg(sw + int64_t(m) * p.nb * p.kb + kbi);
        }
#pragma unroll
        for (int n = 0; n < kNT; ++n) {
          uint4 b0 = make_uint4(0, 0, 0, 0), b1 = b0;
          if (n * 8 + g < rows) {
            const uint8_t* src = my_act + (n * 8 + g) * stride + j * kBlock + t * 16;
            b0 = *reinterpret_cast<const uint4*>(src);
            b1 = *reinterpret_cast<const uint4*>(src + 64);
          }
          // scales of the rows this lane accumulates: 2t and 2t + 1 of the tile
          const float2 sa = *reinterpret_cast<const float2*>(my_scale + j * kNT * 8 + n * 8 + 2 * t);
          const float sa0 = n * 8 + 2 * t < rows ? sa.x : 0.0f, sa1 = n * 8 + 2 * t + 1 < rows ? sa.y : 0.0f;
#pragma unroll
          for (int m = 0; m < kMats; ++m) {
            const uint4(&w)[4] = buf[d][m];
            float part[4] = {0.f, 0.f, 0.f, 0.f};
            mma_e4m3(part, w[0].x, w[1].x, w[0].y, w[1].y, b0.x, b0.y);
            mma_e4m3(part, w[0].z, w[1].z, w[0].w, w[1].w, b0.z, b0.w);
            mma_e4m3(part, w[2].x, w[3].x, w[2].y, w[3].y, b1.x, b1.y);
            mma_e4m3(part, w[2].z, w[3].z, w[2].w, w[3].w, b1.z, b1.w);
            acc[m][n][0] = fmaf(part[0], w_scale[m] * sa0, acc[m][n][0]);
            acc[m][n][1] = fmaf(part[1], w_scale[m] * sa1, acc[m][n][1]);
            acc[m][n][2] = fmaf(part[2], w_scale[m] * sa0, acc[m][n][2]);
            acc[m][n][3] = fmaf(part[3], w_scale[m] * sa1, acc[m][n][3]);
          }
        }
      }
      issue(buf[d]);
      if (++j == kbw) {
        // end of a row group: the warps' sums meet; two buffers alternate, so one barrier is enough
        j = 0;
#pragma unroll
        for (int m = 0; m < kMats; ++m)
#pragma unroll
          for (int n = 0; n < kNT; ++n) {
            float(*r)[kGvRows] = &red[parity][warp][m][n * 8 + 2 * t];
            r[0][g] = acc[m][n][0], r[1][g] = acc[m][n][1], r[0][g + 8] = acc[m][n][2], r[1][g + 8] = acc[m][n][3];
          }
        clear();
        __syncthreads();
        const int ti = u / p.groups, grp = u - ti * p.groups;
        for (int o = threadIdx.x; o < rows * kGvRows; o += kGvThreads) {
          const int r = o / kGvRows, i = o - r * kGvRows;
          const int n = grp * kGvRows + i;
          float v[kMats];
#pragma unroll
          for (int m = 0; m < kMats; ++m) {
            v[m] = 0.0f;
#pragma unroll
            for (int w = 0; w < kGvWarps; ++w) v[m] += red[parity][w][m][r][i];
          }
          if constexpr (kGated) {
            // rows of h are whole sixteens: columns past N come from clamped rows and are zero
            const float h = n < p.N ? __fdividef(v[0], 1.0f + __expf(-v[0])) * v[1] : 0.0f;
            if (n < p.ldy32) p.y32[int64_t(row0 + r) * p.ldy32 + n] = h;
          } else if constexpr (kOut == kGemvF32) {
            if (n < p.N) p.y32[int64_t(row0 + r) * p.ldy32 + n] = v[0];
          } else if (n < p.N) {
            if (p.bias != nullptr) v[0] += bf16_bits_to_float(p.bias[n]);
            p.y[int64_t(row0 + r) * p.ldy + n] = __bfloat16_as_ushort(__float2bfloat16_rn(v[0]));
          }
        }
        parity ^= 1;
        ++u;
      }
    }
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

namespace {

constexpr int kSmemCap = 227 * 1024;
PerDeviceCache<const void*, int> g_gemv_attr;

size_t act_bytes(int64_t rows, int64_t kbw, int nt) {
  return size_t(kGvWarps) * size_t(rows * (kbw * kBlock + 64) + kbw * nt * 8 * 4);
}
size_t red_bytes(int nt, int mats) { return size_t(2) * kGvWarps * mats * nt * 8 * kGvRows * 4; }
int64_t slice_of(int64_t kb) { return (kb + kGvWarps - 1) / kGvWarps; }

template <int kNT, int kSrc, int kOut>
bool launch_gv(const GemvArgs& a, int num_sms, cudaStream_t st) {
  auto kfn = block_gemv_kernel<kNT, kSrc, kOut>;
  int dev = 0, smem_max = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  if (!g_gemv_attr.get(dev, reinterpret_cast<const void*>(kfn), &smem_max, [&](int* v) {
        cudaFuncAttributes fa = {};
        if (cudaFuncGetAttributes(&fa, kfn) != cudaSuccess) return false;
        *v = kSmemCap - int(fa.sharedSizeBytes);
        return report_cuda(cudaFuncSetAttribute(kfn, cudaFuncAttributeMaxDynamicSharedMemorySize, *v),
                           "block gemv smem attribute") == cudaSuccess;
      }))
    return false;
  GvParams p = {};
  p.a = a.a;
  p.lda = a.lda;
  p.s_a = a.s_a;
  p.lds_a = a.lds_a;
  p.row_src = a.row_src;
  p.tiles = a.tiles;
  p.n_tiles = a.n_tiles;
  p.ids = a.ids;
  p.weights = a.weights;
  p.pairs = a.pairs;
  p.experts = int(a.experts);
  p.M = int(a.tiles ? a.tile_rows : a.ids ? 1 : a.M);
  p.qw = a.qw;
  p.ldw = a.ldw;
  p.s_w = a.s_w;
  p.N = int(a.N);
  p.K = int(a.K);
  p.kb = int(blocks_of(a.K));
  p.nb = int(blocks_of(a.N));
  const int64_t n_out = kOut == kGemvSwiglu ? std::min<int64_t>(a.ldy32, (a.N + kGvRows - 1) / kGvRows * kGvRows) : a.N;
  p.groups = int((n_out + kGvRows - 1) / kGvRows);
  p.kbw = int(slice_of(kOut == kGemvSum ? int64_t(p.kb) * a.pairs : p.kb));
  p.vec = aligned(a.a, 16) && a.lda % 8 == 0;
  p.bias = a.bias;
  p.y = a.y;
  p.ldy = a.ldy;
  p.y32 = a.y32;
  p.ldy32 = a.ldy32;
  const size_t smem = act_bytes(p.M, p.kbw, kNT);
  if (smem > size_t(smem_max)) return false;
  const int64_t units = (kOut == kGemvSum ? 1 : a.tiles ? a.max_tiles : a.ids ? a.pairs : 1) * int64_t(p.groups);
  const int per_sm = smem + red_bytes(kNT, kOut == kGemvSwiglu ? 2 : 1) + 1024 <= size_t(kSmemCap) / 2 ? 2 : 1;
  const int grid = int(std::min<int64_t>(units, int64_t(num_sms) * per_sm));
  return launch(kfn, dim3(grid), dim3(kGvThreads), smem, st, true, dim3(1, 1, 1), p) == FP8_OK;
}

}  // namespace

bool gemv_fits(int64_t rows, int64_t K, int mats) {
  if (rows > kGemvMaxRows) return false;
  const int nt = rows > 8 ? 2 : 1;
  return act_bytes(rows, slice_of(blocks_of(K)), nt) + red_bytes(nt, mats) + 1024 <= size_t(kSmemCap);
}

bool gemv_quantizes(int64_t M, int64_t K) { return M * slice_of(blocks_of(K)) <= 16; }

bool gemv_launch(const GemvArgs& a, GemvOut out, int num_sms, cudaStream_t st) {
  const int64_t rows = a.tiles ? a.tile_rows : a.ids ? 1 : a.M;
  const bool two = rows > 8;
  switch (out) {
    case kGemvBf16:
      if (a.src == kSrcBf16)
        return two ? launch_gv<2, kSrcBf16, kGemvBf16>(a, num_sms, st) : launch_gv<1, kSrcBf16, kGemvBf16>(a, num_sms, st);
      return two ? launch_gv<2, kSrcCodes, kGemvBf16>(a, num_sms, st) : launch_gv<1, kSrcCodes, kGemvBf16>(a, num_sms, st);
    case kGemvSwiglu:
      return two ? launch_gv<2, kSrcBf16, kGemvSwiglu>(a, num_sms, st)
                 : launch_gv<1, kSrcBf16, kGemvSwiglu>(a, num_sms, st);
    case kGemvF32:
      return two ? launch_gv<2, kSrcF32, kGemvF32>(a, num_sms, st) : launch_gv<1, kSrcF32, kGemvF32>(a, num_sms, st);
    case kGemvSum:
      return launch_gv<1, kSrcF32, kGemvSum>(a, num_sms, st);
  }
  return false;
}

}  // namespace block
}  // namespace fp8k
