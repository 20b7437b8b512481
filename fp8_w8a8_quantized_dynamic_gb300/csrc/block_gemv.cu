// Block-scaled FP8 GEMV for sm_103a: the product for few rows, bound by streaming the weights (times here
// and below: graphs that cycle through weights which together pass L2. One row, 4096 x 6144, 25 MB: 7.7 to
// 8.9 us over several GPUs, 2.8 to 3.3 TB/s; 4096 x 28672, 117 MB: 20.2 us, 5.8 TB/s; the start of a launch,
// its first loads and the last sums take 4 us). One token's experts, 8 of 2048 x 1408: 23.3 us for 69 MB in
// two launches.
//
// A warp takes 16 weight rows at a time (kGemvSwiglu: 16 of gate and the same 16 of up) over a slice
// of K in whole 128-wide blocks; 1, 2, 4 or all 8 warps of a CTA share one row group's K. A lane loads
// 32 bytes of two weight rows (four lanes a row's 128) straight into the registers that mma.sync
// m16n8k32 takes as its A operand: its eight words a row are the fragments of four MMAs under a
// permutation of k that the activations follow, so nothing passes through shared memory and nothing
// is rearranged. The loads run kDepth blocks ahead, over the ends of row groups, and the first ones
// are in flight before the kernel waits for its activations. Block partials are added, scaled, in
// fp32; the warps' sums meet in shared memory in a fixed order.
//
// Activations: the warps of a K slice quantize it for every row into shared memory (no barrier where
// each slice has one warp), or copy codes that a kernel before wrote. Rows are 16 modulo 128 bytes
// apart, so a quarter warp's 16-byte reads (two rows, four at every 32 bytes) touch every bank once.

#include "block_gemv.h"

#include <algorithm>

#include "api_common.h"
#include "device_cache.h"
#include "device_common.cuh"
#include "tcgen05.cuh"

namespace fp8k {
namespace block {

constexpr int kGvWarpsLog2 = 3;
constexpr int kGvWarps = 1 << kGvWarpsLog2;
constexpr int kGvThreads = kGvWarps * 32;
constexpr int kGvRows = 16;

struct GvParams {
  const void* a;
  int64_t lda;
  const float* s_a;
  int64_t lds_a;
  int M;
  const int32_t* ids;
  const float* weights;
  int pairs, experts;
  const uint8_t* qw;
  int64_t ldw, mat_bytes;
  const float* s_w;
  int N, K, kb, nb;
  int split_log2;  // warps that share a row group's K; the others take other row groups
  int units;       // of one tile: kGvWarps >> split_log2 row groups each
  int kbw;      // K blocks of one warp
  int vec;      // activation rows are 16-byte aligned
  const uint16_t* bias;
  uint16_t* y;
  int64_t ldy;
  float* y32;
  int64_t ldy32;
};

// Thirty-two bytes of a weight row (32-byte aligned), not kept in L1.
__device__ __forceinline__ void ld_stream(const uint8_t* p, uint32_t (&v)[8]) {
  asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
               : "l"(p));
}
// The same for any row: `left` bytes (whole sixteens) to its end, zero past it. Predicated in one
// statement: a branch would merge the loaded registers with the zeros, and that copy would wait.
__device__ __forceinline__ void ld_ragged(const uint8_t* p, int left, uint32_t (&v)[8]) {
  asm volatile(
      "{\n\t.reg .pred a, b;\n\tsetp.gt.s32 a, %9, 0;\n\tsetp.gt.s32 b, %9, 16;\n\t"
      "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
      "mov.b32 %4, 0;\n\tmov.b32 %5, 0;\n\tmov.b32 %6, 0;\n\tmov.b32 %7, 0;\n\t"
      "@a ld.global.nc.L1::no_allocate.v4.b32 {%0,%1,%2,%3}, [%8];\n\t"
      "@b ld.global.nc.L1::no_allocate.v4.b32 {%4,%5,%6,%7}, [%8+16];\n\t}"
      : "=&r"(v[0]), "=&r"(v[1]), "=&r"(v[2]), "=&r"(v[3]), "=&r"(v[4]), "=&r"(v[5]), "=&r"(v[6]), "=&r"(v[7])
      : "l"(p), "r"(left));
}

__device__ __forceinline__ void mma_e4m3(float (&d)[4], const float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}

// Sixteen values -> codes, any scale.
__device__ __forceinline__ uint4 codes_of_f32(const float (&x)[16], float s) {
  const ExactScale k = make_exact_scale(s);
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = quant4_exact_f32<kFmtE4M3>(pack_f32x2(x[4 * i], x[4 * i + 1]), pack_f32x2(x[4 * i + 2], x[4 * i + 3]), k, s);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// kNT: eight-row activation tiles (1 or 2). kFull: weight rows are whole blocks, 32-byte aligned, and
// loaded 32 bytes at a time (1 x 4096 x 28672 in 20.2 us, 21.7 in predicated 16-byte loads; 1 x 5632 x 2048
// 6.7 and 7.3; 1 x 4096 x 6144 7.7 and 7.9, 8 rows 11.0 and 10.7; 1 x 512 x 28672 6.3 and 5.4).
template <int kNT, int kSrc, int kOut, bool kFull>
__global__ void __launch_bounds__(kGvThreads, 2)
block_gemv_kernel(const __grid_constant__ GvParams p) {
  constexpr bool kGated = kOut == kGemvSwiglu;
  constexpr bool kSum = kOut == kGemvSum;
  constexpr int kMats = kGated ? 2 : 1;
  constexpr int kDepth = kGated ? 2 : 4;  // blocks in flight a lane: 256 bytes either way
  extern __shared__ __align__(16) uint8_t act[];
  __shared__ float red[2][kGvWarps][kMats][kNT * 8][kGvRows + 4];  // + 4: a warp's 32 stores on 32 banks
  __shared__ uint4 zeros[kBlock / 16];  // the codes of rows that a tile does not have
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int kbw = p.kbw, splits = 1 << p.split_log2, per_log2 = kGvWarpsLog2 - p.split_log2;
  const int per_cta = 1 << per_log2;
  const int split = warp & (splits - 1), sub = warp >> p.split_log2;  // K slice, and row group of the unit
  const int kb0 = split * kbw;                        // this warp's blocks [kb0, kb0 + kbw)
  const int total_kb = kSum ? p.kb * p.pairs : p.kb;  // kSum: the pairs' K one after the other
  constexpr bool kPairs = kGated;  // the tiles are the pairs of one token

  // shared memory of a K slice: rows of codes, then scales [kbw][8 kNT]
  const int stride = kbw * kBlock + 16;
  const int rows_held = kSum || kPairs ? 1 : kNT * 8;
  const int rows_max = min(rows_held, p.M);
  const int slice_bytes = (rows_max * stride + kbw * kNT * 8 * 4 + 15) / 16 * 16;
  uint8_t* my_act = act + split * slice_bytes;
  float* my_scale = reinterpret_cast<float*>(my_act + rows_max * stride);

  auto expert_of_pair = [&](int j) {
    const int e = __ldg(p.ids + j);
    return e >= 0 && e < p.experts ? e : -1;
  };
  // unit -> row tile and row group; tile -> expert and rows
  auto tile_of = [&](int ti, int& expert, int& row0, int& rows) {
    if (kSum) {
      expert = 0, row0 = 0, rows = 1;
    } else if (kPairs) {
      expert = expert_of_pair(ti), row0 = ti, rows = 1;
    } else {
      expert = 0, row0 = 0, rows = p.M;
    }
  };

  // dense weights do not depend on the kernel before; kSum's ids are older than it too (the
  // kernel before starts its dependents after its own wait)
  if (kPairs) pdl_wait();
  pdl_trigger();

  const int n_tiles = kPairs ? p.pairs : 1;
  const int units = n_tiles * p.units;
  // contiguous units, so a CTA sees few tiles
  const int first = int(int64_t(units) * blockIdx.x / gridDim.x);
  const int last = int(int64_t(units) * (blockIdx.x + 1) / gridDim.x);
  if (first >= last) return;
  if (threadIdx.x < kBlock / 16) zeros[threadIdx.x] = make_uint4(0, 0, 0, 0);

  // The load side of the pipeline walks (unit, block) kDepth steps ahead. Its pointers move on by a
  // block a step; seek() sets them at the start of a unit (kSum: and of a pair's K). A slot with
  // nothing to load reads the first matrix's first block, and its step is not computed.
  uint32_t buf[kDepth][kMats][2][8];
  float w_scale[kDepth][kMats];  // the blocks' weight scales, loaded with them
  uint32_t live = 0;             // bit d: buf[d] holds a block to compute
  int l_tile = first / p.units, l_unit = first - l_tile * p.units;  // row tile, and unit in it
  int lu = first, lj = 0, l_known = -1, l_expert = 0;
  int l_run = 0;        // blocks until the next seek()
  int l_left = 0;       // ragged: bytes of the row from this lane's 32 on
  int l_step = 0;       // bytes from block to block, 0 for an empty slot
  const uint8_t* l_ptr = nullptr;  // row g; row g + 8 and the second matrix lie l_row8 and p.mat_bytes on
  const float* l_sw = nullptr;
  int64_t l_row8 = 0;
  auto seek = [&]() {
    const int row = ((l_unit << per_log2) + sub) * kGvRows;
    const int kbi = kb0 + lj;
    int kb = kbi;
    bool in = lu < last && row < p.N && kbi < total_kb;
    l_run = kbw - lj;
    if (kSum) {
      const int j = in ? kbi / p.kb : 0;
      kb = kbi - j * p.kb;
      l_expert = in ? expert_of_pair(j) : -1;
      if (in) l_run = min(l_run, p.kb - kb);
    } else {
      if (lu < last && l_tile != l_known) {
        int r0, rows;
        tile_of(l_tile, l_expert, r0, rows);
        l_known = l_tile;
      }
      if (in) l_run = min(l_run, total_kb - kbi);
    }
    in = in && l_expert >= 0;
    if (lu >= last) l_run = 1 << 30;
    const int64_t col = in ? int64_t(kb) * kBlock + t * 32 : kFull ? t * 32 : 0;
    const int64_t mat = in ? int64_t(kMats) * l_expert : 0;
    const int r0 = in ? min(row + g, p.N - 1) : 0, r8 = in ? min(row + g + 8, p.N - 1) : 0;  // past N: not used
    l_left = in ? int(min(p.ldw - col, int64_t(1) << 30)) : 0;
    l_step = in ? kBlock : 0;
    l_ptr = p.qw + mat * p.mat_bytes + int64_t(r0) * p.ldw + col;
    l_row8 = int64_t(r8 - r0) * p.ldw;
    l_sw = in ? p.s_w + (mat * p.nb + row / kBlock) * p.kb + kb : p.s_w;
  };
  auto issue = [&](int d) {
#pragma unroll
    for (int m = 0; m < kMats; ++m) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint8_t* src = l_ptr + (m ? p.mat_bytes : 0) + (h ? l_row8 : 0);
        if constexpr (kFull)
          ld_stream(src, buf[d][m][h]);
        else
          ld_ragged(src, l_left, buf[d][m][h]);
      }
      w_scale[d][m] = __ldg(l_sw + (m ? p.nb * p.kb : 0));
    }
    live = (live & ~(1u << d)) | (l_step ? 1u << d : 0u);
    l_ptr += l_step;
    l_sw += l_step ? 1 : 0;
    if (!kFull) l_left -= kBlock;
    ++lj;
    if (--l_run == 0) {
      if (lj == kbw) {
        lj = 0;
        ++lu;
        if (++l_unit == p.units) l_unit = 0, ++l_tile;
      }
      seek();
    }
  };
  seek();
#pragma unroll
  for (int d = 0; d < kDepth; ++d) issue(d);
  if (!kPairs) pdl_wait();

  int tile = -1, expert = 0, row0 = 0, rows = 0;
  // codes and scales of the K slices for the rows of the current tile; the warps that share a slice
  // share the work. The barrier at the end of a unit has passed: nobody reads the last tile's.
  auto fill = [&]() {
    if constexpr (kSrc == kSrcCodes) {
      const uint8_t* a = static_cast<const uint8_t*>(p.a);
      for (int i = sub * 32 + lane; i < rows * kbw * 8; i += 32 * per_cta) {
        const int r = i / (kbw * 8), c = i - r * kbw * 8;
        const int64_t col = int64_t(kb0) * kBlock + c * 16;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (col < p.lda && kb0 + c / 8 < p.kb) v = *reinterpret_cast<const uint4*>(a + int64_t(row0 + r) * p.lda + col);
        *reinterpret_cast<uint4*>(my_act + r * stride + c * 16) = v;
      }
      for (int i = sub * 32 + lane; i < kbw * kNT * 8; i += 32 * per_cta) {
        const int kb = i / (kNT * 8), r = i - kb * kNT * 8;
        my_scale[i] = r < rows && kb0 + kb < p.kb ? p.s_a[int64_t(kb0 + kb) * p.lds_a + row0 + r] : 0.0f;
      }
    } else {
      for (int i = sub * 32 + lane; i < kbw * kNT * 8; i += 32 * per_cta)
        if ((i & (kNT * 8 - 1)) >= rows) my_scale[i] = 0.0f;
      // eight lanes quantize one block of one row, sixteen values each
      const int items = rows * kbw;
      for (int i0 = sub * 4; i0 < items; i0 += 4 * per_cta) {
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
        if (kPairs) src_row = 0;
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
    if (per_cta > 1)
      __syncthreads();
    else
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

  // fragments of row 8 n + g: its codes, or zeros
  const uint8_t* b_ptr[kNT];
  int b_step[kNT];
  int c_tile = first / p.units, c_unit = first - c_tile * p.units, j = 0, parity = 0;
  const int steps = (last - first) * kbw;
  __syncthreads();  // zeros
  for (int s0 = 0; s0 < steps; s0 += kDepth) {
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
      if (s0 + d >= steps) break;
      if (j == 0) {
        if (c_tile != tile) {
          tile = c_tile;
          tile_of(c_tile, expert, row0, rows);
          fill();
        }
#pragma unroll
        for (int n = 0; n < kNT; ++n) {
          const bool has = n * 8 + g < rows;
          b_ptr[n] = (has ? my_act + (n * 8 + g) * stride : reinterpret_cast<const uint8_t*>(zeros)) + t * 32;
          b_step[n] = has ? kBlock : 0;
        }
      }
      if (live & (1u << d)) {
#pragma unroll
        for (int n = 0; n < kNT; ++n) {
          const uint4 b0 = *reinterpret_cast<const uint4*>(b_ptr[n]);
          const uint4 b1 = *reinterpret_cast<const uint4*>(b_ptr[n] + 16);
          // scales of the rows this lane accumulates: 2t and 2t + 1 of the tile
          const float2 sa = *reinterpret_cast<const float2*>(my_scale + j * kNT * 8 + n * 8 + 2 * t);
#pragma unroll
          for (int m = 0; m < kMats; ++m) {
            const uint32_t(&w0)[8] = buf[d][m][0];  // rows g and g + 8
            const uint32_t(&w1)[8] = buf[d][m][1];
            const float none[4] = {0.f, 0.f, 0.f, 0.f};
            float part[4];
            mma_e4m3(part, none, w0[0], w1[0], w0[1], w1[1], b0.x, b0.y);
            mma_e4m3(part, part, w0[2], w1[2], w0[3], w1[3], b0.z, b0.w);
            mma_e4m3(part, part, w0[4], w1[4], w0[5], w1[5], b1.x, b1.y);
            mma_e4m3(part, part, w0[6], w1[6], w0[7], w1[7], b1.z, b1.w);
            const float s0w = w_scale[d][m] * sa.x, s1w = w_scale[d][m] * sa.y;
            acc[m][n][0] = fmaf(part[0], s0w, acc[m][n][0]);
            acc[m][n][1] = fmaf(part[1], s1w, acc[m][n][1]);
            acc[m][n][2] = fmaf(part[2], s0w, acc[m][n][2]);
            acc[m][n][3] = fmaf(part[3], s1w, acc[m][n][3]);
          }
        }
      }
#pragma unroll
      for (int n = 0; n < kNT; ++n) b_ptr[n] += b_step[n];
      issue(d);
      if (++j == kbw) {
        // end of a row group: the warps' sums meet; two buffers alternate, so one barrier is enough
        j = 0;
#pragma unroll
        for (int m = 0; m < kMats; ++m)
#pragma unroll
          for (int n = 0; n < kNT; ++n) {
            float(*r)[kGvRows + 4] = &red[parity][warp][m][n * 8 + 2 * t];
            r[0][g] = acc[m][n][0], r[1][g] = acc[m][n][1], r[0][g + 8] = acc[m][n][2], r[1][g + 8] = acc[m][n][3];
          }
        clear();
        __syncthreads();
        const int first_row = c_unit << (per_log2 + 4);
        for (int o = threadIdx.x; o < (rows << (per_log2 + 4)); o += kGvThreads) {
          const int r = o >> (per_log2 + 4), i = o & ((kGvRows << per_log2) - 1);
          const int n = first_row + i;
          float v[kMats];
#pragma unroll
          for (int m = 0; m < kMats; ++m) {
            v[m] = 0.0f;
            for (int w = 0; w < splits; ++w) v[m] += red[parity][((i >> 4) << p.split_log2) + w][m][r][i & 15];
          }
          if constexpr (kGated) {
            // rows of h are whole sixteens: columns past N come from clamped rows and are zero
            const float h = n < p.N ? swiglu(v[0], v[1]) : 0.0f;
            if (n < p.ldy32) p.y32[int64_t(row0 + r) * p.ldy32 + n] = h;
          } else if (n < p.N) {
            if (p.bias != nullptr) v[0] += bf16_bits_to_float(p.bias[n]);
            p.y[int64_t(row0 + r) * p.ldy + n] = __bfloat16_as_ushort(__float2bfloat16_rn(v[0]));
          }
        }
        parity ^= 1;
        if (++c_unit == p.units) c_unit = 0, ++c_tile;
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

size_t act_bytes(int64_t rows, int64_t kbw, int splits, int nt) {
  return size_t(splits) * size_t(round_up16(rows * (kbw * kBlock + 16) + kbw * nt * 8 * 4));
}
size_t red_bytes(int nt, int mats) { return size_t(2) * kGvWarps * mats * nt * 8 * (kGvRows + 4) * 4; }
// Warps that share a row group's K (1, 2, 4 or 8): the split with the fewest steps of the busiest
// warp, a unit counting its blocks and one more for its barrier and output; of equals the smaller, which
// takes fewer CTAs. Few row groups take all eight and so the whole GPU (one row, K 4096, N 1024: 3.9 us,
// 5.2 with four, 12.3 with one), many take fewer and longer slices (K 512, N 28672: 6.3 us, 8.8 with eight).
int splits_of(int64_t kb, int64_t tiles, int64_t groups, int num_sms) {
  int best = kGvWarps;
  int64_t best_cost = -1;
  for (int s = kGvWarps; s >= 1; s /= 2) {
    const int64_t units = tiles * ((groups * s + kGvWarps - 1) / kGvWarps);
    const int64_t per_cta = (units + 2 * num_sms - 1) / (2 * num_sms);
    const int64_t cost = per_cta * ((kb + s - 1) / s + 1);
    if (best_cost < 0 || cost <= best_cost) best = s, best_cost = cost;
  }
  return best;
}

template <int kNT, int kSrc, int kOut, bool kFull>
bool launch_as(const GemvArgs& a, int num_sms, cudaStream_t st) {
  auto kfn = block_gemv_kernel<kNT, kSrc, kOut, kFull>;
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
  p.ids = a.ids;
  p.weights = a.weights;
  p.pairs = a.pairs;
  p.experts = int(a.experts);
  p.M = int(a.ids ? 1 : a.M);
  p.qw = a.qw;
  p.ldw = a.ldw;
  p.mat_bytes = a.N * a.ldw;
  p.s_w = a.s_w;
  p.N = int(a.N);
  p.K = int(a.K);
  p.kb = int(blocks_of(a.K));
  p.nb = int(blocks_of(a.N));
  // (SwiGLU: the rows of h are whole sixteens)
  const int64_t groups = (std::min<int64_t>(kOut == kGemvSwiglu ? a.ldy32 : a.N, round_up16(a.N)) + kGvRows - 1) / kGvRows;
  const int64_t total_kb = kOut == kGemvSum ? int64_t(p.kb) * a.pairs : p.kb;
  const int64_t tiles = kOut == kGemvSwiglu ? a.pairs : 1;
  const int splits = splits_of(total_kb, tiles, groups, num_sms);
  while ((1 << p.split_log2) < splits) ++p.split_log2;
  p.units = int((groups * splits + kGvWarps - 1) / kGvWarps);
  p.kbw = int((total_kb + splits - 1) / splits);
  p.vec = aligned(a.a, 16) && a.lda % 8 == 0;
  p.bias = a.bias;
  p.y = a.y;
  p.ldy = a.ldy;
  p.y32 = a.y32;
  p.ldy32 = a.ldy32;
  const size_t smem = act_bytes(p.M, p.kbw, splits, kNT);
  if (smem > size_t(smem_max)) return false;
  const int64_t units = tiles * p.units;
  const int per_sm = smem + red_bytes(kNT, kOut == kGemvSwiglu ? 2 : 1) + 1024 <= size_t(kSmemCap) / 2 ? 2 : 1;
  const int grid = int(std::min<int64_t>(units, int64_t(num_sms) * per_sm));
  return launch(kfn, dim3(grid), dim3(kGvThreads), smem, st, true, dim3(1, 1, 1), p) == FP8_OK;
}

template <int kNT, int kSrc, int kOut>
bool launch_gv(const GemvArgs& a, int num_sms, cudaStream_t st) {
  if (a.ldw % kBlock == 0 && a.K > a.ldw - kBlock && aligned(a.qw, 32)) return launch_as<kNT, kSrc, kOut, true>(a, num_sms, st);
  return launch_as<kNT, kSrc, kOut, false>(a, num_sms, st);
}

}  // namespace

bool gemv_fits(int64_t rows, int64_t K, int mats) {
  if (rows > kGemvMaxRows) return false;
  const int nt = rows > 8 ? 2 : 1;
  return act_bytes(rows, (blocks_of(K) + kGvWarps - 1) / kGvWarps, kGvWarps, nt) + red_bytes(nt, mats) + 1024 <= size_t(kSmemCap);
}

// The fill of a K slice by every CTA against a second launch and codes through L2 (us, in the kernel /
// before it): M 1 K 4096 N 6144 8.2 / 9.8, M 2 9.0 / 9.9, M 4 10.9 / 10.6, M 8 15.3 / 11.0; M 4 K 5632 N 2048
// 10.2 / 8.6; K 1000 N 1027 M 8 3.5 / 4.6, M 16 5.6 / 5.8. Where the two are level the one launch is less
// work for the host.
bool gemv_quantizes(int64_t M, int64_t K) { return M * ((blocks_of(K) + kGvWarps - 1) / kGvWarps) <= 16; }

bool gemv_launch(const GemvArgs& a, GemvOut out, int num_sms, cudaStream_t st) {
  const bool two = a.M > 8;  // dense rows
  switch (out) {
    case kGemvBf16:
      if (a.src == kSrcBf16)
        return two ? launch_gv<2, kSrcBf16, kGemvBf16>(a, num_sms, st) : launch_gv<1, kSrcBf16, kGemvBf16>(a, num_sms, st);
      return two ? launch_gv<2, kSrcCodes, kGemvBf16>(a, num_sms, st) : launch_gv<1, kSrcCodes, kGemvBf16>(a, num_sms, st);
    case kGemvSwiglu:
      return launch_gv<1, kSrcBf16, kGemvSwiglu>(a, num_sms, st);
    case kGemvSum:
      return launch_gv<1, kSrcF32, kGemvSum>(a, num_sms, st);
  }
  return false;
}

}  // namespace block
}  // namespace fp8k
