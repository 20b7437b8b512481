// Low-rank adapters of many requests beside a projection they share, for sm_103a:
//
//   out[m] = bf16( y[m] + s[e] * B[e] (A[e] x[m]) ),  e = ids[m]; rows without an adapter are copied.
//
// Two forms. Few tokens (tokens_kernel): a cluster of CTAs a token, one launch; the adapter's
// matrices are read once a token, by wide loads. Many tokens (shrink_kernel, expand_kernel): rows are
// sorted by adapter and tiles of up to 128 of them pass the tensor cores, first v = A x over all of K, then
// y + s B v, whose time is the stream of y. v is fp32 between the two; the tensor core takes it as the sum of three bf16
// numbers of eight bits each, all that v has, against B's exact bf16 values.
//
// MMAs are issued by one lane of a warp that stays together (elect.sync), never by a lane that runs a loop of its own: that
// form, with the MMAs of a step in straight code, ended in an illegal instruction.
//
// Every wait is bounded; on expiry the kernel records an error, leaves its loop and stores nothing more.

#include "lora.h"

#include <algorithm>
#include <cfloat>

#include "any_rows.cuh"
#include "api_common.h"
#include "device_cache.h"
#include "device_common.cuh"
#include "gemm_tcgen05.h"
#include "tcgen05.cuh"

namespace fp8k {
namespace lora {

__device__ unsigned int g_lora_error;

// ---------------------------------------------------------------------------
// few tokens: a cluster a token
// ---------------------------------------------------------------------------

constexpr int kCluster = 8;
constexpr int kTokenThreads = 256;
constexpr int kTokenWarps = kTokenThreads / 32;

struct TokenParams {
  Args a;
  int k_slice;              // of a CTA of the cluster, a multiple of 8
  int n_slice;              // columns of a CTA
};

__device__ __forceinline__ void unpack8(uint4 v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) f[2 * i] = bf16_lo(w[i]), f[2 * i + 1] = bf16_hi(w[i]);
}

__device__ __forceinline__ float dot8(uint4 v, const float (&f)[8], float sum) {
  float g[8];
  unpack8(v, g);
#pragma unroll
  for (int i = 0; i < 8; ++i) sum = fmaf(g[i], f[i], sum);
  return sum;
}

// Sums of kValues values over the kLanes lanes (a power of two) that share them: each halving step exchanges half of the
// values, so that a lane ends with one of them in p[0], that of halving_index; past that all lanes add.
template <int kLanes, int kValues>
__device__ __forceinline__ void sum_halving(float (&p)[kValues], int lane) {
  int left = kValues;
#pragma unroll
  for (int m = kLanes / 2; m > 0; m >>= 1) {
    if (left > 1) {
      left >>= 1;
      const bool upper = (lane & m) != 0;
#pragma unroll
      for (int i = 0; i < kValues / 2; ++i) {
        if (i < left) {
          const float send = upper ? p[i] : p[i + left];
          const float keep = upper ? p[i + left] : p[i];
          p[i] = keep + __shfl_xor_sync(0xffffffffu, send, m);
        }
      }
    } else {
      p[0] += __shfl_xor_sync(0xffffffffu, p[0], m);
    }
  }
}
template <int kLanes, int kValues>
__device__ __forceinline__ int halving_index(int lane) {
  int mine = 0, left = kValues;
#pragma unroll
  for (int m = kLanes / 2; m > 0; m >>= 1) {
    if (left > 1) {
      left >>= 1;
      mine += (lane & m) != 0 ? left : 0;
    }
  }
  return mine;
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// kLpr lanes share a row of B (eight values of the rank each). Cluster rank c sums K slice c of v = A x
// and sends it to all of the cluster; then every CTA adds the slices in order and computes its columns.
// Bounds: latency for one token (4096 to 6144 at rank 16, 2.8 us); the L2 for more, which hands out an adapter's matrices to each
// of its tokens (64 tokens, 51 of them with one of 32 adapters, 4096 to 4096 at rank 64: 11.2 us, 54 MB at 4.8 TB/s, 29 MB of them
// from HBM).
// kVec: all rows start on 16-byte boundaries and are whole eights. Values beyond `end` are zeros. (What was loaded is shifted into
// place where it is used: until then more loads go out. 26 tokens, 128 to 12544 at rank 47: 28.5 us when each was shifted at once,
// 20.2
// so.)
template <bool kVec>
struct Eight {
  Raw8 v;
  __device__ __forceinline__ void clear() { v.a = v.b = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void load(const uint16_t* row, int c, int end, bool live) {
    v = load8_raw(row, off_piece(row), c, live ? end : 0);
  }
  __device__ __forceinline__ uint4 get(int at, int c, int end) const { return values8(v, at, c, end); }
};
template <>
struct Eight<true> {
  uint4 v;
  __device__ __forceinline__ void clear() { v = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void load(const uint16_t* row, int c, int, bool live) {
    v = live ? ld_nc_v4(row + c) : make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ uint4 get(int, int, int) const { return v; }
};

template <int kLpr, int kLoads, bool kVec>
__global__ void __launch_bounds__(kTokenThreads, kLoads == 8 || !kVec ? 2 : 4)
tokens_kernel(const __grid_constant__ TokenParams p) {
  constexpr int kU = kLpr < kLoads ? kLpr : kLoads;  // loads of a batch; a lane ends with one column of it
  constexpr int kBatches = kLoads / kU;              // batches in flight
  constexpr int kHalves = kLoads / 4;                // pieces of A's rows in flight
  constexpr int kRowsPerLoad = 32 / kLpr;
  constexpr int kBatchCols = kU * kRowsPerLoad;
  constexpr int kStepCols = kBatches * kBatchCols;  // of a warp
  __shared__ float part[kCluster][kMaxRank];
  __shared__ float v[kMaxRank];
  pdl_trigger();
  pdl_wait();
  cluster_arrive();  // waited for before the first store into another CTA: by then it runs
  const Args& g = p.a;
  const int64_t m = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = int(cluster_rank());
  const int N = int(g.N), K = int(g.K), r = g.rank;
  const int n0 = min(N, int(blockIdx.x) * p.n_slice), n1 = min(N, n0 + p.n_slice);
  const int e = g.ids[m];
  const uint16_t* y = g.y + m * g.ldy;
  uint16_t* out = g.out + m * g.ldo;
  if (e < 0 || e >= g.adapters) {  // (the whole cluster)
    if (out != y)
      for (int n = n0 + threadIdx.x; n < n1; n += kTokenThreads) out[n] = y[n];
    cluster_wait();
    return;
  }
  const uint16_t* A = g.a + int64_t(e) * r * K;
  const uint16_t* B = g.b + int64_t(e) * N * r;
  const int sub = lane % kLpr, row_in_load = lane / kLpr;
  // the first loads of B and y are under way while v is summed
  Eight<kVec> bv[kLoads];
  uint16_t yv[kBatches];
  const int my_u = halving_index<kLpr, kU>(lane);
  auto col_of = [&](int base, int b) { return base + b * kBatchCols + my_u * kRowsPerLoad + row_in_load; };
  auto row_of = [&](int base, int q) { return base + (q / kU) * kBatchCols + (q % kU) * kRowsPerLoad + row_in_load; };
  auto load_b = [&](int base) {
#pragma unroll
    for (int q = 0; q < kLoads; ++q) {
      const int n = row_of(base, q);
      bv[q].clear();  // (rows past the last cost no address arithmetic: 12.2 against 11.2 us for 64 tokens)
      if (n < n1 && sub * 8 < r) bv[q].load(B + int64_t(n) * r, sub * 8, r, true);
    }
#pragma unroll
    for (int b = 0; b < kBatches; ++b) yv[b] = col_of(base, b) < n1 ? y[col_of(base, b)] : uint16_t(0);
  };
  load_b(n0 + warp * kStepCols);
  const float scale = g.scales ? g.scales[e] : 1.0f;

  const int k0 = min(K, rank * p.k_slice), k1 = min(K, k0 + p.k_slice);
  const uint16_t* x = g.x + m * g.ldx;
  cluster_wait();
  const int per_warp = (r + kTokenWarps - 1) / kTokenWarps, i_end = min(r, (warp + 1) * per_warp);
  for (int i0 = warp * per_warp; i0 < i_end; i0 += 4) {
    float acc[4] = {};
    for (int k = k0 + lane * 8; k < k1; k += 256 * kHalves) {  // four rows at a time
      Eight<kVec> xv[kHalves], av[kHalves][4];
#pragma unroll
      for (int h = 0; h < kHalves; ++h) {
        const int kh = k + 256 * h;
        xv[h].load(x, kh, k1, kh < k1);
#pragma unroll
        for (int i = 0; i < 4; ++i) av[h][i].load(A + int64_t(i0 + i) * K, kh, k1, kh < k1 && i0 + i < i_end);
      }
#pragma unroll
      for (int h = 0; h < kHalves; ++h) {
        const int kh = k + 256 * h;
        float f[8];
        unpack8(xv[h].get(off_piece(x), kh, k1), f);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          acc[i] = dot8(av[h][i].get(off_piece(A + int64_t(i0 + i) * K), kh, i0 + i < i_end ? k1 : 0), f, acc[i]);
      }
    }
    // eight lanes end with the sum of a row: each sends it to one of the cluster's CTAs
    const int i = i0 + halving_index<32, 4>(lane);
    sum_halving<32, 4>(acc, lane);
    if (i < i_end) st_cluster_u32(map_to_rank(smem_u32(&part[rank][i]), lane & 7), __float_as_uint(acc[0]));
  }
  pair_sync();
  for (int i = threadIdx.x; i < kMaxRank; i += kTokenThreads) {
    float s = 0.0f;
    if (i < r)
      for (int c = 0; c < kCluster; ++c) s += part[c][i];
    v[i] = s;
  }
  __syncthreads();
  float f[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = v[sub * 8 + j];
  for (int base = n0 + warp * kStepCols; base < n1; base += kTokenWarps * kStepCols) {
    float sum[kBatches][kU], was[kBatches];
#pragma unroll
    for (int q = 0; q < kLoads; ++q) {
      const int n = row_of(base, q);
      sum[q / kU][q % kU] = dot8(bv[q].get(off_piece(B + int64_t(n) * r), sub * 8, n < n1 ? r : 0), f, 0.0f);
    }
#pragma unroll
    for (int b = 0; b < kBatches; ++b) was[b] = bf16_bits_to_float(yv[b]);
    if (base + kTokenWarps * kStepCols < n1) load_b(base + kTokenWarps * kStepCols);
#pragma unroll
    for (int b = 0; b < kBatches; ++b) {
      sum_halving<kLpr, kU>(sum[b], lane);
      const int n = col_of(base, b);
      if (n < n1 && (sub & (kLpr / kU - 1)) == 0)
        out[n] = __bfloat16_as_ushort(__float2bfloat16_rn(fmaf(scale, sum[b][0], was[b])));
    }
  }
}

template <int kLpr, int kLoads, bool kVec>
bool launch_tokens_of(const TokenParams& p, int64_t groups, cudaStream_t st) {
  return launch(tokens_kernel<kLpr, kLoads, kVec>, dim3(unsigned(kCluster * groups), unsigned(p.a.M)), dim3(kTokenThreads), 0, st, true,
                dim3(kCluster, 1, 1), p) == FP8_OK;
}
template <int kLoads, bool kVec>
bool launch_tokens_by_rank(const TokenParams& p, int64_t groups, cudaStream_t st) {
  if (p.a.rank <= 8) return launch_tokens_of<1, kLoads, kVec>(p, groups, st);
  if (p.a.rank <= 16) return launch_tokens_of<2, kLoads, kVec>(p, groups, st);
  if (p.a.rank <= 32) return launch_tokens_of<4, kLoads, kVec>(p, groups, st);
  if (p.a.rank <= 64) return launch_tokens_of<8, kLoads, kVec>(p, groups, st);
  return p.a.rank <= 128 ? launch_tokens_of<16, kLoads, kVec>(p, groups, st) : launch_tokens_of<32, kLoads, kVec>(p, groups, st);
}

bool launch_tokens(const Args& a, int num_sms, cudaStream_t st) {
  TokenParams p = {};
  p.a = a;
  p.k_slice = int(((a.K + 7) / 8 + kCluster - 1) / kCluster * 8);
  const bool vec = aligned(a.x, 16) && (a.M <= 1 || a.ldx % 8 == 0) && aligned(a.a, 16) && a.K % 8 == 0 &&
                   aligned(a.b, 16) && a.rank % 8 == 0;
  // few tokens: several clusters a token, each with all of v and a share of the columns, for as many CTAs as the SMs hold
  const int64_t groups = std::max<int64_t>(1, std::min<int64_t>({4, 2 * num_sms / (kCluster * a.M), a.N / (kCluster * 128)}));
  p.n_slice = int((a.N + kCluster * groups - 1) / (kCluster * groups));
  if (!vec) return launch_tokens_by_rank<4, false>(p, groups, st);
  // two CTAs of the deep form fit an SM, four of the other
  return a.M * kCluster <= 2 * num_sms ? launch_tokens_by_rank<8, true>(p, groups, st) : launch_tokens_by_rank<4, true>(p, groups, st);
}

// ---------------------------------------------------------------------------
// many tokens: tiles of rows sorted by adapter, on tensor cores
// ---------------------------------------------------------------------------

constexpr int kTileRows = block::kRowTile;  // 128, the MMA's M
constexpr int kTileThreads = 256;
constexpr int kBk = 64;                     // bf16 values of K in a 128-byte swizzled row
constexpr uint32_t kXBytes = kTileRows * 128;
constexpr int kShrinkMaxStages = 6;
constexpr int kShrinkThreads = kTileThreads + 32;

// kWithhold (the failure-path self-test): the first CTA does without one load, so the waits for it run out, after kWithheldNs.
constexpr unsigned long long kWithheldNs = 20000000ull;

__device__ __forceinline__ void mma_bf16(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
      :: "r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate));
}

// The same with A in tensor memory: row i in lane i, two values of K a column.
__device__ __forceinline__ void mma_bf16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
      :: "r"(d_tmem), "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate));
}

// D fp32, A and B bf16, both K-major, M = 128.
__host__ __device__ constexpr uint32_t idesc_of(int n) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (uint32_t(n >> 3) << 17) | (uint32_t(kTileRows >> 4) << 24);
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];"
      :: "r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z) : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void sts128(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" :: "r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// Pieces of 16 or 4 bytes.
template <int kBytes>
struct PieceOf;
template <>
struct PieceOf<16> {
  using type = uint4;
};
template <>
struct PieceOf<4> {
  using type = uint32_t;
};
__device__ __forceinline__ void ld_shared_piece(uint4& v, uint32_t a) { v = lds128(a); }
__device__ __forceinline__ void ld_shared_piece(uint32_t& v, uint32_t a) {
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
}
template <int kBytes>
__device__ __forceinline__ void copy_async(uint32_t dst, const uint16_t* src) {
  if constexpr (kBytes == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" :: "r"(dst), "l"(src), "n"(kBytes) : "memory");
}

// A barrier of `threads` of the block's threads; whether ok holds for all of them.
__device__ __forceinline__ bool barrier_all(int id, int threads, bool ok) {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.and.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
               : "=r"(r) : "r"(uint32_t(ok)), "r"(id), "r"(threads) : "memory");
  return r != 0;
}

// The larger; NaN if either is.
__device__ __forceinline__ float max_or_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// Two fp32 to bf16, the first in the low half.
__device__ __forceinline__ uint32_t cvt_bf16x2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

// Byte offset of 16-byte piece c of row r in a tile of 128-byte rows with the 128-byte swizzle.
__device__ __forceinline__ uint32_t swizzled(int r, int c) { return uint32_t(r) * 128u + uint32_t((c ^ (r & 7)) << 4); }

// Eight values of a row from k on into shared memory, zeros where they are not live, by an asynchronous copy.
__device__ __forceinline__ void copy8_async(uint32_t dst, const uint16_t* row, bool live, int k) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
               :: "r"(dst), "l"(live ? row + k : row), "r"(live ? 16u : 0u) : "memory");
}
// Four bytes, or zeros where bytes is 0.
__device__ __forceinline__ void copy4_async(uint32_t dst, const uint16_t* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" :: "r"(dst), "l"(src), "r"(bytes) : "memory");
}
// What this thread wrote to shared memory becomes visible to the tensor core (after the barrier that follows).
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// n / d for 0 <= n < 4096, d <= 32 and inv = 1 / d: the half keeps the product clear of whole numbers.
__device__ __forceinline__ int quotient(int n, float inv) { return int((float(n) + 0.5f) * inv); }

// A place in a ring of barriers, and the parity of its turn.
struct Place {
  int i = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void next(int n) {
    if (++i == n) i = 0, parity ^= 1u;
  }
};

struct TileParams {
  Args a;
  Sorted s;
  int rp;                   // rank rounded up to 16
  int kb, kb_slice;         // blocks of 64 of K, and of one split
  int stages;               // shrink
  int slots, b_bufs;        // expand: of y, of B
  int vec, vec_b;           // rows of x and A, of B, on 16-byte boundaries
  uint32_t tmem_cols;
};

// v between the two kernels: four values at a time of each row, [split][rank / 4][row], so that 32 lanes with a row each pass whole
// lines (with a row's values side by side 8192 x 14336 at rank 64 took 134 us against 124, then).
__device__ __forceinline__ float4* four_of_v(const TileParams& p, int split, int four, int64_t row) {
  return reinterpret_cast<float4*>(p.s.v) + (int64_t(split) * (p.rp / 4) + four) * p.a.M + row;
}

constexpr int kCopyThreads = 256;  // expand: those that copy y and out
constexpr int kCopyRows = kTileRows / (kCopyThreads / 32);  // of a warp

struct TileCtl {
  uint64_t done[8];    // MMAs of a stage (shrink), of a step (expand)
  uint64_t loaded[8];  // A of a stage, B of a step
  uint64_t read[2];    // expand: the warps that have read a step's sums
  uint64_t y_in[4], y_out[4];  // expand: a slot holds y, holds out
  uint64_t freed[4];           // expand: B's buffer has been multiplied
  uint32_t tmem_base;
  int abort_flag;
};

__device__ __forceinline__ uint32_t align1024(uint32_t a) { return (a + 1023u) & ~1023u; }

// The start and end that both kernels share: barriers and tensor memory. The trigger for the next kernel comes after the
// tensor memory is held, so that no CTA of a later kernel can hold it while one of this kernel waits for it.
// (loads: arrivals on a load's barrier; warps: those that join sums with y)
__device__ __forceinline__ void tile_begin(TileCtl* ctl, uint32_t cols, int loads, int warps) {
  if (threadIdx.x == 0) {
    for (int i = 0; i < 8; ++i) {
      mbar_init(smem_u32(&ctl->done[i]), 1);
      mbar_init(smem_u32(&ctl->loaded[i]), uint32_t(loads));
    }
    for (int i = 0; i < 2; ++i) mbar_init(smem_u32(&ctl->read[i]), uint32_t(warps));
    for (int i = 0; i < 4; ++i) {
      mbar_init(smem_u32(&ctl->y_in[i]), kCopyThreads);
      mbar_init(smem_u32(&ctl->y_out[i]), uint32_t(warps));
      mbar_init(smem_u32(&ctl->freed[i]), 1);
    }
    ctl->abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_async();
  }
  if (threadIdx.x < 32) {
    __syncwarp();
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                 :: "r"(smem_u32(&ctl->tmem_base)), "r"(cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  pdl_trigger();
  pdl_wait();
}
__device__ __forceinline__ void tile_end(TileCtl* ctl, uint32_t cols) {
  asm volatile("cp.async.wait_all;" ::: "memory");
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  if (threadIdx.x < 32)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(ctl->tmem_base), "r"(cols) : "memory");
}

// v[split][row] = A[e] x[row's token] over the split's K, for a tile's rows. Warps 0 to 7 copy the tile's rows of x (any
// tokens: eight threads a 128-byte piece of a row, asynchronous 16-byte copies) and, by TMA, A's into a ring of stages, whose
// barrier counts the copies' completion; warp 8 issues the MMAs. (With a fence for the tensor core in the copying
// threads, which waits for their copies in flight, a step took a load's latency: 27 us for 8192 x 4096 at rank 64.)
// Bounds: the first wave's fill and the stream of x (8192 x 4096 at rank 64: 19 us, 3.9 TB/s; the tensor cores are busy for 10
// percent). A tile of 128 rows is an MMA's; K splits fill the SMs (splits_of).
// kPiece: the bytes of a copy, as many as all rows of x and A start and end on. 4: a warp copies 128 bytes of a row. 2: whole
// pieces are loaded and shifted into place. A tile whose wait ran out gets NaN for its rows, so that the second product leaves
// nothing of an earlier call's v.
template <int kPiece, bool kWithhold>
__global__ void __launch_bounds__(kShrinkThreads, 2)
shrink_kernel(const __grid_constant__ CUtensorMap tmap_a, const __grid_constant__ TileParams p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ TileCtl ctl;
  const uint32_t base = align1024(smem_u32(smem_raw));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  tile_begin(&ctl, p.tmem_cols, kTileThreads + 1, 1);
  const int tile = blockIdx.x;
  const Args& g = p.a;
  const int K = int(g.K), r = g.rank;
  [[maybe_unused]] __shared__ const uint16_t* x_row[kPiece == 4 ? kTileRows : 1];
  if (tile < *p.s.n_tiles) {
    const block::RowTile t = p.s.tiles[tile];
    if constexpr (kPiece == 4) {
      const int row = t.row0 + int(threadIdx.x);
      if (threadIdx.x < kTileRows && row < t.row_end) x_row[threadIdx.x] = g.x + int64_t(p.s.order[row]) * g.ldx;
      __syncthreads();
    }
    const int kb0 = int(blockIdx.y) * p.kb_slice, steps = min(p.kb, kb0 + p.kb_slice) - kb0;
    if (t.expert < g.adapters && steps > 0) {
      const int rows = min(kTileRows, t.row_end - t.row0);
      const uint32_t stage_bytes = kXBytes + uint32_t(p.rp) * 128u;
      auto wait = [&](uint64_t* bars, int step) {
        return mbar_wait_short(smem_u32(bars + step % p.stages), uint32_t(step / p.stages) & 1u, &ctl.abort_flag,
                               &g_lora_error, kWithhold ? kWithheldNs : kWaitLimitNs);
      };
      bool ok = true;
      int filled = 0;
      if (warp == kTileThreads / 32) {
        for (int i = 0; i < steps; ++i) {
          if (!(ok = __all_sync(0xffffffffu, wait(ctl.loaded, i)))) break;
          fence_async();  // what the copying threads wrote becomes visible to the tensor core
          tmem_fence_after();
          if (elect_one()) {
            const uint32_t st = base + uint32_t(i % p.stages) * stage_bytes;
            const uint64_t ad = make_sdesc(st), bd = make_sdesc(st + kXBytes);
#pragma unroll
            for (int kk = 0; kk < kBk / 16; ++kk)
              mma_bf16(ctl.tmem_base, ad + uint64_t(kk * 2), bd + uint64_t(kk * 2), idesc_of(p.rp), i != 0 || kk != 0);
            mma_commit<false>(smem_u32(&ctl.done[i % p.stages]));
          }
          __syncwarp();
        }
      } else {
        // eight threads a row; this thread's rows of x
        const int piece = threadIdx.x & 7, first = threadIdx.x >> 3;
        const uint16_t* x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = first + 32 * i;
          x[i] = row < rows ? g.x + int64_t(p.s.order[t.row0 + row]) * g.ldx : g.x;
        }
        const uint16_t* A = g.a + int64_t(t.expert) * r * K;
        auto a_row = [&](int i) { return A + int64_t(min(first + 32 * i, r - 1)) * K; };
        if constexpr (kPiece == 4) {
          // (rows of x past the tile's leave nothing in others' sums: they are not copied)
          for (; filled < steps; ++filled) {
            if (filled >= p.stages && !(ok = wait(ctl.done, filled - p.stages))) break;
            const uint32_t st = base + uint32_t(filled % p.stages) * stage_bytes;
            const uint32_t bar = smem_u32(&ctl.loaded[filled % p.stages]);
            const int k = (kb0 + filled) * kBk + 2 * lane, bytes = k < K ? 4 : 0, k_in = k < K ? k : 0;
            const uint32_t word = uint32_t(lane & 3) * 4u;
#pragma unroll 4
            for (int row = warp; row < rows; row += kTileThreads / 32)
              copy4_async(st + swizzled(row, lane >> 2) + word, x_row[row] + k_in, bytes);
#pragma unroll 4
            for (int row = warp; row < p.rp; row += kTileThreads / 32)
              copy4_async(st + kXBytes + swizzled(row, lane >> 2) + word, A + int64_t(min(row, r - 1)) * K + k_in,
                          row < r ? bytes : 0);
            if (threadIdx.x == 0) mbar_arrive(bar);  // (in place of the arrival that announces A's bytes)
            asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" :: "r"(bar) : "memory");
          }
        } else if constexpr (kPiece == 16) {
          for (; filled < steps; ++filled) {
            if (filled >= p.stages && !(ok = wait(ctl.done, filled - p.stages))) break;
            const uint32_t st = base + uint32_t(filled % p.stages) * stage_bytes;
            const uint32_t bar = smem_u32(&ctl.loaded[filled % p.stages]);
            if (threadIdx.x == 0 && !(kWithhold && blockIdx.x == 0 && blockIdx.y == 0 && filled == steps - 1)) {
              mbar_arrive_expect_tx(bar, uint32_t(p.rp) * 128u);
              tma_load_3d(st + kXBytes, &tmap_a, bar, (kb0 + filled) * 128, 0, t.expert);
            }
            const int k = (kb0 + filled) * kBk + piece * 8;
#pragma unroll
            for (int i = 0; i < 4; ++i)
              copy8_async(st + swizzled(first + 32 * i, piece), x[i], first + 32 * i < rows && k < K, k);
            asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" :: "r"(bar) : "memory");
          }
        } else {
          // rows that start or end anywhere: whole pieces, loaded a step ahead and shifted into place. (The distance from a piece
          // is one for a row: K steps are whole pieces.)
          constexpr int kAhead = 4;  // rows of A whose loads run ahead; the others', of ranks over 128, do not
          int x_at[4], a_at[kAhead];
          Raw8 xr[4], ar[kAhead];
          auto load = [&](int step) {
            const int k = (kb0 + step) * kBk + piece * 8;
#pragma unroll
            for (int i = 0; i < 4; ++i) xr[i] = load8_raw(x[i], x_at[i], k, first + 32 * i < rows ? K : 0);
#pragma unroll
            for (int i = 0; i < kAhead; ++i) ar[i] = load8_raw(a_row(i), a_at[i], k, first + 32 * i < r ? K : 0);
          };
#pragma unroll
          for (int i = 0; i < 4; ++i) x_at[i] = off_piece(x[i]), a_at[i] = off_piece(a_row(i));
          load(0);
          for (; filled < steps; ++filled) {
            if (filled >= p.stages && !(ok = wait(ctl.done, filled - p.stages))) break;
            const uint32_t st = base + uint32_t(filled % p.stages) * stage_bytes;
            const uint32_t bar = smem_u32(&ctl.loaded[filled % p.stages]);
            const int k = (kb0 + filled) * kBk + piece * 8;
#pragma unroll
            for (int i = 0; i < 4; ++i)
              sts128(st + swizzled(first + 32 * i, piece), values8(xr[i], x_at[i], k, first + 32 * i < rows ? K : 0));
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
              if (first + 32 * i < p.rp)
                sts128(st + kXBytes + swizzled(first + 32 * i, piece), values8(ar[i], a_at[i], k, first + 32 * i < r ? K : 0));
            for (int row = first + 32 * kAhead; row < p.rp; row += 32)
              sts128(st + kXBytes + swizzled(row, piece),
                     row < r && k < K ? load8_any(A + int64_t(row) * K, k, K) : make_uint4(0, 0, 0, 0));
            fence_async();  // (before the next loads: it waits for what is in flight)
            if (threadIdx.x == 0) mbar_arrive(bar);  // (in place of the arrival that announces A's bytes)
            mbar_arrive(bar);
            if (filled + 1 < steps) load(filled + 1);
          }
        }
      }
      if (ok) ok = wait(ctl.done, steps - 1);
      if (__syncthreads_and(ok)) {
        tmem_fence_after();
        // four warps hold the tile's rows, the other four the second half of the columns
        const int row = (warp & 3) * 32 + lane;
        float4* dst = four_of_v(p, blockIdx.y, 0, t.row0 + row);
        const uint32_t from = ctl.tmem_base + (uint32_t((warp & 3) * 32) << 16);
        for (int c = (warp >> 2) * 32; warp < kTileThreads / 32 && c < p.rp; c += 64) {
          uint32_t f[32];
          __syncwarp();
          tmem_ld32(from + c, f);
          if (row < rows) {
#pragma unroll
            for (int q = 0; q < 8; ++q)
              if (c + 4 * q < p.rp)
                *reinterpret_cast<uint4*>(dst + (c / 4 + q) * g.M) = make_uint4(f[4 * q], f[4 * q + 1], f[4 * q + 2], f[4 * q + 3]);
          }
        }
      } else {
        if (int(threadIdx.x) < rows) {
          const float nan = __uint_as_float(0x7FC00000u);
          *four_of_v(p, blockIdx.y, 0, t.row0 + threadIdx.x) = make_float4(nan, nan, nan, nan);
        }
        if (threadIdx.x == 0)  // nothing of a load may land after the CTA has left
          for (int i = max(0, filled - p.stages); i < filled; ++i)
            mbar_wait_bounded(smem_u32(&ctl.loaded[i % p.stages]), uint32_t(i / p.stages) & 1u, nullptr, &g_lora_error,
                              kWithhold ? kWithheldNs : kWaitLimitNs);
      }
    }
  }
  tile_end(&ctl, p.tmem_cols);
}

// v of a tile's rows, the sum of the splits in order, as the sum of three bf16 numbers: eight bits each, so that nothing of v's 24
// is lost (above 2^-133, the smallest bf16 number). The first two go to swizzled tiles of shared memory, the third to tensor memory
// (as the operand of the same MMAs: three tiles of rank 256 leave no room for B and y, and at rank 64 one would cost a slot of y).
// `groups` of four warps share out the pieces of eight values; in a warp with few rows several lanes share a row's. (Where each
// lane passed all of its row's pieces, one after the other, 64 tokens of 32 adapters took 67 us at K = N = 8192 and rank 128, 54 so.)
// kSteps: addresses by steps from the first, for kernels of 72 registers (8192 x 14336 at rank 64: 120 us, 131 otherwise); else each
// by itself, so that no load waits for another's address (2048 x 4096 at rank 128: 46 us against 49).
// nan_row gets `tag` for the rows with a NaN.
template <bool kSteps>
__device__ __forceinline__ void put_v(const TileParams& p, const block::RowTile& t, int rows, uint32_t v_hi, uint32_t v_mid,
                                      uint32_t v_lo_tmem, int groups, int* nan_row, int tag) {
  const int lane = threadIdx.x & 31, quarter = int(threadIdx.x >> 5) & 3, group = int(threadIdx.x) / kTileRows;
  const int live = min(32, rows - quarter * 32);  // rows of this warp's 32 places
  if (live <= 0) return;  // (what lies in places without a row reaches no other row's sums)
  const int mine = (p.rp / 8 - group + groups - 1) / groups;  // pieces of this group
  const int shift = live > 1 ? __clz(live - 1) - 27 : 5, share = 1 << shift;  // lanes of a row
  const int at = lane >> shift;
  const int64_t M = p.a.M, split = p.rp / 4 * M;
  const int64_t row = t.row0 + quarter * 32 + at;
  const float4* from = four_of_v(p, 0, 2 * (group + (lane & (share - 1)) * groups), row);
  const uint32_t to_row = uint32_t(quarter * 32 + at) * 128u;
  const uint32_t to_tmem = v_lo_tmem + (uint32_t(quarter * 32) << 16);
  for (int k0 = 0; k0 < mine; k0 += share, from += int64_t(2 * share * groups) * M) {
    const int k = k0 + (lane & (share - 1)), c = group + k * groups;
    const bool have = at < live && k < mine;
    float f[8] = {};
    if (have) {
      const float4* next = from;
      for (int s0 = 0; s0 < p.s.splits; s0 += 4, next += 4 * split) {  // four splits' loads at once, added in order
        float4 in[4][2];
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const float4* four = kSteps ? next + s * split : four_of_v(p, s0 + s, 2 * c, row);
          const bool more = s0 + s < p.s.splits;
          in[s][0] = more ? four[0] : make_float4(0.f, 0.f, 0.f, 0.f);
          in[s][1] = more ? four[M] : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          f[0] += in[s][0].x, f[1] += in[s][0].y, f[2] += in[s][0].z, f[3] += in[s][0].w;
          f[4] += in[s][1].x, f[5] += in[s][1].y, f[6] += in[s][1].z, f[7] += in[s][1].w;
        }
      }
    }
    if (c * 8 + 8 > p.a.rank) {  // (behind the rank an infinity of x times zero is NaN)
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = c * 8 + i < p.a.rank ? f[i] : 0.0f;
    }
    float most = f[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) most = max_or_nan(most, f[i]);
    if (most != most) nan_row[quarter * 32 + at] = tag;  // (more than one lane may say so)
    // the next eight bits of each, and what they leave (where that is infinite or NaN the sums are, and are taken again)
    uint32_t w[4];
    auto next8 = [&]() {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        w[j] = cvt_bf16x2(f[2 * j], f[2 * j + 1]);
        f[2 * j] -= bf16_lo(w[j]);
        f[2 * j + 1] -= bf16_hi(w[j]);
      }
    };
    const uint32_t to = uint32_t(c >> 3) * kXBytes + to_row + uint32_t(((c & 7) ^ (at & 7)) << 4);
    next8();
    if (have) sts128(v_hi + to, make_uint4(w[0], w[1], w[2], w[3]));
    next8();
    if (have) sts128(v_mid + to, make_uint4(w[0], w[1], w[2], w[3]));
    next8();
    if (share == 1) {
      tmem_st4(to_tmem + uint32_t(c) * 4u, w);
      continue;
    }
    for (int j = 0; j < share && k0 + j < mine; ++j) {  // a row's third parts to the lane of its place
      uint32_t l[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) l[i] = __shfl_sync(0xffffffffu, w[i], (lane << shift) + j);
      tmem_st4(to_tmem + uint32_t(group + (k0 + j) * groups) * 4u, l);
    }
  }
  tmem_wait_st();
}

// Whether any of a thread's sums is not finite, and which.
__device__ __forceinline__ bool any_not_finite(const uint32_t (&f)[32]) {
  uint64_t z[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 16; ++i)
    z[i & 1] = fma_f32x2(pack_f32x2(__uint_as_float(f[2 * i]), __uint_as_float(f[2 * i + 1])), 0, z[i & 1]);
  return !(lo_of(z[0]) + hi_of(z[0]) + lo_of(z[1]) + hi_of(z[1]) == 0.0f);
}
__device__ __forceinline__ uint32_t not_finite(const uint32_t (&f)[32]) {
  uint32_t bad = 0;
#pragma unroll
  for (int i = 0; i < 32; ++i) bad |= fabsf(__uint_as_float(f[i])) <= FLT_MAX ? 0u : 1u << i;
  return bad;
}

// One sum in fp32, from v's splits as put_v adds them and a row of B; a NaN ends it.
__device__ __forceinline__ float sum_again(const TileParams& p, int64_t row, const uint16_t* b) {
  float sum = 0.0f;
#pragma unroll 1
  for (int j = 0; j < p.a.rank && sum == sum; j += 4) {
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
    for (int s = 0; s < p.s.splits; ++s) {
      const float4 in = *four_of_v(p, s, j >> 2, row);
      v.x += in.x, v.y += in.y, v.z += in.z, v.w += in.w;
    }
    const int n = p.a.rank - j;
    sum = fmaf(bf16_bits_to_float(b[j]), v.x, sum);
    if (n > 1) sum = fmaf(bf16_bits_to_float(b[j + 1]), v.y, sum);
    if (n > 2) sum = fmaf(bf16_bits_to_float(b[j + 2]), v.z, sum);
    if (n > 3) sum = fmaf(bf16_bits_to_float(b[j + 3]), v.w, sum);
  }
  return sum;
}

// The parts of v lose what the formula has where a number is not finite: an infinity of B times a part that is 0 or of the other
// sign, or a v that rounds to an infinite bf16 number. Such sums of a warp's rows and columns (`bad`: this lane's row's) are
// taken once more, from v and B themselves, and put in their places in tensor memory: a lane a column where the rows are far fewer
// (a token's infinity), else a lane a row (an infinity in B). What is NaN all the same is left: rows with a NaN in v are not
// among `bad`, and a column whose B starts with a NaN is passed over. `row0`: the warp's first row of v, `b`: the first column's of
// B. (2048 tokens of four adapters, 4096 to 8192 at rank 64: 36 us when all is finite and with NaN tokens or adapters, 66 with an
// infinite token, 52 with an infinite value in B, 1.2 ms with an adapter whose B is infinite throughout.)
__device__ __forceinline__ void sums_again(const TileParams& p, uint32_t taddr, uint32_t bad, int64_t row0, const uint16_t* b) {
  const int lane = threadIdx.x & 31, rank = p.a.rank;
  uint32_t columns = __reduce_or_sync(0xffffffffu, bad);
  const float first = (columns >> lane) & 1u ? bf16_bits_to_float(b[lane * rank]) : 0.0f;
  columns &= ~__ballot_sync(0xffffffffu, first != first);
  bad &= columns;
  const uint32_t rows = __ballot_sync(0xffffffffu, bad != 0);
  if (__popc(rows) * 4 <= __popc(columns)) {
#pragma unroll 1
    for (uint32_t left = rows; left != 0; left &= left - 1) {
      const int r = __ffs(left) - 1;
      const uint32_t of_row = __shfl_sync(0xffffffffu, bad, r);
      const float sum = (of_row >> lane) & 1u ? sum_again(p, row0 + r, b + lane * rank) : 0.0f;
      __syncwarp();
#pragma unroll 1
      for (uint32_t c = of_row; c != 0; c &= c - 1) {
        const int column = __ffs(c) - 1;
        const float mine = __shfl_sync(0xffffffffu, sum, column);
        const uint32_t was = tmem_ld1(taddr + column);
        tmem_st1(taddr + column, lane == r ? __float_as_uint(mine) : was);
        tmem_wait_st();
      }
    }
  } else {
#pragma unroll 1
    for (uint32_t c = columns; c != 0; c &= c - 1) {
      const int column = __ffs(c) - 1;
      uint32_t sum = tmem_ld1(taddr + column);
      if ((bad >> column) & 1u) sum = __float_as_uint(sum_again(p, row0 + lane, b + column * rank));
      __syncwarp();
      tmem_st1(taddr + column, sum);
    }
    tmem_wait_st();
  }
}

// out = y + s B[e] v. The CTAs share out
// (tile, kBn columns) steps in equal runs, so that a CTA passes along the columns of one tile and perhaps on to the next.
//   joining warps  32 rows and 32 columns each: a thread reads its row of a step's sums from tensor memory, joins it with y in
//                  a slot of shared memory and writes the result over y there. Sums that are not finite are taken again in fp32
//                  first (sums_again; looking for them takes no time that shows, 122.4 us for the call with 8192 tokens either way).
//   issuing warp   loads B by TMA, two or three steps ahead, and issues the MMAs. Where the rows of B do not start on 16-byte
//                  boundaries (a rank that is no multiple of eight), four warps more load it in whole pieces.
//   copying warps  y into the slots, by asynchronous copies of kPiece bytes (2: rows of any alignment, by loads) as far ahead as
//                  there are slots, and out from them: every eighth row each, whole lines at a time (the rows of a tile may be
//                  any tokens).
// What was measured for 8192 x 14336: rows loaded and stored by the joining threads, 32 bytes of a row at a time, 111 us
// (each asks the L2 for a single sector); a bulk copy of 256 bytes a row each way 470 us (some 60 cycles a copy).
// Slot rows lie 16 bytes further apart than they are long, so that eight lanes' accesses down the rows take all banks.
// Bounds: the stream of y in and out (8192 x 14336 at rank 64 in 16 adapters: 97 us, 4.8 TB/s; the tensor cores are busy for 21
// percent of it); one CTA an SM, whose copying warps are its loads in flight (two CTAs of 64 columns: 138 us for the call
// against 128, then).
constexpr int join_threads(int bn) { return bn * 4; }
constexpr int kBThreads = 128;
constexpr int expand_threads(int bn, bool tma) { return join_threads(bn) + 32 + kCopyThreads + (tma ? 0 : kBThreads); }

template <int kBn, int kPiece, bool kTma, bool kWithhold>
__global__ void __launch_bounds__(kBn * 4 + 32 + kCopyThreads + (kTma ? 0 : kBThreads), 1)
expand_kernel(const __grid_constant__ CUtensorMap tmap_b, const __grid_constant__ TileParams p) {
  constexpr int kJoin = kBn * 4, kJoinWarps = kJoin / 32;
  constexpr int kMostK = kBn == 128 ? 4 : kBn == 64 ? 12 : 16;  // K steps of the ranks that take this width (launch_sorted)
  constexpr uint32_t kPitch = kBn * 2 + 16, kSlotBytes = kTileRows * kPitch;
  constexpr unsigned long long kLimit = kWithhold ? kWithheldNs : kWaitLimitNs;
  extern __shared__ uint8_t smem_raw[];
  __shared__ TileCtl ctl;
  __shared__ int nan_row[kTileRows];  // the tile, plus one, whose row there has a NaN in v
  const uint32_t base = align1024(smem_u32(smem_raw));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x < kTileRows) nan_row[threadIdx.x] = 0;
  tile_begin(&ctl, p.tmem_cols, kTma ? 1 : kBThreads, kJoinWarps);
  const Args& g = p.a;
  const int N = int(g.N);
  const int steps = (N + kBn - 1) / kBn;
  const int64_t total = int64_t(*p.s.n_tiles) * steps, run = (total + gridDim.x - 1) / gridDim.x;
  const int64_t begin = run * blockIdx.x, end = min(total, run * (blockIdx.x + 1));
  const int rk = (p.rp + kBk - 1) / kBk;  // 128-byte rows that the rank fills
  const uint32_t v_hi = base, v_mid = base + uint32_t(rk) * kXBytes, b_at = v_mid + uint32_t(rk) * kXBytes;
  const uint32_t v_lo_tmem = ctl.tmem_base + 2 * kBn;  // behind two steps' sums
  const uint32_t b_bytes = uint32_t(rk) * (kBn * 128u);
  const uint32_t slots_at = b_at + uint32_t(p.b_bufs) * b_bytes;
  auto wait = [&](uint64_t* bar, uint32_t it) {  // the it-th step's phase of a pair of barriers
    return mbar_wait_short(smem_u32(bar + (it & 1u)), (it >> 1) & 1u, &ctl.abort_flag, &g_lora_error, kLimit);
  };
  auto wait_at = [&](uint64_t* bars, const Place& a) {
    return mbar_wait_short(smem_u32(bars + a.i), a.parity, &ctl.abort_flag, &g_lora_error, kLimit);
  };
  auto withheld = [&](const Place& b) { return kWithhold && blockIdx.x == 0 && b.i == 1 && b.parity == 0; };  // the second B

  constexpr int kCopyWarps = kCopyThreads / 32;
  if (!kTma && warp > kJoinWarps + kCopyWarps) {
    // ---------------- B where TMA cannot load it ----------------
    const int pieces = p.rp / 8, n_pieces = kBn * pieces;
    const float inv_pieces = 1.0f / float(pieces);
    const int me = threadIdx.x - (kJoinWarps + 1 + kCopyWarps) * 32;
    Place at, last;  // a buffer is free once its last turn's MMAs are done
    int untouched = p.b_bufs;
    bool ok = true;
    for (int64_t u = begin; ok && u < end;) {
      const int tile = int(u / steps), s0 = int(u - int64_t(tile) * steps), s1 = int(min(int64_t(steps), s0 + (end - u)));
      u += s1 - s0;
      const block::RowTile t = p.s.tiles[tile];
      if (t.expert >= g.adapters) continue;
      const uint16_t* B = g.b + int64_t(t.expert) * N * g.rank;
      for (int s = s0; s < s1; ++s, at.next(p.b_bufs)) {
        if (untouched > 0) {
          --untouched;
        } else {
          if (!(ok = wait_at(ctl.freed, last))) break;
          last.next(p.b_bufs);
        }
        const uint32_t to = b_at + uint32_t(at.i) * b_bytes;
        for (int i0 = me; i0 < n_pieces; i0 += 4 * kBThreads) {  // four loads at once
          Raw8 v[4];
          int where[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int i = min(i0 + j * kBThreads, n_pieces - 1), row = quotient(i, inv_pieces), c = i - row * pieces;
            const int n = min(s * kBn + row, N - 1);
            const uint16_t* from = B + int64_t(n) * g.rank;
            where[j] = row * 32 + c;
            v[j] = load8_raw(from, off_piece(from), c * 8, s * kBn + row < N ? g.rank : 0);
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int row = where[j] / 32, c = where[j] % 32;
            const uint16_t* from = B + int64_t(min(s * kBn + row, N - 1)) * g.rank;
            sts128(to + uint32_t(c >> 3) * (kBn * 128u) + swizzled(row, c & 7),
                   values8(v[j], off_piece(from), c * 8, s * kBn + row < N ? g.rank : 0));
          }
        }
        fence_async();
        if (!withheld(at) || me != 0) mbar_arrive(smem_u32(&ctl.loaded[at.i]));
      }
    }
  } else if (warp > kJoinWarps) {
    // ---------------- copies of y and out: a warp has every eighth row, lane l knows the token of the l-th ----------------
    // (so that the few rows of a short tile are shared out)
    constexpr int kCols = kPiece == 2 ? 8 : kPiece / 2;                     // of a lane
    constexpr int kLanes = kBn / kCols < 32 ? kBn / kCols : 32;             // of a row
    constexpr int kRowsAt = 32 / kLanes, kParts = kBn / kCols / kLanes;     // rows at a time, parts of a row
    constexpr int kTimes = kCopyRows / kRowsAt * kParts;
    constexpr int kBatch = kPiece == 4 ? (kTimes < 16 ? kTimes : 16) : (kTimes < 4 ? kTimes : 4);
    const int first = warp - kJoinWarps - 1, at_row = lane / kLanes, at_col = (lane % kLanes) * kCols;
    struct Walk {
      int64_t u;      // the step after this part of a tile
      int s, s1;      // columns of the next step, and where the part ends
      int token, rows;  // .. of the warp, behind which there is nothing to copy
    };
    auto enter = [&](Walk& w) {  // the next part of a tile with something to do; false behind the last
      while (w.u < end) {
        const int tile = int(w.u / steps);
        w.s = int(w.u - int64_t(tile) * steps);
        w.s1 = int(min(int64_t(steps), w.s + (end - w.u)));
        w.u += w.s1 - w.s;
        const block::RowTile t = p.s.tiles[tile];
        if (t.expert >= g.adapters && g.out == g.y) continue;
        w.rows = (min(kTileRows, t.row_end - t.row0) - first + kCopyWarps - 1) / kCopyWarps;
        w.token = lane < w.rows ? p.s.order[t.row0 + first + lane * kCopyWarps] : -1;
        return true;
      }
      return false;
    };
    constexpr uint32_t kRowPitch = kCopyWarps * kPitch;  // from a warp's row to its next
    const uint32_t mine = slots_at + uint32_t(first) * kPitch + uint32_t(at_row) * kRowPitch + at_col * 2u;
    // the i-th access of a lane: a row of the warp's, a part of it
    auto row_of = [&](int i) { return i / kParts * kRowsAt; };
    auto part_of = [&](int i) { return i % kParts * kLanes * kCols; };
    Walk in = {begin}, out = {begin};
    bool more = enter(in), left = enter(out);
    Place in_at, out_at;
    int held = 0;  // slots that were loaded and not yet stored
    while (left) {
      for (; more && held < p.slots; ++held, in_at.next(p.slots)) {
        const uint32_t to = mine + uint32_t(in_at.i) * kSlotBytes, bar = smem_u32(&ctl.y_in[in_at.i]);
        const int col = in.s * kBn + at_col;
        if constexpr (kPiece >= 4) {
#pragma unroll
          for (int i = 0; i < kTimes; ++i) {
            const int token = __shfl_sync(0xffffffffu, in.token, row_of(i) + at_row), n = col + part_of(i);
            if (token >= 0 && n < N) copy_async<kPiece>(to + uint32_t(row_of(i)) * kRowPitch + part_of(i) * 2u, g.y + token * g.ldy + n);
          }
          asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" :: "r"(bar) : "memory");
        } else {
          // rows that start off 4-byte boundaries: whole pieces, shifted into place
#pragma unroll 1
          for (int i0 = 0; i0 < kTimes && row_of(i0) < in.rows; i0 += kBatch) {
            Raw8 v[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
              const int token = __shfl_sync(0xffffffffu, in.token, row_of(i0 + i) + at_row);
              const uint16_t* row = g.y + (token >= 0 ? token * g.ldy : 0);
              v[i] = load8_raw(row, off_piece(row), col, token >= 0 ? N : 0);  // (col is whole eights)
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
              const int token = __shfl_sync(0xffffffffu, in.token, row_of(i0 + i) + at_row);
              const uint16_t* row = g.y + (token >= 0 ? token * g.ldy : 0);
              sts128(to + uint32_t(row_of(i0 + i)) * kRowPitch, values8(v[i], off_piece(row), col, token >= 0 ? N : 0));
            }
          }
          mbar_arrive(bar);
        }
        if (++in.s == in.s1) more = enter(in);
      }
      if (!__all_sync(0xffffffffu, wait_at(ctl.y_out, out_at))) break;
      const uint32_t from = mine + uint32_t(out_at.i) * kSlotBytes;
      const int col = out.s * kBn + at_col;
      using Piece = typename PieceOf<kPiece == 2 ? 16 : kPiece>::type;
#pragma unroll 1
      for (int i0 = 0; i0 < kTimes && row_of(i0) < out.rows; i0 += kBatch) {
        Piece v[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
          ld_shared_piece(v[i], from + uint32_t(row_of(i0 + i)) * kRowPitch + part_of(i0 + i) * 2u);
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int token = __shfl_sync(0xffffffffu, out.token, row_of(i0 + i) + at_row), n = col + part_of(i0 + i);
          if constexpr (kPiece == 2)
            store8_run(g.out + (token >= 0 ? token * g.ldo : 0), n, N, v[i], token >= 0 && n < N, lane % kLanes > 0,
                       lane % kLanes < kLanes - 1 && n + 8 < N);
          else if (token >= 0 && n < N)
            *reinterpret_cast<Piece*>(g.out + token * g.ldo + n) = v[i];
        }
      }
      --held;
      out_at.next(p.slots);
      if (++out.s == out.s1) left = enter(out);
    }
  } else {
    uint32_t it = 0;        // steps with an adapter so far
    Place slot, filled, used;  // of all steps that pass the slots; of B, filled and multiplied
    // descriptors of v and of B; K steps of 16 and tiles of 64 lie at fixed distances (in 16-byte units)
    const uint64_t v_desc = make_sdesc(v_hi), b_desc = make_sdesc(b_at);
    const uint32_t mid_part = uint32_t(rk) * (kXBytes >> 4);
    bool ok = true;
    for (int64_t u = begin; u < end;) {
      const int tile = int(u / steps), s0 = int(u - int64_t(tile) * steps), s1 = int(min(int64_t(steps), s0 + (end - u)));
      u += s1 - s0;
      const block::RowTile t = p.s.tiles[tile];
      const int rows = min(kTileRows, t.row_end - t.row0);
      if (t.expert >= g.adapters) {  // no adapter: y passes the slots as it is
        if (g.out != g.y && warp < kJoinWarps)
          for (int s = s0; ok && s < s1; ++s, slot.next(p.slots)) {
            if (!(ok = __all_sync(0xffffffffu, wait_at(ctl.y_in, slot)))) break;
            if (lane == 0) mbar_arrive(smem_u32(&ctl.y_out[slot.i]));
          }
        continue;
      }
      auto fill = [&](int step) {  // by the issuing warp
        if (kTma && !withheld(filled) && elect_one()) {
          const uint32_t bar = smem_u32(&ctl.loaded[filled.i]);
          mbar_arrive_expect_tx(bar, b_bytes);
          for (int i = 0; i < rk; ++i)
            tma_load_3d(b_at + uint32_t(filled.i) * b_bytes + uint32_t(i) * (kBn * 128u), &tmap_b, bar, i * 128, step * kBn,
                        t.expert);
        }
        __syncwarp();
        filled.next(p.b_bufs);
      };
      if (warp == kJoinWarps) {
        // the buffers are free behind the last tile's last MMAs
        ok = __all_sync(0xffffffffu, ok && (it == 0 || wait(ctl.done, it - 1)));
        for (int i = 0; ok && i < p.b_bufs - 1 && s0 + i < s1; ++i) fill(s0 + i);
      } else {
        // all of the last tile's MMAs are done: each warp waited for its last step
        put_v<kBn == 128>(p, t, rows, v_hi, v_mid, v_lo_tmem, kJoin / kTileRows, nan_row, tile + 1);
        fence_async();
        tmem_fence_before();
      }
      if (!barrier_all(1, kJoin + 32, ok)) {
        ok = false;
        break;
      }
      if (warp == kJoinWarps) {
        // (the warp stays together around the one lane that issues)
        for (int s = s0; s < s1; ++s, ++it) {
          ok = __all_sync(0xffffffffu, wait_at(ctl.loaded, used) && (it < 2 || wait(ctl.read, it - 2)));
          if (!ok) break;
          tmem_fence_after();
          if (elect_one()) {
            // (straight code: a thread's chain of address arithmetic around eight MMAs took 2000 cycles a step)
            const uint64_t b = b_desc + uint32_t(used.i) * (b_bytes >> 4);
            const uint32_t d = ctl.tmem_base + (it & 1u) * kBn;
#pragma unroll
            for (int i = 0; i < kMostK; ++i) {
              if (i < p.rp / 16) {
                const uint64_t a = v_desc + uint32_t((i >> 2) * (kXBytes >> 4) + (i & 3) * 2);
                const uint64_t bi = b + uint32_t((i >> 2) * (kBn * 128 >> 4) + (i & 3) * 2);
                mma_bf16(d, a, bi, idesc_of(kBn), i != 0);
                mma_bf16(d, a + mid_part, bi, idesc_of(kBn), 1);
                mma_bf16_ta(d, v_lo_tmem + uint32_t(i) * 8u, bi, idesc_of(kBn), 1);
              }
            }
            mma_commit<false>(smem_u32(&ctl.done[it & 1u]));
            if (!kTma) mma_commit<false>(smem_u32(&ctl.freed[used.i]));
          }
          __syncwarp();
          used.next(p.b_bufs);
          // B as far ahead as there are buffers: the next to fill is that of the step before this one
          const int ahead = s + p.b_bufs - 1;
          if (ahead < s1) {
            if (s > s0) ok = __all_sync(0xffffffffu, wait(ctl.done, it - 1));
            if (!ok) break;
            fill(ahead);
          }
        }
        continue;
      }
      const int row = (warp & 3) * 32 + lane, group = warp >> 2;  // columns [32 group, 32 group + 32)
      const float scale = g.scales ? g.scales[t.expert] : 1.0f;
      const bool watched = row < rows && nan_row[row] != tile + 1;  // (all sums of a row with a NaN are NaN)
      for (int s = s0; s < s1; ++s, ++it, slot.next(p.slots)) {
        ok = ok && wait(ctl.done, it);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        tmem_fence_after();
        uint32_t f[32];
        const uint32_t sums = ctl.tmem_base + (it & 1u) * kBn + (uint32_t((warp & 3) * 32) << 16) + group * 32;
        tmem_ld32(sums, f);
        if (__any_sync(0xffffffffu, watched && any_not_finite(f))) {
          const int n = s * kBn + group * 32;  // columns past the last are no one's
          const uint32_t mask = N - n >= 32 ? ~0u : N > n ? (1u << (N - n)) - 1u : 0u;
          sums_again(p, sums, watched ? not_finite(f) & mask : 0u, t.row0 + (warp & 3) * 32,
                     g.b + (int64_t(t.expert) * N + n) * g.rank);
          tmem_ld32(sums, f);
        }
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&ctl.read[it & 1u]));
        if (!(ok = __all_sync(0xffffffffu, wait_at(ctl.y_in, slot)))) break;
        const uint32_t at = slots_at + uint32_t(slot.i) * kSlotBytes + uint32_t(row) * kPitch + uint32_t(group) * 64u;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4 v = lds128(at + i * 16);
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
          uint32_t o[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            o[j] = cvt_bf16x2(fmaf(scale, __uint_as_float(f[8 * i + 2 * j]), bf16_lo(w[j])),
                              fmaf(scale, __uint_as_float(f[8 * i + 2 * j + 1]), bf16_hi(w[j])));
          sts128(at + i * 16, make_uint4(o[0], o[1], o[2], o[3]));
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&ctl.y_out[slot.i]));
      }
    }
    if (kTma && !ok && threadIdx.x == kJoin)  // nothing of a load may land after the CTA has left
      for (; used.i != filled.i || used.parity != filled.parity; used.next(p.b_bufs))
        mbar_wait_bounded(smem_u32(&ctl.loaded[used.i]), used.parity, nullptr, &g_lora_error, kLimit);
  }
  __syncwarp();
  tile_end(&ctl, p.tmem_cols);
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

namespace {
PerDeviceCache<const void*, int> g_smem_cache;

bool allow_smem(const void* kfn) {
  int dev = 0, set = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  return g_smem_cache.get(dev, kfn, &set, [&](int* v) {
    *v = 1;
    cudaFuncAttributes at = {};
    return report_cuda(cudaFuncGetAttributes(&at, kfn), "lora attributes") == cudaSuccess &&
           report_cuda(cudaFuncSetAttribute(kfn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                            232448 - int(at.sharedSizeBytes)),
                       "lora smem attribute") == cudaSuccess;
  });
}
}  // namespace

// K splits of the first product: CTAs for the SMs, each with at least four blocks of K (two where rows are shifted into place),
// and no more than pay for themselves: a block takes 0.65 us (where rows start anywhere 1.5 to 2.2), and each split of a tile's
// sums about 0.01 us a rank to read in the second product. It goes by sizes alone, and by a GB300's 152 SMs: the
// workspace, which holds the splits, is asked for before there is an address or a device.
constexpr int kSms = 152;
int splits_of(int64_t M, int64_t K, int64_t adapters, int64_t rank) {
  const int64_t tiles = (M + kTileRows - 1) / kTileRows + std::min(M, adapters) / 2;
  const int64_t kb = (K + kBk - 1) / kBk;
  int64_t want = std::max<int64_t>(1, std::min<int64_t>(K % 8 == 0 ? kb / 4 : kb / 2, 2 * kSms / tiles));
  while (want > 1 && want * want * padded_rank(rank) > (K % 8 == 0 ? 65 : 150) * kb) --want;
  const int64_t slice = (kb + want - 1) / want;
  return int(std::max<int64_t>(1, (kb + slice - 1) / std::max<int64_t>(slice, 1)));
}

template <int kBn, int kPiece, bool kTma, bool kWithhold = false>
bool launch_expand_of(TileParams p, const CUtensorMap& map_b, int num_sms, cudaStream_t st) {
  auto kernel = expand_kernel<kBn, kPiece, kTma, kWithhold>;
  if (!allow_smem(reinterpret_cast<const void*>(kernel))) return false;
  const int rk = (p.rp + kBk - 1) / kBk;
  const size_t v = size_t(rk) * 2 * kXBytes, buf = size_t(rk) * kBn * 128, slot = size_t(kTileRows) * (kBn * 2 + 16);
  const size_t room = 232448 - 1024 - 1024 - v;  // (the control block and the alignment)
  p.b_bufs = room >= 4 * (buf + slot) ? 4 : 3;
  p.slots = int(std::min<size_t>(4, (room - p.b_bufs * buf) / slot));
  const int64_t units = p.s.max_tiles * ((p.a.N + kBn - 1) / kBn);
  p.tmem_cols = 32;
  while (int(p.tmem_cols) < 2 * kBn + p.rp / 2) p.tmem_cols *= 2;  // two steps' sums and v's last bits
  return launch(kernel, dim3(unsigned(std::min<int64_t>(units, num_sms))), dim3(expand_threads(kBn, kTma)),
                1024 + v + size_t(p.b_bufs) * buf + size_t(p.slots) * slot, st, true, dim3(1, 1, 1), map_b, p) == FP8_OK;
}

template <int kBn, bool kTma>
bool launch_expand(const TileParams& p, int piece, const CUtensorMap& map_b, int num_sms, cudaStream_t st) {
  return piece == 16  ? launch_expand_of<kBn, 16, kTma>(p, map_b, num_sms, st)
         : piece == 4 ? launch_expand_of<kBn, 4, kTma>(p, map_b, num_sms, st)
                      : launch_expand_of<kBn, 2, kTma>(p, map_b, num_sms, st);
}

bool launch_sorted(const Args& a, const Sorted& s, int num_sms, cudaStream_t st, Withhold withhold) {
  TileParams p = {};
  p.a = a;
  p.s = s;
  p.rp = padded_rank(a.rank);
  p.kb = int((a.K + kBk - 1) / kBk);
  p.kb_slice = (p.kb + s.splits - 1) / s.splits;
  p.vec = aligned(a.x, 16) && (a.M <= 1 || a.ldx % 8 == 0) && aligned(a.a, 16) && a.K % 8 == 0;
  p.vec_b = aligned(a.b, 16) && a.rank % 8 == 0;
  const bool words = aligned(a.x, 4) && (a.M <= 1 || a.ldx % 2 == 0) && aligned(a.a, 4) && a.K % 2 == 0;
  auto shrink = p.vec ? shrink_kernel<16, false> : words ? shrink_kernel<4, false> : shrink_kernel<2, false>;
  if (withhold == Withhold::kFirst) shrink = shrink_kernel<16, true>;
  if (!allow_smem(reinterpret_cast<const void*>(shrink))) return false;
  const int stage_bytes = int(kXBytes) + p.rp * 128;
  p.stages = std::max(3, std::min(kShrinkMaxStages, 108 * 1024 / stage_bytes));
  p.tmem_cols = 32;
  while (int(p.tmem_cols) < p.rp) p.tmem_cols *= 2;
  CUtensorMap map_a = {}, map_b = {};
  // (rows of 128 bytes; what lies past the rank or past K reads as zeros)
  if ((p.vec && !make_fp8_tensor_map_3d(&map_a, reinterpret_cast<const uint8_t*>(a.a), a.adapters, a.rank, a.K * 2,
                                          a.K * 2, uint32_t(p.rp))) ||
      (p.vec_b && !make_fp8_tensor_map_3d(&map_b, reinterpret_cast<const uint8_t*>(a.b), a.adapters, a.N,
                                          int64_t(a.rank) * 2, int64_t(a.rank) * 2, p.rp <= kBk ? 128 : p.rp <= 3 * kBk ? 64 : 32)))
    return false;
  if (launch(shrink, dim3(unsigned(s.max_tiles), unsigned(s.splits)), dim3(kShrinkThreads),
             size_t(p.stages) * stage_bytes + 1024, st, true, dim3(1, 1, 1), map_a, p) != FP8_OK)
    return false;
  auto on = [&](int bytes) {
    return aligned(a.y, bytes) && aligned(a.out, bytes) && a.N * 2 % bytes == 0 &&
           (a.M <= 1 || (a.ldy * 2 % bytes == 0 && a.ldo * 2 % bytes == 0));
  };
  const int piece = on(16) ? 16 : on(4) ? 4 : 2;
  if (withhold == Withhold::kSecond) return launch_expand_of<128, 16, true, true>(p, map_b, num_sms, st);
  if (withhold == Withhold::kSecondByWarps) return launch_expand_of<64, 2, false, true>(p, map_b, num_sms, st);
  if (p.vec_b) {
    if (p.rp <= kBk) return launch_expand<128, true>(p, piece, map_b, num_sms, st);
    return p.rp <= 3 * kBk ? launch_expand<64, true>(p, piece, map_b, num_sms, st)
                           : launch_expand<32, true>(p, piece, map_b, num_sms, st);
  }
  return p.rp <= 3 * kBk ? launch_expand<64, false>(p, piece, map_b, num_sms, st)
                         : launch_expand<32, false>(p, piece, map_b, num_sms, st);
}

unsigned int read_and_clear_error() {
  unsigned int v = 0;
  const unsigned int zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_lora_error, sizeof(v)) != cudaSuccess) return 0;
  if (v) cudaMemcpyToSymbol(g_lora_error, &zero, sizeof(zero));
  return v;
}

}  // namespace lora
}  // namespace fp8k
