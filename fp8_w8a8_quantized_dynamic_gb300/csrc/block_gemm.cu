// Block-scaled FP8 GEMM for sm_103a on the 5th-generation tensor cores.
//
//   Y[m, n] = sum_b s_a[b, m] * s_w[n / 128, b] * sum_{k in block b} qA[m, k] qW[n, k]
//
// over blocks b of 128 values of K. The scale changes every 128 values of K, so the tensor core
// sums one block at a time (four tcgen05.mma of K = 32 into a fresh tensor-memory accumulator)
// and the sum over blocks is kept in registers: each thread owns one row of the tile and adds
// s_a * s_w times the block's partial to its fp32 accumulators, one fma an element. Both sums
// are fp32.
//
// The rows are either those of one matrix, or (grouped) the rows of many experts sorted by
// expert, with one weight matrix an expert and a table of row tiles in device memory.
//
// Structure (persistent, one CTA per SM, output tiles of 128 x BN):
//   warp 0      TMA producer: activation tile [128 x 128 B] and weight tile [BN x 128 B] of a K
//               block into a ring of 128B-swizzled shared memory stages.
//   warps 1, 3  MMA issuers, for the K blocks of even and odd number; the block partials rotate
//               through 512 / BN tensor-memory buffers (at most four). One block's waits, MMAs and
//               commits take a thread about 650 cycles and the tensor core 512 (BN = 256), so one
//               issuer would set the pace (measured: 740 cycles a block with one, 556 with two).
//               Warp 1 also allocates the tensor memory.
//   warp 2      scale loader: the rows' scales and the weight blocks' scales of kScaleKb K blocks a
//               slot, by bulk copies and cp.async into a ring of its own (a load from L2 takes longer
//               than a block, and the ring runs ahead over the ends of tiles).
//   warps 4 on  promotion: warpgroups with 64 columns each (32 at BN = 64); a thread reads its row of
//               the partial (tcgen05.ld, at most 32 columns at a time; a read and its wait take some
//               30 cycles, which the scheduler's other warps fill, and keeping reads in flight behind
//               the additions costs more in copied registers) and adds it, scaled, in registers.
//               After the last K block the same threads write the tile out, a 32-byte sector a
//               store. Four warpgroups of 64 columns keep four warps a scheduler busy: 16384 x 4096 x
//               28672 in 1410 us (2.73 PFLOP/s; two warpgroups of 128 columns 1560).
// Ragged sizes need no padding: TMA fills out-of-range rows and columns with zeros and the
// stores are predicated.
//
// Few tiles (kSplit): a cluster of 2, 4 or 8 CTAs shares a tile's K; each sends its sums to the CTAs
// that own their columns (distributed shared memory), which add them in order and write them out
// (200 x 5632 x 2048 in 11.1 us, 14.9 unsplit; 17 rows 8.4 and 14.4).
//
// One CTA computes 128 x 256 by itself. The two-SM MMA on 256 x 256 (half the weight traffic from L2)
// was built and measured slower, 540 against 300 us at 8192 x 4096 x 8192: its commits and the peer's
// arrivals cross the cluster in every block, and two tensor-memory buffers cannot hide that.
//
// Every wait is bounded; on expiry the kernel records an error and each role leaves its loops at the
// first wait of its own that gives up: nothing is issued for a slot that was not handed back, and a
// warp whose waits did not all succeed stores nothing of its tile (with SwiGLU none of the warps that
// meet for its rows does, in a split tile none of the cluster's CTAs). Copies and MMAs in flight are
// drained, and the tensor memory is freed.

#include "block_gemm.h"

#include <algorithm>
#include <type_traits>
#include <utility>

#include "api_common.h"
#include "device_cache.h"
#include "device_common.cuh"
#include "gemm_tcgen05.h"
#include "tcgen05.cuh"

namespace fp8k {
namespace block {

__device__ unsigned int g_block_gemm_error;

constexpr int BM = kRowTile;
constexpr int BK = kBlock;
constexpr int kFirstPromoWarp = 4;
constexpr int kScaleKb = 4;     // K blocks of one slot of the scale ring
constexpr int kScaleSlots = 4;
// 640 threads (BN = 256) start with 96 registers each; 64 + 4 * 104 = 5 * 96
constexpr int kLaunchRegs = 96, kIssueRegs = 64, kPromoRegs = 104;
static_assert(kIssueRegs + 4 * kPromoRegs <= 5 * kLaunchRegs, "register shares of the five warpgroups");
constexpr uint32_t kABytes = BM * BK;
constexpr uint32_t kRingBytes = 194 * 1024;  // four stages of 48 KB; or of 32 KB beside 66 KB of exchanged sums
constexpr int kMaxStages = 8;
constexpr int kMaxBufs = 4;

// kSplit: a cluster's CTAs share a tile's K; part of the ring holds the sums they exchange.
template <int BN, bool kSplit>
struct Tile {
  static constexpr uint32_t stage_bytes = kABytes + BN * BK;
  static constexpr uint32_t exchange_bytes = kSplit ? BN * (BM + 4) * 4 : 0;
  static constexpr int stages = int((kRingBytes - exchange_bytes) / stage_bytes);  // 4, 6, 8 for BN = 256, 128, 64
  static constexpr int bufs = 512 / BN < kMaxBufs ? 512 / BN : kMaxBufs;
  static constexpr int cols = bufs * BN;  // tensor-memory columns (a power of two)
  static constexpr int groups = BN == 256 ? 4 : 2;  // promotion warpgroups, BN / groups columns each
  static constexpr int promo_warps = 4 * groups;
  static constexpr int threads = 128 + 128 * groups;
  static_assert(stages <= kMaxStages && stages * stage_bytes + exchange_bytes <= kRingBytes, "ring");
};

struct SharedCtl {
  uint64_t full[kMaxStages];
  uint64_t empty[kMaxStages];
  uint64_t tfull[kMaxBufs];
  uint64_t tempty[kMaxBufs];
  uint64_t drain;
  uint32_t tmem_base;
  int abort_flag;
  uint64_t sfull[kScaleSlots];
  uint64_t sempty[kScaleSlots];
  uint32_t hmax[2][4][BM];  // SwiGLU: row maxima of the groups' columns, by tile parity
  uint32_t staged[16][32][9];  // a promotion warp's 32 rows of 16 bf16 (+ 2: its lanes' writes on 32 banks)
  alignas(16) float s_row[kScaleSlots][kScaleKb][BM + 4];  // from the tile's first row rounded down to 4
  alignas(16) float s_col[kScaleSlots][kScaleKb][4];  // [half of the columns][gate, up]
};
constexpr size_t kSmemBytes = 1024 + kRingBytes + sizeof(SharedCtl);
static_assert(kSmemBytes <= 232448, "ring and control block must fit the 227 KB per-block limit");
static_assert(2 * kSmemBytes > 233472, "two GEMM CTAs must never share an SM (tensor memory)");

struct Params {
  int rows, N, kb;
  const float* s_a;
  int64_t lds_a;
  int bulk_scales;  // s_a's rows start on 16-byte boundaries (16384 x 4096 x 28672: 1413 us, 1423 by cp.async)
  const float* s_w;
  int nb;  // scale rows of one weight matrix
  const RowTile* tiles;
  const int* n_row_tiles;
  int m_tiles, n_tiles, group_n;
  int split_log2, kb_slice;  // kSplit: CTAs of a cluster, K blocks of one
  const uint16_t* bias;
  uint16_t* y;
  int64_t ldy;
  int vec;  // alignment of the bf16 output's rows: 32 bytes or less
  float* y32;
  int64_t ldy32;
  uint8_t* qh;
  int64_t ldh;
  float* s_h;
  int64_t lds_h;
};

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z,
                                            uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4, %5}], [%2], %6;"
      :: "r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z), "l"(policy) : "memory");
}

__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
      :: "r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate));
}

__host__ __device__ constexpr int ilog2(int n) { return n <= 1 ? 0 : 1 + ilog2(n / 2); }

// Copies `bytes` (a multiple of 16, both addresses 16-byte aligned) and completes them on the barrier.
__device__ __forceinline__ void bulk_load(uint32_t dst, const float* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
               :: "r"(dst), "l"(src), "r"(bytes), "r"(bar) : "memory");
}

// A predicated arrival, without a branch.
__device__ __forceinline__ void arrive_if(uint32_t bar, bool p) {
  asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %1, 0;\n\t@q mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}"
               :: "r"(bar), "r"(uint32_t(p)) : "memory");
}

// One lane of a converged warp (the compiler keeps the branch uniform).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

__device__ __forceinline__ void cp_async4(uint32_t dst, const float* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" :: "r"(dst), "l"(src) : "memory");
}
// Arrives on the barrier when this thread's copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" :: "r"(bar) : "memory");
}

// Reads 32 or 16 columns of this warp's tensor-memory lanes and waits for them.
__device__ __forceinline__ void tmem_read(uint32_t taddr, uint32_t (&r)[32]) { tmem_ld32(taddr, r); }
__device__ __forceinline__ void tmem_read(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// acc += s2 * r (kN columns, in pairs).
template <int kN>
__device__ __forceinline__ void add_scaled(uint64_t* acc, const uint32_t (&r)[kN], uint64_t s2) {
#pragma unroll
  for (int j = 0; j < kN / 2; ++j)
    acc[j] = fma_f32x2(pack_f32x2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1])), s2, acc[j]);
}

__device__ __forceinline__ void st_global_v8(void* p, uint32_t a, uint32_t b, uint32_t c, uint32_t d, uint32_t e,
                                             uint32_t f, uint32_t g, uint32_t h) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
               :: "l"(p), "r"(a), "r"(b), "r"(c), "r"(d), "r"(e), "r"(f), "r"(g), "r"(h) : "memory");
}

constexpr int kOutBf16Any = 3;  // kOutBf16 with rows of any alignment and width

// kWithhold (the failure-path self-test): CTA 0 does not load the last K block of its first tile, so the
// waits for it run out, after kWithheldNs.
constexpr unsigned long long kWithheldNs = 20000000ull;

template <int BN, int kOut, bool kSplit, bool kWithhold>
__global__ void __launch_bounds__(Tile<BN, kSplit>::threads, 1)
block_gemm_kernel(const __grid_constant__ CUtensorMap tmap_a, const __grid_constant__ CUtensorMap tmap_b,
                  const __grid_constant__ Params p) {
  constexpr int kStages = Tile<BN, kSplit>::stages;
  constexpr int kBufs = Tile<BN, kSplit>::bufs;
  constexpr int kGroups = Tile<BN, kSplit>::groups;
  constexpr int kPromoWarps = Tile<BN, kSplit>::promo_warps;
  constexpr int kCols = BN / kGroups;                              // columns of one promotion group
  constexpr int kChunk = kCols < 32 || kOut == kOutSwiglu ? 16 : 32;  // read at a time (SwiGLU: its second scale takes
                                                                      // the registers of the other 16)
  constexpr int kTileN = kOut == kOutSwiglu ? BN / 2 : BN;         // output columns of a tile
  static_assert(kOut != kOutSwiglu || BN == 256, "a SwiGLU tile is one 128-wide block of h");
  static_assert(!kSplit || (kOut != kOutSwiglu && BN <= 128), "sums of K slices are linear outputs of narrow tiles");
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  SharedCtl* ctl = reinterpret_cast<SharedCtl*>(smem + kRingBytes);
  const uint32_t smem_base = smem_u32(smem);
  float* exchange = reinterpret_cast<float*>(smem + kStages * Tile<BN, kSplit>::stage_bytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort_flag = &ctl->abort_flag;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return mbar_wait_short(smem_u32(bar), parity, abort_flag, &g_block_gemm_error,
                           kWithhold ? kWithheldNs : kWaitLimitNs);
  };
  // for a whole warp: whether all of its lanes' waits succeeded
  auto wait_all = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, wait(bar, parity)); };

  if (threadIdx.x == 0) {
    asm volatile("prefetch.tensormap [%0];" :: "l"(reinterpret_cast<uint64_t>(&tmap_a)) : "memory");
    asm volatile("prefetch.tensormap [%0];" :: "l"(reinterpret_cast<uint64_t>(&tmap_b)) : "memory");
    for (int s = 0; s < kStages; ++s) {
      mbar_init(smem_u32(&ctl->full[s]), 1);
      mbar_init(smem_u32(&ctl->empty[s]), 1);
    }
    for (int b = 0; b < kBufs; ++b) {
      mbar_init(smem_u32(&ctl->tfull[b]), 1);
      mbar_init(smem_u32(&ctl->tempty[b]), kPromoWarps);
    }
    mbar_init(smem_u32(&ctl->drain), 2);
    for (int i = 0; i < kScaleSlots; ++i) {
      mbar_init(smem_u32(&ctl->sfull[i]), 33);  // each lane's cp.async, and the bulk copies
      mbar_init(smem_u32(&ctl->sempty[i]), kPromoWarps);
    }
    ctl->abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                 :: "r"(smem_u32(&ctl->tmem_base)), "n"(Tile<BN, kSplit>::cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tmem_fence_before();
  __syncthreads();
  if (kSplit) pair_sync();  // the cluster's other CTAs run: their shared memory may be written
  tmem_fence_after();
  const uint32_t tmem_base = ctl->tmem_base;

  pdl_trigger();
  pdl_wait();  // qA, s_a and the tile table come from the preceding kernels

  const bool grouped = p.tiles != nullptr;
  const int m_tiles = grouped ? *p.n_row_tiles : p.m_tiles;
  const int units = m_tiles * p.n_tiles;
  // unit -> expert, first row, end of the expert's rows, column tile. Within a group of column
  // tiles the column runs fastest, so a group's weights stay in L2 while the row tiles pass.
  auto decode = [&](int u, int& expert, int& row0, int& row_end, int& n_idx) {
    const int per_group = p.group_n * m_tiles;
    const int g = u / per_group;
    const int r = u - g * per_group;
    const int gn = min(p.group_n, p.n_tiles - g * p.group_n);
    const int m_idx = r / gn;
    n_idx = g * p.group_n + (r - m_idx * gn);
    if (grouped) {
      const int4 t = *reinterpret_cast<const int4*>(p.tiles + m_idx);
      expert = t.x, row0 = t.y, row_end = t.z;
    } else {
      expert = 0, row0 = m_idx * BM, row_end = p.rows;
    }
  };

  // K slice and work units: all of K and every gridDim.x-th tile, or (kSplit) a cluster a tile and
  // rank r's share of its K
  auto rank_of = [&]() { return kSplit ? int(cluster_rank()) : 0; };
  auto kb_begin = [&]() { return kSplit ? min(p.kb, rank_of() * p.kb_slice) : 0; };
  auto kb_end = [&]() { return kSplit ? min(p.kb, (rank_of() + 1) * p.kb_slice) : p.kb; };
  auto first_unit = [&]() { return kSplit ? int(blockIdx.x) >> p.split_log2 : int(blockIdx.x); };
  auto unit_stride = [&]() { return kSplit ? int(gridDim.x) >> p.split_log2 : int(gridDim.x); };

  if (warp < kFirstPromoWarp) {
   if constexpr (BN == 256) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(kIssueRegs));
   if (warp == 0) {
    if (lane == 0) {
      // ---------------- TMA producer ----------------
      const uint64_t pol = l2_policy(kHintNormal);
      uint32_t it = 0;
      for (int u = first_unit(); u < units; u += unit_stride()) {
        int expert, row0, row_end, n_idx;
        decode(u, expert, row0, row_end, n_idx);
        const int n0 = n_idx * kTileN;
        bool ok = true;
        for (int kb = kb_begin(); kb < kb_end(); ++kb, ++it) {
          const int s = it % kStages;
          if (!wait(&ctl->empty[s], ((it / kStages) & 1u) ^ 1u) ||
              (kWithhold && blockIdx.x == 0 && kb == kb_end() - 1)) {
            ok = false;
            break;
          }
          const uint32_t fb = smem_u32(&ctl->full[s]);
          const uint32_t dst = smem_base + s * Tile<BN, kSplit>::stage_bytes;
          mbar_arrive_expect_tx(fb, Tile<BN, kSplit>::stage_bytes);
          tma_load_2d(dst, &tmap_a, fb, kb * BK, row0, pol);
          if (kOut == kOutSwiglu) {
            // 64 columns of gate, then the same 64 of up, twice
#pragma unroll
            for (int h = 0; h < 4; ++h)
              tma_load_3d(dst + kABytes + h * (64 * BK), &tmap_b, fb, kb * BK, n0 + (h >> 1) * 64, 2 * expert + (h & 1),
                          pol);
          } else {
            tma_load_3d(dst + kABytes, &tmap_b, fb, kb * BK, n0, expert, pol);
          }
        }
        if (!ok) break;
      }
      // the last fill of every stage must land before the CTA's memory is released
      for (uint32_t j = it > uint32_t(kStages) ? it - kStages : 0u; j < it; ++j)
        mbar_wait_bounded(smem_u32(&ctl->full[j % kStages]), (j / kStages) & 1u, nullptr, &g_block_gemm_error);
    }
   } else if (warp != 2) {
    // ---------------- MMA issuers: warps 1 and 3, K blocks of even and odd number ----------------
    // D fp32, A and B e4m3, both K-major, N = BN, M = 128
    constexpr uint32_t idesc =
        (1u << 4) | (uint32_t(BN >> 3) << 17) | (uint32_t(BM >> 4) << 24);
    const int mine = units > first_unit() ? (units - first_unit() + unit_stride() - 1) / unit_stride() : 0;
    const uint32_t total = uint32_t(mine) * uint32_t(kb_end() - kb_begin());  // blocks of all of this CTA's tiles
    for (uint32_t it = warp >> 1; it < total; it += 2) {
      const int b = it % kBufs, s = it % kStages;
      // the operands are there long before the buffer is free: what follows the last wait is
      // what counts
      bool ok = wait(&ctl->full[s], (it / kStages) & 1u);
      ok = wait(&ctl->tempty[b], ((it / kBufs) & 1u) ^ 1u) && ok;
      if (!__all_sync(0xffffffffu, ok)) break;
      tmem_fence_after();
      if (elect_one()) {
        const uint64_t adesc = make_sdesc(smem_base + s * Tile<BN, kSplit>::stage_bytes);
        const uint64_t bdesc = make_sdesc(smem_base + s * Tile<BN, kSplit>::stage_bytes + kABytes);
        const uint32_t d = tmem_base + b * BN;
#pragma unroll
        for (int kk = 0; kk < BK / 32; ++kk)
          mma_f8(d, adesc + uint64_t(kk * 32 >> 4), bdesc + uint64_t(kk * 32 >> 4), idesc, kk != 0);
        mma_commit<false>(smem_u32(&ctl->tfull[b]));
        mma_commit<false>(smem_u32(&ctl->empty[s]));
      }
      __syncwarp();
    }
    if (elect_one()) mma_commit<false>(smem_u32(&ctl->drain));
    __syncwarp();
    // all MMAs done before the tensor memory is released
    mbar_wait_bounded(smem_u32(&ctl->drain), 0, nullptr, &g_block_gemm_error);
   } else if (warp == 2) {
    // ---------------- scale loader ----------------
    uint32_t slot_no = 0;
    bool ok = true;
    for (int u = first_unit(); ok && u < units; u += unit_stride()) {
      int expert, row0, row_end, n_idx;
      decode(u, expert, row0, row_end, n_idx);
      const int n0 = n_idx * kTileN;
      // lane % 4: the weight scale row of (half of the columns, matrix)
      const int mat = kOut == kOutSwiglu ? 2 * expert + (lane & 1) : expert;
      const int col = kOut == kOutSwiglu ? n0 : n0 + ((lane >> 1) & 1) * (BN / 2);
      const float* sw = p.s_w + (int64_t(mat) * p.nb + min(col / kBlock, p.nb - 1)) * p.kb;
      for (int kb0 = kb_begin(); kb0 < kb_end(); kb0 += kScaleKb, ++slot_no) {
        const int slot = slot_no % kScaleSlots;
        // (a slot that was not handed back may still expect bytes of its last fill: never filled again)
        if (!(ok = wait_all(&ctl->sempty[slot], ((slot_no / kScaleSlots) & 1u) ^ 1u))) break;
        const uint32_t bar = smem_u32(&ctl->sfull[slot]);
        if (p.bulk_scales) {
          // one bulk copy a block: rows [a0, a0 + n), whole 16-byte pieces that each hold one of the
          // rows (so nothing past the buffer of a view is read)
          const int a0 = row0 & ~3;
          const uint32_t bytes = uint32_t(min(BM + 4, ((p.rows + 3) & ~3) - a0)) * 4u;
          const int blocks = min(kScaleKb, kb_end() - kb0);
          if (lane == 0) mbar_arrive_expect_tx(bar, bytes * blocks);
          __syncwarp();
          if (lane < blocks)
            bulk_load(smem_u32(&ctl->s_row[slot][lane][0]), p.s_a + int64_t(kb0 + lane) * p.lds_a + a0, bytes, bar);
        } else {
#pragma unroll
          for (int j = 0; j < kScaleKb; ++j) {
            const int kb = min(kb0 + j, kb_end() - 1);
#pragma unroll
            for (int i = 0; i < BM / 32; ++i) {
              const int row = row0 + lane + i * 32;  // rows past the tile's repeat its first
              cp_async4(smem_u32(&ctl->s_row[slot][j][(row0 & 3) + lane + i * 32]),
                        p.s_a + int64_t(kb) * p.lds_a + (row < row_end ? row : row0));
            }
          }
          if (lane == 0) mbar_arrive(bar);
        }
        if (lane < 4 * kScaleKb)
          cp_async4(smem_u32(&ctl->s_col[slot][lane >> 2][lane & 3]), sw + min(kb0 + (lane >> 2), kb_end() - 1));
        cp_async_arrive(bar);
      }
    }
    // nothing of the last slots may land after the CTA has left
    for (uint32_t i = slot_no > uint32_t(kScaleSlots) ? slot_no - kScaleSlots : 0u; i < slot_no; ++i)
      mbar_wait_bounded(smem_u32(&ctl->sfull[i % kScaleSlots]), (i / kScaleSlots) & 1u, nullptr, &g_block_gemm_error);
    asm volatile("cp.async.wait_all;" ::: "memory");
   }
  } else {
    // ---------------- promotion and epilogue: warps 4 on ----------------
    if constexpr (BN == 256) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(kPromoRegs));
    const int group = (warp - kFirstPromoWarp) >> 2;  // of columns
    const int quarter = warp & 3;        // tensor-memory lanes this warp may access
    const int row_in_tile = quarter * 32 + lane;
    // first column of the group, and from one 32-column read to the next (SwiGLU: 32 columns of gate
    // and the same 32 of up, 64 on)
    const uint32_t tbase = tmem_base + (uint32_t(quarter * 32) << 16) +
                           (kOut == kOutSwiglu ? (group >> 1) * 128 + (group & 1) * 32 : group * kCols);
    uint32_t it = 0, tile_no = 0, slot_no = 0;
    int u = first_unit();
    for (; u < units; u += unit_stride(), ++tile_no) {
      int expert, row0, row_end, n_idx;
      decode(u, expert, row0, row_end, n_idx);
      const int n0 = n_idx * kTileN;
      const int row = row0 + row_in_tile;
      const bool live = row < row_end;
      uint64_t acc[kCols / 2];
#pragma unroll
      for (int j = 0; j < kCols / 2; ++j) acc[j] = 0;
      uint64_t g2 = 0, u2 = 0;  // this block's scales of the group's first and second half of columns
      // the scales of block kb; the slot is handed back with its last block. False: they did not come.
      auto next_scales = [&](int kb) {
        const int slot = slot_no % kScaleSlots, j = (kb - kb_begin()) % kScaleKb;
        if (j == 0 && !wait_all(&ctl->sfull[slot], (slot_no / kScaleSlots) & 1u)) return false;
        const float sa = ctl->s_row[slot][j][(row0 & 3) + row_in_tile];
        const float2 sw = *reinterpret_cast<const float2*>(&ctl->s_col[slot][j][2 * (group / (kGroups / 2))]);
        const float g = sa * sw.x, u = kOut == kOutSwiglu ? sa * sw.y : g;
        if (j == kScaleKb - 1 || kb == kb_end() - 1) {
          // The slot goes back only when the loads of every lane have delivered: the arriving lane depends on
          // their values. The barrier alone does not order them before the bulk copy that fills the slot again
          // (another proxy): behind the stores of other warps a load waits for microseconds, and an arrival
          // that was merely issued after it gave wrong scales at K of one to three blocks, where the tiles
          // before this one are still being stored.
          const float all = kOut == kOutSwiglu ? g + u : g;
          if (lane == (__any_sync(0xffffffffu, all == all) ? 0 : 1)) mbar_arrive(smem_u32(&ctl->sempty[slot]));
          ++slot_no;
        }
        g2 = pack_f32x2(g, g);
        u2 = kOut == kOutSwiglu ? pack_f32x2(u, u) : g2;
        return true;
      };
      bool ok = true;
      for (int kb = kb_begin(); kb < kb_end(); ++kb, ++it) {
        constexpr int kChunks = kCols / kChunk;
        const int b = it % kBufs;
        if (!(ok = next_scales(kb) && wait_all(&ctl->tfull[b], (it / kBufs) & 1u))) break;
        tmem_fence_after();
        const uint32_t tempty = smem_u32(&ctl->tempty[b]);
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
          uint32_t part[kChunk];
          tmem_read(tbase + b * BN + (kOut == kOutSwiglu ? (c >> 1) * 64 + (c & 1) * 16 : c * kChunk), part);
          if (c == kChunks - 1) {  // the last read has landed: the buffer is free before its columns are added
            tmem_fence_before();
            arrive_if(tempty, lane == 0);
          }
          add_scaled(acc + c * (kChunk / 2), part, 2 * c < kChunks ? g2 : u2);
        }
      }
      if (!ok) break;
      if constexpr (kSplit) {
        // this slice's sums go to the CTAs that own their columns: [slice][column][row], columns far enough
        // apart that a warp's loads of whole rows below fall on 32 banks, as its stores here do
        const int own_log2 = ilog2(BN) - p.split_log2;
        const uint32_t column_bytes = (BM + (1u << max(0, 5 - own_log2))) * 4u;
        const uint32_t at = smem_u32(exchange) + (uint32_t(rank_of()) << own_log2) * column_bytes + row_in_tile * 4u;
#pragma unroll
        for (int q = 0; q < kCols / 8; ++q) {  // eight columns have one owner
          const uint32_t c = group * kCols + 8 * q;
          uint32_t dst = map_to_rank(at, c >> own_log2) + (c & ((1u << own_log2) - 1u)) * column_bytes;
#pragma unroll
          for (int j = 4 * q; j < 4 * q + 4; ++j) {
            st_cluster_u32(dst, uint32_t(acc[j]));
            st_cluster_u32(dst + column_bytes, uint32_t(acc[j] >> 32));
            dst += 2 * column_bytes;
          }
        }
        continue;
      }
      // each thread writes its row's columns, a 32-byte sector a store
      if constexpr (kOut == kOutSwiglu) {
        // columns [32 group, 32 group + 32) of the tile's 128-wide block of h
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const float h0 = swiglu(lo_of(acc[j]), lo_of(acc[16 + j])), h1 = swiglu(hi_of(acc[j]), hi_of(acc[16 + j]));
          m = max(m, max(__float_as_uint(fabsf(h0)), __float_as_uint(fabsf(h1))));  // keeps a NaN
          acc[j] = pack_f32x2(h0, h1);
        }
        ctl->hmax[tile_no & 1][group][row_in_tile] = m;
        // the warps that hold the same 32 rows meet; two tiles' maxima alternate, so one meeting a
        // tile is enough
        asm volatile("bar.sync %0, %1;" :: "r"(1 + quarter), "n"(32 * kGroups) : "memory");
#pragma unroll
        for (int o = 0; o < kGroups; ++o) m = max(m, ctl->hmax[tile_no & 1][o][row_in_tile]);
        const float s = scale_from_amax<kFmtE4M3>(__uint_as_float(m));
        const ExactScale k = make_exact_scale(s);
        // a warp whose waits gave up comes to the meeting without a maximum, after it raised (saw) the flag
        if (*abort_flag == 0 && live) {
          uint32_t w[8];
#pragma unroll
          for (int v = 0; v < 8; ++v) w[v] = quant4_exact_f32<kFmtE4M3>(acc[v * 2], acc[v * 2 + 1], k, s);
          const int col = n0 + group * 32;  // columns past N hold zeros (zero weight rows)
          uint8_t* dst = p.qh + int64_t(row) * p.ldh + col;
          if (col < p.ldh) *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
          if (col + 16 < p.ldh) *reinterpret_cast<uint4*>(dst + 16) = make_uint4(w[4], w[5], w[6], w[7]);
          if (group == 0) p.s_h[int64_t(n_idx) * p.lds_h + row] = s;
        }
      } else if constexpr (kOut == kOutF32) {
        const int col0 = n0 + group * kCols;
        float* dst = p.y32 + int64_t(row) * p.ldy32 + col0;
        if (live) {
#pragma unroll
          for (int q = 0; q < kCols / 8; ++q) {
            const uint64_t* a = acc + q * 4;
            if (col0 + q * 8 < p.ldy32)  // ldy32: N rounded up to 8
              st_global_v8(dst + q * 8, uint32_t(a[0]), uint32_t(a[0] >> 32), uint32_t(a[1]), uint32_t(a[1] >> 32),
                           uint32_t(a[2]), uint32_t(a[2] >> 32), uint32_t(a[3]), uint32_t(a[3] >> 32));
          }
        }
      } else {
        const int col0 = n0 + group * kCols;
        // sixteen columns as bf16 pairs
        auto packed = [&](int q, uint32_t (&w)[8]) {
          const int col = col0 + q * 16;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const uint64_t a = acc[q * 8 + j];
            float lo = lo_of(a), hi = hi_of(a);
            if (p.bias) {
              lo += bf16_bits_to_float(__ldg(p.bias + min(col + 2 * j, p.N - 1)));
              hi += bf16_bits_to_float(__ldg(p.bias + min(col + 2 * j + 1, p.N - 1)));
            }
            w[j] = pack_bf16x2(lo, hi);
          }
        };
        if constexpr (kOut == kOutBf16) {
          uint16_t* dst = p.y + int64_t(row) * p.ldy + col0;
          if (live) {
#pragma unroll
            for (int q = 0; q < kCols / 16; ++q) {
              if (col0 + q * 16 >= p.N) break;  // N: whole eights
              uint32_t w[8];
              packed(q, w);
              const bool both = col0 + q * 16 + 16 <= p.N;
              if (p.vec >= 32 && both) {
                st_global_v8(dst + q * 16, w[0], w[1], w[2], w[3], w[4], w[5], w[6], w[7]);
              } else {
                *reinterpret_cast<uint4*>(dst + q * 16) = make_uint4(w[0], w[1], w[2], w[3]);
                if (both) *reinterpret_cast<uint4*>(dst + q * 16 + 8) = make_uint4(w[4], w[5], w[6], w[7]);
              }
            }
          }
        } else {
          // rows that start and end anywhere: through shared memory, two rows' 16 columns a store (8192 x 4096 x
          // 8191: 285 us; two bytes of 32 rows a store: 768)
          uint32_t(&mine)[32][9] = ctl->staged[warp - kFirstPromoWarp];
          const int c = lane & 15;
#pragma unroll
          for (int q = 0; q < kCols / 16; ++q) {
            uint32_t w[8];
            packed(q, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) mine[lane][j] = w[j];
            __syncwarp();
            const int col = col0 + q * 16 + c;
#pragma unroll 1
            for (int r = lane >> 4; r < 32; r += 2) {
              const int to = row0 + quarter * 32 + r;
              if (to < row_end && col < p.N)
                p.y[int64_t(to) * p.ldy + col] = reinterpret_cast<const uint16_t*>(mine[r])[c];
            }
            __syncwarp();
          }
        }
      }
    }
    // a warp that left early still comes to the meetings of its remaining tiles, where the others wait
    if constexpr (kOut == kOutSwiglu)
      for (; u < units; u += unit_stride())
        asm volatile("bar.sync %0, %1;" :: "r"(1 + quarter), "n"(32 * kGroups) : "memory");
  }

  if constexpr (kSplit) {
    // a slice that is not whole is nobody's to add: the threads that know raise every CTA's flag
    if (*abort_flag != 0)
      for (int r = 0; r < (1 << p.split_log2); ++r) st_cluster_u32(map_to_rank(smem_u32(&ctl->abort_flag), r), 1u);
    __syncwarp();
    pair_sync();  // all threads of the cluster: every slice's sums (or flags) have arrived
    if (warp >= kFirstPromoWarp && first_unit() < units && *abort_flag == 0) {
      // the owner adds the slices in order: a thread four columns of every `step`-th row, neighbouring
      // threads neighbouring columns
      int expert, row0, row_end, n_idx;
      decode(first_unit(), expert, row0, row_end, n_idx);
      const int own_log2 = ilog2(BN) - p.split_log2;
      const int column = BM + (1 << max(0, 5 - own_log2));
      const int t = threadIdx.x - kFirstPromoWarp * 32, c = (t & ((1 << (own_log2 - 2)) - 1)) * 4;
      const int step = kPromoWarps * 32 >> (own_log2 - 2);
      const int n = n_idx * kTileN + (rank_of() << own_log2) + c;
      const int rows = n < p.N ? min(BM, row_end - row0) : 0;
      float bias[4] = {0.f, 0.f, 0.f, 0.f};
      if (kOut != kOutF32 && p.bias && n < p.N)
#pragma unroll
        for (int i = 0; i < 4; ++i) bias[i] = bf16_bits_to_float(__ldg(p.bias + min(n + i, p.N - 1)));
      for (int r = t >> (own_log2 - 2); r < rows; r += step) {
        float v[4] = {0.f, 0.f, 0.f, 0.f};
        const float* from = exchange + c * column + r;
#pragma unroll 2
        for (int k = 0; k < (1 << p.split_log2); ++k, from += column << own_log2)
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] += from[i * column];
        const int64_t row = row0 + r;
        if constexpr (kOut == kOutF32) {  // ldy32: N rounded up to 8
          *reinterpret_cast<float4*>(p.y32 + row * p.ldy32 + n) = make_float4(v[0], v[1], v[2], v[3]);
        } else {
          uint16_t* dst = p.y + row * p.ldy + n;
          const uint32_t lo = pack_bf16x2(v[0] + bias[0], v[1] + bias[1]);
          const uint32_t hi = pack_bf16x2(v[2] + bias[2], v[3] + bias[3]);
          if (p.vec >= 8 && n + 4 <= p.N) {
            *reinterpret_cast<uint2*>(dst) = make_uint2(lo, hi);
          } else {
            dst[0] = uint16_t(lo);
            if (n + 1 < p.N) dst[1] = uint16_t(lo >> 16);
            if (n + 2 < p.N) dst[2] = uint16_t(hi);
            if (n + 3 < p.N) dst[3] = uint16_t(hi >> 16);
          }
        }
      }
    }
  }
  __syncwarp();
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  if (warp == 1) {
    __syncwarp();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(tmem_base), "n"(Tile<BN, kSplit>::cols)
                 : "memory");
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

namespace {

PerDeviceCache<std::pair<const void*, int>, int> g_slot_cache;

// CTAs of the kernel that run at once in clusters of `split`, its attributes set; 0: it cannot run.
int slots_of(const void* kfn, int threads, int split, int num_sms) {
  int dev = 0, slots = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  g_slot_cache.get(dev, std::make_pair(kfn, split), &slots, [&](int* v) {
    if (report_cuda(cudaFuncSetAttribute(kfn, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kSmemBytes)),
                    "block gemm smem attribute") != cudaSuccess)
      return false;
    *v = num_sms;
    if (split > 1) {
      cudaLaunchConfig_t cfg = {};
      cfg.blockDim = dim3(unsigned(threads));
      cfg.dynamicSmemBytes = kSmemBytes;
      cfg.gridDim = dim3(split * 64);
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = split;
      attr[0].val.clusterDim.y = 1;
      attr[0].val.clusterDim.z = 1;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      int clusters = 0;
      if (report_cuda(cudaOccupancyMaxActiveClusters(&clusters, kfn, &cfg), "block gemm clusters") != cudaSuccess) {
        cudaGetLastError();
        return false;
      }
      *v = clusters * split;
    }
    return true;
  });
  return slots;
}

template <int BN, int kOut, bool kSplit = false, bool kWithhold = false>
bool launch_tile(const GemmArgs& a, int split, int num_sms, cudaStream_t st) {
  auto kfn = block_gemm_kernel<BN, kOut, kSplit, kWithhold>;
  const int slots = slots_of(reinterpret_cast<const void*>(kfn), Tile<BN, kSplit>::threads, split, num_sms);
  if (slots <= 0) return false;
  Params p = {};
  p.rows = int(a.rows);
  p.N = int(a.N);
  p.kb = int(blocks_of(a.K));
  p.s_a = a.s_a;
  p.lds_a = a.lds_a;
  p.bulk_scales = aligned(a.s_a, 16) && a.lds_a % 4 == 0;
  p.s_w = a.s_w;
  p.nb = int(blocks_of(a.N));
  p.split_log2 = ilog2(split);
  p.kb_slice = (p.kb + split - 1) / split;
  p.tiles = a.tiles;
  p.n_row_tiles = a.n_tiles;
  constexpr int kTileN = kOut == kOutSwiglu ? BN / 2 : BN;
  p.m_tiles = int((a.rows + BM - 1) / BM);
  p.n_tiles = int((a.N + kTileN - 1) / kTileN);
  // Weights of a raster group: about 28 MB, which L2 holds beside the activations that stream
  // past. Grouped: the row tiles of an expert follow one another, so all of its columns.
  const int64_t tile_bytes = int64_t(BN) * a.ldw;
  p.group_n = a.tiles ? p.n_tiles : int(std::min<int64_t>(p.n_tiles, std::max<int64_t>(1, (28 << 20) / tile_bytes)));
  p.bias = a.bias;
  p.y = a.y;
  p.ldy = a.ldy;
  p.y32 = a.y32;
  p.ldy32 = a.ldy32;
  p.qh = a.qh;
  p.ldh = a.ldh;
  p.s_h = a.s_h;
  p.lds_h = a.lds_h;
  p.vec = 32;
  while (p.vec > 2 && !(aligned(a.y, p.vec) && a.ldy * 2 % p.vec == 0)) p.vec /= 2;
  const int64_t units = (a.tiles ? a.max_tiles : int64_t(p.m_tiles)) * p.n_tiles;
  if (units > kMaxDim) return false;
  CUtensorMap ma, mb;
  if (!make_fp8_tensor_map(&ma, a.qa, std::max(a.rows, a.held_rows), a.K, a.lda, BM) ||
      !make_fp8_tensor_map_3d(&mb, a.qw, a.mats, a.N, a.K, a.ldw, kOut == kOutSwiglu ? 64 : BN))
    return false;
  // a split tile's cluster comes and goes with it; otherwise the CTAs stay and walk the tiles
  const int64_t grid = kSplit ? units * split : std::min<int64_t>(units, slots);
  return launch(kfn, dim3(unsigned(grid)), dim3(Tile<BN, kSplit>::threads), kSmemBytes, st, true, dim3(split, 1, 1), ma, mb, p) == FP8_OK;
}

// Tile width and K split, by the time of the busiest CTA in us: waves of CTAs, each the blocks of its
// K slice and about one for its start and end, and an exchange of sums where K is split. Measured on
// a GB300: a block of a 128 x 64, 128 x 128 and 128 x 256 tile takes 0.30, 0.36 and 0.50.
struct TileChoice {
  int bn, split;
};

template <int kOut>
TileChoice choose_tile(int64_t m_tiles, int64_t N, int64_t kb, int num_sms) {
  TileChoice best = {256, 1};
  double best_us = -1;
  auto consider = [&](int bn, int split, int slots, double block_us) {
    if (slots < split || (split > 1 && (kb + split - 1) / split * (split - 1) >= kb)) return;  // an empty slice
    const int64_t units = m_tiles * ((N + bn - 1) / bn);
    const int64_t waves = (units * split + slots - 1) / slots;
    if (split > 1 && waves > 1) return;
    const double us = double(waves) * (double((kb + split - 1) / split) * block_us + 1.0) + (split > 1 ? 1.2 : 0.0);
    if (best_us < 0 || us < best_us) best = {bn, split}, best_us = us;
  };
  consider(256, 1, num_sms, 0.50);
  consider(128, 1, num_sms, 0.36);
  consider(64, 1, num_sms, 0.30);
  for (int split = 2; split <= 8; split *= 2) {
    consider(128, split, slots_of(reinterpret_cast<const void*>(block_gemm_kernel<128, kOut, true, false>), Tile<128, true>::threads, split, num_sms), 0.36);
    consider(64, split, slots_of(reinterpret_cast<const void*>(block_gemm_kernel<64, kOut, true, false>), Tile<64, true>::threads, split, num_sms), 0.30);
  }
  return best;
}

template <int kOut>
bool launch_any(const GemmArgs& a, int num_sms, cudaStream_t st) {
  if constexpr (kOut == kOutSwiglu) {
    return launch_tile<256, kOut>(a, 1, num_sms, st);
  } else {
    const int64_t m_tiles = a.tiles ? a.max_tiles : (a.rows + BM - 1) / BM;
    const TileChoice c = choose_tile<kOut>(m_tiles, a.N, blocks_of(a.K), num_sms);
    if (c.split > 1)
      return c.bn == 128 ? launch_tile<128, kOut, true>(a, c.split, num_sms, st)
                         : launch_tile<64, kOut, true>(a, c.split, num_sms, st);
    auto whole = [&](auto out) {
      constexpr int kHow = decltype(out)::value;
      if (c.bn == 256) return launch_tile<256, kHow>(a, 1, num_sms, st);
      return c.bn == 128 ? launch_tile<128, kHow>(a, 1, num_sms, st) : launch_tile<64, kHow>(a, 1, num_sms, st);
    };
    // whole sectors are stored at once where the rows allow it
    if (kOut == kOutBf16 && !(aligned(a.y, 16) && a.ldy % 8 == 0 && a.N % 8 == 0))
      return whole(std::integral_constant<int, kOutBf16Any>{});
    return whole(std::integral_constant<int, kOut>{});
  }
}

}  // namespace

int64_t gemm_held_rows(int64_t rows, int64_t ld) { return std::max(rows, (128 * 1024 + ld - 1) / ld); }

bool gemm_launch(const GemmArgs& a, Out out, int num_sms, cudaStream_t stream) {
  switch (out) {
    case kOutBf16: return launch_any<kOutBf16>(a, num_sms, stream);
    case kOutSwiglu: return launch_any<kOutSwiglu>(a, num_sms, stream);
    case kOutF32: return launch_any<kOutF32>(a, num_sms, stream);
  }
  return false;
}

bool gemm_launch_withheld(const GemmArgs& a, Out out, int split, int num_sms, cudaStream_t stream) {
  switch (out) {
    case kOutBf16:
      return split > 1 ? launch_tile<64, kOutBf16, true, true>(a, split, num_sms, stream)
                       : launch_tile<256, kOutBf16, false, true>(a, 1, num_sms, stream);
    case kOutSwiglu: return launch_tile<256, kOutSwiglu, false, true>(a, 1, num_sms, stream);
    case kOutF32: break;
  }
  return false;
}

unsigned int gemm_read_and_clear_error() {
  unsigned int v = 0;
  const unsigned int zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_block_gemm_error, sizeof(v)) != cudaSuccess) return 0;
  if (v) cudaMemcpyToSymbol(g_block_gemm_error, &zero, sizeof(zero));
  return v;
}

}  // namespace block
}  // namespace fp8k
