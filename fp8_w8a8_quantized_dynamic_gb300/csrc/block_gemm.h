// Internal interface of the block-scaled FP8 GEMM (one scale per row and 128 values of K of the
// activations, one per 128 x 128 block of the weights), dense or over the rows of many experts.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

namespace fp8k {
namespace block {

constexpr int kBlock = 128;      // values of K, and rows of W, that share a scale
constexpr int kRowTile = 128;    // activation rows of one output tile

inline int64_t blocks_of(int64_t n) { return (n + kBlock - 1) / kBlock; }

// What the tile's accumulators become.
enum Out : int {
  kOutBf16 = 0,    // y = bf16(acc (+ bias))
  kOutSwiglu = 1,  // W holds gate and up matrices: h = silu(gate) * up, quantized 1 x 128 into qh, s_h
  kOutF32 = 2      // unrounded fp32 rows
};

// A row tile of the grouped product: rows [row0, row_end) of the sorted activations belong to
// `expert`; a tile covers the first of them (kRowTile in the GEMM). Written by the routing plan kernel.
struct RowTile {
  int expert, row0, row_end, pad;
};

struct GemmArgs {
  // activations: codes [rows, lda] and scales [K blocks][lds_a]
  const uint8_t* qa;
  int64_t rows, lda;
  int64_t held_rows;  // rows that qa's buffer has room for, where that is more: see gemm_held_rows
  const float* s_a;
  int64_t lds_a;
  // weights: mats matrices of codes [N, ldw], each with scales [N blocks][K blocks]; with
  // kOutSwiglu two matrices (gate, up) an expert and N is the width of one of them
  const uint8_t* qw;
  int64_t mats, ldw;
  const float* s_w;
  int64_t N, K;
  // grouped: the row tiles and how many (device memory; at most max_tiles), else null
  const RowTile* tiles;
  const int* n_tiles;
  int64_t max_tiles;
  const uint16_t* bias;  // kOutBf16, may be null
  uint16_t* y;           // kOutBf16
  int64_t ldy;
  float* y32;            // kOutF32
  int64_t ldy32;
  uint8_t* qh;           // kOutSwiglu
  int64_t ldh;
  float* s_h;
  int64_t lds_h;
};

// Rows to make room for in a workspace's codes of `rows` rows. Loads through the tensor map of less than
// 128 KB take about twice as long (rows x 4096 x 6144: 17 rows 27.2 us, 32 rows 12.9), so a small buffer
// is made as long as that and its map covers all of it (17 rows 11.4). What the rows past the last hold
// does not matter: no result of theirs is stored.
int64_t gemm_held_rows(int64_t rows, int64_t ld);

// Enqueues the product. False when a tensor map could not be encoded or the launch failed.
bool gemm_launch(const GemmArgs& a, Out out, int num_sms, cudaStream_t stream);

// The product with one load withheld from its waits, for the failure-path self-test: whole tiles of 256
// columns, 64 with K shared by `split` CTAs, or SwiGLU.
bool gemm_launch_withheld(const GemmArgs& a, Out out, int split, int num_sms, cudaStream_t stream);

// Device-side error bits recorded by this file's kernels on the current device (read, then cleared).
unsigned int gemm_read_and_clear_error();

}  // namespace block
}  // namespace fp8k
