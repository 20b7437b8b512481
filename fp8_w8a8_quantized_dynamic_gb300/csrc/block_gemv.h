// Internal interface of the block-scaled FP8 GEMV: products of at most 16 rows with streamed
// weights, or of one token with its experts.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "block_gemm.h"

namespace fp8k {
namespace block {

constexpr int kGemvMaxRows = 16;

// Where the activations come from: bf16 or fp32 rows quantized in the kernel, or codes.
enum Src : int { kSrcBf16 = 0, kSrcF32 = 1, kSrcCodes = 2 };

struct GemvArgs {
  Src src;
  const void* a;          // bf16 / fp32 rows, or codes
  int64_t lda;            // elements (bytes for codes)
  const float* s_a;       // kSrcCodes: [K blocks][lds_a]
  int64_t lds_a;
  int64_t M;              // dense: rows
  // one token: the tiles are its pairs, expert ids[j] and row j; with kGemvSum K runs over all pairs
  const int32_t* ids;
  const float* weights;
  int pairs;
  int64_t experts;
  const uint8_t* qw;      // matrices [N, ldw], as GemmArgs
  int64_t ldw;
  const float* s_w;
  int64_t N, K;
  const uint16_t* bias;
  uint16_t* y;            // bf16 output
  int64_t ldy;
  float* y32;             // fp32 output, rows of ldy32 (whole sixteens)
  int64_t ldy32;
};

enum GemvOut : int {
  kGemvBf16 = 0,    // y = bf16(acc (+ bias))
  kGemvSwiglu = 1,  // one token: gate and up matrices of its pairs' experts: y32 = silu(gate) * up
  kGemvSum = 2      // one token: y = bf16(sum over pairs of weight * acc)
};

// Whether the GEMV holds `rows` rows of K columns beside the sums of `mats` matrices in one SM's
// shared memory.
bool gemv_fits(int64_t rows, int64_t K, int mats);
// Whether quantizing in the kernel (every CTA its K slices) beats a kernel of its own before it.
bool gemv_quantizes(int64_t M, int64_t K);

bool gemv_launch(const GemvArgs& a, GemvOut out, int num_sms, cudaStream_t stream);

}  // namespace block
}  // namespace fp8k
