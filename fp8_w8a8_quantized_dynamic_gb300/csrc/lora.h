// Internal interface of the low-rank adapters beside a projection (lora.cu):
//   out[m] = y[m] + s[e] * B[e] (A[e] x[m]),  e = ids[m] (outside [0, adapters): out[m] = y[m])
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "block_gemm.h"

namespace fp8k {
namespace lora {

constexpr int kMaxRank = 256;

struct Args {
  const uint16_t* y;
  int64_t M, N, ldy;
  const uint16_t* x;
  int64_t K, ldx;
  const uint16_t* a;  // [adapters][rank][K]
  const uint16_t* b;  // [adapters][N][rank]
  int adapters, rank;
  const int32_t* ids;
  const float* scales;  // null: 1
  uint16_t* out;
  int64_t ldo;
};

// A token at a time: one kernel, no workspace. For few tokens.
bool launch_tokens(const Args& p, int num_sms, cudaStream_t st);

// Rows sorted by adapter, on tensor cores: tiles (and how many) and the token of each sorted row, in
// device memory; `adapters` itself stands for no adapter there. v: fp32 [splits][rank rounded up to 16, / 4][M][4].
struct Sorted {
  const block::RowTile* tiles;
  const int* n_tiles;
  int64_t max_tiles;
  const int* order;
  float* v;
  int splits;
};
int splits_of(int64_t M, int64_t K, int64_t adapters, int64_t rank);
inline int padded_rank(int64_t rank) { return int((rank + 15) / 16 * 16); }

// The failure-path self-test: a load withheld from the waits of the first product (rows of x and A on 16-byte boundaries), or of
// the second, whose B comes by TMA (rows on 16-byte boundaries, rank up to 64) or by warps (rank up to 192).
enum class Withhold : int { kNone = -1, kFirst, kSecond, kSecondByWarps };
bool launch_sorted(const Args& p, const Sorted& s, int num_sms, cudaStream_t st, Withhold withhold = Withhold::kNone);

unsigned int read_and_clear_error();

}  // namespace lora
}  // namespace fp8k
