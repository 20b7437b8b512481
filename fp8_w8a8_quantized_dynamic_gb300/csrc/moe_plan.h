// Internal interface of the stable sort of pairs by expert (plan_kernel in moe.cuh), which the experts, the tokens' way
// to them and the adapters share.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "api_common.h"
#include "block_gemm.h"

namespace fp8k {
namespace moe {

// Workspace for the counts of many pairs' CTAs (0 for few pairs, which need none).
size_t plan_counts_bytes(int64_t pairs, int64_t experts);

struct Plan {
  const int32_t* ids;
  int64_t pairs;
  int experts;
  int spare;               // the expert that any id outside [0, experts) counts as; -1: such pairs have no row
  int* counts;             // plan_counts_bytes(pairs, experts)
  int* pos;                // row of each pair
  // what else is wanted; null where not
  int* order;              // pair of each row
  block::RowTile* tiles;
  int* n_tiles;
  int* offsets;            // [experts + 1] first rows
};

fp8_status launch_plan(const Plan& p, cudaStream_t st);

}  // namespace moe
}  // namespace fp8k
