// Host-side pieces shared by the C-ABI translation units: device check, kernel launch, argument
// validation.
#pragma once

#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <mutex>

#include "fp8w8a8.h"

#define FP8_API extern "C" __attribute__((visibility("default")))

#define FP8_TRY(expr)                  \
  do {                                 \
    const fp8_status _s = (expr);      \
    if (_s != FP8_OK) return _s;       \
  } while (0)

namespace fp8k {

constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1;

// ---------------------------------------------------------------------------
// device properties (cached per device)
// ---------------------------------------------------------------------------

struct DevInfo {
  int checked = 0;
  int supported = 0;
  int sms = 0;
};

inline std::mutex g_dev_mu;
inline DevInfo g_dev[64];

inline fp8_status current_device(int* sms) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return FP8_ERR_CUDA;
  std::lock_guard<std::mutex> lock(g_dev_mu);
  DevInfo& d = g_dev[dev];
  if (!d.checked) {
    int major = 0, minor = 0, n = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return FP8_ERR_CUDA;
    d.supported = (major == 10 && minor == 3);
    d.sms = n;
    d.checked = 1;
  }
  if (!d.supported) return FP8_ERR_UNSUPPORTED_DEVICE;
  *sms = d.sms;
  return FP8_OK;
}

inline int64_t round_up16(int64_t k) { return (k + 15) / 16 * 16; }

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Passes `e` through; with FP8W8A8_DEBUG set, a failure is also described on stderr.
inline cudaError_t report_cuda(cudaError_t e, const char* where) {
  static const bool debug = std::getenv("FP8W8A8_DEBUG") != nullptr;
  if (e != cudaSuccess && debug) std::fprintf(stderr, "fp8w8a8: %s: %s\n", where, cudaGetErrorString(e));
  return e;
}

// ---------------------------------------------------------------------------
// launch
// ---------------------------------------------------------------------------

template <typename... KArgs, typename... Args>
fp8_status launch(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, bool pdl,
                  dim3 cluster, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  int n = 0;
  if (pdl) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  if (cluster.x * cluster.y * cluster.z > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = cluster.x;
    attr[n].val.clusterDim.y = cluster.y;
    attr[n].val.clusterDim.z = cluster.z;
    ++n;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  return report_cuda(cudaLaunchKernelEx(&cfg, kernel, args...), "kernel launch") == cudaSuccess ? FP8_OK
                                                                                       : FP8_ERR_CUDA;
}

struct BF16Mat {
  const uint16_t* p;
  int64_t rows, cols, ld;
  int contiguous() const { return ld == cols && aligned(p, 16); }
  int vec() const { return aligned(p, 16) && ld % 8 == 0; }
};

// ---------------------------------------------------------------------------
// validation
// ---------------------------------------------------------------------------

inline fp8_status check_bf16_mat(const void* p, int64_t rows, int64_t cols, int64_t ld) {
  if (rows < 0 || cols < 0 || rows > kMaxDim || cols > kMaxDim) return FP8_ERR_INVALID_ARG;
  if (ld < std::max<int64_t>(cols, 1)) return FP8_ERR_INVALID_ARG;
  if (rows > 0 && cols > 0 && p == nullptr) return FP8_ERR_INVALID_ARG;
  if (!aligned(p, 2)) return FP8_ERR_MISALIGNED;
  return FP8_OK;
}

// Whether an output is written over an input with another row stride, so that rows fall on other rows.
inline bool crosses(const void* out, int64_t ldo, const void* in, int64_t ldi, int64_t rows) {
  return out != nullptr && out == in && rows > 1 && ldo != ldi;
}

inline fp8_status check_fp8_mat(const void* p, int64_t rows, int64_t cols, int64_t ld) {
  if (rows < 0 || cols < 0 || rows > kMaxDim || cols > kMaxDim) return FP8_ERR_INVALID_ARG;
  if (ld < std::max<int64_t>(round_up16(cols), 16)) return FP8_ERR_INVALID_ARG;
  if (ld % FP8_LD_ALIGN != 0) return FP8_ERR_MISALIGNED;
  if (rows > 0 && p == nullptr) return FP8_ERR_INVALID_ARG;
  if (!aligned(p, 16)) return FP8_ERR_MISALIGNED;
  return FP8_OK;
}

// Scales of rows: fp32 [K blocks][lds], lds >= rows.
inline fp8_status check_row_scales(const float* s, int64_t rows, int64_t K, int64_t lds) {
  if (lds < std::max<int64_t>(rows, 1)) return FP8_ERR_INVALID_ARG;
  if (rows > 0 && K > 0 && s == nullptr) return FP8_ERR_INVALID_ARG;
  return aligned(s, 4) ? FP8_OK : FP8_ERR_MISALIGNED;
}

inline fp8_status check_ws(const void* ws, size_t ws_bytes, size_t need) {
  if (need == 0) return FP8_OK;
  if (ws == nullptr || ws_bytes < need) return FP8_ERR_WORKSPACE;
  if (!aligned(ws, 256)) return FP8_ERR_WORKSPACE;
  return FP8_OK;
}

inline size_t round_up_256(size_t b) { return (b + 255) / 256 * 256; }

// Hands out the parts of a workspace.
struct Carver {
  size_t at = 0;
  size_t take(size_t bytes) {
    const size_t p = at;
    at = round_up_256(at + bytes);
    return p;
  }
};

}  // namespace fp8k
