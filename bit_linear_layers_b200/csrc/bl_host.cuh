// Host-side helpers shared by the library's translation units: argument checks,
// launch status, occupancy of persistent kernels, launches with programmatic
// serialisation.
#pragma once

#include <algorithm>
#include <atomic>
#include <cstdint>
#include <type_traits>

#include "bl_common.cuh"

namespace bl {

// one-time set-up of the current device (bl_api.cu); *num_sms where given
int library_device(int* num_sms);
// bytes of workspace of bl_layer_norm_backward (bl_norm_grad.cu)
size_t norm_workspace_bytes(int64_t M, int64_t K);

namespace {

constexpr int kMaxDevices = 64;
constexpr int64_t kMaxProduct = int64_t(1) << 40;
constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1;

inline size_t align256(size_t v) { return (v + 255) & ~size_t(255); }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

template <typename Kernel>
inline bool set_smem(Kernel k, int bytes) {
  return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) == cudaSuccess;
}

inline int launch_status() {
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? BL_OK : BL_ERR_CUDA;
}

constexpr int64_t kMaxIds = (int64_t(1) << 31) - 1;

inline bool type_ok(int type) { return type == BL_TYPE_BF16 || type == BL_TYPE_F32; }
inline int type_bytes(int type) { return type == BL_TYPE_F32 ? 4 : 2; }
inline bool aligned_to(const void* p, int bytes) { return reinterpret_cast<uintptr_t>(p) % uintptr_t(bytes) == 0; }

// rows of K elements with a pitch of ld elements, all below 2^40 elements
inline int check_rows(int64_t M, int64_t K, int64_t ld) {
  if (ld < K) return BL_ERR_INVALID_ARG;
  if (ld > kMaxProduct || (M > 0 && ld >= kMaxProduct / M)) return BL_ERR_UNSUPPORTED;
  return BL_OK;
}

inline int check_norm_shape(int64_t M, int64_t K) {
  if (M < 0 || K < 1) return BL_ERR_INVALID_ARG;
  return M > kMaxDim || K > kMaxDim ? BL_ERR_UNSUPPORTED : BL_OK;
}

// rows that `elems` elements at a time can be read or written of
inline bool rows_aligned(const void* p, int type, int64_t ld, int64_t K, int64_t M, int elems) {
  return K % elems == 0 && (M <= 1 || ld % elems == 0) && aligned_to(p, elems * type_bytes(type));
}

template <int V>
using Int = std::integral_constant<int, V>;

// CTAs per SM of a kernel on the current device, looked up once per device
// (and its dynamic shared memory allowed)
template <auto Kernel>
int ctas_per_sm(int threads, int smem) {
  static std::atomic<int> known[kMaxDevices];
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
    cudaGetLastError();
    return 0;
  }
  int n = known[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    if ((smem > 0 && !set_smem(Kernel, smem)) ||
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, Kernel, threads, size_t(smem)) != cudaSuccess) {
      cudaGetLastError();
      return 0;
    }
    known[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

// CTAs of a persistent kernel over `units`: as many as fit at once, evenly loaded
inline int64_t persistent_grid(int ctas_per_sm, int sms, int64_t units, int64_t most) {
  const int64_t cap = std::min<int64_t>(int64_t(ctas_per_sm) * sms, most);
  return units <= cap ? units : cdiv(units, cdiv(units, cap));
}

// launch with programmatic serialisation: the kernel may be scheduled while
// the one before it runs, and waits for it by itself
template <typename... Params, typename... Args>
int launch_after(void (*kernel)(Params...), dim3 grid, int threads, int smem, cudaStream_t s, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kernel, args...) != cudaSuccess) {
    cudaGetLastError();
    return BL_ERR_CUDA;
  }
  return launch_status();
}

// f(uint16_t or float of `a`, of `b`)
template <typename F>
inline int with_types(int a, int b, F&& f) {
  if (a == BL_TYPE_F32) return b == BL_TYPE_F32 ? f(float{}, float{}) : f(float{}, uint16_t{});
  return b == BL_TYPE_F32 ? f(uint16_t{}, float{}) : f(uint16_t{}, uint16_t{});
}

}  // namespace
}  // namespace bl
