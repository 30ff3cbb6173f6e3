// The 2-norm over many gradient tensors, and the gradients scaled down to a
// largest norm:
//   n = sqrt(sum g^2 over all tensors), c = min(1, max_norm / (n + 1e-6)), out = c g
//
// Squares of fp32 and bf16 values span twice the type's exponents, so an fp32
// sum overflows from |g| = 1.8e19 on and loses what is below 1e-19. The values
// of one 16-byte access are squared and added in fp32; the result is added to
// a double where it is far inside the range, and formed again in doubles
// where it is not (rare, and exact enough at any scale). The CTAs' sums are
// stored in order and added in order by every CTA of the second kernel, so the
// norm does not depend on the order of execution.
#pragma once

#include "bl_elem.cuh"

namespace bl {

constexpr int kGcThreads = 256;
constexpr int kGcVecs = 8;                           // 16-byte accesses per thread and chunk
constexpr int kGcChunkVecs = kGcThreads * kGcVecs;   // a chunk is 32 KB of one tensor
constexpr int kGcMaxTensors = 1024;                  // per launch: descriptors travel as kernel parameters
constexpr int kGcMaxCtas = 1024;                     // partial sums per launch

struct GcTensor {
  const void* g;
  void* out;
  int64_t numel;
};
template <int CAP>
struct GcParams {
  GcTensor t[CAP];
  int32_t chunk0[CAP + 1];  // first chunk of each tensor
  uint8_t f32[CAP];
  int32_t n;
};

// tensor of chunk c: the last one that starts at or before it
template <int CAP>
__device__ __forceinline__ int gc_find(const GcParams<CAP>& P, int c) {
  int lo = 0, hi = P.n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (P.chunk0[mid] <= c)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

template <typename T>
__device__ __forceinline__ float gc_value(uint32_t word, int j);
template <>
__device__ __forceinline__ float gc_value<float>(uint32_t word, int) {
  return __uint_as_float(word);
}
template <>
__device__ __forceinline__ float gc_value<uint16_t>(uint32_t word, int j) {
  return j == 0 ? __uint_as_float(word << 16) : __uint_as_float(word & 0xFFFF0000u);
}

// sum of squares of one 16-byte access
template <typename T>
__device__ __forceinline__ double gc_squares(const uint4& v) {
  constexpr int PER = 4 / sizeof(T);
  const uint32_t h[4] = {v.x, v.y, v.z, v.w};
  if (((v.x | v.y | v.z | v.w) & (sizeof(T) == 4 ? 0x7FFFFFFFu : 0x7FFF7FFFu)) == 0u) return 0.0;
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const float f = gc_value<T>(h[i], j);
      s = fmaf(f, f, s);
    }
  // 2^-60: a square lost below the smallest normal, 2^-126, is nothing next to it
  if (s > 0x1p-60f && s < 0x1p120f) return static_cast<double>(s);
  double t = 0.0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const double f = static_cast<double>(gc_value<T>(h[i], j));
      t = fma(f, f, t);
    }
  return t;
}

// f(first element, number of elements): the 16-byte aligned pieces of chunk
// `rel` of a tensor; pieces cut by the tensor's ends are shorter. The pieces
// are counted from the aligned address at or below the tensor's first byte.
template <typename T, typename Whole, typename Cut>
__device__ __forceinline__ void gc_for_chunk(const void* g, int64_t numel, int rel, Whole&& whole, Cut&& cut) {
  constexpr int PER = 16 / sizeof(T);
  const int mis = static_cast<int>((reinterpret_cast<uintptr_t>(g) & 15u) / sizeof(T));
  const int64_t v0 = static_cast<int64_t>(rel) * kGcChunkVecs + threadIdx.x;
#pragma unroll
  for (int u = 0; u < kGcVecs; ++u) {
    const int64_t e = (v0 + u * kGcThreads) * PER - mis;
    if (e >= 0 && e + PER <= numel)
      whole(u, e);
    else if (e < numel && e + PER > 0)
      cut(e < 0 ? 0 : e, e + PER < numel ? e + PER : numel);
  }
}

template <typename T>
__device__ __forceinline__ double gc_norm_chunk(const GcTensor& t, int rel) {
  const T* g = static_cast<const T*>(t.g);
  double s = 0.0;
  gc_for_chunk<T>(
      t.g, t.numel, rel,
      [&](int, int64_t e) { s += gc_squares<T>(*reinterpret_cast<const uint4*>(g + e)); },
      [&](int64_t a, int64_t b) {
        for (int64_t i = a; i < b; ++i) {
          float f[1];
          Elem<T, 1>::load(g + i, f);
          s = fma(static_cast<double>(f[0]), static_cast<double>(f[0]), s);
        }
      });
  return s;
}

// CTA sum of doubles, the total in thread 0
__device__ __forceinline__ double gc_block_sum(double v, double* sh) {
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
  __syncthreads();
  double t = sh[0];
  for (int w = 1; w < kGcThreads / 32; ++w) t += sh[w];
  return t;
}

template <int CAP>
__global__ void __launch_bounds__(kGcThreads)
    grad_norm_kernel(const __grid_constant__ GcParams<CAP> P, double* __restrict__ sums) {
  __shared__ double sh[kGcThreads / 32];
  const int chunks = P.chunk0[P.n];
  const int c0 = static_cast<int>(static_cast<int64_t>(chunks) * blockIdx.x / gridDim.x);
  const int c1 = static_cast<int>(static_cast<int64_t>(chunks) * (blockIdx.x + 1) / gridDim.x);
  double s = 0.0;
  if (c0 < c1) {
    int i = gc_find(P, c0);
    for (int c = c0; c < c1; ++c) {
      while (P.chunk0[i + 1] <= c) ++i;
      const int rel = c - P.chunk0[i];
      s += P.f32[i] ? gc_norm_chunk<float>(P.t[i], rel) : gc_norm_chunk<uint16_t>(P.t[i], rel);
    }
  }
  s = gc_block_sum(s, sh);
  if (threadIdx.x == 0) sums[blockIdx.x] = s;
}

template <typename T>
__device__ __forceinline__ void gc_scale_chunk(const GcTensor& t, int rel, float coef) {
  const T* g = static_cast<const T*>(t.g);
  T* out = static_cast<T*>(t.out);
  constexpr int PER = 16 / sizeof(T);
  const bool same = ((reinterpret_cast<uintptr_t>(g) ^ reinterpret_cast<uintptr_t>(out)) & 15u) == 0;
  auto single = [&](int64_t a, int64_t b) {
    for (int64_t i = a; i < b; ++i) {
      float f[1];
      Elem<T, 1>::load(g + i, f);
      f[0] *= coef;
      Elem<T, 1>::store(out + i, f);
    }
  };
  gc_for_chunk<T>(
      t.g, t.numel, rel,
      [&](int, int64_t e) {
        if (!same) return single(e, e + PER);
        const uint4 v = *reinterpret_cast<const uint4*>(g + e);
        uint32_t h[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (sizeof(T) == 4) {
            h[i] = __float_as_uint(__uint_as_float(h[i]) * coef);
          } else {
            h[i] = static_cast<uint32_t>(float_to_bf16_bits(gc_value<T>(h[i], 0) * coef)) |
                   (static_cast<uint32_t>(float_to_bf16_bits(gc_value<T>(h[i], 1) * coef)) << 16);
          }
        }
        *reinterpret_cast<uint4*>(out + e) = make_uint4(h[0], h[1], h[2], h[3]);
      },
      single);
}

// stats[0] = norm, stats[1] = coefficient; then the tensors of this launch
template <int CAP>
__global__ void __launch_bounds__(kGcThreads)
    grad_scale_kernel(const __grid_constant__ GcParams<CAP> P, const double* __restrict__ sums, int num_sums,
                      float max_norm, float* __restrict__ stats) {
  __shared__ double sh[kGcThreads / 32];
  double s = 0.0;
  for (int i = threadIdx.x; i < num_sums; i += kGcThreads) s += sums[i];
  const double norm = sqrt(gc_block_sum(s, sh));
  double c = static_cast<double>(max_norm) / (norm + 1e-6);
  c = c > 1.0 ? 1.0 : c;  // NaN stays NaN
  const float coef = static_cast<float>(c);
  if (stats && blockIdx.x == 0 && threadIdx.x == 0) {
    stats[0] = static_cast<float>(norm);
    stats[1] = coef;
  }
  const int chunks = P.chunk0[P.n];
  const int c0 = static_cast<int>(static_cast<int64_t>(chunks) * blockIdx.x / gridDim.x);
  const int c1 = static_cast<int>(static_cast<int64_t>(chunks) * (blockIdx.x + 1) / gridDim.x);
  if (c0 >= c1) return;
  int i = gc_find(P, c1 - 1);
  for (int ch = c1 - 1; ch >= c0; --ch) {
    while (P.chunk0[i] > ch) --i;
    const GcTensor& t = P.t[i];
    if (!t.out || (coef == 1.0f && t.out == t.g)) continue;  // nothing to write
    const int rel = ch - P.chunk0[i];
    if (P.f32[i])
      gc_scale_chunk<float>(t, rel, coef);
    else
      gc_scale_chunk<uint16_t>(t, rel, coef);
  }
}

}  // namespace bl
