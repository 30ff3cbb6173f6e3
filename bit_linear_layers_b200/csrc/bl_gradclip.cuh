// The 2-norm over many gradient tensors, and the gradients scaled down to a
// largest norm:
//   n = sqrt(sum g^2 over all tensors), c = min(1, max_norm / (n + 1e-6)), out = c g
// (c = 1 where max_norm is infinite and n no NaN).
//
// Squares of fp32 and bf16 values span twice the type's exponents, so an fp32
// sum overflows from |g| = 1.8e19 on and loses what is below 1e-19. The values
// of one 16-byte access are squared and added in fp32; the result is added to
// a double where it is far inside the range, and formed again in doubles
// where it is not (rare, and exact enough at any scale). The CTAs' sums are
// stored in order and added in order by every CTA of the second kernel, so the
// norm does not depend on the order of execution. Both kernels are bound by
// memory: all loads of a chunk are issued before the first is used. The second
// reading of the gradients is what clipping costs beyond the copy: the norm has
// to be known first, and only the last 126 MB can still be in L2. The 202 million
// fp32 gradients of a 7B-shaped layer take 390 us (2.43 GB moved at 6.2 TB/s, 95% of
// the copy rate), 180 tensors of 6 million elements 17 us.
#pragma once

#include "bl_elem.cuh"

namespace bl {

constexpr int kGcThreads = 256;
// 16-byte accesses per thread and chunk: a chunk is 16 KB of one tensor, 32 KB from
// 96 MB of gradients on (808 MB 410 and 390 us, 80 MB 46 and 49 us, 24 MB 17 and 20 us)
constexpr int kGcVecs = 4, kGcVecsMany = 8;
constexpr int64_t kGcManyBytes = int64_t(96) << 20;
constexpr int kGcMaxTensors = 900;                   // per launch: descriptors travel as kernel parameters
constexpr int kGcMaxCtas = 1184;                     // partial sums per launch

struct GcTensor {
  const void* g;
  void* out;
  int64_t numel;
};
// CTA b takes the chunks from gc_begin(b) to gc_begin(b + 1). Parameters are read through
// the constant cache, a miss at a time: the tensor of a CTA's first chunk is
// looked up by the host (a search over the table took longer than the sums of a
// small model).
template <int CAP>
struct GcParams {
  GcTensor t[CAP];
  int32_t chunk0[CAP + 1];     // first chunk of each tensor
  uint16_t first[kGcMaxCtas + 1];  // tensor of CTA b's first chunk; [grid]: of the last chunk
  uint8_t f32[CAP];
};

// first chunk of CTA b: the first chunks % grid CTAs have one more than the others
__host__ __device__ inline int gc_begin(int chunks, int b, int grid) {
  const int q = chunks / grid, r = chunks - q * grid;
  return b * q + (b < r ? b : r);
}

template <typename T>
__device__ __forceinline__ float gc_value(uint32_t word, int j) {
  if constexpr (sizeof(T) == 4) return __uint_as_float(word);
  return j == 0 ? __uint_as_float(word << 16) : __uint_as_float(word & 0xFFFF0000u);
}

// squares of one 16-byte access added in fp32; `good` unless that may have left the range
template <typename T>
__device__ __forceinline__ float gc_squares(const uint4& v, bool& good) {
  constexpr int PER = 4 / sizeof(T);
  const uint32_t h[4] = {v.x, v.y, v.z, v.w};
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const float f = gc_value<T>(h[i], j);
      s = fmaf(f, f, s);
    }
  // 2^-60: a square lost below the smallest normal, 2^-126, is nothing next to it
  const uint32_t any = (v.x | v.y | v.z | v.w) & (sizeof(T) == 4 ? 0x7FFFFFFFu : 0x7FFF7FFFu);
  good = good && ((s > 0x1p-60f && s < 0x1p120f) || any == 0u);
  return s;
}
template <typename T>
__device__ __noinline__ double gc_squares_exact(uint4 v) {
  constexpr int PER = 4 / sizeof(T);
  const uint32_t h[4] = {v.x, v.y, v.z, v.w};
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

// A thread's share of chunk `rel` of a tensor: the 16-byte pieces v0 + u *
// kGcThreads, counted from the aligned address at or below the tensor's first
// byte, so piece v begins at element v * PER - mis. Pieces that lie within the
// tensor are accessed whole; those that its ends cut (two at most) element by
// element, by the one thread that has them.
template <typename T, int VECS>
struct GcShare {
  static constexpr int PER = 16 / sizeof(T);
  int64_t e0;  // first element of piece 0
  int64_t numel;
  __device__ __forceinline__ GcShare(const GcTensor& t, int rel) {
    const int mis = static_cast<int>((reinterpret_cast<uintptr_t>(t.g) & 15u) / sizeof(T));
    e0 = (static_cast<int64_t>(rel) * (kGcThreads * VECS) + threadIdx.x) * PER - mis;
    numel = t.numel;
  }
  __device__ __forceinline__ int64_t at(int u) const { return e0 + u * (kGcThreads * PER); }
  __device__ __forceinline__ bool whole(int u) const { return at(u) >= 0 && at(u) + PER <= numel; }
  // f(first element, end) of the pieces that the ends cut
  template <typename F>
  __device__ __forceinline__ void cut(F&& f) const {
    if (e0 >= 0 && at(VECS - 1) + PER <= numel) return;
#pragma unroll 1
    for (int u = 0; u < VECS; ++u) {
      const int64_t e = at(u);
      if (!whole(u) && e < numel && e + PER > 0) f(e < 0 ? 0 : e, e + PER < numel ? e + PER : numel);
    }
  }
};

__device__ __forceinline__ uint4 gc_load(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

template <typename T, int VECS>
__device__ __forceinline__ double gc_norm_chunk(const GcTensor& t, int rel) {
  const T* g = static_cast<const T*>(t.g);
  const GcShare<T, VECS> sh(t, rel);
  uint4 v[VECS];
#pragma unroll
  for (int u = 0; u < VECS; ++u) v[u] = sh.whole(u) ? gc_load(g + sh.at(u)) : make_uint4(0u, 0u, 0u, 0u);
  bool good = true;
  float f[VECS];
#pragma unroll
  for (int u = 0; u < VECS; ++u) f[u] = gc_squares<T>(v[u], good);
  double s = 0.0;
  if (good) {
#pragma unroll
    for (int u = 0; u < VECS; u += 2) s += static_cast<double>(f[u]) + static_cast<double>(f[u + 1]);
  } else {
#pragma unroll
    for (int u = 0; u < VECS; ++u) s += gc_squares_exact<T>(v[u]);
  }
  sh.cut([&](int64_t a, int64_t b) {
    for (int64_t i = a; i < b; ++i) {
      float e[1];
      Elem<T, 1>::load(g + i, e);
      s = fma(static_cast<double>(e[0]), static_cast<double>(e[0]), s);
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

template <int CAP, int VECS>
__global__ void __launch_bounds__(kGcThreads)
    grad_norm_kernel(const __grid_constant__ GcParams<CAP> P, int chunks, double* __restrict__ sums) {
  __shared__ double sh[kGcThreads / 32];
  const int c0 = gc_begin(chunks, blockIdx.x, gridDim.x), c1 = gc_begin(chunks, blockIdx.x + 1, gridDim.x);
  grid_begin();
  double s = 0.0;
  if (c0 < c1) {
    int i = P.first[blockIdx.x];
    for (int c = c0; c < c1; ++c) {
      while (P.chunk0[i + 1] <= c) ++i;
      const int rel = c - P.chunk0[i];
      s += P.f32[i] ? gc_norm_chunk<float, VECS>(P.t[i], rel) : gc_norm_chunk<uint16_t, VECS>(P.t[i], rel);
    }
  }
  s = gc_block_sum(s, sh);
  if (threadIdx.x == 0) sums[blockIdx.x] = s;
}

template <typename T, int VECS>
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
  const GcShare<T, VECS> sh(t, rel);
  uint4 v[VECS];
#pragma unroll
  for (int u = 0; u < VECS; ++u) v[u] = sh.whole(u) ? gc_load(g + sh.at(u)) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
  for (int u = 0; u < VECS; ++u) {
    uint32_t h[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 4) {
        h[i] = __float_as_uint(__uint_as_float(h[i]) * coef);
      } else {
        const __nv_bfloat162 b = __floats2bfloat162_rn(gc_value<T>(h[i], 0) * coef, gc_value<T>(h[i], 1) * coef);
        h[i] = *reinterpret_cast<const uint32_t*>(&b);
      }
    }
    if (!sh.whole(u)) continue;
    T* o = out + sh.at(u);
    if (same) {
      *reinterpret_cast<uint4*>(o) = make_uint4(h[0], h[1], h[2], h[3]);
    } else {
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        if constexpr (sizeof(T) == 4)
          o[j] = __uint_as_float(h[j]);
        else
          o[j] = static_cast<uint16_t>(h[j / 2] >> (16 * (j & 1)));
      }
    }
  }
  sh.cut(single);
}

// stats[0] = norm, stats[1] = coefficient; then the tensors of this launch
template <int CAP, int VECS>
__global__ void __launch_bounds__(kGcThreads)
    grad_scale_kernel(const __grid_constant__ GcParams<CAP> P, int chunks, const double* __restrict__ sums,
                      int num_sums, float max_norm, float* __restrict__ stats) {
  __shared__ double sh[kGcThreads / 32];
  grid_begin();
  double s = 0.0;
  for (int i = threadIdx.x; i < num_sums; i += kGcThreads) s += sums[i];
  const double norm = sqrt(gc_block_sum(s, sh));
  double c = static_cast<double>(max_norm) / (norm + 1e-6);
  // 1 also where both are infinite: no norm is above an infinite bound. A NaN norm stays NaN
  if (!(c <= 1.0) && !isnan(norm)) c = 1.0;
  const float coef = static_cast<float>(c);
  if (stats && blockIdx.x == 0 && threadIdx.x == 0) {
    stats[0] = static_cast<float>(norm);
    stats[1] = coef;
  }
  const int c0 = gc_begin(chunks, blockIdx.x, gridDim.x), c1 = gc_begin(chunks, blockIdx.x + 1, gridDim.x);
  if (c0 >= c1) return;
  // from the last chunk down: what the norm's pass read last is still in L2
  int i = P.first[blockIdx.x + 1];
  for (int ch = c1 - 1; ch >= c0; --ch) {
    while (P.chunk0[i] > ch) --i;
    const GcTensor& t = P.t[i];
    if (!t.out || (coef == 1.0f && t.out == t.g)) continue;  // nothing to write
    const int rel = ch - P.chunk0[i];
    if (P.f32[i])
      gc_scale_chunk<float, VECS>(t, rel, coef);
    else
      gc_scale_chunk<uint16_t, VECS>(t, rel, coef);
  }
}

}  // namespace bl
