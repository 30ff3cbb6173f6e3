// Element access of the full-precision operators (layer norm, embedding,
// gradient clipping): bf16 (raw uint16_t patterns) and fp32 values in memory,
// fp32 in registers, E consecutive elements per access.
#pragma once

#include "bl_common.cuh"

namespace bl {

// E elements of T in one access (two 16-byte ones for eight fp32); p must be
// aligned to E * sizeof(T) or to 16 bytes, whichever is less
template <typename T, int E>
struct Elem;

template <>
struct Elem<uint16_t, 1> {
  static __device__ __forceinline__ void load(const uint16_t* p, float (&f)[1]) { f[0] = bf16_bits_to_float(*p); }
  static __device__ __forceinline__ void store(uint16_t* p, const float (&f)[1]) { *p = float_to_bf16_bits(f[0]); }
};
template <>
struct Elem<float, 1> {
  static __device__ __forceinline__ void load(const float* p, float (&f)[1]) { f[0] = *p; }
  static __device__ __forceinline__ void store(float* p, const float (&f)[1]) { *p = f[0]; }
};
template <>
struct Elem<uint16_t, 8> {
  static __device__ __forceinline__ void load(const uint16_t* p, float (&f)[8]) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    const uint32_t h[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[2 * j] = __uint_as_float(h[j] << 16);
      f[2 * j + 1] = __uint_as_float(h[j] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ void store(uint16_t* p, const float (&f)[8]) {
    uint32_t h[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * j], f[2 * j + 1]);
      h[j] = static_cast<uint32_t>(__bfloat16_as_ushort(b.x)) | (static_cast<uint32_t>(__bfloat16_as_ushort(b.y)) << 16);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(h[0], h[1], h[2], h[3]);
  }
};
template <>
struct Elem<float, 8> {
  static __device__ __forceinline__ void load(const float* p, float (&f)[8]) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
    f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  }
  static __device__ __forceinline__ void store(float* p, const float (&f)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
  }
};

// NS sums over a CTA of WARPS warps; every thread gets the totals. sh holds
// WARPS * NS floats and may be reused by the next call.
template <int WARPS, int NS>
__device__ __forceinline__ void block_sums(float (&v)[NS], float* sh) {
#pragma unroll
  for (int i = 0; i < NS; ++i) v[i] = warp_sum(v[i]);
  if constexpr (WARPS > 1) {
    __syncthreads();  // sh may still be read from a previous reduction
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
      for (int i = 0; i < NS; ++i) sh[(threadIdx.x >> 5) * NS + i] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      float t = sh[i];
#pragma unroll
      for (int w = 1; w < WARPS; ++w) t += sh[w * NS + i];
      v[i] = t;
    }
  }
}

}  // namespace bl
