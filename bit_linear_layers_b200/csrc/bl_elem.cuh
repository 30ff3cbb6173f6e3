// Element access of the full-precision operators (layer norm, embedding,
// gradient clipping): bf16 (raw uint16_t patterns) and fp32 values in memory,
// fp32 in registers, E consecutive elements per access.
#pragma once

#include "bl_common.cuh"

namespace bl {

// E elements of T in one access; p must be aligned to E * sizeof(T)
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
    asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=f"(f[0]), "=f"(f[1]), "=f"(f[2]), "=f"(f[3]), "=f"(f[4]), "=f"(f[5]), "=f"(f[6]), "=f"(f[7])
                 : "l"(p));
  }
  static __device__ __forceinline__ void store(float* p, const float (&f)[8]) {
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(f[0]), "f"(f[1]), "f"(f[2]),
                 "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7])
                 : "memory");
  }
};

// E elements as they lie in memory, and their values; raw loads are held
// across a row's passes so that a bf16 row costs half the registers. One
// access each (16 bytes for eight bf16, 32 for eight fp32, aligned so), and
// loaded once: a row may be overwritten in place after it.
template <typename T, int E>
struct Raw;
template <>
struct Raw<uint16_t, 8> {
  uint4 v;
  __device__ __forceinline__ void load(const uint16_t* p) {
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
  }
  __device__ __forceinline__ void zero() { v = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    const uint32_t h[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[2 * j] = __uint_as_float(h[j] << 16);
      f[2 * j + 1] = __uint_as_float(h[j] & 0xFFFF0000u);
    }
  }
};
template <>
struct Raw<float, 8> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    asm volatile("ld.global.L1::no_allocate.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=f"(a.x), "=f"(a.y), "=f"(a.z), "=f"(a.w), "=f"(b.x), "=f"(b.y), "=f"(b.z), "=f"(b.w)
                 : "l"(p));
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
    f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  }
};
template <>
struct Raw<uint16_t, 1> {
  uint16_t v;
  __device__ __forceinline__ void load(const uint16_t* p) { v = *p; }
  __device__ __forceinline__ void zero() { v = 0; }
  __device__ __forceinline__ void get(float (&f)[1]) const { f[0] = bf16_bits_to_float(v); }
};
template <>
struct Raw<float, 1> {
  float v;
  __device__ __forceinline__ void load(const float* p) { v = *p; }
  __device__ __forceinline__ void zero() { v = 0.f; }
  __device__ __forceinline__ void get(float (&f)[1]) const { f[0] = v; }
};

// E values added as a tree
template <int E>
__device__ __forceinline__ float tree_sum(const float (&f)[E]) {
  if constexpr (E == 1) {
    return f[0];
  } else {
    float h[E / 2];
#pragma unroll
    for (int j = 0; j < E / 2; ++j) h[j] = f[2 * j] + f[2 * j + 1];
    return tree_sum<E / 2>(h);
  }
}

// NS sums over a CTA of WARPS warps; every thread gets the totals. sh holds
// WARPS * NS floats that no thread still reads when the call begins.
template <int WARPS, int NS>
__device__ __forceinline__ void block_sums(float (&v)[NS], float* sh) {
#pragma unroll
  for (int i = 0; i < NS; ++i) v[i] = warp_sum(v[i]);
  if constexpr (WARPS > 1) {
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
      for (int i = 0; i < NS; ++i) sh[i * WARPS + (threadIdx.x >> 5)] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      float t = sh[i * WARPS];
#pragma unroll
      for (int w = 1; w < WARPS; ++w) t += sh[i * WARPS + w];
      v[i] = t;
    }
  }
}

}  // namespace bl
