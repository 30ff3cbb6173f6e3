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
struct Elem<uint16_t, 2> {
  static __device__ __forceinline__ void load(const uint16_t* p, float (&f)[2]) {
    const uint32_t v = *reinterpret_cast<const uint32_t*>(p);
    f[0] = __uint_as_float(v << 16), f[1] = __uint_as_float(v & 0xFFFF0000u);
  }
  static __device__ __forceinline__ void store(uint16_t* p, const float (&f)[2]) {
    *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(f[0], f[1]);
  }
};
template <>
struct Elem<uint16_t, 4> {
  static __device__ __forceinline__ void load(const uint16_t* p, float (&f)[4]) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    f[0] = __uint_as_float(v.x << 16), f[1] = __uint_as_float(v.x & 0xFFFF0000u);
    f[2] = __uint_as_float(v.y << 16), f[3] = __uint_as_float(v.y & 0xFFFF0000u);
  }
  static __device__ __forceinline__ void store(uint16_t* p, const float (&f)[4]) {
    __nv_bfloat162 h[2] = {__floats2bfloat162_rn(f[0], f[1]), __floats2bfloat162_rn(f[2], f[3])};
    *reinterpret_cast<uint2*>(p) = *reinterpret_cast<const uint2*>(h);
  }
};
template <>
struct Elem<float, 2> {
  static __device__ __forceinline__ void load(const float* p, float (&f)[2]) {
    const float2 v = *reinterpret_cast<const float2*>(p);
    f[0] = v.x, f[1] = v.y;
  }
  static __device__ __forceinline__ void store(float* p, const float (&f)[2]) {
    *reinterpret_cast<float2*>(p) = make_float2(f[0], f[1]);
  }
};
template <>
struct Elem<float, 4> {
  static __device__ __forceinline__ void load(const float* p, float (&f)[4]) {
    const float4 v = *reinterpret_cast<const float4*>(p);
    f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
  }
  static __device__ __forceinline__ void store(float* p, const float (&f)[4]) {
    *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
  }
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

// ---------------------------------------------------------------------------
// Pairs of fp32 values, two IEEE operations per instruction (each rounded as a
// scalar one would be).
__device__ __forceinline__ uint64_t f2_bits(float2 a) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a.x), "f"(a.y));
  return d;
}
__device__ __forceinline__ float2 f2_of(uint64_t d) {
  float2 a;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a.x), "=f"(a.y) : "l"(d));
  return a;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(f2_bits(a)), "l"(f2_bits(b)));
  return f2_of(d);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(f2_bits(a)), "l"(f2_bits(b)));
  return f2_of(d);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(f2_bits(a)), "l"(f2_bits(b)), "l"(f2_bits(c)));
  return f2_of(d);
}
__device__ __forceinline__ float2 both(float a) { return make_float2(a, a); }
__device__ __forceinline__ float2 bf16_pair(uint32_t h) {
  return make_float2(__uint_as_float(h << 16), __uint_as_float(h & 0xFFFF0000u));
}

// N pairs added as a tree
template <int N>
__device__ __forceinline__ float2 tree_sum2(const float2 (&f)[N]) {
  if constexpr (N == 1) {
    return f[0];
  } else {
    float2 h[N / 2];
#pragma unroll
    for (int j = 0; j < N / 2; ++j) h[j] = add2(f[2 * j], f[2 * j + 1]);
    return tree_sum2<N / 2>(h);
  }
}

// ---------------------------------------------------------------------------
// Rows of a matrix staged in shared memory by asynchronous copies, and read
// from there E elements at a time. E = 1 takes rows of any alignment, E = 2 those
// of an even width: the copy keeps the row's offset within 16 bytes, so that all
// of it but the ends moves in 16-byte pieces whatever the width of the matrix.
template <typename T, int E>
struct StagedRow {
  static constexpr bool OFFSET = E <= 2;            // rows keep their offset
  static constexpr int PAIRS = E == 1 ? 1 : E / 2;  // pairs of a unit (E = 1: two elements `stride` apart)
  static constexpr int PAD = OFFSET ? 32 : 0;       // bytes of a slot beyond its columns

  // T threads (tid their index) copy K <= KP elements from g into the slot.
  // cut_head, cut_tail: the memory just ahead of / behind the row may not be read
  // (the matrix's first and last row).
  template <int KP, int T_>
  static __device__ __forceinline__ void copy(uint8_t* slot_ptr, const T* g, int K, bool cut_head, bool cut_tail,
                                              int tid) {
    constexpr int threads = T_;
    const uint32_t slot = smem_u32(slot_ptr);
    const int bytes = K * static_cast<int>(sizeof(T));
    if constexpr (!OFFSET) {
      const uint8_t* src = reinterpret_cast<const uint8_t*>(g) + tid * 16;
      constexpr int PIECES = (KP * int(sizeof(T)) + T_ * 16 - 1) / (T_ * 16);
#pragma unroll
      for (int j = 0; j < PIECES; ++j)
        if ((tid + j * T_) * 16 < bytes) copy16(slot + (tid + j * T_) * 16, src + j * (T_ * 16));
    } else {
      const uintptr_t a = reinterpret_cast<uintptr_t>(g), end = a + bytes, base = a & ~uintptr_t(15);
      const uintptr_t a16 = (a + 15) & ~uintptr_t(15), e16 = end & ~uintptr_t(15);
      for (uintptr_t i = a16 + tid * 16; i + 16 <= end; i += threads * 16)
        copy16(slot + static_cast<uint32_t>(i - base), reinterpret_cast<const void*>(i));
      if (tid < 8) {  // up to four words ahead of the whole pieces, up to four behind them
        const bool head = tid < 4;
        const uintptr_t w = head ? (a & ~uintptr_t(3)) + 4 * tid : e16 + 4 * (tid - 4);
        if (head ? w < (a16 < end ? a16 : end) : (e16 >= a16 && w < end)) {
          const uint32_t dst = slot + static_cast<uint32_t>(w - base);
          if (sizeof(T) == 2 && ((w < a && cut_head) || (w + 4 > end && cut_tail))) {
#pragma unroll
            for (int j = 0; j < 2; ++j)
              if (w + 2 * j >= a && w + 2 * j < end)
                asm volatile("st.shared.u16 [%0], %1;" ::"r"(dst + 2 * j),
                             "h"(*reinterpret_cast<const volatile uint16_t*>(w + 2 * j))
                             : "memory");
          } else {
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(w) : "memory");
          }
        }
      }
    }
  }
  static __device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  }
  // zeros behind the row's columns, once: the copies never reach there (with an
  // offset they do: what is read from there is replaced)
  template <int KP, int T_>
  static __device__ __forceinline__ void clear_pad(uint8_t* slot, int K, int tid) {
    if constexpr (!OFFSET)
      for (int i = K * int(sizeof(T)) + tid * 16; i < KP * int(sizeof(T)); i += T_ * 16)
        *reinterpret_cast<uint4*>(slot + i) = make_uint4(0u, 0u, 0u, 0u);
  }
  // element 0 within the slot
  static __device__ __forceinline__ const uint8_t* first(const uint8_t* slot, const T* g) {
    return OFFSET ? slot + (reinterpret_cast<uintptr_t>(g) & 15u) : slot;
  }
  // the unit with zeros behind the row's columns
  static __device__ __forceinline__ void get_or_zero(const uint8_t* row, int k, int stride, int K, float2 (&f)[PAIRS]) {
    get(row, k, stride, f);
    if constexpr (E == 1) f[0] = make_float2(k < K ? f[0].x : 0.f, k + stride < K ? f[0].y : 0.f);
    if constexpr (E == 2) f[0] = k < K ? f[0] : make_float2(0.f, 0.f);
  }
  // the unit at column k (E = 1: columns k and k + stride) of a row in shared memory
  static __device__ __forceinline__ void get(const uint8_t* row, int k, int stride, float2 (&f)[PAIRS]) {
    const T* p = reinterpret_cast<const T*>(row) + k;
    if constexpr (E == 1) {
      if constexpr (sizeof(T) == 4)
        f[0] = make_float2(p[0], p[stride]);
      else
        f[0] = make_float2(bf16_bits_to_float(p[0]), bf16_bits_to_float(p[stride]));
    } else if constexpr (E == 2) {
      if constexpr (sizeof(T) == 4)
        f[0] = *reinterpret_cast<const float2*>(p);
      else
        f[0] = bf16_pair(*reinterpret_cast<const uint32_t*>(p));
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int j = 0; j < E / 4; ++j) {
        const float4 v = reinterpret_cast<const float4*>(p)[j];
        f[2 * j] = make_float2(v.x, v.y);
        f[2 * j + 1] = make_float2(v.z, v.w);
      }
    } else if constexpr (E == 8) {
      const uint4 v = *reinterpret_cast<const uint4*>(p);
      f[0] = bf16_pair(v.x), f[1] = bf16_pair(v.y), f[2] = bf16_pair(v.z), f[3] = bf16_pair(v.w);
    } else {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      f[0] = bf16_pair(v.x), f[1] = bf16_pair(v.y);
    }
  }
};

// The unit at column k of a row in global memory (E = 1: k and k + stride, each
// where it is below K)
template <typename T, int E>
__device__ __forceinline__ void put_unit(T* row, int k, int stride, int K, const float2 (&f)[E == 1 ? 1 : E / 2]) {
  if constexpr (E == 1) {
    const float a[1] = {f[0].x}, b[1] = {f[0].y};
    if (k < K) Elem<T, 1>::store(row + k, a);
    if (k + stride < K) Elem<T, 1>::store(row + k + stride, b);
  } else {
    float o[E];
#pragma unroll
    for (int j = 0; j < E / 2; ++j) {
      o[2 * j] = f[j].x;
      o[2 * j + 1] = f[j].y;
    }
    Elem<T, E>::store(row + k, o);
  }
}

// 1 / sqrt(v): the fast estimate and a Newton step (half an ulp or so; infinity and NaN pass through)
__device__ __forceinline__ float inv_sqrt(float v) {
  const float r = rsqrtf(v);
  const float e = fmaf(-v * r, r, 1.0f);
  return isfinite(e) ? fmaf(0.5f * r, e, r) : r;
}

__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

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

// barrier of W warps (W = 1: of the warp); id 0 is the CTA's own
template <int W>
__device__ __forceinline__ void group_sync(int id) {
  if constexpr (W == 1)
    __syncwarp();
  else
    asm volatile("bar.sync %0, %1;" ::"r"(id), "n"(W * 32) : "memory");
}

// NS sums over a group of W warps; every thread gets the totals. sh holds
// W * NS floats that no thread still reads when the call begins.
template <int W, int NS>
__device__ __forceinline__ void group_sums(float (&v)[NS], float* sh, int warp, int id) {
#pragma unroll
  for (int i = 0; i < NS; ++i) v[i] = warp_sum(v[i]);
  if constexpr (W > 1) {
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
      for (int i = 0; i < NS; ++i) sh[i * W + warp] = v[i];
    }
    group_sync<W>(id);
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      float t = sh[i * W];
#pragma unroll
      for (int w = 1; w < W; ++w) t += sh[i * W + w];
      v[i] = t;
    }
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
