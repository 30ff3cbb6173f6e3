// Layer norm with an affine part and its gradient, the full-precision norm
// in front of the binarized linears when they are trained.
//
//   mu = mean_k x, var = mean_k (x - mu)^2, rstd = (var + eps)^-1/2
//   y_k = (x_k - mu) * rstd * w_k + b_k
//
// With z_k = (x_k - mu) * rstd and g_k = dy_k * w_k the gradient is
//   dx_k = rstd * (g_k - mean_k g - z_k * mean_k (g z))
//   dw_k = sum_m dy_mk z_mk,  db_k = sum_m dy_mk
//
// Sums are fp32. A row far from zero loses its small deviations when a
// rounded mean is subtracted, so both passes shift first and correct after:
// with c the rounded mean and d = x - c (exact or nearly so), the mean is
// c + mean d and the variance mean d^2 - (mean d)^2, where mean d is a rounding
// of the mean only and the subtraction cancels nothing.
#pragma once

#include "bl_elem.cuh"

namespace bl {

constexpr int kNormThreads = 256;
constexpr int kNormWarps = kNormThreads / 32;
constexpr int kNormMaxParts = 148 * 8;  // partial rows of dweight and dbias
constexpr int kNormMaxK = 16384;        // widest rows staged on chip (forward)
constexpr int kNormGradMaxK = 8192;     // ... (gradient)

// Rows staged on chip. A group of W warps takes a row: the row is copied into
// shared memory S - 1 rows ahead of its use, CPT columns per thread in units of
// E, unpacked once, and passed over three times in registers (2048 x 11007 bf16:
// 41 us, 88 us while 32 single columns per thread were indexed at run time and so
// lay in local memory). A few warps per row leave little beside the arithmetic
// itself: with eight, the sums' shuffles and barriers took more instructions than
// the row. The weight and the bias stay in registers up to 16
// columns per thread, else in shared memory (in planes of four columns, so that
// a warp's 16-byte reads meet no bank twice); read again for each row they would
// cost more L2 traffic than the row. The CTAs stay and their groups take rows in
// turn.
// fp32 rows from 256 columns on are bound by memory (65536 x 256: 20.7 us, 16384 x
// 1024: 19.5 us, the copy rate); narrower ones and bf16 rows by the latency of the
// two sums with 16 warps per SM, and bf16 rows of 4096 also by the one row per
// group that is on its way meanwhile (S = 2: 32 KB per SM; 4096 x 4096 bf16: 15.0
// us, 4.5 TB/s). One row of 4096 takes 2.7 us in bf16, 2.2 us in fp32.
template <typename TX, int E, int CPT, int W>
struct NormCfg {
  static_assert(CPT <= 32, "a thread's columns stay in registers");
  static constexpr int KP = CPT * W * 32;  // columns a group covers
  static constexpr int SLOT = KP * int(sizeof(TX)) + StagedRow<TX, E>::PAD;
  static constexpr int S = SLOT <= 2080 ? 4 : SLOT <= 4128 ? 3 : 2;
  // fp32 rows of 16384 leave no room for them: read from L2 with each row
  static constexpr bool WB_MEM = SLOT > 48 * 1024, WB_SMEM = CPT > 16 && !WB_MEM;
  static constexpr int WB = WB_SMEM ? 8 * KP : 0;
  // groups per CTA: up to 16 warps, two CTAs per SM where that takes no more than half of them away
  static constexpr int fit(int kb) { return (kb * 1024 - WB) / (S * SLOT); }
  static constexpr int least(int a, int b) { return a < b ? a : b; }
  static constexpr int MOST = W == 1 ? 8 : 16 / W;
  static constexpr int GROUPS = least(MOST, fit(112) >= (MOST + 1) / 2 ? fit(112) : fit(226));
  static constexpr int smem(int groups) { return WB + groups * S * SLOT; }
};

// The mean to keep. Values of few bits (bf16) differ from c by numbers that all
// round the same way within a binade, so md has a bias of up to half a step of
// the deviations: the correction is better than the sum's rounding only where the
// mean is larger than they are (4 x 13056 bf16, means of 0.02 deviations: relative
// errors of 1e-7, with the correction 2e-6). What is left of the mean is taken out
// of z and, from the kept mean, in the gradient all the same.
__device__ __forceinline__ float kept_mean(float c, float md, float var) { return c * c > var ? c + md : c; }

// place of column k among the planes
template <int E>
__device__ __forceinline__ int wb_at(int k, int kp) {
  return E == 8 ? ((k >> 2) & 1) * (kp / 2) + (k >> 3) * 4 + (k & 3) : k;
}

template <typename TX, typename TY, int E, int CPT, int W>
__global__ void __launch_bounds__((NormCfg<TX, E, CPT, W>::GROUPS * W * 32))
    layer_norm_rows_kernel(const TX* __restrict__ x, int64_t ldx, const float* __restrict__ w,
                           const float* __restrict__ b, TY* __restrict__ y, int64_t ldy, float* __restrict__ mean,
                           float* __restrict__ rstd, int64_t M, int K, float eps) {
  using C = NormCfg<TX, E, CPT, W>;
  using Row = StagedRow<TX, E>;
  constexpr int PAIRS = Row::PAIRS, UNIT = E == 1 ? 2 : E, NU = CPT / UNIT, T = W * 32, S = C::S;
  constexpr bool WB_REGS = !C::WB_SMEM && !C::WB_MEM;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ float sh[16][3 * W];
  const int groups = blockDim.x / T, group = threadIdx.x / T, tid = threadIdx.x % T, warp = tid >> 5;
  const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
  int64_t m = static_cast<int64_t>(blockIdx.x) * groups + group;
  uint8_t* ring = smem + C::WB + group * (S * C::SLOT);
#pragma unroll
  for (int i = 0; i < S; ++i) Row::template clear_pad<C::KP, T>(ring + i * C::SLOT, K, tid);
  grid_begin();
  const TX* ahead = x + m * ldx;  // the row fetched next
  int64_t m_ahead = m;
  auto fetch = [&](int slot) {
    if (m_ahead < M)
      Row::template copy<C::KP, T>(ring + slot * C::SLOT, ahead, K, m_ahead == 0, m_ahead == M - 1, tid);
    cp_async_commit();
    m_ahead += step;
    ahead += step * ldx;
  };
#pragma unroll
  for (int i = 0; i < S - 1; ++i) fetch(i);

  // first column of unit u; E = 1: a unit is columns k and k + T
  auto column = [&](int u) { return E == 1 ? tid + 2 * u * T : (tid + u * T) * E; };
  constexpr int NR = WB_REGS ? NU : 1;
  float2 wr[NR][PAIRS], br[NR][PAIRS];
  float* wb = reinterpret_cast<float*>(smem);
  auto wb_load = [&](int k) { return make_float2(w && k < K ? w[k] : 1.f, b && k < K ? b[k] : 0.f); };
  if constexpr (C::WB_SMEM) {
    for (int k = threadIdx.x; k < C::KP; k += blockDim.x) {
      const float2 v = wb_load(k);
      wb[wb_at<E>(k, C::KP)] = v.x;
      wb[C::KP + wb_at<E>(k, C::KP)] = v.y;
    }
    __syncthreads();
  } else if constexpr (WB_REGS) {
#pragma unroll
    for (int u = 0; u < NU; ++u)
#pragma unroll
      for (int j = 0; j < PAIRS; ++j) {
        const int k = column(u) + (E == 1 ? 0 : 2 * j);
        const float2 v0 = wb_load(k), v1 = wb_load(k + (E == 1 ? T : 1));
        wr[u][j] = make_float2(v0.x, v1.x);
        br[u][j] = make_float2(v0.y, v1.y);
      }
  }
  auto wb_get = [&](const float* plane, int k, float2(&f)[PAIRS]) {
    if constexpr (E <= 2) {
      f[0] = make_float2(plane[k], plane[k + (E == 1 ? T : 1)]);
    } else {
#pragma unroll
      for (int j = 0; j < PAIRS / 2; ++j) {
        const float4 v = *reinterpret_cast<const float4*>(plane + wb_at<E>(k + 4 * j, C::KP));
        f[2 * j] = make_float2(v.x, v.y);
        f[2 * j + 1] = make_float2(v.z, v.w);
      }
    }
  };

  const float inv_k = 1.0f / static_cast<float>(K);
  constexpr int ALL = NU > 8 ? NU : 8;  // every unit: `held` is in registers only where no index is left
  int slot = 0;
  const TX* xr = x + m * ldx;
  TY* yr = y + m * ldy;
  for (; m < M; m += step, xr += step * ldx, yr += step * ldy) {
    cp_async_wait<S - 2>();
    group_sync<W>(1 + group);  // the whole row has arrived; the slot of the row before is free
    fetch(slot == 0 ? S - 1 : slot - 1);
    const uint8_t* row = Row::first(ring + slot * C::SLOT, xr);
    float2 held[NU][PAIRS];
    float2 acc = both(0.f);
#pragma unroll ALL
    for (int u = 0; u < NU; ++u) {
      float2 f[PAIRS];
      Row::get_or_zero(row, column(u), T, K, f);
      acc = add2(acc, tree_sum2<PAIRS>(f));
#pragma unroll
      for (int j = 0; j < PAIRS; ++j) held[u][j] = f[j];
    }
    float s[1] = {acc.x + acc.y};
    group_sums<W>(s, sh[group], warp, 1 + group);
    const float c = s[0] * inv_k;
    float2 a1 = both(0.f), a2[2] = {both(0.f), both(0.f)};
#pragma unroll ALL
    for (int u = 0; u < NU; ++u) {
      float2 f[PAIRS];
#pragma unroll
      for (int j = 0; j < PAIRS; ++j) f[j] = held[u][j];
      const int k = column(u);
      // behind the columns 0 - 0
      const float2 cu = make_float2(k < K ? -c : 0.f, (E == 1 ? k + T : k) < K ? -c : 0.f);
#pragma unroll
      for (int j = 0; j < PAIRS; ++j) {
        f[j] = add2(f[j], cu);
        held[u][j] = f[j];
        a2[j & 1] = fma2(f[j], f[j], a2[j & 1]);
      }
      a1 = add2(a1, tree_sum2<PAIRS>(f));
    }
    a2[0] = add2(a2[0], a2[1]);
    float q[2] = {a1.x + a1.y, a2[0].x + a2[0].y};
    group_sums<W>(q, sh[group] + W, warp, 1 + group);
    const float md = q[0] * inv_k;
    float var = q[1] * inv_k - md * md;
    var = var < 0.f ? 0.f : var;  // a rounding below zero; NaN stays NaN
    const float r = inv_sqrt(var + eps);
    if (tid == 0) {
      if (mean) mean[m] = kept_mean(c, md, var);
      if (rstd) rstd[m] = r;
    }
    const float2 shift = both(-md * r);
#pragma unroll ALL
    for (int u = 0; u < NU; ++u) {
      const int k = column(u);
      float2 f[PAIRS], wv[PAIRS], bv[PAIRS];
#pragma unroll
      for (int j = 0; j < PAIRS; ++j) f[j] = held[u][j];
      if constexpr (C::WB_SMEM) {
        wb_get(wb, k, wv);
        wb_get(wb + C::KP, k, bv);
      }
#pragma unroll
      for (int j = 0; j < PAIRS; ++j) {
        if constexpr (C::WB_MEM) {
          const int k0 = k + (E == 1 ? 0 : 2 * j);
          const float2 v0 = wb_load(k0), v1 = wb_load(k0 + (E == 1 ? T : 1));
          wv[j] = make_float2(v0.x, v1.x);
          bv[j] = make_float2(v0.y, v1.y);
        }
        const float2 z = fma2(f[j], both(r), shift);
        f[j] = WB_REGS ? fma2(z, wr[WB_REGS ? u : 0][j], br[WB_REGS ? u : 0][j]) : fma2(z, wv[j], bv[j]);
      }
      if (k < K) put_unit<TY, E>(yr, k, T, K, f);
    }
    slot = slot + 1 == S ? 0 : slot + 1;
  }
}

// Rows too long for that: one CTA per row, three passes over the row (the
// later ones from L1/L2).
template <typename TX, typename TY>
__global__ void __launch_bounds__(kNormThreads)
    layer_norm_kernel(const TX* __restrict__ x, int64_t ldx, const float* __restrict__ w, const float* __restrict__ b,
                      TY* __restrict__ y, int64_t ldy, float* __restrict__ mean, float* __restrict__ rstd, int64_t K,
                      float eps) {
  __shared__ float sh[3 * kNormWarps];
  grid_begin();
  const int64_t m = blockIdx.x;
  const TX* xr = x + m * ldx;
  TY* yr = y + m * ldy;
  float f[1];
  float s[1] = {0.f};
  for (int64_t k = threadIdx.x; k < K; k += kNormThreads) {
    Elem<TX, 1>::load(xr + k, f);
    s[0] += f[0];
  }
  block_sums<kNormWarps>(s, sh);
  const float inv_k = 1.0f / static_cast<float>(K);
  const float c = s[0] * inv_k;
  float q[2] = {0.f, 0.f};
  for (int64_t k = threadIdx.x; k < K; k += kNormThreads) {
    Elem<TX, 1>::load(xr + k, f);
    const float d = f[0] - c;
    q[0] += d;
    q[1] = fmaf(d, d, q[1]);
  }
  block_sums<kNormWarps>(q, sh + kNormWarps);
  const float md = q[0] * inv_k;
  float var = q[1] * inv_k - md * md;
  var = var < 0.f ? 0.f : var;  // a rounding below zero; NaN stays NaN
  const float r = inv_sqrt(var + eps);
  if (threadIdx.x == 0) {
    if (mean) mean[m] = kept_mean(c, md, var);
    if (rstd) rstd[m] = r;
  }
  for (int64_t k = threadIdx.x; k < K; k += kNormThreads) {
    Elem<TX, 1>::load(xr + k, f);
    f[0] = ((f[0] - c) - md) * r;
    if (w) f[0] *= w[k];
    if (b) f[0] += b[k];
    Elem<TY, 1>::store(yr + k, f);
  }
}

}  // namespace bl
