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

// One CTA per row, three passes over the row (the later ones from L1/L2).
template <typename TX, typename TY>
__global__ void __launch_bounds__(kNormThreads)
    layer_norm_kernel(const TX* __restrict__ x, int64_t ldx, const float* __restrict__ w, const float* __restrict__ b,
                      TY* __restrict__ y, int64_t ldy, float* __restrict__ mean, float* __restrict__ rstd, int64_t K,
                      float eps) {
  __shared__ float sh[2 * kNormWarps];
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
  block_sums<kNormWarps>(q, sh);
  const float md = q[0] * inv_k;
  float var = q[1] * inv_k - md * md;
  var = var < 0.f ? 0.f : var;  // a rounding below zero; NaN stays NaN
  const float r = 1.0f / sqrtf(var + eps);
  if (threadIdx.x == 0) {
    if (mean) mean[m] = c + md;
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

// One CTA per row: dx (where wanted) and the row's correction of the kept mean.
template <typename TX, typename TY>
__global__ void __launch_bounds__(kNormThreads)
    layer_norm_dx_kernel(const TX* __restrict__ x, int64_t ldx, const float* __restrict__ w,
                         const float* __restrict__ mean, const float* __restrict__ rstd, const TY* __restrict__ dy,
                         int64_t lddy, TX* __restrict__ dx, int64_t lddx, float* __restrict__ shift, int64_t K) {
  __shared__ float sh[3 * kNormWarps];
  const int64_t m = blockIdx.x;
  const TX* xr = x + m * ldx;
  const TY* gr = dy + m * lddy;
  const float c = mean[m], r = rstd[m];
  float s[3] = {0.f, 0.f, 0.f};  // sums of d, g and g d
  float fx[1], fg[1];
  for (int64_t k = threadIdx.x; k < K; k += kNormThreads) {
    Elem<TX, 1>::load(xr + k, fx);
    Elem<TY, 1>::load(gr + k, fg);
    const float d = fx[0] - c, g = w ? fg[0] * w[k] : fg[0];
    s[0] += d;
    s[1] += g;
    s[2] = fmaf(g, d, s[2]);
  }
  block_sums<kNormWarps>(s, sh);
  const float inv_k = 1.0f / static_cast<float>(K);
  const float md = s[0] * inv_k;
  const float mg = s[1] * inv_k, mgz = r * (s[2] - md * s[1]) * inv_k;
  if (shift && threadIdx.x == 0) shift[m] = md;
  if (!dx) return;
  for (int64_t k = threadIdx.x; k < K; k += kNormThreads) {
    Elem<TX, 1>::load(xr + k, fx);
    Elem<TY, 1>::load(gr + k, fg);
    const float z = ((fx[0] - c) - md) * r, g = w ? fg[0] * w[k] : fg[0];
    fx[0] = r * (g - mg - z * mgz);
    Elem<TX, 1>::store(dx + m * lddx + k, fx);
  }
}

// Partial sums of dy z and dy over the rows m = p, p + P, ...: CTA (column
// block, p), one column per lane, the rows dealt to the warps.
template <typename TX, typename TY>
__global__ void __launch_bounds__(kNormThreads)
    layer_norm_dw_kernel(const TX* __restrict__ x, int64_t ldx, const float* __restrict__ mean,
                         const float* __restrict__ rstd, const float* __restrict__ shift, const TY* __restrict__ dy,
                         int64_t lddy, float* __restrict__ part, int64_t M, int64_t K) {
  __shared__ float sh[2][kNormWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t k = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  const int64_t p = blockIdx.y, P = gridDim.y;
  float sw = 0.f, sb = 0.f;
  if (k < K) {
    float fx[1], fg[1];
    for (int64_t m = p + warp * P; m < M; m += P * kNormWarps) {
      Elem<TX, 1>::load(x + m * ldx + k, fx);
      Elem<TY, 1>::load(dy + m * lddy + k, fg);
      sw = fmaf(fg[0], ((fx[0] - mean[m]) - shift[m]) * rstd[m], sw);
      sb += fg[0];
    }
  }
  sh[0][warp][lane] = sw;
  sh[1][warp][lane] = sb;
  __syncthreads();
  if (warp < 2 && k < K) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < kNormWarps; ++i) t += sh[warp][i][lane];
    part[(warp * P + p) * K + k] = t;
  }
}

// dweight and dbias: the P partial rows added in order
__global__ void __launch_bounds__(kNormThreads)
    layer_norm_dw_sum_kernel(const float* __restrict__ part, int64_t P, int64_t K, float* __restrict__ dw,
                             float* __restrict__ db) {
  __shared__ float sh[kNormWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t k = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  float* out = blockIdx.y == 0 ? dw : db;
  if (!out) return;  // uniform per CTA
  const float* src = part + static_cast<int64_t>(blockIdx.y) * P * K;
  float t = 0.f;
  if (k < K)
    for (int64_t p = warp; p < P; p += kNormWarps) t += src[p * K + k];
  sh[warp][lane] = t;
  __syncthreads();
  if (warp == 0 && k < K) {
    t = 0.f;
#pragma unroll
    for (int i = 0; i < kNormWarps; ++i) t += sh[i][lane];
    out[k] = t;
  }
}

}  // namespace bl
