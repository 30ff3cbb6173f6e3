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

// Rows in registers. W warps share a row; each of their threads holds NV
// accesses of E elements of it, and the weight and bias of its columns for all
// rows it meets (read again for each row they would cost more L2 traffic than
// the row itself). CTAs stay and take rows in turn, the next row's loads in
// flight while this one is reduced. W = 1: eight rows per CTA, no barriers.
constexpr int rows_per_cta(int W) { return W == 1 ? 8 : 1; }
constexpr int row_threads(int W) { return W == 1 ? 256 : W * 32; }

template <typename TX, typename TY, int E, int NV, int W>
__global__ void __launch_bounds__(row_threads(W))
    layer_norm_rows_kernel(const TX* __restrict__ x, int64_t ldx, const float* __restrict__ w,
                           const float* __restrict__ b, TY* __restrict__ y, int64_t ldy, float* __restrict__ mean,
                           float* __restrict__ rstd, int64_t M, int K, float eps) {
  __shared__ float sh[3 * W];
  constexpr int RPC = rows_per_cta(W);
  const int tid = W == 1 ? threadIdx.x & 31 : threadIdx.x;
  const int64_t step = static_cast<int64_t>(gridDim.x) * RPC;
  int64_t m = static_cast<int64_t>(blockIdx.x) * RPC + (W == 1 ? threadIdx.x >> 5 : 0);
  Raw<TX, E> cur[NV], nxt[NV];
  auto fetch = [&](Raw<TX, E>(&r)[NV], int64_t row) {
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      const int k = (tid + u * W * 32) * E;
      if (k < K)
        r[u].load(x + row * ldx + k);
      else
        r[u].zero();
    }
  };
  if (m < M) fetch(cur, m);
  float wr[NV][E], br[NV][E];
#pragma unroll
  for (int u = 0; u < NV; ++u)
#pragma unroll
    for (int j = 0; j < E; ++j) {
      const int k = (tid + u * W * 32) * E + j;
      wr[u][j] = w && k < K ? w[k] : 1.f;
      br[u][j] = b && k < K ? b[k] : 0.f;
    }
  const float inv_k = 1.0f / static_cast<float>(K);
  for (; m < M; m += step) {
    if (m + step < M) fetch(nxt, m + step);
    float f[E];
    float s[1] = {0.f};
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      cur[u].get(f);
      s[0] += tree_sum<E>(f);
    }
    block_sums<W>(s, sh);
    const float c = s[0] * inv_k;
    float q[2] = {0.f, 0.f};
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      if ((tid + u * W * 32) * E < K) {
        cur[u].get(f);
        float d2[E];
#pragma unroll
        for (int j = 0; j < E; ++j) {
          f[j] -= c;
          d2[j] = f[j] * f[j];
        }
        q[0] += tree_sum<E>(f);
        q[1] += tree_sum<E>(d2);
      }
    }
    block_sums<W>(q, sh + W);
    const float md = q[0] * inv_k;
    float var = q[1] * inv_k - md * md;
    var = var < 0.f ? 0.f : var;  // a rounding below zero; NaN stays NaN
    const float r = 1.0f / sqrtf(var + eps);
    if (tid == 0) {
      if (mean) mean[m] = c + md;
      if (rstd) rstd[m] = r;
    }
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      const int k = (tid + u * W * 32) * E;
      if (k < K) {
        cur[u].get(f);
#pragma unroll
        for (int j = 0; j < E; ++j) f[j] = fmaf(((f[j] - c) - md) * r, wr[u][j], br[u][j]);
        Elem<TY, E>::store(y + m * ldy + k, f);
      }
    }
#pragma unroll
    for (int u = 0; u < NV; ++u) cur[u] = nxt[u];
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

// The gradient, rows in registers as in the forward pass: one pass over x and
// dy gives dx, and each thread adds up dy z and dy of its columns over its rows;
// a CTA ends with one partial row of both, which the kernel below adds up in
// order. The mean is corrected as in the forward pass: md = mean (x - kept mean).
template <typename TX, typename TG, int E, int NV, int W>
__global__ void __launch_bounds__(row_threads(W))
    layer_norm_grad_rows_kernel(const TX* __restrict__ x, int64_t ldx, const float* __restrict__ w,
                                const float* __restrict__ mean, const float* __restrict__ rstd,
                                const TG* __restrict__ dy, int64_t lddy, TX* __restrict__ dx, int64_t lddx,
                                float* __restrict__ part, int64_t M, int K) {
  __shared__ float sh[2][3 * W];
  constexpr int RPC = rows_per_cta(W);
  const int tid = W == 1 ? threadIdx.x & 31 : threadIdx.x;
  const int64_t step = static_cast<int64_t>(gridDim.x) * RPC;
  int64_t m = static_cast<int64_t>(blockIdx.x) * RPC + (W == 1 ? threadIdx.x >> 5 : 0);
  Raw<TX, E> cx[NV], nx[NV];
  Raw<TG, E> cg[NV], ng[NV];
  auto fetch = [&](Raw<TX, E>(&rx)[NV], Raw<TG, E>(&rg)[NV], int64_t row) {
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      const int k = (tid + u * W * 32) * E;
      if (k < K) {
        rx[u].load(x + row * ldx + k);
        rg[u].load(dy + row * lddy + k);
      } else {
        rx[u].zero();
        rg[u].zero();
      }
    }
  };
  if (m < M) fetch(cx, cg, m);
  float wr[NV][E], aw[NV][E], ab[NV][E];
#pragma unroll
  for (int u = 0; u < NV; ++u)
#pragma unroll
    for (int j = 0; j < E; ++j) {
      const int k = (tid + u * W * 32) * E + j;
      wr[u][j] = w && k < K ? w[k] : 1.f;
      aw[u][j] = ab[u][j] = 0.f;
    }
  const float inv_k = 1.0f / static_cast<float>(K);
  int buf = 0;
  for (; m < M; m += step) {
    const float c = mean[m], r = rstd[m];
    if (m + step < M) fetch(nx, ng, m + step);
    float fx[E], fg[E];
    float s[3] = {0.f, 0.f, 0.f};  // sums of d, g and g d
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      if ((tid + u * W * 32) * E < K) {
        cx[u].get(fx);
        cg[u].get(fg);
        float gd[E];
#pragma unroll
        for (int j = 0; j < E; ++j) {
          fx[j] -= c;
          fg[j] *= wr[u][j];
          gd[j] = fx[j] * fg[j];
        }
        s[0] += tree_sum<E>(fx);
        s[1] += tree_sum<E>(fg);
        s[2] += tree_sum<E>(gd);
      }
    }
    block_sums<W>(s, sh[buf]);
    buf ^= 1;
    const float md = s[0] * inv_k, mg = s[1] * inv_k, mgz = r * (s[2] - md * s[1]) * inv_k;
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      const int k = (tid + u * W * 32) * E;
      if (k < K) {
        cx[u].get(fx);
        cg[u].get(fg);
#pragma unroll
        for (int j = 0; j < E; ++j) {
          const float z = ((fx[j] - c) - md) * r;
          aw[u][j] = fmaf(fg[j], z, aw[u][j]);
          ab[u][j] += fg[j];
          fx[j] = r * (fmaf(fg[j], wr[u][j], -mg) - z * mgz);
        }
        if (dx) Elem<TX, E>::store(dx + m * lddx + k, fx);
      }
    }
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      cx[u] = nx[u];
      cg[u] = ng[u];
    }
  }
  if (!part) return;
  // partial rows: [0, P) dweight, [P, 2P) dbias
  float* pw = part + static_cast<int64_t>(blockIdx.x) * K;
  float* pb = pw + static_cast<int64_t>(gridDim.x) * K;
  if constexpr (W == 1) {
    constexpr int COLS = 32 * E * NV;
    __shared__ float acc[8][2][COLS];
    const int warp = threadIdx.x >> 5;
#pragma unroll
    for (int u = 0; u < NV; ++u)
#pragma unroll
      for (int j = 0; j < E; ++j) {
        acc[warp][0][(tid + u * 32) * E + j] = aw[u][j];
        acc[warp][1][(tid + u * 32) * E + j] = ab[u][j];
      }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * COLS; i += 256) {
      const int k = i % COLS;
      if (k < K) {
        float t = acc[0][i / COLS][k];
#pragma unroll
        for (int v = 1; v < 8; ++v) t += acc[v][i / COLS][k];
        (i < COLS ? pw : pb)[k] = t;
      }
    }
  } else {
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      const int k = (tid + u * W * 32) * E;
      if (k < K) {
#pragma unroll
        for (int j = 0; j < E; ++j) {
          pw[k + j] = aw[u][j];
          pb[k + j] = ab[u][j];
        }
      }
    }
  }
}

// Rows too long for that: dx and the weight's gradient separately, from two
// readings of x and dy. One CTA per row: dx (where wanted) and the row's correction of the kept mean.
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
