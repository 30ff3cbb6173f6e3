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
// shared memory S - 1 rows ahead of its use and read from there by each of the
// three passes, CPT columns per thread in units of E. Few warps per row leave
// little beside the arithmetic itself (W = 1: no barrier, one set of shuffles per
// row; eight warps per row executed more instructions for the sums than for the
// rows), so W is 1 wherever there are rows enough. The weight and the bias stay
// in registers up to 16 columns per thread, else in shared memory (in planes of
// four columns, so that a warp's 16-byte reads meet no bank twice).
// The CTAs stay and their groups take rows in turn.
template <typename TX, int E, int CPT, int W>
struct NormCfg {
  static constexpr int KP = CPT * W * 32;  // columns a group covers
  static constexpr int SLOT = KP * int(sizeof(TX)) + StagedRow<TX, E>::PAD;
  static constexpr int S = SLOT <= 2080 ? 4 : SLOT <= 4128 ? 3 : 2;
  // fp32 rows of 16384 leave no room for them: read from L2 with each row
  static constexpr bool WB_MEM = SLOT > 48 * 1024, WB_SMEM = CPT > 16 && !WB_MEM;
  static constexpr int WB = WB_SMEM ? 8 * KP : 0;
  // groups per CTA: two CTAs per SM where each holds at least four rows
  static constexpr int fit(int kb) { return (kb * 1024 - WB) / (S * SLOT); }
  static constexpr int least(int a, int b) { return a < b ? a : b; }
  static constexpr int GROUPS = W > 1 ? least(fit(226), W >= 8 ? 1 : 4) : least(8, fit(112) >= 4 ? fit(112) : fit(226));
  static constexpr int smem(int groups) { return WB + groups * S * SLOT; }
};

// place of column k among the planes
template <int E>
__device__ __forceinline__ int wb_at(int k, int kp) {
  return E == 8 ? ((k >> 2) & 1) * (kp / 2) + (k >> 3) * 4 + (k & 3) : k;
}

template <typename TX, typename TY, int E, int CPT, int W>
__global__ void __launch_bounds__(512)
    layer_norm_rows_kernel(const TX* __restrict__ x, int64_t ldx, const float* __restrict__ w,
                           const float* __restrict__ b, TY* __restrict__ y, int64_t ldy, float* __restrict__ mean,
                           float* __restrict__ rstd, int64_t M, int K, float eps) {
  using C = NormCfg<TX, E, CPT, W>;
  using Row = StagedRow<TX, E>;
  constexpr int PAIRS = Row::PAIRS, UNIT = E == 1 ? 2 : E, NU = CPT / UNIT, T = W * 32, S = C::S;
  constexpr bool WB_REGS = !C::WB_SMEM && !C::WB_MEM;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float sh[16][3 * W];
  const int groups = blockDim.x / T, group = threadIdx.x / T, tid = threadIdx.x % T, warp = tid >> 5;
  const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
  int64_t m = static_cast<int64_t>(blockIdx.x) * groups + group;
  uint8_t* ring = smem + C::WB + group * (S * C::SLOT);
#pragma unroll
  for (int i = 0; i < S; ++i) Row::template clear_pad<C::KP, T>(ring + i * C::SLOT, K, tid);
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
    if constexpr (E == 1) {
      f[0] = make_float2(plane[k], plane[k + T]);
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
  int slot = 0;
  const TX* xr = x + m * ldx;
  TY* yr = y + m * ldy;
  // the unit of a row, `fill` behind its columns
  auto unit = [&](const uint8_t* row, int u, float fill, float2(&f)[PAIRS]) {
    const int k = column(u);
    Row::get(row, k, T, f);
    if constexpr (E == 1) f[0] = make_float2(k < K ? f[0].x : fill, k + T < K ? f[0].y : fill);
  };
  constexpr bool HOLD = NU * UNIT <= 16;  // few columns: read once, held
  for (; m < M; m += step, xr += step * ldx, yr += step * ldy) {
    cp_async_wait<S - 2>();
    group_sync<W>(1 + group);  // the whole row has arrived; the slot of the row before is free
    fetch(slot == 0 ? S - 1 : slot - 1);
    const uint8_t* row = Row::first(ring + slot * C::SLOT, xr);
    float2 held[HOLD ? NU : 1][PAIRS];
    float2 acc = both(0.f);
#pragma unroll 8
    for (int u = 0; u < NU; ++u) {
      float2 f[PAIRS];
      unit(row, u, 0.f, f);
      acc = add2(acc, tree_sum2<PAIRS>(f));
      if constexpr (HOLD) {
#pragma unroll
        for (int j = 0; j < PAIRS; ++j) held[u][j] = f[j];
      }
    }
    float s[1] = {acc.x + acc.y};
    group_sums<W>(s, sh[group], warp, 1 + group);
    const float c = s[0] * inv_k;
    float2 a1 = both(0.f), a2 = both(0.f);
#pragma unroll 8
    for (int u = 0; u < NU; ++u) {
      float2 f[PAIRS], d2[PAIRS];
      if constexpr (HOLD) {
#pragma unroll
        for (int j = 0; j < PAIRS; ++j) f[j] = held[u][j];
      } else {
        unit(row, u, 0.f, f);
      }
      const int k = column(u);
      // behind the columns 0 - 0
      const float2 cu = make_float2(k < K ? -c : 0.f, (E == 1 ? k + T : k) < K ? -c : 0.f);
#pragma unroll
      for (int j = 0; j < PAIRS; ++j) {
        f[j] = add2(f[j], cu);
        if constexpr (HOLD) held[u][j] = f[j];
        d2[j] = mul2(f[j], f[j]);
      }
      a1 = add2(a1, tree_sum2<PAIRS>(f));
      a2 = add2(a2, tree_sum2<PAIRS>(d2));
    }
    float q[2] = {a1.x + a1.y, a2.x + a2.y};
    group_sums<W>(q, sh[group] + W, warp, 1 + group);
    const float md = q[0] * inv_k;
    float var = q[1] * inv_k - md * md;
    var = var < 0.f ? 0.f : var;  // a rounding below zero; NaN stays NaN
    const float r = inv_sqrt(var + eps);
    if (tid == 0) {
      if (mean) mean[m] = c + md;
      if (rstd) rstd[m] = r;
    }
    const float2 shift = both(-md * r);
#pragma unroll 8
    for (int u = 0; u < NU; ++u) {
      const int k = column(u);
      float2 f[PAIRS], wv[PAIRS], bv[PAIRS];
      if constexpr (HOLD) {
#pragma unroll
        for (int j = 0; j < PAIRS; ++j) f[j] = held[u][j];
      } else {
        Row::get(row, k, T, f);
      }
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
        const float2 z = fma2(HOLD ? f[j] : add2(f[j], both(-c)), both(r), shift);
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

// The gradient in one pass over x and dy, which are staged on chip as in the
// forward pass. Two kinds of work meet: a row's sums run along the row, the
// weight's gradient runs across rows, each thread adding up dy z and dy of its
// own columns. The mean is corrected as in the forward pass: md = mean (x - kept
// mean). A CTA ends with one partial row of dweight and of dbias, which
// layer_norm_dw_sum_kernel adds up in order.

// Up to 512 columns: a warp per row does both, its lanes' columns in registers.
template <typename TX, typename TG, int E, int CPT>
struct NormGradRowCfg {
  static constexpr int KP = CPT * 32, WARPS = 8;
  static constexpr int SLOT_X = KP * int(sizeof(TX)) + StagedRow<TX, E>::PAD;
  static constexpr int SLOT = SLOT_X + KP * int(sizeof(TG)) + StagedRow<TG, E>::PAD;
  static constexpr int S = SLOT <= 2112 ? 4 : 3;
  static constexpr int ACC = WARPS * 2 * KP * 4;
  static constexpr int SMEM = S * WARPS * SLOT > ACC ? S * WARPS * SLOT : ACC;
};

template <typename TX, typename TG, int E, int CPT>
__global__ void __launch_bounds__(256)
    layer_norm_grad_rows_kernel(const TX* __restrict__ x, int64_t ldx, const float* __restrict__ w,
                                const float* __restrict__ mean, const float* __restrict__ rstd,
                                const TG* __restrict__ dy, int64_t lddy, TX* __restrict__ dx, int64_t lddx,
                                float* __restrict__ part, int64_t M, int K) {
  using C = NormGradRowCfg<TX, TG, E, CPT>;
  using RowX = StagedRow<TX, E>;
  using RowG = StagedRow<TG, E>;
  constexpr int PAIRS = RowX::PAIRS, UNIT = E == 1 ? 2 : E, NU = CPT / UNIT, S = C::S;
  extern __shared__ __align__(16) uint8_t smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t step = static_cast<int64_t>(gridDim.x) * C::WARPS;
  int64_t m = static_cast<int64_t>(blockIdx.x) * C::WARPS + warp;
  uint8_t* ring = smem + warp * (S * C::SLOT);
#pragma unroll
  for (int i = 0; i < S; ++i) {
    RowX::template clear_pad<C::KP, 32>(ring + i * C::SLOT, K, lane);
    RowG::template clear_pad<C::KP, 32>(ring + i * C::SLOT + C::SLOT_X, K, lane);
  }
  auto fetch = [&](int slot, int64_t row) {
    if (row < M) {
      uint8_t* at = ring + slot * C::SLOT;
      RowX::template copy<C::KP, 32>(at, x + row * ldx, K, row == 0, row == M - 1, lane);
      RowG::template copy<C::KP, 32>(at + C::SLOT_X, dy + row * lddy, K, row == 0, row == M - 1, lane);
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < S - 1; ++i) fetch(i, m + i * step);
  float c = 0.f, r = 0.f;
  if (m < M) c = mean[m], r = rstd[m];
  auto column = [&](int u) { return E == 1 ? lane + 64 * u : (lane + u * 32) * E; };
  float2 wr[NU][PAIRS], aw[NU][PAIRS], ab[NU][PAIRS];
#pragma unroll
  for (int u = 0; u < NU; ++u)
#pragma unroll
    for (int j = 0; j < PAIRS; ++j) {
      const int k0 = column(u) + (E == 1 ? 0 : 2 * j), k1 = k0 + (E == 1 ? 32 : 1);
      wr[u][j] = make_float2(w && k0 < K ? w[k0] : 1.f, w && k1 < K ? w[k1] : 1.f);
      aw[u][j] = ab[u][j] = both(0.f);
    }
  const float inv_k = 1.0f / static_cast<float>(K);
  int slot = 0;
  for (; m < M; m += step) {
    cp_async_wait<S - 2>();
    __syncwarp();
    fetch(slot == 0 ? S - 1 : slot - 1, m + (S - 1) * step);
    float c_next = 0.f, r_next = 0.f;
    if (m + step < M) c_next = mean[m + step], r_next = rstd[m + step];
    const uint8_t* at = ring + slot * C::SLOT;
    const uint8_t *xs = RowX::first(at, x + m * ldx), *gs = RowG::first(at + C::SLOT_X, dy + m * lddy);
    float2 fx[NU][PAIRS], fg[NU][PAIRS];
    float2 s0 = both(0.f), s1 = both(0.f), s2 = both(0.f);  // sums of d, g and g d
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      const int k = column(u);
      RowX::get(xs, k, 32, fx[u]);
      RowG::get(gs, k, 32, fg[u]);
      if constexpr (E == 1) {
        fx[u][0] = make_float2(k < K ? fx[u][0].x : 0.f, k + 32 < K ? fx[u][0].y : 0.f);
        fg[u][0] = make_float2(k < K ? fg[u][0].x : 0.f, k + 32 < K ? fg[u][0].y : 0.f);
      }
      // behind the columns 0 - 0
      const float2 cu = make_float2(k < K ? -c : 0.f, (E == 1 ? k + 32 : k) < K ? -c : 0.f);
      float2 g[PAIRS], gd[PAIRS];
#pragma unroll
      for (int j = 0; j < PAIRS; ++j) {
        fx[u][j] = add2(fx[u][j], cu);
        g[j] = mul2(fg[u][j], wr[u][j]);
        gd[j] = mul2(g[j], fx[u][j]);
      }
      s0 = add2(s0, tree_sum2<PAIRS>(fx[u]));
      s1 = add2(s1, tree_sum2<PAIRS>(g));
      s2 = add2(s2, tree_sum2<PAIRS>(gd));
    }
    const float t0 = warp_sum(s0.x + s0.y), t1 = warp_sum(s1.x + s1.y), t2 = warp_sum(s2.x + s2.y);
    const float md = t0 * inv_k, mg = t1 * inv_k, mgz = r * (t2 - md * t1) * inv_k;
    const float2 zs = both(-md * r), o0 = both(-r * mg), o1 = both(-r * mgz);
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      const int k = column(u);
#pragma unroll
      for (int j = 0; j < PAIRS; ++j) {
        const float2 z = fma2(fx[u][j], both(r), zs);
        aw[u][j] = fma2(fg[u][j], z, aw[u][j]);
        ab[u][j] = add2(ab[u][j], fg[u][j]);
        fx[u][j] = fma2(mul2(fg[u][j], wr[u][j]), both(r), fma2(z, o1, o0));
      }
      if (dx && k < K) put_unit<TX, E>(dx + m * lddx, k, 32, K, fx[u]);
    }
    c = c_next;
    r = r_next;
    slot = slot + 1 == S ? 0 : slot + 1;
  }
  if (!part) return;
  grid_dependents_launch();  // the kernel that adds the partial rows up may be scheduled; it waits for them
  cp_async_wait<0>();
  __syncthreads();  // the ring is free: the warps' sums meet there
  float* acc = reinterpret_cast<float*>(smem);  // [warp][dweight | dbias][KP]
#pragma unroll
  for (int u = 0; u < NU; ++u)
#pragma unroll
    for (int j = 0; j < PAIRS; ++j) {
      const int k0 = column(u) + (E == 1 ? 0 : 2 * j), k1 = k0 + (E == 1 ? 32 : 1);
      acc[(2 * warp) * C::KP + k0] = aw[u][j].x;
      acc[(2 * warp) * C::KP + k1] = aw[u][j].y;
      acc[(2 * warp + 1) * C::KP + k0] = ab[u][j].x;
      acc[(2 * warp + 1) * C::KP + k1] = ab[u][j].y;
    }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * C::KP; i += 256) {
    const int k = i % C::KP, which = i / C::KP;
    if (k < K) {
      float t = 0.f;
#pragma unroll
      for (int v = 0; v < C::WARPS; ++v) t += acc[(2 * v + which) * C::KP + k];
      part[(static_cast<int64_t>(which) * gridDim.x + blockIdx.x) * K + k] = t;
    }
  }
}

// More columns: a CTA of W warps takes R rows at a time. First the rows' sums, W / R
// warps to a row; then, each thread holding CPT columns, dx and the columns'
// sums for all R rows. The sums of the next tile are formed before the
// columns of this one, so that one barrier per tile serves both, and the tile
// after that is on its way. (With the columns' threads also forming the row's
// sums, every warp spent 15 shuffles and a barrier on each row, as much as on its
// 8 columns.)
template <typename TX, typename TG, int E, int CPT, int W>
struct NormGradTileCfg {
  static constexpr int KP = CPT * W * 32, THREADS = W * 32;
  static constexpr int SLOT_X = KP * int(sizeof(TX)) + StagedRow<TX, E>::PAD;
  static constexpr int SLOT = SLOT_X + KP * int(sizeof(TG)) + StagedRow<TG, E>::PAD;
  // three tiles on chip, of as many rows as leave room for 4, 2 or 1 CTAs per SM
  static constexpr int S = 3, LIMIT = (W <= 4 ? 50 : W <= 8 ? 100 : 200) * 1024;
  static constexpr int R = S * 4 * SLOT <= LIMIT ? 4 : S * 2 * SLOT <= LIMIT ? 2 : 1;
  static constexpr int TILE = R * SLOT;
  static constexpr int SMEM = S * TILE;
};

template <typename TX, typename TG, int E, int CPT, int W>
__global__ void __launch_bounds__(W * 32)
    layer_norm_grad_tile_kernel(const TX* __restrict__ x, int64_t ldx, const float* __restrict__ w,
                                const float* __restrict__ mean, const float* __restrict__ rstd,
                                const TG* __restrict__ dy, int64_t lddy, TX* __restrict__ dx, int64_t lddx,
                                float* __restrict__ part, int64_t M, int K) {
  using C = NormGradTileCfg<TX, TG, E, CPT, W>;
  using RowX = StagedRow<TX, E>;
  using RowG = StagedRow<TG, E>;
  constexpr int R = C::R, S = C::S;
  static_assert(W % R == 0 && W <= 32 && S >= 3, "");
  constexpr int P = W / R;  // warps to a row's sums
  constexpr int PAIRS = RowX::PAIRS, UNIT = E == 1 ? 2 : E, NU = CPT / UNIT, T = W * 32;
  constexpr int NS = R * CPT / UNIT, TS = 32;  // the sums' units per lane
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float4 sums[2][W];     // of d, g and g d, by warp
  __shared__ float2 kept[2][R];     // mean and rstd
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int my_row = warp / P, my_part = warp % P;
  const int64_t tiles = (M + R - 1) / R;
  uint8_t* ring = smem;

  auto fetch = [&](int slot, int64_t tile) {
    if (tile < tiles) {
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const int64_t m = tile * R + i;
        if (m < M) {
          uint8_t* at = ring + slot * C::TILE + i * C::SLOT;
          RowX::template copy<C::KP, T>(at, x + m * ldx, K, m == 0, m == M - 1, tid);
          RowG::template copy<C::KP, T>(at + C::SLOT_X, dy + m * lddy, K, m == 0, m == M - 1, tid);
        }
      }
    }
    cp_async_commit();
  };
  // what the forward pass kept of this warp's row of a tile
  auto kept_of = [&](int64_t tile) {
    const int64_t m = tile * R + my_row;
    return tile < tiles && m < M ? make_float2(mean[m], rstd[m]) : make_float2(0.f, 0.f);
  };
  const int64_t step = gridDim.x;
  int64_t tile = blockIdx.x;
#pragma unroll
  for (int i = 0; i < S * R; ++i) {
    RowX::template clear_pad<C::KP, T>(ring + i * C::SLOT, K, tid);
    RowG::template clear_pad<C::KP, T>(ring + i * C::SLOT + C::SLOT_X, K, tid);
  }
#pragma unroll
  for (int i = 0; i < S - 1; ++i) fetch(i, tile + i * step);

  // columns of the sums: a contiguous share of the row per warp
  auto sum_column = [&](int u) {
    return my_part * (C::KP / P) + (E == 1 ? lane + 64 * u : (lane + 32 * u) * E);
  };
  auto column = [&](int u) { return E == 1 ? tid + 2 * u * T : (tid + u * T) * E; };
  auto weight_pair = [&](int k, int j, int stride) {
    const int k0 = k + (E == 1 ? 0 : 2 * j), k1 = k0 + (E == 1 ? stride : 1);
    return make_float2(w && k0 < K ? w[k0] : 1.f, w && k1 < K ? w[k1] : 1.f);
  };
  float2 ws[NS][PAIRS], wr[NU][PAIRS], aw[NU][PAIRS], ab[NU][PAIRS];
#pragma unroll
  for (int u = 0; u < NS; ++u)
#pragma unroll
    for (int j = 0; j < PAIRS; ++j) ws[u][j] = weight_pair(sum_column(u), j, TS);
#pragma unroll
  for (int u = 0; u < NU; ++u)
#pragma unroll
    for (int j = 0; j < PAIRS; ++j) {
      wr[u][j] = weight_pair(column(u), j, T);
      aw[u][j] = ab[u][j] = both(0.f);
    }
  const float inv_k = 1.0f / static_cast<float>(K);

  // sums of this warp's share of its row of the tile in `slot`
  auto row_sums = [&](int64_t t, int slot, int buf, float2 k) {
    const int64_t m = t * R + my_row;
    if (t >= tiles || m >= M) return;
    const uint8_t* at = ring + slot * C::TILE + my_row * C::SLOT;
    const uint8_t *xs = RowX::first(at, x + m * ldx), *gs = RowG::first(at + C::SLOT_X, dy + m * lddy);
    float2 s0 = both(0.f), s1 = both(0.f), s2 = both(0.f);
#pragma unroll
    for (int u = 0; u < NS; ++u) {
      const int col = sum_column(u);
      float2 fx[PAIRS], fg[PAIRS];
      RowX::get(xs, col, TS, fx);
      RowG::get(gs, col, TS, fg);
      if constexpr (E == 1) {
        fx[0] = make_float2(col < K ? fx[0].x : 0.f, col + TS < K ? fx[0].y : 0.f);
        fg[0] = make_float2(col < K ? fg[0].x : 0.f, col + TS < K ? fg[0].y : 0.f);
      }
      // behind the columns 0 - 0
      const float2 cu = make_float2(col < K ? -k.x : 0.f, (E == 1 ? col + TS : col) < K ? -k.x : 0.f);
      float2 gd[PAIRS];
#pragma unroll
      for (int j = 0; j < PAIRS; ++j) {
        fx[j] = add2(fx[j], cu);
        fg[j] = mul2(fg[j], ws[u][j]);
        gd[j] = mul2(fg[j], fx[j]);
      }
      s0 = add2(s0, tree_sum2<PAIRS>(fx));
      s1 = add2(s1, tree_sum2<PAIRS>(fg));
      s2 = add2(s2, tree_sum2<PAIRS>(gd));
    }
    const float t0 = warp_sum(s0.x + s0.y), t1 = warp_sum(s1.x + s1.y), t2 = warp_sum(s2.x + s2.y);
    if (lane == 0) {
      sums[buf][warp] = make_float4(t0, t1, t2, 0.f);
      if (my_part == 0) kept[buf][my_row] = k;
    }
  };

  float2 k_next = kept_of(tile);
  cp_async_wait<S - 2>();
  __syncthreads();
  row_sums(tile, 0, 0, k_next);
  k_next = kept_of(tile + step);
  int slot = 0, buf = 0;
  for (; tile < tiles; tile += step) {
    cp_async_wait<S - 3>();
    __syncthreads();  // the next tile has arrived, this one's sums are there, the last one's slot is free
    const int next = slot + 1 == S ? 0 : slot + 1;
    fetch(slot == 0 ? S - 1 : slot - 1, tile + (S - 1) * step);
    const float2 k_cur = k_next;
    k_next = kept_of(tile + 2 * step);
    row_sums(tile + step, next, buf ^ 1, k_cur);

    // lane l: the sums of warp l; after the exchange, of row l / P
    float4 v = sums[buf][lane % W];
#pragma unroll
    for (int o = 1; o < P; o <<= 1) {
      v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
      v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
      v.z += __shfl_xor_sync(0xffffffffu, v.z, o);
    }
    const float2 kr = kept[buf][(lane % W) / P];
    const float md = v.x * inv_k, mg = v.y * inv_k, mgz = kr.y * (v.z - md * v.y) * inv_k;
    const float l_zs = -md * kr.y, l_o0 = -kr.y * mg, l_o1 = -kr.y * mgz;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int64_t m = tile * R + i;
      const float c = __shfl_sync(0xffffffffu, kr.x, i * P), r = __shfl_sync(0xffffffffu, kr.y, i * P);
      const float2 zs = both(__shfl_sync(0xffffffffu, l_zs, i * P));
      const float2 o0 = both(__shfl_sync(0xffffffffu, l_o0, i * P)), o1 = both(__shfl_sync(0xffffffffu, l_o1, i * P));
      if (m >= M) break;
      const uint8_t* at = ring + slot * C::TILE + i * C::SLOT;
      const uint8_t *xs = RowX::first(at, x + m * ldx), *gs = RowG::first(at + C::SLOT_X, dy + m * lddy);
#pragma unroll
      for (int u = 0; u < NU; ++u) {
        const int k = column(u);
        float2 fx[PAIRS], fg[PAIRS];
        RowX::get(xs, k, T, fx);
        RowG::get(gs, k, T, fg);
#pragma unroll
        for (int j = 0; j < PAIRS; ++j) {
          const float2 z = fma2(add2(fx[j], both(-c)), both(r), zs);
          aw[u][j] = fma2(fg[j], z, aw[u][j]);
          ab[u][j] = add2(ab[u][j], fg[j]);
          fx[j] = fma2(mul2(fg[j], wr[u][j]), both(r), fma2(z, o1, o0));
        }
        if (dx && k < K) put_unit<TX, E>(dx + m * lddx, k, T, K, fx);
      }
    }
    slot = next;
    buf ^= 1;
  }
  if (!part) return;
  grid_dependents_launch();
  float* pw = part + static_cast<int64_t>(blockIdx.x) * K;
  float* pb = pw + static_cast<int64_t>(gridDim.x) * K;
#pragma unroll
  for (int u = 0; u < NU; ++u)
#pragma unroll
    for (int j = 0; j < PAIRS; ++j) {
      const int k0 = column(u) + (E == 1 ? 0 : 2 * j), k1 = k0 + (E == 1 ? T : 1);
      if (k0 < K) pw[k0] = aw[u][j].x, pb[k0] = ab[u][j].x;
      if (k1 < K) pw[k1] = aw[u][j].y, pb[k1] = ab[u][j].y;
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

// dweight and dbias: the P partial rows added in order, 32 columns per CTA, a
// contiguous share of the rows per warp, eight of them in flight. (With one load
// at a time this took 17 us for 389 rows of 1001 columns, three times the pass
// over x and dy.)
constexpr int kNormSumThreads = 512;

__global__ void __launch_bounds__(kNormSumThreads)
    layer_norm_dw_sum_kernel(const float* __restrict__ part, int P, int64_t K, float* __restrict__ dw,
                             float* __restrict__ db) {
  constexpr int WARPS = kNormSumThreads / 32;
  __shared__ float sh[WARPS][32];
  grid_dependency_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t k = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  float* out = blockIdx.y == 0 ? dw : db;
  if (!out) return;  // uniform per CTA
  const float* src = part + static_cast<int64_t>(blockIdx.y) * P * K + k;
  const int per = (P + WARPS - 1) / WARPS, p1 = min(P, (warp + 1) * per);
  float t = 0.f;
  if (k < K)
    for (int p = warp * per; p < p1; p += 8) {
      float f[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = p + i < p1 ? src[(p + i) * K] : 0.f;
      t += tree_sum<8>(f);
    }
  sh[warp][lane] = t;
  __syncthreads();
  if (warp == 0 && k < K) {
    t = 0.f;
#pragma unroll
    for (int i = 0; i < WARPS; ++i) t += sh[i][lane];
    out[k] = t;
  }
}

}  // namespace bl
