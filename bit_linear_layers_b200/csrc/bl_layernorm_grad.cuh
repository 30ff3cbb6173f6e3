// The gradient of the layer norm: dx, and dweight and dbias summed over the rows
// (the formulas are with the forward pass).
#pragma once

#include "bl_layernorm.cuh"

namespace bl {

// The gradient in one pass over x and dy, which are staged on chip as in the
// forward pass. Two kinds of work meet: a row's sums run along the row, the
// weight's gradient runs across rows, each thread adding up dy z and dy of its
// own columns. The mean is corrected as in the forward pass: md = mean (x - kept
// mean). A CTA ends with one partial row of dweight and of dbias, which
// layer_norm_dw_sum_kernel adds up in order.

// Up to 512 columns: a warp per row does both, its lanes' columns in registers
// (32768 x 512 fp32: 34 us, 5.9 TB/s).
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
  extern __shared__ __align__(1024) uint8_t smem[];
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
  grid_dependency_wait();
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
      RowX::get_or_zero(xs, k, 32, K, fx[u]);
      RowG::get_or_zero(gs, k, 32, K, fg[u]);
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
  grid_dependents_launch();  // the kernel that adds the partial rows up may be scheduled; it waits for them
  if (!part) return;
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

// More columns: a CTA of W warps takes tiles of R rows, two on chip, one of them
// on its way. First the rows' sums, each warp whole rows (or a share of one);
// then, each thread holding CPT columns, dx and the columns' sums for all R rows.
// What a tile costs beside its elements (the sums' shuffles, the copies'
// addresses, the rows' constants) is paid per warp, so the tile is as large as
// fits and the warps are few: up to 64 elements per thread and tile. (With 16,
// and a third tile on chip to form the next sums ahead, 38 instructions went
// into an element, of which the arithmetic needs 13.)
// Measured: 16384 x 2048 from fp32 x and bf16 dy 60 us (5.6 TB/s), 4096 x 4096
// bf16 29 us: there 16 warps per SM wait for the sums between the tile's two
// halves. Rows that are read element by element (1001 columns, 8192 rows: 29 us)
// are bound by their instructions.
template <typename TX, typename TG, int E, int CPT, int W>
struct NormGradTileCfg {
  static constexpr int KP = CPT * W * 32, THREADS = W * 32;
  static constexpr int SLOT_X = KP * int(sizeof(TX)) + StagedRow<TX, E>::PAD;
  static constexpr int SLOT = SLOT_X + KP * int(sizeof(TG)) + StagedRow<TG, E>::PAD;
  // rows of any alignment take more instructions per element: more warps, smaller tiles
  static constexpr int CTAS = E <= 2 ? (W <= 4 ? 5 : W <= 10 && CPT == 8 ? 2 : 1) : W <= 4 ? 3 : 1;
  static constexpr int LIMIT = 222 * 1024 / CTAS - KP * 4;
  static constexpr int R = 2 * 8 * SLOT <= LIMIT ? 8 : 2 * 4 * SLOT <= LIMIT ? 4 : 2 * 2 * SLOT <= LIMIT ? 2 : 1;
  static constexpr int TILE = R * SLOT;
  static constexpr int SMEM = 2 * TILE + KP * 4;
};

template <typename TX, typename TG, int E, int CPT, int W>
__global__ void __launch_bounds__(W * 32, (NormGradTileCfg<TX, TG, E, CPT, W>::CTAS))
    layer_norm_grad_tile_kernel(const TX* __restrict__ x, int64_t ldx, const float* __restrict__ w,
                                const float* __restrict__ mean, const float* __restrict__ rstd,
                                const TG* __restrict__ dy, int64_t lddy, TX* __restrict__ dx, int64_t lddx,
                                float* __restrict__ part, int64_t M, int K, int height) {
  using C = NormGradTileCfg<TX, TG, E, CPT, W>;
  using RowX = StagedRow<TX, E>;
  using RowG = StagedRow<TG, E>;
  constexpr int R = C::R;
  constexpr int P = W > R ? W / R : 1, Q = R > W ? (R + W - 1) / W : 1;  // warps to a row's sums, rows to a warp
  constexpr int PAIRS = RowX::PAIRS, UNIT = E == 1 ? 2 : E, NU = CPT / UNIT, T = W * 32;
  static_assert(C::KP % (P * 32 * UNIT) == 0, "a whole number of units per lane");
  constexpr int NS = C::KP / P / 32 / UNIT, TS = 32;  // the sums' units per lane and row
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ float4 sums[R * P];       // of d, g and g d
  __shared__ float2 kept[R];           // mean and rstd
  __shared__ float4 consts[R];         // -c, r, -md r, -r mean g
  __shared__ float consts1[R];         // -r mean(g z)
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // this warp's rows of a tile: my_row + q * W
  const int my_row = P > 1 ? warp / P : warp, my_part = P > 1 ? warp % P : 0;
  const int64_t tiles = (M + height - 1) / height;  // of `height` <= R rows
  float* wplane = reinterpret_cast<float*>(smem);  // the weight, in planes of four columns
  uint8_t* ring = smem + C::KP * 4;

  const int64_t step = gridDim.x;
  int64_t tile = blockIdx.x;
#pragma unroll
  for (int i = 0; i < 2 * R; ++i) {
    RowX::template clear_pad<C::KP, T>(ring + i * C::SLOT, K, tid);
    RowG::template clear_pad<C::KP, T>(ring + i * C::SLOT + C::SLOT_X, K, tid);
  }
  auto fetch = [&](int slot, int64_t t) {
    const int rows = t >= tiles ? 0 : static_cast<int>(M - t * height < height ? M - t * height : height);
    const TX* xt = x + t * height * ldx;
    const TG* gt = dy + t * height * lddy;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (i < rows) {
        const bool first = t == 0 && i == 0, last = t == tiles - 1 && i == rows - 1;
        uint8_t* at = ring + slot * C::TILE + i * C::SLOT;
        RowX::template copy<C::KP, T>(at, xt, K, first, last, tid);
        RowG::template copy<C::KP, T>(at + C::SLOT_X, gt, K, first, last, tid);
      }
      xt += ldx;
      gt += lddy;
    }
    cp_async_commit();
  };
  // what the forward pass kept of this warp's rows of a tile
  float2 k_cur[Q], k_next[Q];
  auto kept_of = [&](int64_t t, float2(&k)[Q]) {
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int row = my_row + q * W;
      const int64_t m = t * height + row;
      k[q] = row < height && m < M ? make_float2(mean[m], rstd[m]) : make_float2(0.f, 0.f);
    }
  };
  grid_dependency_wait();
  fetch(0, tile);
  kept_of(tile, k_next);

  // columns of the sums: a contiguous share of the row per warp
  auto sum_column = [&](int u) {
    return my_part * (C::KP / P) + (E == 1 ? lane + 64 * u : (lane + 32 * u) * E);
  };
  auto column = [&](int u) { return E == 1 ? tid + 2 * u * T : (tid + u * T) * E; };
  auto weights = [&](int k, int stride, float2(&f)[PAIRS]) {
    if constexpr (E <= 2) {
      f[0] = make_float2(wplane[k], wplane[k + (E == 1 ? stride : 1)]);
    } else {
#pragma unroll
      for (int j = 0; j < PAIRS / 2; ++j) {
        const float4 v = *reinterpret_cast<const float4*>(wplane + wb_at<E>(k + 4 * j, C::KP));
        f[2 * j] = make_float2(v.x, v.y);
        f[2 * j + 1] = make_float2(v.z, v.w);
      }
    }
  };
  for (int k = tid; k < C::KP; k += T) wplane[wb_at<E>(k, C::KP)] = w && k < K ? w[k] : 1.f;
  __syncthreads();
  float2 wr[NU][PAIRS], aw[NU][PAIRS], ab[NU][PAIRS];
#pragma unroll
  for (int u = 0; u < NU; ++u) {
    weights(column(u), T, wr[u]);
#pragma unroll
    for (int j = 0; j < PAIRS; ++j) aw[u][j] = ab[u][j] = both(0.f);
  }
  const float inv_k = 1.0f / static_cast<float>(K);
  // a row's constants from its sums
  auto finish = [&](int row, float4 v, float2 k) {
    const float md = v.x * inv_k, mg = v.y * inv_k, mgz = k.y * (v.z - md * v.y) * inv_k;
    consts[row] = make_float4(-k.x, k.y, -md * k.y, -k.y * mg);
    consts1[row] = -k.y * mgz;
  };

  int slot = 0;
  for (; tile < tiles; tile += step) {
    const int rows = static_cast<int>(M - tile * height < height ? M - tile * height : height);
    const TX* xt = x + tile * height * ldx;
    const TG* gt = dy + tile * height * lddy;
    cp_async_wait<0>();
    __syncthreads();  // the tile has arrived; the other slot and the constants are free
    fetch(slot ^ 1, tile + step);
#pragma unroll
    for (int q = 0; q < Q; ++q) k_cur[q] = k_next[q];
    kept_of(tile + step, k_next);

#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int row = my_row + q * W;
      if (row < rows) {
        const uint8_t* at = ring + slot * C::TILE + row * C::SLOT;
        const uint8_t *xs = RowX::first(at, xt + row * ldx), *gs = RowG::first(at + C::SLOT_X, gt + row * lddy);
        float2 s0[2], s1[2], s2[2];
        s0[0] = s0[1] = s1[0] = s1[1] = s2[0] = s2[1] = both(0.f);
        const float c = k_cur[q].x;
#pragma unroll 8
        for (int u = 0; u < NS; ++u) {
          const int col = sum_column(u);
          float2 fx[PAIRS], fg[PAIRS], ws[PAIRS];
          RowX::get_or_zero(xs, col, TS, K, fx);
          RowG::get_or_zero(gs, col, TS, K, fg);
          weights(col, TS, ws);
          // behind the columns 0 - 0
          const float2 cu = make_float2(col < K ? -c : 0.f, (E == 1 ? col + TS : col) < K ? -c : 0.f);
#pragma unroll
          for (int j = 0; j < PAIRS; ++j) {
            const int h = PAIRS > 1 ? j & 1 : u & 1;
            fx[j] = add2(fx[j], cu);
            fg[j] = mul2(fg[j], ws[j]);
            s0[h] = add2(s0[h], fx[j]);
            s1[h] = add2(s1[h], fg[j]);
            s2[h] = fma2(fg[j], fx[j], s2[h]);
          }
        }
        s0[0] = add2(s0[0], s0[1]);
        s1[0] = add2(s1[0], s1[1]);
        s2[0] = add2(s2[0], s2[1]);
        float4 v = make_float4(warp_sum(s0[0].x + s0[0].y), warp_sum(s1[0].x + s1[0].y), warp_sum(s2[0].x + s2[0].y), 0.f);
        if (lane == 0) {
          if constexpr (P == 1) {
            finish(row, v, k_cur[q]);
          } else {
            sums[warp] = v;
            if (my_part == 0) kept[row] = k_cur[q];
          }
        }
      }
    }
    __syncthreads();  // the sums
    if constexpr (P > 1) {
      if (tid < R) {
        float4 v = sums[tid * P];
#pragma unroll
        for (int i = 1; i < P; ++i) {
          const float4 a = sums[tid * P + i];
          v.x += a.x;
          v.y += a.y;
          v.z += a.z;
        }
        finish(tid, v, kept[tid]);
      }
      __syncthreads();
    }
    TX* dxt = dx + (dx ? tile * height * lddx : 0);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (i >= rows) break;
      const float4 q = consts[i];
      const float2 c = both(q.x), r = both(q.y), zs = both(q.z), o0 = both(q.w), o1 = both(consts1[i]);
      const uint8_t* at = ring + slot * C::TILE + i * C::SLOT;
      const uint8_t *xs = RowX::first(at, xt + i * ldx), *gs = RowG::first(at + C::SLOT_X, gt + i * lddy);
#pragma unroll
      for (int u = 0; u < NU; ++u) {
        const int k = column(u);
        float2 fx[PAIRS], fg[PAIRS];
        RowX::get(xs, k, T, fx);
        RowG::get(gs, k, T, fg);
#pragma unroll
        for (int j = 0; j < PAIRS; ++j) {
          const float2 z = fma2(add2(fx[j], c), r, zs);
          aw[u][j] = fma2(fg[j], z, aw[u][j]);
          ab[u][j] = add2(ab[u][j], fg[j]);
          fx[j] = fma2(mul2(fg[j], wr[u][j]), r, fma2(z, o1, o0));
        }
        if (dx && k < K) put_unit<TX, E>(dxt + i * lddx, k, T, K, fx);
      }
    }
    slot ^= 1;
  }
  grid_dependents_launch();  // the kernel that adds the partial rows up may be scheduled; it waits for them
  if (!part) return;
  float* pw = part + static_cast<int64_t>(blockIdx.x) * K;
  float* pb = pw + static_cast<int64_t>(gridDim.x) * K;
#pragma unroll
  for (int u = 0; u < NU; ++u) {
    const int k = column(u);
    if constexpr (E == 1) {
      if (k < K) pw[k] = aw[u][0].x, pb[k] = ab[u][0].x;
      if (k + T < K) pw[k + T] = aw[u][0].y, pb[k + T] = ab[u][0].y;
    } else if (E == 2 && k < K) {
      *reinterpret_cast<float2*>(pw + k) = aw[u][0];
      *reinterpret_cast<float2*>(pb + k) = ab[u][0];
    } else if (E > 2 && k < K) {  // K is a multiple of four here
#pragma unroll
      for (int j = 0; j + 1 < PAIRS; j += 2) {
        *reinterpret_cast<float4*>(pw + k + 2 * j) = make_float4(aw[u][j].x, aw[u][j].y, aw[u][j + 1].x, aw[u][j + 1].y);
        *reinterpret_cast<float4*>(pb + k + 2 * j) = make_float4(ab[u][j].x, ab[u][j].y, ab[u][j + 1].x, ab[u][j + 1].y);
      }
    }
  }
}

// Rows too long for that: dx and the weight's gradient separately, from two
// readings of x and dy, E elements per access (2048 x 16384 bf16 85 us, 1024 x 11008
// 36 us; element by element 2347 x 9386 took 93 us, in pairs 67 us). One CTA per
// row: dx (where wanted) and the row's correction of the kept mean.
constexpr int kNormLongThreads = 512;

template <typename TX, typename TY, int E>
__global__ void __launch_bounds__(kNormLongThreads)
    layer_norm_dx_kernel(const TX* __restrict__ x, int64_t ldx, const float* __restrict__ w,
                         const float* __restrict__ mean, const float* __restrict__ rstd, const TY* __restrict__ dy,
                         int64_t lddy, TX* __restrict__ dx, int64_t lddx, float* __restrict__ shift, int64_t K) {
  constexpr int WARPS = kNormLongThreads / 32;
  __shared__ float sh[3 * WARPS];
  grid_begin();
  const int64_t m = blockIdx.x;
  const TX* xr = x + m * ldx;
  const TY* gr = dy + m * lddy;
  const float c = mean[m], r = rstd[m];
  const bool w16 = (reinterpret_cast<uintptr_t>(w) & 15u) == 0;
  auto weights = [&](int64_t k, float(&f)[E]) {
    if constexpr (E >= 4) {
      if (w && w16) {
#pragma unroll
        for (int j = 0; j < E; j += 4) {
          const float4 v = *reinterpret_cast<const float4*>(w + k + j);
          f[j] = v.x, f[j + 1] = v.y, f[j + 2] = v.z, f[j + 3] = v.w;
        }
        return;
      }
    }
#pragma unroll
    for (int j = 0; j < E; ++j) f[j] = w ? w[k + j] : 1.f;
  };
  float s[3] = {0.f, 0.f, 0.f};  // sums of d, g and g d
#pragma unroll 4
  for (int64_t k = threadIdx.x * E; k < K; k += kNormLongThreads * E) {
    float fx[E], fg[E], fw[E];
    Elem<TX, E>::load(xr + k, fx);
    Elem<TY, E>::load(gr + k, fg);
    weights(k, fw);
#pragma unroll
    for (int j = 0; j < E; ++j) {
      const float d = fx[j] - c, g = fg[j] * fw[j];
      s[0] += d;
      s[1] += g;
      s[2] = fmaf(g, d, s[2]);
    }
  }
  block_sums<WARPS>(s, sh);
  const float inv_k = 1.0f / static_cast<float>(K);
  const float md = s[0] * inv_k;
  const float mg = s[1] * inv_k, mgz = r * (s[2] - md * s[1]) * inv_k;
  if (shift && threadIdx.x == 0) shift[m] = md;
  if (!dx) return;
#pragma unroll 4
  for (int64_t k = threadIdx.x * E; k < K; k += kNormLongThreads * E) {
    float fx[E], fg[E], fw[E];
    Elem<TX, E>::load(xr + k, fx);
    Elem<TY, E>::load(gr + k, fg);
    weights(k, fw);
#pragma unroll
    for (int j = 0; j < E; ++j) {
      const float z = ((fx[j] - c) - md) * r, g = fg[j] * fw[j];
      fx[j] = r * (g - mg - z * mgz);
    }
    Elem<TX, E>::store(dx + m * lddx + k, fx);
  }
}

// Partial sums of dy z and dy over the rows m = p, p + P, ...: CTA (column
// block, p), E columns per lane, the rows dealt to the warps, four in flight.
template <typename TX, typename TY, int E>
__global__ void __launch_bounds__(kNormThreads)
    layer_norm_dw_kernel(const TX* __restrict__ x, int64_t ldx, const float* __restrict__ mean,
                         const float* __restrict__ rstd, const float* __restrict__ shift, const TY* __restrict__ dy,
                         int64_t lddy, float* __restrict__ part, int64_t M, int64_t K) {
  __shared__ float sh[2][kNormWarps][32 * E];
  grid_begin();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t k0 = static_cast<int64_t>(blockIdx.x) * (32 * E), k = k0 + lane * E;
  const int64_t p = blockIdx.y, P = gridDim.y;
  float sw[E] = {}, sb[E] = {};
  if (k < K) {
#pragma unroll 4
    for (int64_t m = p + warp * P; m < M; m += P * kNormWarps) {
      float fx[E], fg[E];
      Elem<TX, E>::load(x + m * ldx + k, fx);
      Elem<TY, E>::load(dy + m * lddy + k, fg);
      const float c = mean[m], md = shift[m], r = rstd[m];
#pragma unroll
      for (int j = 0; j < E; ++j) {
        sw[j] = fmaf(fg[j], ((fx[j] - c) - md) * r, sw[j]);
        sb[j] += fg[j];
      }
    }
  }
#pragma unroll
  for (int j = 0; j < E; ++j) {
    sh[0][warp][j * 32 + lane] = sw[j];
    sh[1][warp][j * 32 + lane] = sb[j];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 64 * E; i += kNormThreads) {
    const int which = i / (32 * E), col = i % (32 * E);
    if (k0 + col >= K) continue;
    float t = 0.f;
#pragma unroll
    for (int v = 0; v < kNormWarps; ++v) t += sh[which][v][(col % E) * 32 + col / E];
    part[(which * P + p) * K + k0 + col] = t;
  }
}

// dweight and dbias: the P partial rows added in order, 32 columns per CTA, a
// contiguous share of the rows per warp, eight of them in flight: 3 us. (With one
// load at a time 17 us for 389 rows of 1001 columns, three times the pass over x
// and dy.)
constexpr int kNormSumThreads = 512;

__global__ void __launch_bounds__(kNormSumThreads)
    layer_norm_dw_sum_kernel(const float* __restrict__ part, int P, int64_t K, float* __restrict__ dw,
                             float* __restrict__ db) {
  constexpr int WARPS = kNormSumThreads / 32;
  __shared__ float sh[WARPS][32];
  grid_begin();
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
