// bl_layer_norm and bl_layer_norm_backward: argument checks and dispatch. A
// translation unit of its own, since its kernels are most of the library's
// compile time.
#include "bl_host.cuh"
#include "bl_layernorm.cuh"

namespace bl {
namespace {

int check_norm_shape(int64_t M, int64_t K) {
  if (M < 0 || K < 1) return BL_ERR_INVALID_ARG;
  return M > kMaxDim || K > kMaxDim ? BL_ERR_UNSUPPORTED : BL_OK;
}

struct NormWs {
  int64_t parts;  // partial rows of dweight and of dbias there is room for
  size_t shift, part, bytes;
};
NormWs norm_ws(int64_t M, int64_t K) {
  NormWs w{};
  if (M < 1 || K < 1 || M > kMaxDim || K > kMaxDim || M >= kMaxProduct / K) return w;
  w.parts = std::min<int64_t>(M, K <= 1024 ? kNormMaxParts : kNormMaxParts / 2);
  w.shift = 0;
  w.part = align256(size_t(M) * 4);
  w.bytes = w.part + align256(size_t(2 * w.parts) * size_t(K) * 4);
  return w;
}

// rows that `elems` elements at a time can be read or written of
inline bool rows_aligned(const void* p, int type, int64_t ld, int64_t K, int64_t M, int elems) {
  return K % elems == 0 && (M <= 1 || ld % elems == 0) && aligned_to(p, elems * type_bytes(type));
}
// rows whose 16-byte pieces can be copied whole
inline bool rows_in_pieces(const void* p, int type, int64_t ld, int64_t K, int64_t M) {
  return rows_aligned(p, type, ld, K, M, 16 / type_bytes(type));
}

// The layer norm's tiling: f(CPT, W) (columns per thread, warps per row) of the
// smallest tile that holds a row.
// Rows read 16 bytes at a time: 32 columns per thread, fewer where the rows are
// so few (`few`) that spreading each over a CTA is what fills the GPU.
template <typename F>
int with_wide_tile(int64_t K, bool few, F&& f) {
  if (few && K <= 8192) {
    if (K <= 1024) return f(Int<8>{}, Int<4>{});
    if (K <= 2048) return f(Int<16>{}, Int<4>{});
    if (K <= 4096) return f(Int<16>{}, Int<8>{});
    return f(Int<16>{}, Int<16>{});
  }
  if (K <= 256) return f(Int<8>{}, Int<1>{});
  if (K <= 512) return f(Int<16>{}, Int<1>{});
  if (K <= 1024) return f(Int<32>{}, Int<1>{});
  if (K <= 2048) return f(Int<32>{}, Int<2>{});
  if (K <= 4096) return f(Int<32>{}, Int<4>{});
  if (K <= 6144) return f(Int<32>{}, Int<6>{});
  if (K <= 8192) return f(Int<32>{}, Int<8>{});
  return f(Int<32>{}, Int<16>{});
}
// Rows of any alignment, read element by element: 16 columns per thread, in
// finer steps, since a thread without columns costs as much as one with them
// (5001 columns: 22 us in a tile of 8192, 14 us in one of 5120).
template <typename F>
int with_narrow_tile(int64_t K, F&& f) {
  if (K <= 256) return f(Int<8>{}, Int<1>{});
  if (K <= 1024) return f(Int<8>{}, Int<4>{});
  if (K <= 2048) return f(Int<16>{}, Int<4>{});
  if (K <= 2560) return f(Int<16>{}, Int<5>{});
  if (K <= 4096) return f(Int<16>{}, Int<8>{});
  if (K <= 5120) return f(Int<16>{}, Int<10>{});
  if (K <= 6144) return f(Int<16>{}, Int<12>{});
  if (K <= 7168) return f(Int<16>{}, Int<14>{});
  if (K <= 8192) return f(Int<16>{}, Int<16>{});
  return f(Int<32>{}, Int<16>{});
}

}  // namespace

size_t norm_workspace_bytes(int64_t M, int64_t K) { return norm_ws(M, K).bytes; }

}  // namespace bl

using namespace bl;

extern "C" {

int bl_layer_norm(const void* x, int x_type, int64_t ldx, const float* weight, const float* bias, void* y, int y_type,
                  int64_t ldy, float* mean, float* rstd, int64_t M, int64_t K, float eps, void* stream) {
  int rc = check_norm_shape(M, K);
  if (rc != BL_OK) return rc;
  if (!type_ok(x_type) || !type_ok(y_type) || !(eps > 0.f) || !(eps < INFINITY)) return BL_ERR_INVALID_ARG;
  if ((rc = check_rows(M, K, ldx)) != BL_OK || (rc = check_rows(M, K, ldy)) != BL_OK) return rc;
  if (M == 0) return BL_OK;
  if (!x || !y || !aligned_to(x, type_bytes(x_type)) || !aligned_to(y, type_bytes(y_type)) || !aligned_to(weight, 4) ||
      !aligned_to(bias, 4) || !aligned_to(mean, 4) || !aligned_to(rstd, 4))
    return BL_ERR_INVALID_ARG;
  if (x == y && (x_type != y_type || ldx != ldy)) return BL_ERR_INVALID_ARG;
  int sms = 0;
  rc = library_device(&sms);
  if (rc != BL_OK) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return with_types(x_type, y_type, [&](auto tx, auto ty) {
    using TX = decltype(tx);
    using TY = decltype(ty);
    if (K > kNormMaxK) {
      return launch_after(layer_norm_kernel<TX, TY>, dim3(unsigned(M)), kNormThreads, 0, s, static_cast<const TX*>(x), ldx,
                          weight, bias, static_cast<TY*>(y), ldy, mean, rstd, K, eps);
    }
    constexpr int WIDE = 16 / int(sizeof(TX));
    const bool wide = rows_aligned(x, x_type, ldx, K, M, WIDE) && rows_aligned(y, y_type, ldy, K, M, WIDE);
    auto run = [&](auto e, auto cpt, auto warps) {
      constexpr int E = decltype(e)::value, CPT = decltype(cpt)::value, W = decltype(warps)::value;
      using C = NormCfg<TX, E, CPT, W>;
      constexpr auto kernel = layer_norm_rows_kernel<TX, TY, E, CPT, W>;
      const int groups = int(std::min<int64_t>(C::GROUPS, cdiv(M, sms)));
      // with fewer groups more CTAs fit, but then there are no rows for them
      const int n = ctas_per_sm<kernel>(C::GROUPS * W * 32, C::smem(C::GROUPS));
      if (n < 1) return int(BL_ERR_CUDA);
      const int64_t grid = persistent_grid(n, sms, cdiv(M, groups), kMaxDim);
      return launch_after(kernel, dim3(unsigned(grid)), groups * W * 32, C::smem(groups), s, static_cast<const TX*>(x), ldx,
                          weight, bias, static_cast<TY*>(y), ldy, mean, rstd, M, int(K), eps);
    };
    if (wide)
      return with_wide_tile(K, M <= 2 * int64_t(sms), [&](auto cpt, auto warps) { return run(Int<WIDE>{}, cpt, warps); });
    return with_narrow_tile(K, [&](auto cpt, auto warps) { return run(Int<1>{}, cpt, warps); });
  });
}

int bl_layer_norm_backward(const void* x, int x_type, int64_t ldx, const float* weight, const float* mean,
                           const float* rstd, const void* dy, int dy_type, int64_t lddy, void* dx, int64_t lddx,
                           float* dweight, float* dbias, int64_t M, int64_t K, void* ws, size_t ws_bytes, void* stream) {
  int rc = check_norm_shape(M, K);
  if (rc != BL_OK) return rc;
  if (!type_ok(x_type) || !type_ok(dy_type)) return BL_ERR_INVALID_ARG;
  if ((rc = check_rows(M, K, ldx)) != BL_OK || (rc = check_rows(M, K, lddy)) != BL_OK ||
      (dx && (rc = check_rows(M, K, lddx)) != BL_OK))
    return rc;
  if (!aligned_to(weight, 4) || !aligned_to(dweight, 4) || !aligned_to(dbias, 4)) return BL_ERR_INVALID_ARG;
  if (dweight && dweight == dbias) return BL_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (M == 0) {  // an empty batch: zero gradients of the weight and the bias
    for (float* g : {dweight, dbias})
      if (g && cudaMemsetAsync(g, 0, size_t(K) * 4, s) != cudaSuccess) {
        cudaGetLastError();
        return BL_ERR_CUDA;
      }
    return BL_OK;
  }
  if (!x || !mean || !rstd || !dy || !aligned_to(x, type_bytes(x_type)) || !aligned_to(dy, type_bytes(dy_type)) ||
      !aligned_to(dx, type_bytes(x_type)) || !aligned_to(mean, 4) || !aligned_to(rstd, 4) || dx == x ||
      (dx && dx == dy))
    return BL_ERR_INVALID_ARG;
  const bool want_dw = dweight || dbias;
  if (!dx && !want_dw) return BL_OK;
  const NormWs w = norm_ws(M, K);
  if (w.bytes == 0) return BL_ERR_UNSUPPORTED;
  if (want_dw && (!ws || !aligned16(ws) || ws_bytes < w.bytes)) return BL_ERR_INVALID_ARG;
  int sms = 0;
  rc = library_device(&sms);
  if (rc != BL_OK) return rc;
  float* shift = want_dw ? reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + w.shift) : nullptr;
  float* part = want_dw ? reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + w.part) : nullptr;
  return with_types(x_type, dy_type, [&](auto tx, auto ty) {
    using TX = decltype(tx);
    using TY = decltype(ty);
    const auto* xp = static_cast<const TX*>(x);
    const auto* gp = static_cast<const TY*>(dy);
    auto* dxp = static_cast<TX*>(dx);
    auto sum_parts = [&](int64_t parts) {
      return launch_after(layer_norm_dw_sum_kernel, dim3(unsigned(cdiv(K, 32)), 2), kNormSumThreads, 0, s,
                          static_cast<const float*>(part), int(parts), K, dweight, dbias);
    };
    if (K > kNormGradMaxK) {
      int st = launch_after(layer_norm_dx_kernel<TX, TY>, dim3(unsigned(M)), kNormThreads, 0, s, xp, ldx, weight, mean,
                            rstd, gp, lddy, dxp, lddx, shift, K);
      if (st != BL_OK || !want_dw) return st;
      const int64_t parts = std::min<int64_t>(cdiv(M, 64), 128);
      st = launch_after(layer_norm_dw_kernel<TX, TY>, dim3(unsigned(cdiv(K, 32)), unsigned(parts)), kNormThreads, 0, s, xp,
                        ldx, mean, rstd, static_cast<const float*>(shift), gp, lddy, part, M, K);
      return st != BL_OK ? st : sum_parts(parts);
    }
    auto launch = [&](auto kernel, int64_t grid, int threads, int smem, auto... more) {
      const int st = launch_after(kernel, dim3(unsigned(grid)), threads, smem, s, xp, ldx, weight, mean, rstd, gp, lddy,
                                  dxp, lddx, part, M, int(K), more...);
      return st != BL_OK || !want_dw ? st : sum_parts(grid);
    };
    const int64_t most = want_dw ? w.parts : kMaxDim;
    constexpr int WIDE = sizeof(TX) == 2 && sizeof(TY) == 2 ? 8 : 4;
    const bool wide = rows_in_pieces(x, x_type, ldx, K, M) && rows_in_pieces(dy, dy_type, lddy, K, M) &&
                      (!dx || rows_in_pieces(dx, x_type, lddx, K, M));
    auto by_width = [&](auto e) {
      constexpr int E = decltype(e)::value;
      auto rows = [&](auto cpt) {
        constexpr int CPT = decltype(cpt)::value;
        using C = NormGradRowCfg<TX, TY, E, CPT>;
        constexpr auto kernel = layer_norm_grad_rows_kernel<TX, TY, E, CPT>;
        const int n = ctas_per_sm<kernel>(C::WARPS * 32, C::SMEM);
        if (n < 1) return int(BL_ERR_CUDA);
        return launch(kernel, persistent_grid(n, sms, cdiv(M, C::WARPS), most), C::WARPS * 32, C::SMEM);
      };
      auto tiles = [&](auto cpt, auto warps) {
        constexpr int CPT = decltype(cpt)::value, W = decltype(warps)::value;
        using C = NormGradTileCfg<TX, TY, E, CPT, W>;
        constexpr auto kernel = layer_norm_grad_tile_kernel<TX, TY, E, CPT, W>;
        const int n = ctas_per_sm<kernel>(C::THREADS, C::SMEM);
        if (n < 1) return int(BL_ERR_CUDA);
        // rows per tile: the height whose rounds take least, a round costing its rows and about one more, the partial
        // rows about one per 130 (777 x 1001: 13.2 us with the tallest tile, 98 CTAs of them)
        int height = 1;
        int64_t best = INT64_MAX, grid = 1;
        for (int h = 1; h <= C::R; ++h) {
          const int64_t tiles_h = cdiv(M, h), g = persistent_grid(n, sms, tiles_h, most);
          const int64_t cost = 130 * cdiv(tiles_h, g) * (h + 1) + g;
          if (cost <= best) best = cost, height = h, grid = g;
        }
        return launch(kernel, grid, C::THREADS, C::SMEM, height);
      };
      if (K <= 256) return rows(Int<8>{});
      if (K <= 512) return rows(Int<16>{});
      if (K <= 1024) return tiles(Int<8>{}, Int<4>{});
      if (K <= 2048) return tiles(Int<8>{}, Int<8>{});
      if (K <= 2560) return tiles(Int<8>{}, Int<10>{});
      if (K <= 4096) return tiles(Int<8>{}, Int<16>{});
      if (K <= 5120) return tiles(Int<16>{}, Int<10>{});
      if (K <= 6144) return tiles(Int<16>{}, Int<12>{});
      return tiles(Int<32>{}, Int<8>{});
    };
    return wide ? by_width(Int<WIDE>{}) : by_width(Int<1>{});
  });
}

}  // extern "C"
