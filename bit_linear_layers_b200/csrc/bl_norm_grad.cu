// bl_layer_norm_backward: argument checks, workspace and dispatch.
#include "bl_host.cuh"
#include "bl_layernorm_grad.cuh"

namespace bl {
namespace {

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

// rows whose 16-byte pieces can be copied whole
inline bool rows_in_pieces(const void* p, int type, int64_t ld, int64_t K, int64_t M) {
  return rows_aligned(p, type, ld, K, M, 16 / type_bytes(type));
}

}  // namespace

size_t norm_workspace_bytes(int64_t M, int64_t K) { return norm_ws(M, K).bytes; }

}  // namespace bl

using namespace bl;

extern "C" {

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
    constexpr int WIDE = sizeof(TX) == 2 && sizeof(TY) == 2 ? 8 : 4;
    const bool wide = rows_in_pieces(x, x_type, ldx, K, M) && rows_in_pieces(dy, dy_type, lddy, K, M) &&
                      (!dx || rows_in_pieces(dx, x_type, lddx, K, M));
    // even widths in pairs (4096 x 2050: 28 us, element by element 30 to 32 us)
    const bool pairs = rows_aligned(x, x_type, ldx, K, M, 2) && rows_aligned(dy, dy_type, lddy, K, M, 2) &&
                       (!dx || rows_aligned(dx, x_type, lddx, K, M, 2));
    auto in_width = [&](auto f) { return wide ? f(Int<WIDE>{}) : pairs ? f(Int<2>{}) : f(Int<1>{}); };
    if (K > kNormGradMaxK)
      return in_width([&](auto e) {
        constexpr int E = decltype(e)::value;
        int st = launch_after(layer_norm_dx_kernel<TX, TY, E>, dim3(unsigned(M)), kNormLongThreads, 0, s, xp, ldx, weight,
                              mean, rstd, gp, lddy, dxp, lddx, shift, K);
        if (st != BL_OK || !want_dw) return st;
        // about one round of eight CTAs per SM, of 32 rows or more (2048 x 16384: 18 parts 85 us, 64 parts 123 us with
        // single loads of the weight)
        const int64_t blocks = cdiv(K, 32 * E);
        const int64_t parts = std::min<int64_t>(std::min<int64_t>(cdiv(M, 32), 128), std::max<int64_t>(1, sms * 8 / blocks));
        st = launch_after(layer_norm_dw_kernel<TX, TY, E>, dim3(unsigned(blocks), unsigned(parts)), kNormThreads, 0, s,
                          xp, ldx, mean, rstd, static_cast<const float*>(shift), gp, lddy, part, M, K);
        return st != BL_OK ? st : sum_parts(parts);
      });
    auto launch = [&](auto kernel, int64_t grid, int threads, int smem, auto... more) {
      const int st = launch_after(kernel, dim3(unsigned(grid)), threads, smem, s, xp, ldx, weight, mean, rstd, gp, lddy,
                                  dxp, lddx, part, M, int(K), more...);
      return st != BL_OK || !want_dw ? st : sum_parts(grid);
    };
    const int64_t most = want_dw ? w.parts : kMaxDim;
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
      if constexpr (E <= 2)  // read element by element a column without data costs as much as any: a finer step
        if (K <= 768) return tiles(Int<6>{}, Int<4>{});
      if (K <= 1024) return tiles(Int<8>{}, Int<4>{});
      if constexpr (E <= 2)
        if (K <= 1536) return tiles(Int<8>{}, Int<6>{});
      if (K <= 2048) return tiles(Int<8>{}, Int<8>{});
      if (K <= 2560) return tiles(Int<8>{}, Int<10>{});
      if (K <= 4096) return tiles(Int<8>{}, Int<16>{});
      if (K <= 5120) return tiles(Int<16>{}, Int<10>{});
      if (K <= 6144) return tiles(Int<16>{}, Int<12>{});
      return tiles(Int<32>{}, Int<8>{});
    };
    return in_width(by_width);
  });
}

}  // extern "C"
