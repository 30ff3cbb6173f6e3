// bl_layer_norm: argument checks and dispatch. The layer norm and its gradient
// have a translation unit each, since their kernels are most of the library's
// compile time.
#include "bl_host.cuh"
#include "bl_layernorm.cuh"

namespace bl {
namespace {

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
// Rows of any alignment, read element by element: up to 16 columns per thread,
// in finer steps, since a thread without columns costs as much as one with them
// (1537 x 5001: 22 us in a tile of 8192, 14 us in one of 5120), and as few warps
// as that allows (30000 x 301: 43 us with four, 20 us with one). Reading even
// widths in pairs gains nothing here (4096 x 2050: 17 and 17 us from bf16, 21 and
// 19 us from fp32); the gradient does so.
template <typename F>
int with_narrow_tile(int64_t K, F&& f) {
  if (K <= 256) return f(Int<8>{}, Int<1>{});
  if (K <= 384) return f(Int<12>{}, Int<1>{});
  if (K <= 512) return f(Int<16>{}, Int<1>{});
  if (K <= 768) return f(Int<12>{}, Int<2>{});
  if (K <= 1024) return f(Int<16>{}, Int<2>{});
  if (K <= 1536) return f(Int<16>{}, Int<3>{});
  if (K <= 2048) return f(Int<16>{}, Int<4>{});
  if (K <= 2560) return f(Int<16>{}, Int<5>{});
  if (K <= 3584) return f(Int<16>{}, Int<7>{});
  if (K <= 4096) return f(Int<16>{}, Int<8>{});
  if (K <= 5120) return f(Int<16>{}, Int<10>{});
  if (K <= 6144) return f(Int<16>{}, Int<12>{});
  if (K <= 7168) return f(Int<16>{}, Int<14>{});
  if (K <= 8192) return f(Int<16>{}, Int<16>{});
  return f(Int<32>{}, Int<16>{});
}

}  // namespace

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

}  // extern "C"
