// Attention over a paged cache for few rows: kernel instances.
#include "paged_token.cuh"

namespace rope_gb300 {

namespace {
template <class T, int HD, int NB>
PagedTokenKernel pick() {
  using C = PagedTokenCfg<HD, NB>;
  return {(const void*)paged_token_kernel_t<T, HD, NB>, (const void*)paged_join_kernel_t<T>, C::kSmem,
          C::kSmem + C::kClusterPart};
}
template <class T>
PagedTokenKernel pick_head(int H, bool few) {
  if (H <= 64) return few ? pick<T, 64, 1>() : pick<T, 64, 2>();
  if (H <= 128) return few ? pick<T, 128, 1>() : pick<T, 128, 2>();
  return few ? pick<T, 256, 1>() : pick<T, 256, 2>();
}
}  // namespace

PagedTokenKernel paged_token_kernel(int dtype, int H, bool few) {
  return dtype == 1 ? pick_head<__half>(H, few) : pick_head<__nv_bfloat16>(H, few);
}

}  // namespace rope_gb300
