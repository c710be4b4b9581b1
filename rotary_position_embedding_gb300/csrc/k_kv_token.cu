// Attention over a key/value cache for few rows: kernel instances.
#include "kv_token.cuh"

namespace rope_gb300 {

namespace {
template <class T, bool FP8, int HD>
KvTokenKernel pick(bool two) {
  if (two)
    return {(const void*)kv_token_kernel_t<T, FP8, HD, 2>, (const void*)kv_join_kernel_t<T>,
            TokenCfg<T, FP8, HD, 2>::kSmem};
  return {(const void*)kv_token_kernel_t<T, FP8, HD, 1>, (const void*)kv_join_kernel_t<T>,
          TokenCfg<T, FP8, HD, 1>::kSmem};
}
template <class T, bool FP8>
KvTokenKernel pick_head(int H, bool two) {
  return H <= 64 ? pick<T, FP8, 64>(two) : H <= 128 ? pick<T, FP8, 128>(two) : pick<T, FP8, 256>(two);
}
}  // namespace

KvTokenKernel kv_token_kernel(int dtype, bool fp8, int H, bool two) {
  if (dtype == 1) return fp8 ? pick_head<__half, true>(H, two) : pick_head<__half, false>(H, two);
  return fp8 ? pick_head<__nv_bfloat16, true>(H, two) : pick_head<__nv_bfloat16, false>(H, two);
}

}  // namespace rope_gb300
