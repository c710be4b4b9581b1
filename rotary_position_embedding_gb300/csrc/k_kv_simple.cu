// Attention over a key/value cache on CUDA cores, and the joining of splits:
// kernel instances.
#include "kv_simple.cuh"

namespace rope_gb300 {

namespace {

template <class T, bool FP8>
const void* pick(int H, bool few) {
  if (H <= 64) return few ? (const void*)kv_simple_kernel_t<T, FP8, 1, 1> : (const void*)kv_simple_kernel_t<T, FP8, 1, 4>;
  if (H <= 128) return few ? (const void*)kv_simple_kernel_t<T, FP8, 2, 1> : (const void*)kv_simple_kernel_t<T, FP8, 2, 4>;
  return few ? (const void*)kv_simple_kernel_t<T, FP8, 4, 1> : (const void*)kv_simple_kernel_t<T, FP8, 4, 4>;
}

}  // namespace

KvSimpleKernel kv_simple_kernel(int dtype, bool fp8, int H, int64_t R) {
  const bool few = kv_simple_rows(R) == 16;
  const void* fn = dtype == 0   ? (fp8 ? pick<float, true>(H, few) : pick<float, false>(H, few))
                   : dtype == 1 ? (fp8 ? pick<__half, true>(H, few) : pick<__half, false>(H, few))
                                : (fp8 ? pick<__nv_bfloat16, true>(H, few) : pick<__nv_bfloat16, false>(H, few));
  const size_t HP = (H + 3) / 4 * 4 + 4, rows = kv_simple_rows(R);
  return {fn, ((rows + 2 * kSimpleCols) * HP + rows * kSimpleP) * sizeof(float)};
}

const void* kv_combine_kernel(int dtype) {
  if (dtype == 0) return (const void*)kv_combine_kernel_t<float>;
  if (dtype == 1) return (const void*)kv_combine_kernel_t<__half>;
  return (const void*)kv_combine_kernel_t<__nv_bfloat16>;
}

}  // namespace rope_gb300
