// Attention over a paged cache on CUDA cores, and the joining of splits: kernel
// instances.
#include "paged_simple.cuh"

namespace rope_gb300 {

namespace {
template <class T>
const void* pick(int H, bool few) {
  if (H <= 64) return few ? (const void*)paged_simple_kernel_t<T, 1, 1> : (const void*)paged_simple_kernel_t<T, 1, 4>;
  if (H <= 128) return few ? (const void*)paged_simple_kernel_t<T, 2, 1> : (const void*)paged_simple_kernel_t<T, 2, 4>;
  return few ? (const void*)paged_simple_kernel_t<T, 4, 1> : (const void*)paged_simple_kernel_t<T, 4, 4>;
}
}  // namespace

KvSimpleKernel paged_simple_kernel(int dtype, int H, bool few) {
  const void* fn = dtype == 0 ? pick<float>(H, few) : dtype == 1 ? pick<__half>(H, few) : pick<__nv_bfloat16>(H, few);
  const size_t HP = (H + 3) / 4 * 4 + 4, rows = few ? 16 : 64;
  return {fn, ((rows + 2 * kSimpleCols) * HP + rows * kSimpleP) * sizeof(float)};
}

const void* paged_combine_kernel(int dtype) {
  if (dtype == 0) return (const void*)paged_combine_kernel_t<float>;
  if (dtype == 1) return (const void*)paged_combine_kernel_t<__half>;
  return (const void*)paged_combine_kernel_t<__nv_bfloat16>;
}

}  // namespace rope_gb300
