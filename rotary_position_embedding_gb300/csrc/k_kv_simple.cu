// Attention over a key/value cache on CUDA cores, and the joining of splits:
// kernel instances.
#include "kv_simple.cuh"

namespace rope_gb300 {

const void* kv_simple_kernel(int dtype, bool fp8) {
  if (dtype == 0) return fp8 ? (const void*)kv_simple_kernel_t<float, true> : (const void*)kv_simple_kernel_t<float, false>;
  if (dtype == 1) return fp8 ? (const void*)kv_simple_kernel_t<__half, true> : (const void*)kv_simple_kernel_t<__half, false>;
  return fp8 ? (const void*)kv_simple_kernel_t<__nv_bfloat16, true> : (const void*)kv_simple_kernel_t<__nv_bfloat16, false>;
}

size_t kv_simple_smem(int H) {
  const size_t HP = (H + 3) / 4 * 4 + 4;
  return ((kKvSimpleRows + kSimpleCols) * HP + kKvSimpleRows * 33) * sizeof(float);
}

const void* kv_combine_kernel(int dtype) {
  if (dtype == 0) return (const void*)kv_combine_kernel_t<float>;
  if (dtype == 1) return (const void*)kv_combine_kernel_t<__half>;
  return (const void*)kv_combine_kernel_t<__nv_bfloat16>;
}

}  // namespace rope_gb300
