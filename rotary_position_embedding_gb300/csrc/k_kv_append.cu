// Q and K rotation with the append to 8-bit caches: kernel instances.
#include "kv_append.cuh"

namespace rope_gb300 {

namespace {
template <class T, int V>
const void* pick(bool inter, bool norm) {
  if (inter)
    return norm ? (const void*)kv_append_kernel_t<T, V, true, true> : (const void*)kv_append_kernel_t<T, V, true, false>;
  return norm ? (const void*)kv_append_kernel_t<T, V, false, true> : (const void*)kv_append_kernel_t<T, V, false, false>;
}
}  // namespace

const void* kv_append_kernel(int dtype, bool vec, bool inter, bool norm) {
  if (dtype == 0) return vec ? pick<float, 4>(inter, norm) : pick<float, 1>(inter, norm);
  if (dtype == 1) return vec ? pick<__half, 8>(inter, norm) : pick<__half, 1>(inter, norm);
  return vec ? pick<__nv_bfloat16, 8>(inter, norm) : pick<__nv_bfloat16, 1>(inter, norm);
}

}  // namespace rope_gb300
