// Q and K rotation with the append to 8-bit caches: kernel instances.
#include "kv_append.cuh"

namespace rope_gb300 {

namespace {
template <class T, int V, bool FAST>
const void* pick(bool inter, bool norm) {
  if (inter)
    return norm ? (const void*)kv_append_kernel_t<T, V, true, true, FAST>
                : (const void*)kv_append_kernel_t<T, V, true, false, FAST>;
  return norm ? (const void*)kv_append_kernel_t<T, V, false, true, FAST>
              : (const void*)kv_append_kernel_t<T, V, false, false, FAST>;
}
template <class T, int V>
const void* pick_vec(bool inter, bool norm, bool fast) {
  return fast ? pick<T, V, true>(inter, norm) : pick<T, V, false>(inter, norm);
}
}  // namespace

const void* kv_append_kernel(int dtype, bool vec, bool inter, bool norm, bool fast) {
  if (dtype == 0) return vec ? pick_vec<float, 4>(inter, norm, fast) : pick<float, 1, false>(inter, norm);
  if (dtype == 1) return vec ? pick_vec<__half, 8>(inter, norm, fast) : pick<__half, 1, false>(inter, norm);
  return vec ? pick_vec<__nv_bfloat16, 8>(inter, norm, fast) : pick<__nv_bfloat16, 1, false>(inter, norm);
}

}  // namespace rope_gb300
