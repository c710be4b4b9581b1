// Q and K rotation with the append to paged caches: kernel instances.
#include "paged_append.cuh"
#include "paged_append_heads.cuh"

namespace rope_gb300 {

namespace {
template <class T, int V>
const void* pick(bool inter, bool norm) {
  if (inter)
    return norm ? (const void*)paged_append_kernel_t<T, V, true, true> : (const void*)paged_append_kernel_t<T, V, true, false>;
  return norm ? (const void*)paged_append_kernel_t<T, V, false, true> : (const void*)paged_append_kernel_t<T, V, false, false>;
}
}  // namespace

const void* paged_append_kernel(int dtype, bool vec, bool inter, bool norm) {
  if (dtype == 0) return vec ? pick<float, 4>(inter, norm) : pick<float, 1>(inter, norm);
  if (dtype == 1) return vec ? pick<__half, 8>(inter, norm) : pick<__half, 1>(inter, norm);
  return vec ? pick<__nv_bfloat16, 8>(inter, norm) : pick<__nv_bfloat16, 1>(inter, norm);
}

namespace {
template <class T, int HPT>
const void* pick_heads(bool inter, bool norm) {
  if (norm) {
    if constexpr (HPT > 2) return nullptr;
    else
      return inter ? (const void*)paged_append_heads_kernel_t<T, true, true, HPT>
                   : (const void*)paged_append_heads_kernel_t<T, false, true, HPT>;
  }
  return inter ? (const void*)paged_append_heads_kernel_t<T, true, false, HPT>
               : (const void*)paged_append_heads_kernel_t<T, false, false, HPT>;
}
}  // namespace

const void* paged_append_heads_kernel(int dtype, bool inter, bool norm, int hpt) {
  if (dtype == 0) return hpt == 2 ? pick_heads<float, 2>(inter, norm) : nullptr;
  if (dtype == 1) return hpt == 2 ? pick_heads<__half, 2>(inter, norm) : pick_heads<__half, 4>(inter, norm);
  return hpt == 2 ? pick_heads<__nv_bfloat16, 2>(inter, norm) : pick_heads<__nv_bfloat16, 4>(inter, norm);
}

}  // namespace rope_gb300
