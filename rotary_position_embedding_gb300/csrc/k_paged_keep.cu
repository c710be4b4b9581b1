// Accepted drafts' rows of a paged cache: kernel instances.
#include "paged_keep.cuh"

namespace rope_gb300 {

const void* paged_keep_kernel(int unit_bytes) {
  if (unit_bytes == 16) return (const void*)paged_keep_kernel_t<uint4>;
  if (unit_bytes == 4) return (const void*)paged_keep_kernel_t<uint32_t>;
  return (const void*)paged_keep_kernel_t<unsigned short>;
}

}  // namespace rope_gb300
