// Attention over a key/value cache for many rows (tcgen05): instances for
// bfloat16 queries over 8-bit caches.
#include "kv_tile.cuh"

namespace rope_gb300 {

KvTileKernel kv_tile_kernel_bf16_fp8(int H, int kind) {
  return kv_tile_pick<__nv_bfloat16, true>(H, kind);
}

}  // namespace rope_gb300
