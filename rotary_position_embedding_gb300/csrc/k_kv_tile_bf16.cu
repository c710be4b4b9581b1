// Attention over a key/value cache for many rows (tcgen05): instances for
// bfloat16 queries.
#include "kv_tile.cuh"

namespace rope_gb300 {

KvTileKernel kv_tile_kernel_bf16(int H, int kind) {
  return kv_tile_pick<__nv_bfloat16, false>(H, kind);
}

}  // namespace rope_gb300
