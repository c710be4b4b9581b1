// Attention over a paged cache for many rows (tcgen05): instances for bfloat16.
#include "paged_tile.cuh"

namespace rope_gb300 {

PagedTileKernel paged_tile_kernel_bf16(int H, int kind) { return paged_tile_pick<__nv_bfloat16>(H, kind); }

}  // namespace rope_gb300
