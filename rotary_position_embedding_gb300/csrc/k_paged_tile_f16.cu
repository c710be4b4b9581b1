// Attention over a paged cache for many rows (tcgen05): instances for float16.
#include "paged_tile.cuh"

namespace rope_gb300 {

PagedTileKernel paged_tile_kernel_f16(int H, int kind) { return paged_tile_pick<__half>(H, kind); }

}  // namespace rope_gb300
