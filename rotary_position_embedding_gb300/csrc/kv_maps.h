// Tensor maps of the 16-bit caches for kv_tile_kernel (internal).
#pragma once

#include <cuda.h>
#include <stdint.h>

namespace rope_gb300 {

struct KvTileMaps {
  CUtensorMap k, v;
};

// Map of a cache (planes, len, H) of 16-bit elements in boxes of 64 elements x
// `rows` rows, 128-byte swizzle, zeros outside. False where it cannot be made.
bool encode_kv_map(CUtensorMap* m, bool bf16, const void* base, int64_t H, int64_t len, int64_t planes, int rows);

}  // namespace rope_gb300
