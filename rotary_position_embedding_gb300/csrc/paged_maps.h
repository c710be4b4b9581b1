// Tensor maps of paged caches (internal).
#pragma once

#include <cuda.h>
#include <stdint.h>

namespace rope_gb300 {

struct PagedMaps {
  CUtensorMap k, v;
};

// K and V in boxes of several rows, V of 8 and of one too; Q (T, Nq, H) in boxes of the
// heads of a group and the tokens of an item.
struct PagedTileMaps {
  CUtensorMap k, v, v_eight, v_row, q;
};

// Map of pages (num, Nkv, ps, H) of 16-bit elements, `stride` elements apart, in
// boxes of 64 elements x `rows` rows, 128-byte swizzle, zeros outside. False where it
// cannot be made.
bool encode_paged_map(CUtensorMap* m, bool bf16, const void* base, int64_t H, int64_t ps, int64_t Nkv, int64_t num,
                      int64_t stride, int rows);
bool encode_paged_q_map(CUtensorMap* m, bool bf16, const void* base, int64_t H, int64_t Nq, int64_t T, int G, int tokens);

}  // namespace rope_gb300
