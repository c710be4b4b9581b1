// Internal interface between the C-ABI layer of the paged-cache operators
// (paged_api.cu) and their kernels. Not installed; not part of the public ABI.
#pragma once

#include "kv_internal.h"

namespace rope_gb300 {

// A batch over caches held in pages. Sequence b has the tokens [starts[b],
// starts[b + 1]) of T, or [b S, (b + 1) S); its row j is row j % ps of page
// table[b, j / ps], a page holding (Nkv, ps, H) elements.
struct PagedBatch {
  const int32_t* starts;  // (B + 1), or null
  const int32_t* past;    // (B)
  const int32_t* table;   // (B, max_pages)
  int32_t* status;
  int64_t T, S;
  int64_t page_stride;    // elements between pages
  int64_t rows;           // max_pages * ps, below 2^30
  int32_t B, max_pages, pages, ps;
  int32_t most;           // longer sequences are left out (attention)
  KvDiv by_ps;
};

// Attention. The G query heads of a key/value head and the n tokens of a sequence
// are the n * G rows of one problem (b, kvh); a row of the batch is token * G + its
// head in the group.
struct PagedParams {
  PagedBatch s;
  const void* q;           // (T, Nq*H)
  const void* k;           // pages
  const void* v;
  void* out;               // (T, Nq*H)
  const float* slopes;     // (Nq), or null
  const int64_t* masks;    // (T): bit t: new token t is seen; or null
  float* ws_o;             // partial outputs, (Nkv, splits, T * G, H)
  float2* ws_ml;           // and their (maximum, sum); or (2 * deal, rt, H)
  int4* ws_join;           // (deal): the problem that a CTA leaves unfinished
  int32_t Nq, Nkv, G, H;
  int32_t window;          // keys that a token sees, itself among them; 0: all
  int32_t splits;
  int32_t tiles;           // row tiles of the longest sequence
  int32_t mixed;           // sequences of up to so many rows are paged_token_kernel's, longer ones paged_tile_kernel's (0: all one's)
  int32_t chunk;           // rows of a box: of a page, and of a unit or tile of keys
  int32_t deal, cluster;   // CTAs that the work is dealt to; paged_token_kernel: or those of a cluster a problem
  int32_t rt;              // and rows of a part in the workspace (8 or 16)
  int32_t tpi, items;      // paged_tile_kernel: tokens of an item; items of the batch, at most
  int32_t over_item, over_join;  // what an item weighs beside its key tiles, what joining parts is worth
  int32_t entire;          // paged_tile_kernel: no item is split, whatever the lengths; no workspace
  int32_t shared;          // both kernels run at a time, each on its share of the SMs (see paged_shares)
  int32_t vec;             // 16-byte loads of Q, K and V are aligned
  KvDiv by_g;
  float scale, cap, over;  // factor of q.k; 0: no cap; scale / cap
};

// Kernel entry points; each launch takes (PagedParams).
KvSimpleKernel paged_simple_kernel(int dtype, int H, bool few);
const void* paged_combine_kernel(int dtype);

// Up to kPagedFewRows rows a problem, 16-bit T, PagedParams.vec, ps a multiple of 8.
// `few`: up to 8 rows. Launches take (PagedParams, PagedMaps): grid (deal), or (B * Nkv *
// cluster), or (B * Nkv); then, if dealt, join with (PagedParams), grid (deal, rows that
// take a CTA).
struct PagedTokenKernel {
  const void* fn;
  const void* join;
  size_t smem, cluster_smem;  // without clusters, with them
};
constexpr int kPagedFewRows = 16;
constexpr int kPagedTokenThreads = 192;
constexpr int kPagedBox = 64;  // most rows of a box
constexpr int paged_token_ctas(int64_t H) { return 152 * (H > 128 ? 1 : 2); }  // that are resident
PagedTokenKernel paged_token_kernel(int dtype, int H, bool few);

// Any number of rows, the same types, G up to kv_tile_rows(H): items of PagedParams.tpi
// tokens; the launch takes (PagedParams, PagedTileMaps), grid (deal), and is followed by
// join with (PagedParams, kv_tile_rows(H)), grid (kPagedJoinCtas an SM), unless
// PagedParams.entire; or, with more
// than kPagedItems items or no workspace, grid (items * Nkv).
struct PagedTileKernel {
  const void* fn;
  const void* join;
  size_t smem;
};
constexpr int kPagedItems = 768;
constexpr int kPagedTileBlock = 384;
constexpr int kPagedTileCtas = 152;  // most that are dealt to
constexpr int kPagedJoinThreads = 256, kPagedJoinCtas = 2;  // of the join kernel; its CTAs an SM
// The kernel deals its registers out again (setmaxnreg): 256 x 208 + 128 x 88 = 384 x 168,
// so it must have been launched with 168 a thread.
constexpr int kPagedTileRegisters = 168;
static_assert(256 * 208 + 128 * 88 <= kPagedTileBlock * kPagedTileRegisters, "registers of paged_tile_kernel");
PagedTileKernel paged_tile_kernel_f16(int H, int kind);
PagedTileKernel paged_tile_kernel_bf16(int H, int kind);

// Append: Q and K rotation, K and V to their pages.
struct PagedAppendParams {
  PagedBatch s;
  const void* q;           // (T, Nq*H), or packed (T, (Nq + 2 Nkv)*H)
  const void* k;           // (T, Nkv*H), or null when packed
  const void* v;
  const void* cos;         // (cache_rows, h)
  const void* sin;
  const int64_t* pos;      // (T), or null: the row of the cache
  const void* qw;          // RMSNorm weights (H), or null
  const void* kw;
  void* q_out;             // (T, Nq*H)
  void* k_pages;
  void* v_pages;
  int64_t cache_rows, H;
  int32_t Nq, Nkv, packed;
  int32_t h, rd;           // half rotary width, rotary width
  int32_t U, nP;           // units of a head, pair units among them
  int32_t lanes;           // threads that share a head (a power of two <= 32)
  int32_t groups, tokens;  // paged_append_heads_kernel: groups of heads of a token, tokens of a CTA at a time
  float eps, width;        // width: H
};
constexpr int kPagedAppendThreads = 256;
const void* paged_append_kernel(int dtype, bool vec, bool interleaved, bool rms_norm);
// The same on the 128-bit path for heads of at most 32 units, `hpt` heads of one role a
// thread (4 or 2, with the norm 2; null for others); PagedAppendParams.groups, tokens.
const void* paged_append_heads_kernel(int dtype, bool interleaved, bool rms_norm, int hpt);
constexpr int kPagedHeadsThreads = 512;  // of a CTA at most

// Rows past + kept[b, i] of each sequence to past + i.
struct PagedKeepParams {
  PagedBatch s;
  void* k;
  void* v;
  const int32_t* kept;       // (B, width)
  const int32_t* kept_lens;  // (B)
  int32_t width, Nkv;
  int32_t lanes;             // that share a row (a power of two <= 32)
  int64_t units;             // of a row
};
constexpr int kPagedKeepThreads = 256;
const void* paged_keep_kernel(int unit_bytes);

}  // namespace rope_gb300
