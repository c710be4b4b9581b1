// C ABI of the operators over paged caches: rope_apply_qkv_paged,
// kv_attention_paged and kv_keep_paged (include/rope.h). Argument checks, choice of
// kernel, launch geometry. Nothing is allocated or kept, nothing waits, and every
// check comes before any CUDA call.
#include <algorithm>

#include "kv_host.h"
#include "paged_internal.h"
#include "paged_maps.h"

using namespace rope_gb300;

namespace {

rope_status check_heads(int64_t batch, int64_t tokens, int32_t num_heads, int32_t kv_num_heads) {
  if (batch < 0 || tokens < 0) return fail(ROPE_ERR_INVALID_ARG, "batch and tokens must be >= 0");
  if (batch > kMaxLen || tokens > kMaxLen) return fail(ROPE_ERR_UNSUPPORTED, "batch and tokens are limited to 2^30");
  if (num_heads < 1 || kv_num_heads < 1)
    return fail(ROPE_ERR_INVALID_ARG, "num_heads (%d) and kv_num_heads (%d) must be >= 1", num_heads, kv_num_heads);
  if (num_heads % kv_num_heads)
    return fail(ROPE_ERR_INVALID_ARG, "kv_num_heads %d does not divide num_heads %d", kv_num_heads, num_heads);
  if (kv_num_heads > 65535) return fail(ROPE_ERR_UNSUPPORTED, "kv_num_heads is limited to 65535");
  return ROPE_OK;
}

rope_status check_table(int64_t batch, int64_t page_size, int64_t max_pages) {
  if (page_size < 1 || max_pages < 1) return fail(ROPE_ERR_INVALID_ARG, "page_size and max_pages must be >= 1");
  if (page_size > kMaxLen || max_pages > kMaxLen || page_size * max_pages > kMaxLen)
    return fail(ROPE_ERR_UNSUPPORTED, "max_pages * page_size is limited to 2^30");
  if (!sizes_fit({batch, max_pages, 4})) return fail(ROPE_ERR_INVALID_ARG, "page_table is too large");
  return ROPE_OK;
}

rope_status check_pages(int32_t kv_num_heads, int64_t head_size, int64_t num_pages, int64_t page_size,
                        int64_t page_stride) {
  if (num_pages < 1) return fail(ROPE_ERR_INVALID_ARG, "num_pages must be >= 1");
  if (num_pages > INT32_MAX) return fail(ROPE_ERR_UNSUPPORTED, "num_pages is limited to 2^31 - 1");
  if (!sizes_fit({kv_num_heads, page_size, head_size}) || page_stride < (int64_t)kv_num_heads * page_size * head_size)
    return fail(ROPE_ERR_INVALID_ARG, "page_stride is below kv_num_heads * page_size * head_size");
  if (!sizes_fit({num_pages, page_stride, 8})) return fail(ROPE_ERR_INVALID_ARG, "the pages have more than 2^59 elements");
  return ROPE_OK;
}

PagedBatch batch_of(int64_t batch, int64_t tokens, const int32_t* past, const int32_t* starts, const int32_t* table,
                    int64_t max_pages, int64_t num_pages, int64_t page_size, int64_t page_stride, int32_t* status) {
  PagedBatch s;
  memset(&s, 0, sizeof(s));
  s.starts = starts;
  s.past = past;
  s.table = table;
  s.status = status;
  s.T = tokens;
  s.S = starts || batch == 0 ? 0 : tokens / batch;
  s.page_stride = page_stride;
  s.rows = max_pages * page_size;
  s.B = (int32_t)batch;
  s.max_pages = (int32_t)max_pages;
  s.pages = (int32_t)num_pages;
  s.ps = (int32_t)page_size;
  s.most = INT32_MAX;
  s.by_ps = div_of(page_size);
  return s;
}

// ---------------------------------------------------------------------------
// Attention
// ---------------------------------------------------------------------------
// In a mixed batch sequences of up to so many rows go to the kernel for few rows: its
// instance for 16 does the arithmetic of 16 for each (95 single tokens of 5 rows beside a
// prompt, capped: 212 us for 139).
constexpr int kMixedRows = 8;

enum class PagedFamily { kSimple, kToken, kTile, kMixed };

struct PagedPlan {
  int64_t tiles = 0;        // kSimple: row tiles of the longest sequence
  bool few = false;         // kSimple: of 16 rows, not 64
  int64_t items = 0;        // kTile: row tiles of all sequences, at most
  int splits = 1;           // kSimple: splits of the keys
  int deal = 0, cluster = 0;  // kToken, kTile: CTAs that are dealt to; kToken: or those of a cluster
  int64_t split_bytes = 0;  // workspace of one split, or of one CTA that is dealt to
  int64_t bytes = 0;
};

// Everything from the sizes alone: the lengths are on the device.

PagedPlan plan_simple(int64_t B, int64_t T, int64_t most, int64_t Nq, int64_t Nkv, int64_t H, int64_t rows) {
  PagedPlan pl;
  const int64_t G = Nq / Nkv, R = most * G;
  // 64 rows a CTA, or 16 where there are no more (16 for more CTAs: 537 float32 tokens of 8
  // heads of 64 53 us instead of 34)
  pl.few = kv_simple_rows(R) == 16;
  const int64_t per = pl.few ? 16 : 64;
  pl.tiles = (R + per - 1) / per;
  int64_t ctas = T * G / per + 1;  // tiles that have rows, at least
  if (ctas < B && B <= T) ctas = B;
  // twice as many as are resident: lengths differ, and a prompt's tiles see half of its keys
  // (float32: 700 tokens 59 -> 51 us, 16 single tokens over up to 2000 keys 201 -> 148)
  int64_t n = 2 * kv_simple_resident(H, pl.few ? 16 : R) * kSms / (ctas * Nkv);
  const int64_t least = pl.few ? 64 : 128;  // keys of a split
  if (n > (rows + least - 1) / least) n = (rows + least - 1) / least;
  if (n > 128) n = 128;
  pl.splits = n < 1 ? 1 : (int)n;
  pl.split_bytes = T * Nq * (H * 4 + 8);
  if (pl.splits > 1) pl.bytes = pl.splits * pl.split_bytes + kWorkspaceSlack;
  return pl;
}

// Few problems of caches that are not long take a cluster of CTAs each, one launch
// instead of two; else units of keys are dealt to as many CTAs as are resident.
PagedPlan plan_token(int64_t B, int64_t most, int64_t Nq, int64_t Nkv, int64_t H, int64_t rows, bool mixed) {
  PagedPlan pl;
  const int64_t R = most * (Nq / Nkv), rt = R > 8 ? 16 : 8;
  const int64_t problems = B * Nkv, units = (rows + 63) / 64;
  pl.split_bytes = 2 * rt * (H * 4 + 8) + 16;
  if (!mixed && units > 1 && rows <= 4096) {
    int n = pow2_at_least(units);
    if (n > kKvClusterMost) n = kKvClusterMost;
    if (problems * n <= kSms) pl.cluster = n;
  }
  if (!pl.cluster && units > 1 && B <= kKvDealMost && problems < (1ll << 30) / (units + 8)) {
    pl.deal = paged_token_ctas(H);
    if (pl.deal > problems * units) pl.deal = (int)(problems * units);
    pl.bytes = pl.deal * pl.split_bytes + kWorkspaceSlack;
  }
  return pl;
}

// One CTA an SM is dealt to, as long as the items fit its tables.
PagedPlan plan_tile(int64_t B, int64_t T, int64_t most, bool ragged, int64_t Nq, int64_t Nkv, int64_t H, int64_t rows) {
  PagedPlan pl;
  const int64_t G = Nq / Nkv, tr = kv_tile_rows(H);
  const int64_t tpi = G < tr ? tr / G : 1, tiles = (most + tpi - 1) / tpi;
  // a sequence has one item more than its tokens fill
  pl.items = B * tiles;
  if (ragged && pl.items > T / tpi + B) pl.items = T / tpi + B;
  pl.split_bytes = 2 * tr * (H * 4 + 8) + 16;
  const int64_t units = (rows + kv_tile_keys(H) - 1) / kv_tile_keys(H);  // of an item
  if (B <= pl.items && pl.items <= kPagedItems && pl.items * Nkv < (1ll << 30) / (units + 8)) {
    pl.deal = kPagedTileCtas;
    if (pl.deal > pl.items * Nkv * units) pl.deal = (int)(pl.items * Nkv * units);
    pl.bytes = pl.deal * pl.split_bytes + kWorkspaceSlack;
  }
  return pl;
}

// The matrix kernels take 16-bit types whose rows are 16-byte aligned, in pages that
// TMA copies in boxes of 8 rows and more. Up to 16 rows of a problem go to the kernel
// for few rows. Where some sequences may have up to kMixedRows and others have more, both
// kernels run, unless the short ones are so few that their CTAs of the kernel for many
// rows fit beside the others', or the tokens are drafts, whose trees are much alike.
PagedFamily choose_paged(bool matrix, int64_t B, int64_t T, int64_t most, bool ragged, bool trees, int64_t G, int64_t Nkv,
                         int64_t H) {
  if (!matrix || rope_get_variant() == ROPE_VARIANT_SIMT) return PagedFamily::kSimple;
  const bool token = B * Nkv <= INT32_MAX / kKvClusterMost;
  if (most * G <= kPagedFewRows) return token ? PagedFamily::kToken : PagedFamily::kSimple;
  const int64_t tr = kv_tile_rows(H);
  if (G > tr || most * G > INT32_MAX || tr * G * Nkv * H > INT32_MAX || (T * G / (tr / 2) + B) * Nkv > INT32_MAX)
    return PagedFamily::kSimple;
  if (!ragged || B == 1 || trees || !token) return PagedFamily::kTile;
  // T <= (B - s) most + s short for s sequences of `short` tokens
  const int64_t shorts = G >= 8 ? 1 : 8 / G;
  const int64_t s = most > shorts ? (B * most - T) / (most - shorts) : B;
  return s * Nkv <= kSms ? PagedFamily::kTile : PagedFamily::kMixed;
}

rope_status check_attention(int64_t batch, int64_t tokens, int64_t max_query_len, int32_t num_heads,
                            int32_t kv_num_heads, int64_t head_size, int64_t page_size, int64_t max_pages) {
  KV_TRY(check_heads(batch, tokens, num_heads, kv_num_heads));
  if (head_size < 1) return fail(ROPE_ERR_INVALID_ARG, "head_size must be >= 1");
  if (head_size > kKvMaxHead)
    return fail(ROPE_ERR_UNSUPPORTED, "head_size %lld exceeds %d", (long long)head_size, kKvMaxHead);
  KV_TRY(check_table(batch, page_size, max_pages));
  if (max_query_len < 0 || max_query_len > tokens)
    return fail(ROPE_ERR_INVALID_ARG, "max_query_len must be within [1, tokens]");
  if (tokens > 0 && batch > 0 && max_query_len < 1)
    return fail(ROPE_ERR_INVALID_ARG, "max_query_len must be within [1, tokens]");
  if (!sizes_fit({tokens, num_heads, head_size, 1024})) return fail(ROPE_ERR_INVALID_ARG, "Q has more than 2^52 elements");
  return ROPE_OK;
}

}  // namespace

extern "C" {

int64_t kv_attention_paged_workspace(rope_dtype dtype, int64_t batch, int64_t tokens, int64_t max_query_len,
                                     int32_t num_heads, int32_t kv_num_heads, int64_t head_size, int64_t page_size,
                                     int64_t max_pages) {
  set_last_error("");
  if (check_dtype(dtype) != ROPE_OK ||
      check_attention(batch, tokens, max_query_len, num_heads, kv_num_heads, head_size, page_size, max_pages) != ROPE_OK)
    return -1;
  if (batch == 0 || tokens == 0) return 0;
  // what the sizes make the call take (tensors that are not 16-byte aligned split less)
  const int64_t rows = page_size * max_pages, G = num_heads / kv_num_heads;
  const bool matrix = dtype != ROPE_F32 && head_size % 8 == 0 && page_size % 8 == 0;
  const bool ragged = batch * max_query_len != tokens;
  const PagedFamily family = choose_paged(matrix, batch, tokens, max_query_len, ragged, false, G, kv_num_heads, head_size);
  if (family == PagedFamily::kSimple)
    return plan_simple(batch, tokens, max_query_len, num_heads, kv_num_heads, head_size, rows).bytes;
  if (family == PagedFamily::kToken) return plan_token(batch, max_query_len, num_heads, kv_num_heads, head_size, rows, false).bytes;
  int64_t n = plan_tile(batch, tokens, max_query_len, ragged, num_heads, kv_num_heads, head_size, rows).bytes;
  if (family == PagedFamily::kMixed && G <= kMixedRows)
    n += plan_token(batch, kMixedRows / G, num_heads, kv_num_heads, head_size, rows, true).bytes;
  return n;
}

rope_status kv_attention_paged(rope_dtype dtype, int64_t batch, int64_t tokens, int64_t max_query_len,
                               int32_t num_heads, int32_t kv_num_heads, int64_t head_size, const void* query,
                               const void* k_pages, const void* v_pages, int64_t num_pages, int64_t page_size,
                               int64_t page_stride, const int32_t* page_table, int64_t max_pages,
                               const int32_t* past_seq_lens, const int32_t* query_starts, float scale, float softcap,
                               int64_t window, const float* alibi_slopes, const int64_t* tree_masks, void* out,
                               int32_t* status_flags, void* workspace, int64_t workspace_bytes, rope_stream_t stream) {
  set_last_error("");
  KV_TRY(check_dtype(dtype));
  if (query_starts && max_query_len > tokens) max_query_len = tokens;  // a server's fixed bound, in a step with fewer
  KV_TRY(check_attention(batch, tokens, max_query_len, num_heads, kv_num_heads, head_size, page_size, max_pages));
  KV_TRY(check_pages(kv_num_heads, head_size, num_pages, page_size, page_stride));
  if (!query_starts && batch * max_query_len != tokens)
    return fail(ROPE_ERR_INVALID_ARG, "without query_starts tokens must be batch * max_query_len");
  if (!(std::fabs(scale) <= 0x1p100f)) return fail(ROPE_ERR_INVALID_ARG, "scale must be finite, at most 2^100 in magnitude");
  if (!(softcap >= 0.0f && softcap < INFINITY))
    return fail(ROPE_ERR_INVALID_ARG, "softcap must be finite and >= 0 (0: no cap)");
  if (window < 0) return fail(ROPE_ERR_INVALID_ARG, "window must be >= 0 (0: none)");
  if (tree_masks && (window > 0 || alibi_slopes))
    return fail(ROPE_ERR_INVALID_ARG, "tree_masks go with neither window nor alibi_slopes");
  if (tree_masks && max_query_len > 64) return fail(ROPE_ERR_INVALID_ARG, "tree_masks: max_query_len is at most 64");
  if (workspace_bytes < 0) return fail(ROPE_ERR_INVALID_ARG, "workspace_bytes is negative");
  if (batch == 0 || tokens == 0) return ROPE_OK;
  const size_t es = dtype == ROPE_F32 ? 4 : 2;
  KV_TRY(check_ptr(query, "query", es));
  KV_TRY(check_ptr(k_pages, "k_pages", es));
  KV_TRY(check_ptr(v_pages, "v_pages", es));
  KV_TRY(check_ptr(page_table, "page_table", 4));
  KV_TRY(check_ptr(past_seq_lens, "past_seq_lens", 4));
  KV_TRY(check_ptr(out, "out", es));
  KV_TRY(check_optional(query_starts, "query_starts", 4));
  KV_TRY(check_optional(alibi_slopes, "alibi_slopes", 4));
  KV_TRY(check_optional(tree_masks, "tree_masks", 8));
  KV_TRY(check_optional(status_flags, "status_flags", 4));
  KV_TRY(check_optional(workspace, "workspace", 16));
  if (out == query || out == k_pages || out == v_pages)
    return fail(ROPE_ERR_INVALID_ARG, "out cannot alias query or the pages");

  PagedParams p;
  memset(&p, 0, sizeof(p));
  p.s = batch_of(batch, tokens, past_seq_lens, query_starts, page_table, max_pages, num_pages, page_size, page_stride,
                 status_flags);
  p.s.most = (int32_t)max_query_len;
  p.q = query;
  p.k = k_pages;
  p.v = v_pages;
  p.out = out;
  p.slopes = alibi_slopes;
  p.masks = tree_masks;
  p.Nq = num_heads;
  p.Nkv = kv_num_heads;
  p.G = num_heads / kv_num_heads;
  p.H = (int32_t)head_size;
  p.window = window > kMaxLen ? 0 : (int32_t)window;
  p.by_g = div_of(p.G);
  const int64_t per16 = 16 / (int64_t)es;
  p.vec = head_size % per16 == 0 && page_stride % per16 == 0 && aligned(query, 16) && aligned(k_pages, 16) &&
          aligned(v_pages, 16) && aligned(out, 16);
  p.scale = scale;
  // as kv_attention: a cap above 2^112 is as good as 2^112, a steepness above 2^125 as that
  p.cap = fminf(softcap, 0x1p112f);
  p.over = softcap > 0.0f ? fminf(fmaxf(scale / p.cap, -0x1p125f), 0x1p125f) : 0.0f;

  const bool ragged = query_starts != nullptr;
  const int64_t rows = p.s.rows;
  const int64_t room = workspace && workspace_bytes > kWorkspaceSlack ? workspace_bytes - kWorkspaceSlack : 0;
  PagedMaps maps;
  memset(&maps, 0, sizeof(maps));
  bool matrix = p.vec && dtype != ROPE_F32 && page_size % 8 == 0;
  PagedFamily family =
      choose_paged(matrix, batch, tokens, max_query_len, ragged, tree_masks != nullptr, p.G, kv_num_heads, head_size);
  if (family != PagedFamily::kSimple) {
    p.chunk = 8;
    while (p.chunk < kPagedBox && page_size % (p.chunk * 2) == 0) p.chunk *= 2;
    if (!encode_paged_map(&maps.k, dtype == ROPE_BF16, k_pages, head_size, page_size, kv_num_heads, num_pages, page_stride, p.chunk) ||
        !encode_paged_map(&maps.v, dtype == ROPE_BF16, v_pages, head_size, page_size, kv_num_heads, num_pages, page_stride, p.chunk))
      family = PagedFamily::kSimple;
  }
  if (family == PagedFamily::kMixed && p.G > kMixedRows) family = PagedFamily::kTile;
  PagedTileMaps tile_maps;
  if (family == PagedFamily::kTile || family == PagedFamily::kMixed) {
    memset(&tile_maps, 0, sizeof(tile_maps));
    const bool bf = dtype == ROPE_BF16;
    p.tpi = kv_tile_rows(head_size) / p.G;
    // in key tiles, which take 1.1 to 1.6 us, capped 2.1 to 2.5: an item (Q, output, a tile
    // or two with hidden keys) 4 to 6 us, joining 8 to 13 us where every SM has parts
    p.over_item = softcap > 0.0f ? 4 : 3;
    p.over_join = softcap > 0.0f ? 5 : 8;
    tile_maps.k = maps.k;
    tile_maps.v = maps.v;
    if (!encode_paged_map(&tile_maps.v_eight, bf, v_pages, head_size, page_size, kv_num_heads, num_pages, page_stride, 8) ||
        !encode_paged_map(&tile_maps.v_row, bf, v_pages, head_size, page_size, kv_num_heads, num_pages, page_stride, 1) ||
        !encode_paged_q_map(&tile_maps.q, bf, query, head_size, num_heads, tokens, p.G, p.tpi))
      family = PagedFamily::kSimple;
  }
  p.mixed = family == PagedFamily::kMixed ? kMixedRows : 0;
  void* args[] = {&p, &maps};
  // Parts in the workspace, `rt` rows each, two a CTA; half of the planned CTAs at least
  // are dealt to, or each takes its own problem.
  auto deal_of = [&](const PagedPlan& pl, int64_t rt, int64_t from) {
    const int64_t fits = (room - from) / pl.split_bytes;
    p.deal = pl.deal <= fits ? pl.deal : fits * 2 >= pl.deal ? (int)fits : 0;
    if (p.deal > 0) {
      const int64_t n = 2 * (int64_t)p.deal * rt;
      p.ws_o = reinterpret_cast<float*>(static_cast<char*>(workspace) + from);
      p.ws_ml = reinterpret_cast<float2*>(p.ws_o + n * head_size);
      p.ws_join = reinterpret_cast<int4*>(p.ws_ml + n);  // 16-byte aligned: n is a multiple of 16
    }
  };
  // The two kernels of a mixed batch run at a time where both are dealt to every SM with a
  // workspace of their own, else one after the other.
  int64_t token_at = 0;  // where paged_token_kernel's begins
  const int64_t token_most = p.mixed ? kMixedRows / p.G : max_query_len;
  if (p.mixed) {
    const PagedPlan tile = plan_tile(batch, tokens, max_query_len, ragged, num_heads, kv_num_heads, head_size, rows);
    const PagedPlan token = plan_token(batch, token_most, num_heads, kv_num_heads, head_size, rows, true);
    p.shared = tile.deal == kSms && token.deal == paged_token_ctas(head_size) && tile.bytes + token.bytes <= room + kWorkspaceSlack;
    if (p.shared) token_at = tile.bytes;
  }
  if (family == PagedFamily::kSimple) {
    const PagedPlan pl = plan_simple(batch, tokens, max_query_len, num_heads, kv_num_heads, head_size, rows);
    if (pl.tiles * pl.splits > INT32_MAX) return fail(ROPE_ERR_UNSUPPORTED, "more than 2^31 row tiles");
    const int64_t fits = room / pl.split_bytes;
    p.splits = pl.splits <= fits ? pl.splits : fits > 1 ? (int)fits : 1;
    p.tiles = (int32_t)pl.tiles;
    if (p.splits > 1) {
      const int64_t n = p.splits * tokens * num_heads;
      p.ws_o = static_cast<float*>(workspace);
      p.ws_ml = reinterpret_cast<float2*>(p.ws_o + n * head_size + (n * head_size & 1));
    }
    const KvSimpleKernel k = paged_simple_kernel(dtype, (int)head_size, pl.few);
    const dim3 grid((unsigned)(pl.tiles * p.splits), kv_num_heads, (unsigned)(batch < 65535 ? batch : 65535));
    KV_TRY(launch(k.fn, grid, kKvSimpleThreads, k.smem, stream, args, "kv_attention_paged launch"));
    if (p.splits > 1) {
      const int64_t n = tokens * num_heads;
      const int per = p.splits > kKvCombineWarpSplits ? 1 : kKvCombineThreads / 32;
      int64_t gc = (n + per - 1) / per;
      if (gc > INT32_MAX) gc = INT32_MAX;
      KV_TRY(launch(paged_combine_kernel(dtype), dim3((unsigned)gc), kKvCombineThreads, 0, stream, args,
                    "kv_attention_paged launch (joining the splits)"));
    }
    set_last_kernel("paged_simple_kernel");
    return ROPE_OK;
  }
  PagedParams tile_p = p;
  const void* tile_join = nullptr;
  auto join_tiles = [&]() -> rope_status {
    if (!tile_p.deal || tile_p.entire) return ROPE_OK;
    int tr = kv_tile_rows(head_size);
    void* jargs[] = {&tile_p, &tr};
    return launch(tile_join, dim3(kSms * kPagedJoinCtas), kPagedJoinThreads, 0, stream, jargs,
                  "kv_attention_paged launch (joining the parts)");
  };
  if (family != PagedFamily::kToken) {
    const PagedPlan pl = plan_tile(batch, tokens, max_query_len, ragged, num_heads, kv_num_heads, head_size, rows);
    const int kind = softcap > 0.0f || !(scale > 0.0f) ? kKvAnyScore : alibi_slopes ? kKvBiased : kKvPlain;
    const PagedTileKernel k =
        dtype == ROPE_F16 ? paged_tile_kernel_f16((int)head_size, kind) : paged_tile_kernel_bf16((int)head_size, kind);
    // Ranges that end at whole items differ by the longest item at most. Where that weighs
    // little more than joining is worth nothing is ever split: no workspace, and one launch
    // less (5 prompts that see 512 keys 36.9 -> 34.8 us, 7 trees over up to 300 keys 17.6 ->
    // 15.9; with 5 more in place of 3 no more gained).
    const int64_t keys = kv_tile_keys(head_size);
    int64_t units = (rows + keys - 1) / keys;
    if (window > 0 && window <= kMaxLen) units = std::min(units, (window + p.tpi - 2) / keys + 2);
    p.entire = pl.deal && !p.shared && units + p.over_item < p.over_join + 3;
    if (p.entire)
      p.deal = pl.deal;
    else
      deal_of(pl, kv_tile_rows(head_size), 0);
    p.items = p.deal ? (int32_t)pl.items : 0;
    void* targs[] = {&p, &tile_maps};
    KV_TRY(launch(k.fn, dim3((unsigned)(p.deal ? p.deal : pl.items * kv_num_heads)), kPagedTileBlock, k.smem, stream, targs,
                  "kv_attention_paged launch (many rows)", kPagedTileRegisters));
    tile_p = p;
    tile_join = k.join;
    if (!p.shared) KV_TRY(join_tiles());
    set_last_kernel("paged_tile_kernel");
  }
  if (family != PagedFamily::kTile) {
    const PagedPlan pl = plan_token(batch, token_most, num_heads, kv_num_heads, head_size, rows, p.mixed != 0);
    p.rt = token_most * p.G > 8 ? 16 : 8;
    p.cluster = pl.cluster;
    deal_of(pl, p.rt, token_at);
    const PagedTokenKernel k = paged_token_kernel(dtype, (int)head_size, p.rt == 8);
    const int64_t grid = p.deal ? p.deal : batch * kv_num_heads * (p.cluster ? p.cluster : 1);
    KV_TRY(launch(k.fn, dim3((unsigned)grid), kPagedTokenThreads, p.cluster ? k.cluster_smem : k.smem, stream, args,
                  "kv_attention_paged launch (few rows)", 0, p.cluster));
    if (p.shared) KV_TRY(join_tiles());
    if (p.deal) {
      // few problems, each of many parts: a CTA a row
      const unsigned n = batch * kv_num_heads * 8 <= p.deal ? (unsigned)p.rt : 1;
      KV_TRY(launch(k.join, dim3((unsigned)p.deal, n), kKvTokenThreads, 0, stream, args,
                    "kv_attention_paged launch (joining the parts)"));
    }
    set_last_kernel("paged_token_kernel");
  }
  return ROPE_OK;
}

rope_status rope_apply_qkv_paged(rope_dtype dtype, int64_t batch, int64_t tokens, int32_t num_heads,
                                 int32_t kv_num_heads, int64_t head_size, const void* query, const void* key,
                                 const void* value, const void* q_norm_weight, const void* k_norm_weight,
                                 float epsilon, const void* cos_cache, const void* sin_cache, int64_t cache_rows,
                                 const int64_t* position_ids, const int32_t* past_seq_lens,
                                 const int32_t* query_starts, const int32_t* page_table, int64_t max_pages,
                                 int32_t interleaved, int32_t rotary_embedding_dim, void* q_out, void* k_pages,
                                 void* v_pages, int64_t num_pages, int64_t page_size, int64_t page_stride,
                                 int32_t* status_flags, rope_stream_t stream) {
  set_last_error("");
  KV_TRY(check_dtype(dtype));
  const bool norm = q_norm_weight || k_norm_weight;
  if (norm && (!q_norm_weight || !k_norm_weight))
    return fail(ROPE_ERR_INVALID_ARG, "RMSNorm needs both q_norm_weight and k_norm_weight");
  if (norm && !(epsilon >= 0.0f && epsilon < INFINITY))
    return fail(ROPE_ERR_INVALID_ARG, "epsilon must be finite and >= 0");
  KV_TRY(check_heads(batch, tokens, num_heads, kv_num_heads));
  if (head_size < 2 || head_size % 2) return fail(ROPE_ERR_INVALID_ARG, "head_size must be even and >= 2");
  if (head_size > INT32_MAX / 4) return fail(ROPE_ERR_UNSUPPORTED, "head_size exceeds 2^29");
  if (num_heads > INT32_MAX / 4) return fail(ROPE_ERR_UNSUPPORTED, "num_heads exceeds 2^29");
  if (interleaved != 0 && interleaved != 1)
    return fail(ROPE_ERR_INVALID_ARG, "interleaved must be 0 or 1 (got %d)", interleaved);
  if (cache_rows < 0) return fail(ROPE_ERR_INVALID_ARG, "cache_rows is negative");
  const int64_t rd = rotary_embedding_dim ? rotary_embedding_dim : head_size;
  if (rd < 2 || rd % 2 || rd > head_size)
    return fail(ROPE_ERR_INVALID_ARG, "rotary_embedding_dim %d must be 0 or even, 0 < rd <= head size %lld",
                rotary_embedding_dim, (long long)head_size);
  KV_TRY(check_table(batch, page_size, max_pages));
  KV_TRY(check_pages(kv_num_heads, head_size, num_pages, page_size, page_stride));
  if (!query_starts && batch > 0 && tokens % batch)
    return fail(ROPE_ERR_INVALID_ARG, "without query_starts batch must divide tokens");
  const int64_t heads = (int64_t)num_heads + 2 * (int64_t)kv_num_heads;
  if (!sizes_fit({tokens, heads, head_size, 8}) || !sizes_fit({cache_rows, rd, 8}))
    return fail(ROPE_ERR_INVALID_ARG, "Q/K/V or the tables have more than 2^59 elements");
  if (batch == 0 || tokens == 0) return ROPE_OK;
  const bool packed = !key && !value;
  if (!packed && (!key || !value)) return fail(ROPE_ERR_INVALID_ARG, "key and value come together (or packed in query)");
  const size_t es = dtype == ROPE_F32 ? 4 : 2;
  KV_TRY(check_ptr(query, "query", es));
  if (!packed) {
    KV_TRY(check_ptr(key, "key", es));
    KV_TRY(check_ptr(value, "value", es));
  }
  KV_TRY(check_ptr(q_out, "q_out", es));
  if (packed && q_out == query)
    return fail(ROPE_ERR_INVALID_ARG, "q_out cannot alias a packed query (different row strides)");
  KV_TRY(check_ptr(k_pages, "k_pages", es));
  KV_TRY(check_ptr(v_pages, "v_pages", es));
  if (k_pages == v_pages || k_pages == q_out || v_pages == q_out)
    return fail(ROPE_ERR_INVALID_ARG, "q_out, k_pages and v_pages cannot alias");
  KV_TRY(check_ptr(page_table, "page_table", 4));
  KV_TRY(check_ptr(past_seq_lens, "past_seq_lens", 4));
  KV_TRY(check_optional(query_starts, "query_starts", 4));
  if (cache_rows > 0) {
    KV_TRY(check_ptr(cos_cache, "cos_cache", es));
    KV_TRY(check_ptr(sin_cache, "sin_cache", es));
  }
  KV_TRY(check_optional(position_ids, "position_ids", 8));
  KV_TRY(check_optional(status_flags, "status_flags", 4));
  if (norm) {
    KV_TRY(check_ptr(q_norm_weight, "q_norm_weight", es));
    KV_TRY(check_ptr(k_norm_weight, "k_norm_weight", es));
  }

  const int64_t V16 = 16 / (int64_t)es;
  bool vec = head_size % V16 == 0 && (rd / 2) % V16 == 0 && page_stride % V16 == 0;
  for (const void* x : {query, key, value, (const void*)q_out, (const void*)k_pages, (const void*)v_pages, cos_cache,
                        sin_cache, q_norm_weight, k_norm_weight})
    vec = vec && aligned(x, 16);
  const int64_t V = vec ? V16 : 1;
  PagedAppendParams p;
  memset(&p, 0, sizeof(p));
  p.s = batch_of(batch, tokens, past_seq_lens, query_starts, page_table, max_pages, num_pages, page_size, page_stride,
                 status_flags);
  p.q = query;
  p.k = key;
  p.v = value;
  p.cos = cos_cache;
  p.sin = sin_cache;
  p.pos = position_ids;
  p.qw = q_norm_weight;
  p.kw = k_norm_weight;
  p.q_out = q_out;
  p.k_pages = k_pages;
  p.v_pages = v_pages;
  p.cache_rows = cache_rows;
  p.H = head_size;
  p.Nq = num_heads;
  p.Nkv = kv_num_heads;
  p.packed = packed;
  p.h = (int32_t)(rd / 2);
  p.rd = (int32_t)rd;
  p.nP = (int32_t)(p.h / V);
  p.U = p.nP + (int32_t)((head_size - rd) / V);
  p.lanes = p.U >= 32 ? 32 : pow2_at_least(p.U);
  p.eps = epsilon;
  p.width = (float)head_size;
  void* args[] = {&p};
  // Several heads of one role a thread where a token's threads fit a CTA: 4 on 16-bit
  // data from 4096 tokens on, else 2 (more, smaller CTAs), as rope_apply_qkv.
  const bool whole_groups = !norm || p.U == p.lanes;  // a head's sum is taken by U lanes side by side
  const int hpt = norm || es == 4 || tokens < 4096 ? 2 : 4;
  const int64_t groups = (num_heads + hpt - 1) / hpt + 2 * ((kv_num_heads + hpt - 1) / hpt);
  if (vec && p.U <= 32 && whole_groups && groups * p.U <= kPagedHeadsThreads) {
    const int per_tok = (int)groups * p.U;
    p.groups = (int32_t)groups;
    p.tokens = per_tok >= 256 ? 1 : 256 / per_tok;
    const int threads = (p.tokens * per_tok + 31) / 32 * 32;
    const void* fn = paged_append_heads_kernel(dtype, interleaved != 0, norm, hpt);
    int resident = 0;
    KV_TRY(resident_ctas(fn, threads, &resident));
    int64_t n = (tokens + p.tokens - 1) / p.tokens;
    if (n > resident * kSms) n = resident * kSms;  // one wave: a thread goes from token to token
    KV_TRY(launch(fn, dim3((unsigned)n), threads, 0, stream, args, "rope_apply_qkv_paged launch"));
    set_last_kernel("paged_append_heads_kernel");
    return ROPE_OK;
  }
  const int64_t per = kPagedAppendThreads / p.lanes;
  int64_t grid = (tokens * heads + per - 1) / per;
  if (grid > INT32_MAX) grid = INT32_MAX;
  KV_TRY(launch(paged_append_kernel(dtype, vec, interleaved != 0, norm), dim3((unsigned)grid), kPagedAppendThreads, 0,
                stream, args, "rope_apply_qkv_paged launch"));
  set_last_kernel("paged_append_kernel");
  return ROPE_OK;
}

rope_status kv_keep_paged(rope_dtype dtype, int64_t batch, int32_t kv_num_heads, int64_t head_size, void* k_pages,
                          void* v_pages, int64_t num_pages, int64_t page_size, int64_t page_stride,
                          const int32_t* page_table, int64_t max_pages, const int32_t* past_seq_lens,
                          const int32_t* kept, int64_t max_kept, const int32_t* kept_lens, int32_t* status_flags,
                          rope_stream_t stream) {
  set_last_error("");
  KV_TRY(check_dtype(dtype));
  KV_TRY(check_heads(batch, 0, kv_num_heads, kv_num_heads));
  if (head_size < 1) return fail(ROPE_ERR_INVALID_ARG, "head_size must be >= 1");
  KV_TRY(check_table(batch, page_size, max_pages));
  KV_TRY(check_pages(kv_num_heads, head_size, num_pages, page_size, page_stride));
  if (max_kept < 0) return fail(ROPE_ERR_INVALID_ARG, "max_kept must be >= 0");
  if (head_size > INT32_MAX / 4 || max_kept > 1 << 20 || !sizes_fit({batch, kv_num_heads, head_size, 1 << 22}))
    return fail(ROPE_ERR_UNSUPPORTED, "batch * kv_num_heads * head_size is limited to 2^40, max_kept to 2^20");
  if (batch == 0 || max_kept == 0) return ROPE_OK;
  const size_t es = dtype == ROPE_F32 ? 4 : 2;
  KV_TRY(check_ptr(k_pages, "k_pages", es));
  KV_TRY(check_ptr(v_pages, "v_pages", es));
  if (k_pages == v_pages) return fail(ROPE_ERR_INVALID_ARG, "k_pages and v_pages are the same");
  KV_TRY(check_ptr(page_table, "page_table", 4));
  KV_TRY(check_ptr(past_seq_lens, "past_seq_lens", 4));
  KV_TRY(check_ptr(kept, "kept", 4));
  KV_TRY(check_ptr(kept_lens, "kept_lens", 4));
  KV_TRY(check_optional(status_flags, "status_flags", 4));

  const int64_t per16 = 16 / (int64_t)es;
  const bool vec = head_size % per16 == 0 && page_stride % per16 == 0 && aligned(k_pages, 16) && aligned(v_pages, 16);
  const int64_t V = vec ? per16 : 1;
  PagedKeepParams p;
  memset(&p, 0, sizeof(p));
  p.s = batch_of(batch, 0, past_seq_lens, nullptr, page_table, max_pages, num_pages, page_size, page_stride / V,
                 status_flags);
  p.k = k_pages;
  p.v = v_pages;
  p.kept = kept;
  p.kept_lens = kept_lens;
  p.width = (int32_t)max_kept;
  p.Nkv = kv_num_heads;
  p.units = head_size / V;
  p.lanes = p.units >= 32 ? 32 : pow2_at_least(p.units);
  int64_t grid = (batch * 2 * kv_num_heads + kPagedKeepThreads / 32 - 1) / (kPagedKeepThreads / 32);
  if (grid > INT32_MAX) grid = INT32_MAX;
  void* args[] = {&p};
  KV_TRY(launch(paged_keep_kernel(vec ? 16 : (int)es), dim3((unsigned)grid), kPagedKeepThreads, 0, stream, args,
                "kv_keep_paged launch"));
  set_last_kernel("paged_keep_kernel");
  return ROPE_OK;
}

}  // extern "C"
