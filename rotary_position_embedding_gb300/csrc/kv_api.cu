// C ABI of the cache operators: rope_apply_qkv_fp8, kv_attention and
// kv_attention_fp8 (include/rope.h). Argument checks, choice of kernel, launch
// geometry. As in rope_api.cu nothing is allocated or kept, nothing waits, and
// every check comes before any CUDA call.
#include "kv_host.h"
#include "kv_maps.h"

using namespace rope_gb300;

static_assert(ROPE_KV_SCALE_BLOCK == kKvBlock, "rope.h and the kernels agree on the rows of a scale");

namespace {

// ---------------------------------------------------------------------------
// Attention
// ---------------------------------------------------------------------------
enum class Family { kSimple, kToken, kTile };

struct Plan {
  int64_t tiles = 0;        // row tiles of a (b, kvh)
  int splits = 1;           // kSimple, kTile: splits of the keys
  int deal = 0;             // kToken: CTAs that the work is dealt to (0: one problem a CTA)
  int cluster = 0;          // kToken: CTAs of a problem, a cluster (0: none)
  int64_t bytes = 0;        // workspace for `splits` or `deal`
  int64_t split_bytes = 0;  // of one split, or of one CTA
};

// CTAs of a cluster that takes one problem of kToken, or 0. Few problems of short
// caches need no second launch that way, as long as all clusters are resident. One
// float16 sequence, 8 key/value heads of 128: 778 keys 7.0 us, dealt out 12.7; 4000
// keys 14.4 against 17.4; but 8000 keys 23.3 against 18.9. In 8 bits 8000 keys 17.8
// against 18.0; 7 such sequences 32.6 against 34.2. 12 sequences of 195 keys, in
// clusters of 4: 7.6 against 11.2.
// The lengths are on the device, so max_len stands for them here and in the plans
// below, whose figures are of caches that are nearly full: 778 keys take 7.2 us in a
// cache of 4096 rows and 13.0 in one of 4097 or 131072.
int token_cluster(bool fp8, int64_t problems, int64_t H, int64_t R, int64_t max_len) {
  if (max_len <= 64 || max_len * (fp8 ? 1 : 2) > 8192) return 0;
  int n = pow2_at_least((max_len + 63) / 64);
  if (n > kKvClusterMost) n = kKvClusterMost;
  return problems * n <= kv_token_ctas(fp8, H, R > 8) ? n : 0;
}

// Row tiles and splits from the sizes alone: the lengths are on the device.
// kSimple and kTile split the keys where the row tiles leave SMs without a CTA;
// kToken deals units of keys to as many CTAs as are resident.
Plan plan_attention(Family family, bool fp8, int64_t B, int64_t S, int64_t Nq, int64_t Nkv, int64_t H, int64_t max_len) {
  Plan pl;
  const int64_t R = S * (Nq / Nkv);
  if (family == Family::kToken) {
    const int rt = R > 8 ? 16 : 8;
    pl.tiles = (R + rt - 1) / rt;
    pl.split_bytes = 2 * rt * (H * 4 + 8) + 16;
    // a (b, kvh) has one tile of up to 16 rows here, or so many tiles that a CTA
    // each is enough
    const int64_t problems = B * Nkv * pl.tiles;
    const int64_t units = (max_len + 63) / 64;
    pl.cluster = token_cluster(fp8, problems, H, R, max_len);
    if (pl.cluster) return pl;
    // Many more problems than CTAs even out by themselves (2048 problems of 1 to 4096
    // keys in 8 bits on 608 places: 225 us one a CTA, 233 us dealt). Between three and
    // six problems a place, one CTA an SM is dealt to twice: 512 problems of 8000
    // 16-bit keys of 256 take 757 us so, 852 one a CTA (of 1 to 8190 keys 455 and 447;
    // dealt to once 751 and 474).
    const int places = kv_token_ctas(fp8, H, rt == 16);
    const int rounds = places == kSms && problems >= 3 * places ? 2 : 1;
    if (problems < 3 * rounds * places && B <= kKvDealMost && max_len > 64 && problems * units < (1ll << 31)) {
      pl.deal = rounds * places;
      if (pl.deal > problems * units) pl.deal = (int)(problems * units);
      pl.bytes = pl.deal * pl.split_bytes + kWorkspaceSlack;
    }
    return pl;
  }
  const int64_t rows = family == Family::kTile ? kv_tile_rows(H) : kv_simple_rows(R);
  pl.tiles = (R + rows - 1) / rows;
  const int64_t ctas = pl.tiles * Nkv * B;
  int64_t n = family == Family::kTile ? kSms / ctas : kv_simple_resident(H, R) * kSms / ctas;
  const int64_t least = family == Family::kTile ? 512 : 128;
  if (n > (max_len + least - 1) / least) n = (max_len + least - 1) / least;
  if (n > 128) n = 128;
  pl.splits = n < 1 ? 1 : (int)n;
  pl.split_bytes = B * Nkv * R * (H * 4 + 8);
  if (pl.splits > 1) pl.bytes = pl.splits * pl.split_bytes + kWorkspaceSlack;
  return pl;
}

// The matrix kernels take 16-bit types whose rows are 16-byte aligned. Up to 16
// rows of a (b, kvh) go to the one for few rows, and more where it has little to
// read or reads codes that the other one has to widen: 20 to 64 rows, one sequence
// of 1000 keys, 8 key/value heads of 128: 11 us against 16 (8 bits: 10 against 18; of
// 8000 keys 27 against 20);
// 32 rows, 8 sequences of 8000 keys in 8 bits 83 us against 131, 48 rows 113 (but one
// such sequence 26 against 20, and in float16 8 of them 118 against 60).
Family choose_family(bool matrix, bool fp8, int64_t B, int64_t S, int64_t G, int64_t Nkv, int64_t H, int64_t max_len) {
  if (!matrix || rope_get_variant() == ROPE_VARIANT_SIMT) return Family::kSimple;
  const int64_t R = S * G;
  const bool grid = B <= 65535 && (R + kv_tile_rows(H) - 1) / kv_tile_rows(H) <= 65535;
  bool few = R <= 16;
  if (!few && R <= 64 && B <= 65535) {  // B * Nkv * max_len stays below 2^62
    const int64_t problems = B * Nkv * ((R + 15) / 16);
    few = (max_len <= 4096 && problems * kKvClusterMost <= kv_token_ctas(fp8, H, true) &&
           token_cluster(fp8, problems, H, R, max_len) > 0) ||
          (fp8 && H <= 128 && R <= 48 && B * Nkv * max_len >= (R <= 32 ? 1 << 18 : 1 << 19));
  }
  if (!few && grid) return Family::kTile;
  return R < ((int64_t)1 << 30) && Nkv * ((R + 7) / 8) <= INT32_MAX ? Family::kToken : Family::kSimple;
}

rope_status check_attention_sizes(int64_t batch, int64_t seq, int32_t num_heads, int32_t kv_num_heads,
                                  int64_t head_size, int64_t max_cache_len) {
  if (batch < 0 || seq < 0) return fail(ROPE_ERR_INVALID_ARG, "batch and seq must be >= 0");
  if (num_heads < 1 || kv_num_heads < 1)
    return fail(ROPE_ERR_INVALID_ARG, "num_heads (%d) and kv_num_heads (%d) must be >= 1", num_heads, kv_num_heads);
  if (num_heads % kv_num_heads)
    return fail(ROPE_ERR_INVALID_ARG, "kv_num_heads %d does not divide num_heads %d", kv_num_heads, num_heads);
  if (head_size < 1) return fail(ROPE_ERR_INVALID_ARG, "head_size must be >= 1");
  if (max_cache_len < 1) return fail(ROPE_ERR_INVALID_ARG, "max_cache_len must be >= 1");
  if (head_size > kKvMaxHead)
    return fail(ROPE_ERR_UNSUPPORTED, "head_size %lld exceeds %d", (long long)head_size, kKvMaxHead);
  if (batch > kMaxLen || seq > kMaxLen || max_cache_len > kMaxLen || kv_num_heads > 65535)
    return fail(ROPE_ERR_UNSUPPORTED, "batch, seq and max_cache_len are limited to 2^30, kv_num_heads to 65535");
  if (!sizes_fit({batch, seq, num_heads, head_size, 1024}) ||
      !sizes_fit({batch, kv_num_heads, max_cache_len, head_size, 8}))
    return fail(ROPE_ERR_INVALID_ARG, "Q has more than 2^52 or the caches more than 2^59 elements");
  return ROPE_OK;
}

rope_status attention_impl(rope_dtype dtype, bool fp8, int64_t batch, int64_t seq, int32_t num_heads,
                           int32_t kv_num_heads, int64_t head_size, const void* query, const void* k_cache,
                           const void* v_cache, const float* k_scale, const float* v_scale,
                           int64_t max_cache_len, const int32_t* past_seq_lens, float scale, float softcap,
                           const float* alibi_slopes, const int32_t* document_ids, const int32_t* prefix_lens,
                           void* out, int32_t* status_flags, void* workspace, int64_t workspace_bytes,
                           rope_stream_t stream) {
  set_last_error("");
  KV_TRY(check_dtype(dtype));
  KV_TRY(check_attention_sizes(batch, seq, num_heads, kv_num_heads, head_size, max_cache_len));
  if (!(std::fabs(scale) <= 0x1p100f)) return fail(ROPE_ERR_INVALID_ARG, "scale must be finite, at most 2^100 in magnitude");
  if (!(softcap >= 0.0f && softcap < INFINITY))
    return fail(ROPE_ERR_INVALID_ARG, "softcap must be finite and >= 0 (0: no cap)");
  if (workspace_bytes < 0) return fail(ROPE_ERR_INVALID_ARG, "workspace_bytes is negative");
  if (batch == 0 || seq == 0) return ROPE_OK;
  const size_t es = dtype == ROPE_F32 ? 4 : 2;
  KV_TRY(check_ptr(query, "query", es));
  KV_TRY(check_ptr(k_cache, "k_cache", fp8 ? 1 : es));
  KV_TRY(check_ptr(v_cache, "v_cache", fp8 ? 1 : es));
  if (fp8) {
    KV_TRY(check_ptr(k_scale, "k_scale", 4));
    KV_TRY(check_ptr(v_scale, "v_scale", 4));
  }
  KV_TRY(check_ptr(past_seq_lens, "past_seq_lens", 4));
  KV_TRY(check_ptr(out, "out", es));
  KV_TRY(check_optional(alibi_slopes, "alibi_slopes", 4));
  KV_TRY(check_optional(document_ids, "document_ids", 4));
  KV_TRY(check_optional(prefix_lens, "prefix_lens", 4));
  KV_TRY(check_optional(status_flags, "status_flags", 4));
  KV_TRY(check_optional(workspace, "workspace", 16));
  if (out == query || out == k_cache || out == v_cache)
    return fail(ROPE_ERR_INVALID_ARG, "out cannot alias query or a cache");

  const bool vec = head_size % (fp8 ? 16 : 16 / es) == 0 && aligned(query, 16) && aligned(k_cache, 16) &&
                   aligned(v_cache, 16) && aligned(out, 16);
  const Family family = choose_family(vec && dtype != ROPE_F32, fp8, batch, seq, num_heads / kv_num_heads,
                                      kv_num_heads, head_size, max_cache_len);
  Plan pl = plan_attention(family, fp8, batch, seq, num_heads, kv_num_heads, head_size, max_cache_len);
  const int64_t fits =
      workspace && workspace_bytes > kWorkspaceSlack ? (workspace_bytes - kWorkspaceSlack) / pl.split_bytes : 0;
  if (pl.splits > fits) pl.splits = fits > 1 ? (int)fits : 1;
  // half of the planned CTAs at least, or each its own problem
  if (pl.deal > fits) pl.deal = fits * 2 >= pl.deal ? (int)fits : 0;

  KvParams p;
  memset(&p, 0, sizeof(p));
  p.q = query;
  p.k = k_cache;
  p.v = v_cache;
  p.ks = k_scale;
  p.vs = v_scale;
  p.out = out;
  p.past = past_seq_lens;
  p.slopes = alibi_slopes;
  p.docs = document_ids;
  p.prefix = prefix_lens;
  p.status = status_flags;
  p.G = num_heads / kv_num_heads;
  p.S = seq;
  p.R = seq * p.G;
  p.max_len = max_cache_len;
  p.nblk = (max_cache_len + kKvBlock - 1) / kKvBlock;
  p.B = (int32_t)batch;
  p.Nq = num_heads;
  p.Nkv = kv_num_heads;
  p.H = (int32_t)head_size;
  p.splits = pl.splits;
  p.tiles = (int32_t)pl.tiles;
  p.rt = p.R > 8 ? 16 : 8;
  p.deal = pl.deal;
  p.cluster = pl.cluster;
  if (family == Family::kToken) {
    p.by_g = div_of(p.G);
    p.by_tiles = div_of(p.tiles);
  }
  if (pl.splits > 1 || pl.deal > 0) {
    const int64_t rows = pl.deal > 0 ? 2 * (int64_t)pl.deal * p.rt : batch * kv_num_heads * pl.splits * p.R;
    p.ws_o = static_cast<float*>(workspace);
    p.ws_ml = reinterpret_cast<float2*>(p.ws_o + rows * head_size + (rows * head_size & 1));
    if (pl.deal > 0) p.ws_join = reinterpret_cast<int4*>(p.ws_ml + rows);  // 16-byte aligned: H and rows are multiples of 8
  }
  p.vec = vec;
  p.scale = scale;
  // A cap above 2^112 is as good as 2^112 (a score below 2^100 is capped by less than
  // 2^-24 of it) and keeps scale / cap a normal number and cap * log2(e) finite. A
  // steepness above 2^125 would be infinite with the kernels' factor, and 0 times it
  // NaN; as |scale| <= 2^100, it comes with a cap, and scores, below 2^-25.
  p.cap = fminf(softcap, 0x1p112f);
  p.over = softcap > 0.0f ? fminf(fmaxf(scale / p.cap, -0x1p125f), 0x1p125f) : 0.0f;

  void* args[] = {&p};
  const int64_t gx = family == Family::kToken ? pl.tiles * kv_num_heads : pl.tiles * pl.splits;
  if (gx > INT32_MAX) return fail(ROPE_ERR_UNSUPPORTED, "more than 2^31 row tiles");
  const dim3 grid((unsigned)gx, kv_num_heads, (unsigned)(batch < 65535 ? batch : 65535));
  if (family == Family::kTile) {
    const int h = (int)head_size;
    const int kind = softcap > 0.0f || !(scale > 0.0f) ? kKvAnyScore : alibi_slopes ? kKvBiased : kKvPlain;
    const KvTileKernel k = dtype == ROPE_F16 ? (fp8 ? kv_tile_kernel_f16_fp8(h, kind) : kv_tile_kernel_f16(h, kind))
                                             : (fp8 ? kv_tile_kernel_bf16_fp8(h, kind) : kv_tile_kernel_bf16(h, kind));
    KvTileMaps maps;
    memset(&maps, 0, sizeof(maps));
    const int64_t planes = batch * kv_num_heads;
    p.tma = !fp8 &&
            encode_kv_map(&maps.k, dtype == ROPE_BF16, k_cache, head_size, max_cache_len, planes, kv_tile_keys(h)) &&
            encode_kv_map(&maps.v, dtype == ROPE_BF16, v_cache, head_size, max_cache_len, planes, kv_tile_keys(h));
    void* targs[] = {&p, &maps};
    const dim3 tg((unsigned)(kv_num_heads * pl.splits), (unsigned)batch, (unsigned)pl.tiles);
    KV_TRY(launch(k.fn, tg, kKvTileThreads, k.smem, stream, targs, "kv_attention launch (many rows)",
                  kKvTileRegisters));
    set_last_kernel("kv_tile_kernel");
  } else if (family == Family::kToken) {
    const KvTokenKernel k = kv_token_kernel(dtype, fp8, (int)head_size, p.rt == 16);
    const dim3 tg = p.deal ? dim3((unsigned)p.deal) : dim3((unsigned)(gx * (p.cluster ? p.cluster : 1)), 1, grid.z);
    KV_TRY(launch(k.fn, tg, kKvTokenThreads, k.smem, stream, args, "kv_attention launch (few rows)", 0, p.cluster));
    if (p.deal) {
      // few problems, each of many parts: a CTA a row
      const unsigned rows = batch * kv_num_heads * pl.tiles * 8 <= p.deal ? (unsigned)(p.R < p.rt ? p.R : p.rt) : 1;
      KV_TRY(launch(k.join, dim3((unsigned)p.deal, rows), kKvTokenThreads, 0, stream, args,
                    "kv_attention launch (joining the parts)"));
    }
    set_last_kernel("kv_token_kernel");
  } else {
    const KvSimpleKernel k = kv_simple_kernel(dtype, fp8, (int)head_size, p.R);
    KV_TRY(launch(k.fn, grid, kKvSimpleThreads, k.smem, stream, args, "kv_attention launch"));
    set_last_kernel("kv_simple_kernel");
  }
  if (pl.splits > 1) {
    const int64_t rows = batch * kv_num_heads * p.R;
    const int per = pl.splits > kKvCombineWarpSplits ? 1 : kKvCombineThreads / 32;
    int64_t gc = (rows + per - 1) / per;
    if (gc > INT32_MAX) gc = INT32_MAX;
    KV_TRY(launch(kv_combine_kernel(dtype), dim3((unsigned)gc), kKvCombineThreads, 0, stream, args,
                  "kv_attention launch (joining the splits)"));
  }
  return ROPE_OK;
}

}  // namespace

extern "C" {

int64_t kv_attention_workspace(int64_t batch, int64_t seq, int32_t num_heads, int32_t kv_num_heads,
                               int64_t head_size, int64_t max_cache_len) {
  set_last_error("");
  if (check_attention_sizes(batch, seq, num_heads, kv_num_heads, head_size, max_cache_len) != ROPE_OK) return -1;
  if (batch == 0 || seq == 0) return 0;
  int64_t most = 0;
  // whichever kernel the types and alignments make the call take
  for (bool fp8 : {false, true})
    for (Family f : {Family::kSimple, choose_family(true, fp8, batch, seq, num_heads / kv_num_heads, kv_num_heads,
                                                    head_size, max_cache_len)}) {
      const Plan pl = plan_attention(f, fp8, batch, seq, num_heads, kv_num_heads, head_size, max_cache_len);
      if (pl.bytes > most) most = pl.bytes;
    }
  return most;
}

rope_status kv_attention(rope_dtype dtype, int64_t batch, int64_t seq, int32_t num_heads, int32_t kv_num_heads,
                         int64_t head_size, const void* query, const void* k_cache, const void* v_cache,
                         int64_t max_cache_len, const int32_t* past_seq_lens, float scale, float softcap,
                         const float* alibi_slopes, const int32_t* document_ids, const int32_t* prefix_lens,
                         void* out, int32_t* status_flags, void* workspace, int64_t workspace_bytes,
                         rope_stream_t stream) {
  return attention_impl(dtype, false, batch, seq, num_heads, kv_num_heads, head_size, query, k_cache, v_cache,
                        nullptr, nullptr, max_cache_len, past_seq_lens, scale, softcap, alibi_slopes, document_ids,
                        prefix_lens, out, status_flags, workspace, workspace_bytes, stream);
}

rope_status kv_attention_fp8(rope_dtype dtype, int64_t batch, int64_t seq, int32_t num_heads,
                             int32_t kv_num_heads, int64_t head_size, const void* query, const void* k_cache,
                             const void* v_cache, const float* k_scale, const float* v_scale,
                             int64_t max_cache_len, const int32_t* past_seq_lens, float scale, float softcap,
                             const float* alibi_slopes, const int32_t* document_ids, const int32_t* prefix_lens,
                             void* out, int32_t* status_flags, void* workspace, int64_t workspace_bytes,
                             rope_stream_t stream) {
  return attention_impl(dtype, true, batch, seq, num_heads, kv_num_heads, head_size, query, k_cache, v_cache,
                        k_scale, v_scale, max_cache_len, past_seq_lens, scale, softcap, alibi_slopes, document_ids,
                        prefix_lens, out, status_flags, workspace, workspace_bytes, stream);
}

rope_status rope_apply_qkv_fp8(rope_dtype dtype, int64_t batch, int64_t seq, int32_t num_heads,
                               int32_t kv_num_heads, int64_t head_size, const void* query, const void* key,
                               const void* value, const void* q_norm_weight, const void* k_norm_weight,
                               float epsilon, const void* cos_cache, const void* sin_cache, int64_t cache_rows,
                               const int64_t* position_ids, const int32_t* past_seq_lens, int32_t interleaved,
                               int32_t rotary_embedding_dim, void* q_out, void* k_cache, void* v_cache,
                               float* k_scale, float* v_scale, int64_t max_cache_len, int32_t* status_flags,
                               rope_stream_t stream) {
  set_last_error("");
  KV_TRY(check_dtype(dtype));
  const bool norm = q_norm_weight || k_norm_weight;
  if (norm && (!q_norm_weight || !k_norm_weight))
    return fail(ROPE_ERR_INVALID_ARG, "RMSNorm needs both q_norm_weight and k_norm_weight");
  if (norm && !(epsilon >= 0.0f && epsilon < INFINITY))
    return fail(ROPE_ERR_INVALID_ARG, "epsilon must be finite and >= 0");
  if (batch < 0 || seq < 0) return fail(ROPE_ERR_INVALID_ARG, "batch and seq must be >= 0");
  if (num_heads < 1 || kv_num_heads < 1)
    return fail(ROPE_ERR_INVALID_ARG, "num_heads (%d) and kv_num_heads (%d) must be >= 1", num_heads, kv_num_heads);
  if (num_heads % kv_num_heads)
    return fail(ROPE_ERR_INVALID_ARG, "kv_num_heads %d does not divide num_heads %d", kv_num_heads, num_heads);
  if (head_size < 2 || head_size % 2) return fail(ROPE_ERR_INVALID_ARG, "head_size must be even and >= 2");
  if (head_size > INT32_MAX / 4) return fail(ROPE_ERR_UNSUPPORTED, "head_size exceeds 2^29");
  if (interleaved != 0 && interleaved != 1)
    return fail(ROPE_ERR_INVALID_ARG, "interleaved must be 0 or 1 (got %d)", interleaved);
  if (cache_rows < 0) return fail(ROPE_ERR_INVALID_ARG, "cache_rows is negative");
  const int64_t rd = rotary_embedding_dim ? rotary_embedding_dim : head_size;
  if (rd < 2 || rd % 2 || rd > head_size)
    return fail(ROPE_ERR_INVALID_ARG, "rotary_embedding_dim %d must be 0 or even, 0 < rd <= head size %lld",
                rotary_embedding_dim, (long long)head_size);
  if (max_cache_len < 1) return fail(ROPE_ERR_INVALID_ARG, "max_cache_len must be >= 1");
  if (max_cache_len > kMaxLen) return fail(ROPE_ERR_UNSUPPORTED, "max_cache_len is limited to 2^30");
  if (!sizes_fit({batch, seq, (int64_t)num_heads + 2 * (int64_t)kv_num_heads, head_size, 8}) ||
      !sizes_fit({batch, kv_num_heads, max_cache_len, head_size, 8}) || !sizes_fit({cache_rows, rd, 8}))
    return fail(ROPE_ERR_INVALID_ARG, "Q/K/V, the caches or the tables have more than 2^59 elements");
  if (batch == 0 || seq == 0) return ROPE_OK;
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
  KV_TRY(check_ptr(k_cache, "k_cache", 1));
  KV_TRY(check_ptr(v_cache, "v_cache", 1));
  KV_TRY(check_ptr(k_scale, "k_scale", 4));
  KV_TRY(check_ptr(v_scale, "v_scale", 4));
  KV_TRY(check_ptr(past_seq_lens, "past_seq_lens", 4));
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

  const int V16 = 16 / (int)es;
  bool vec = head_size % V16 == 0 && (rd / 2) % V16 == 0 && aligned(k_cache, V16) && aligned(v_cache, V16);
  for (const void* x : {query, key, value, (const void*)q_out, cos_cache, sin_cache, q_norm_weight, k_norm_weight})
    vec = vec && aligned(x, 16);
  const int V = vec ? V16 : 1;
  KvAppendParams p;
  memset(&p, 0, sizeof(p));
  p.q = query;
  p.k = key;
  p.v = value;
  p.cos = cos_cache;
  p.sin = sin_cache;
  p.pos = position_ids;
  p.past = past_seq_lens;
  p.qw = q_norm_weight;
  p.kw = k_norm_weight;
  p.q_out = q_out;
  p.k_cache = static_cast<uint8_t*>(k_cache);
  p.v_cache = static_cast<uint8_t*>(v_cache);
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.status = status_flags;
  p.B = batch;
  p.S = seq;
  p.max_len = max_cache_len;
  p.nblk = (max_cache_len + kKvBlock - 1) / kKvBlock;
  p.cache_rows = cache_rows;
  p.H = head_size;
  p.Nq = num_heads;
  p.Nkv = kv_num_heads;
  p.packed = packed;
  p.h = (int32_t)(rd / 2);
  p.rd = (int32_t)rd;
  p.nP = p.h / V;
  p.U = p.nP + (int32_t)((head_size - rd) / V);
  p.eps = epsilon;
  if (norm && p.U > 32)
    return fail(ROPE_ERR_UNSUPPORTED, "RMSNorm: a head has %d units, at most 32 are implemented", p.U);
  p.lanes = p.U >= 32 ? 32 : pow2_at_least(p.U);
  p.rows = pow2_at_least(seq < kKvBlock ? seq : kKvBlock);
  const int rows_wanted = p.rows;
  while (p.lanes * p.rows > kKvAppendThreads) p.rows /= 2;
  const bool fast = p.rows == rows_wanted && p.U <= p.lanes;
  p.wide = head_size % 16 == 0 && aligned(k_cache, 16) && aligned(v_cache, 16);
  p.blocks = (seq + kKvBlock - 2) / kKvBlock + 1;
  // A CTA's first item is within its threads' reach of the last: with these limits
  // the kernel's 32-bit counts do not pass 2^31 (nor does the grid: a CTA takes 8
  // of them at least from Q, and fewer than 2^30 take blocks).
  constexpr int64_t kMostItems = INT32_MAX - kKvAppendThreads;
  p.q_groups = (num_heads + kKvAppendHeads - 1) / kKvAppendHeads;
  const int64_t kv_tasks = sizes_fit({batch, kv_num_heads, p.blocks, 2}) ? batch * kv_num_heads * p.blocks : INT64_MAX;
  const int64_t q_items = batch * seq * p.q_groups;
  if (batch * seq * num_heads > INT32_MAX || q_items > kMostItems || kv_tasks > kMostItems)
    return fail(ROPE_ERR_UNSUPPORTED, "2^31 rows of Q or blocks of the caches, or nearly so many");
  const int per_cta = kKvAppendThreads / (p.lanes * p.rows);
  const int q_per_cta = kKvAppendThreads / p.lanes;
  p.kv_tasks = (int32_t)kv_tasks;
  p.q_items = (int32_t)q_items;
  p.kv_ctas = (p.kv_tasks + per_cta - 1) / per_cta;
  const int64_t grid = p.kv_ctas + ((int64_t)p.q_items + q_per_cta - 1) / q_per_cta;
  p.by_q = div_of(p.q_groups);
  p.by_s = div_of(seq);
  p.by_blocks = div_of(p.blocks);
  p.by_kv = div_of(kv_num_heads);
  void* args[] = {&p};
  KV_TRY(launch(kv_append_kernel(dtype, vec, interleaved != 0, norm, fast), dim3((unsigned)grid), kKvAppendThreads, 0, stream,
                args, "rope_apply_qkv_fp8 launch"));
  set_last_kernel("kv_append_kernel");
  return ROPE_OK;
}

}  // extern "C"
