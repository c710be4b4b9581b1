// Internal interface between the C-ABI layer of the cache operators (kv_api.cu)
// and their kernels. Not installed; not part of the public ABI.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace rope_gb300 {

// Rows of an 8-bit cache that share a scale (ROPE_KV_SCALE_BLOCK in rope.h).
constexpr int kKvBlock = 16;
// Largest head size of the attention kernels.
constexpr int kKvMaxHead = 256;

// Division of 0 <= n < 2^31 by a constant: (n * m) >> shift.
struct KvDiv {
  uint32_t m;
  int32_t shift;
};

// Attention over a key/value cache. The Nq / Nkv = G query heads of a key/value
// head and the S new tokens of a sequence are the R = S * G rows of one problem
// (b, kvh): row r is token r / G, query head kvh * G + r % G, so its Q and its
// output are H consecutive elements of a (B, S, Nq, H) tensor.
struct KvParams {
  const void* q;           // (B, S, Nq*H)
  const void* k;           // (B, Nkv, max_len, H): T, or e4m3 codes
  const void* v;
  const float* ks;         // (B, Nkv, nblk) scales of the 8-bit caches, or null
  const float* vs;
  void* out;               // (B, S, Nq*H)
  const int32_t* past;     // (B)
  const float* slopes;     // (Nq), or null
  const int32_t* docs;     // (B, max_len), or null
  const int32_t* prefix;   // (B), or null
  int32_t* status;
  float* ws_o;             // partial outputs (B*Nkv, splits, R, H), or (2 * deal, rt, H)
  float2* ws_ml;           // and their (maximum, sum)
  int4* ws_join;           // (deal): the problem that a CTA leaves unfinished
  int64_t S, R, max_len, nblk;
  int32_t B, Nq, Nkv, G, H;
  int32_t splits;
  int32_t tiles, rt;       // kv_token_kernel: tiles of a (b, kvh), rows of a tile
  int32_t deal;            // CTAs that the work is dealt to, or 0: one problem a CTA
  KvDiv by_g, by_tiles;   // kv_token_kernel: by G, tiles
  int32_t vec;             // 16-byte loads of Q, K and V are aligned
  int32_t cluster;         // kv_token_kernel: CTAs of a problem that meet in shared memory (0: see deal)
  int32_t tma;             // kv_tile_kernel: the tensor maps are there
  float scale;             // factor of q.k
  float cap;               // 0: no cap
  float over;              // scale / cap
};

// Kernel entry points for cudaLaunchKernel; each launch takes (KvParams).
struct KvSimpleKernel {
  const void* fn;
  size_t smem;
};
KvSimpleKernel kv_simple_kernel(int dtype, bool fp8, int H, int64_t R);
constexpr int kv_simple_rows(int64_t R) { return R <= 16 ? 16 : 64; }  // of a CTA
// CTAs an SM holds (shared memory; registers)
constexpr int kv_simple_resident(int64_t H, int64_t R) {
  return H <= 64 || (H <= 128 && R <= 16) ? 2 : 1;
}
const void* kv_combine_kernel(int dtype);

// Few rows, 16-bit T, KvParams.vec: 8 rows of a (b, kvh) a CTA, or 16. Both
// launches take (KvParams): fn with grid (deal), or (Nkv * tiles, 1, B); then, if
// dealt, join with grid (deal, rows that take a CTA).
struct KvTokenKernel {
  const void* fn;
  const void* join;
  size_t smem;
};
constexpr int kKvTokenThreads = 128;
constexpr int kKvClusterMost = 8;
constexpr int kKvDealMost = 1024;  // sequences whose units a CTA adds up
// CTAs that the work is dealt to: what is resident on 152 SMs (TokenCfg checks it;
// 16-bit rows above H = 128 take 132 KB of shared memory, one CTA an SM).
constexpr int kv_token_ctas(bool fp8, int64_t H, bool two) {
  return 152 * (H > 128 && !fp8 ? 1 : H > 128 || two ? 2 : fp8 ? 4 : 3);
}
KvTokenKernel kv_token_kernel(int dtype, bool fp8, int H, bool two);

// Many rows, 16-bit T, KvParams.vec: 256 rows of a (b, kvh) a CTA (128 above
// H = 128), grid (Nkv * splits, B, row tiles); the launch takes (KvParams,
// KvTileMaps).
struct KvTileKernel {
  const void* fn;
  size_t smem;
};
constexpr int kKvTileThreads = 512;
// The kernel deals its registers out again (setmaxnreg): 256 x 192 + 128 x 88 +
// 128 x 40 = 512 x 128, so it must have been launched with 128 a thread.
constexpr int kKvTileRegisters = 128;
static_assert(256 * 192 + 128 * 88 + 128 * 40 <= kKvTileThreads * kKvTileRegisters, "registers of kv_tile_kernel");
constexpr int kv_tile_keys(int64_t H) { return H <= 128 ? 128 : 64; }
constexpr int kv_tile_rows(int64_t H) { return H <= 128 ? 256 : 128; }
// What scores may hold besides scale * q.k with scale > 0: nothing; a bias by
// distance; anything (a cap, or a scale <= 0 too).
enum { kKvPlain, kKvBiased, kKvAnyScore };
KvTileKernel kv_tile_kernel_f16(int H, int kind);
KvTileKernel kv_tile_kernel_f16_fp8(int H, int kind);
KvTileKernel kv_tile_kernel_bf16(int H, int kind);
KvTileKernel kv_tile_kernel_bf16_fp8(int H, int kind);

constexpr int kKvSimpleThreads = 256;
constexpr int kKvCombineThreads = 128;
constexpr int kKvCombineWarpSplits = 8;  // up to so many splits a warp joins a row alone, above a CTA

// Q and K rotation with the append to 8-bit caches. Rows, blocks and tokens are
// below 2^31.
struct KvAppendParams {
  const void* q;           // (B, S, Nq*H), or packed (B, S, (Nq + 2 Nkv)*H)
  const void* k;           // (B, S, Nkv*H), or null when packed
  const void* v;
  const void* cos;         // (cache_rows, h)
  const void* sin;
  const int64_t* pos;      // (B, S), or null: past + s
  const int32_t* past;     // (B)
  const void* qw;          // RMSNorm weights (H), or null
  const void* kw;
  void* q_out;             // (B, S, Nq*H)
  uint8_t* k_cache;        // (B, Nkv, max_len, H) e4m3 codes
  uint8_t* v_cache;
  float* k_scale;          // (B, Nkv, nblk)
  float* v_scale;
  int32_t* status;
  int64_t B, S, max_len, nblk, cache_rows;
  int64_t H;
  int32_t Nq, Nkv, packed;
  int32_t h, rd;           // half rotary width, rotary width
  int32_t U, nP;           // units of a row, pair units among them
  int32_t lanes;           // lanes that share a row (a power of two)
  int32_t rows;            // rows of a group (a power of two <= 16)
  int32_t wide;            // the caches take 16-byte accesses
  int64_t blocks;          // most blocks that the S rows of a sequence touch
  int32_t kv_tasks;        // blocks of rows, K and V together
  int32_t kv_ctas;
  int32_t q_groups, q_items;  // groups of heads of a token, and of all tokens
  KvDiv by_q, by_s, by_blocks, by_kv;  // by q_groups, S, blocks, Nkv
  float eps;
};
constexpr int kKvAppendThreads = 256;
constexpr int kKvAppendHeads = 2;  // Q heads of a token that `lanes` threads take
const void* kv_append_kernel(int dtype, bool vec, bool interleaved, bool rms_norm, bool fast);

}  // namespace rope_gb300
