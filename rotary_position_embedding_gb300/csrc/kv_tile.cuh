// Attention over a key/value cache for many rows (prompts, chunks): tcgen05.
//
// R = S * G rows of a (b, kvh) (token-major, so the G query heads that share K
// and V sit in one tile), 16-bit T. A CTA takes NT tiles of 128 rows and walks
// the keys in tiles of N; per row tile and key tile
//   S = Q K^T   (128 x N, accumulated in TMEM),
//   P = 2^(x - m) of the scores x (registers), back to TMEM as 16-bit values,
//   O += P V    (A from TMEM, accumulated in TMEM).
// Bound by the tensor cores: 4 H flops a pair of row and key, 1024 clocks a
// row tile and key tile at H = 128, against which the 128 x 128 exponentials and
// what surrounds them have to be hidden. So with NT = 2 the two row tiles take
// turns: while one tile's scores are in registers, the tensor cores work for
// the other. H = 256 fills TMEM with one tile: NT = 1, N = 64, S double-buffered.
//
// Warps (16): 0-3 and 4-7 softmax of row tile 0 and 1, a thread a row (they
// bring Q to shared memory first); 8-11 bring K and V; 12 (one lane) issues
// every MMA; 13-15 only give up their registers.
//   K and V tiles come by TMA; the last one, whose rows behind the keys have to
//   be zeros, by cp.async.
//   8-bit caches: the bringing warps load codes and write float16 (exact); the
//   key scale of each 16 keys multiplies scores, the value scale weights,
//   relative to the largest value scale that the row has seen so far (powers of
//   two); bfloat16 Q rows become float16 after scaling by a power of two that the
//   scores undo. A block of 16 keys none of which a row sees has no part in that
//   row's reference, whatever its scale: the weights there are 0.
// A softmax thread holds its 128 scores in registers from one TMEM load on
// (32 at a time, read twice, the loads' latency was two thirds of a step: 3.3 us
// a step of both row tiles): hence 192 registers a softmax thread, 88 a bringing
// one, 40 a thread of the MMA warps. Where no bias is added, nothing is hidden and
// all of a warp's capped scores have |y| <= 0.4, tanh(y) is a polynomial: 3
// exponential-unit operations a score become one. Scores stay raw there, and the
// maximum is taken before the cap.
// Measured, a step of 128 keys and both row tiles at H = 128: 1.58 us (its MMAs
// alone 1.22), biased 2.00, capped 2.53, over 8-bit caches 2.29, those capped 3.29;
// 1.40 at H = 64, 0.95 for 64 keys and one row tile at H = 256. 4 x 2048 float16
// tokens over up to 4095 keys, 32/8 heads, capped: 405 us, 0.36 of the measured
// bfloat16 rate. Head sizes between run padded: 2 x 2048 bfloat16 tokens over up to
// 4096 keys, 32/8 heads of 64 135 us, 80 148, 96 153, 112 156, 128 161, 160 332, 192
// 339, 256 353.
// Shared memory: Q, two stages of K and two of V, each as slabs of 64 elements
// (128-byte rows, 128-byte swizzle): the K-major form for Q and K, and the same
// bytes read MN-major for V.
// TMEM (512 columns): S (P over its first half), O at 256.
//
// Barriers: k_full, v_full (the bringing threads) and k_free, v_free (commits)
// for each stage; s_full (commit) and p_full (128 threads) for each S buffer;
// o_full at the end; info (documents and scales of a key tile, four slots). A
// commit covers every MMA issued before it, so s_full of step j also says that
// P V of step j - 1 of that row tile is complete: O may be rescaled then. MMAs
// of a CTA run in the order of issue, so S of the next step may overwrite the P
// that P V has yet to read.
// Every wait is bounded (2 s); one that runs out sets status bit 1, and the warp
// goes to the common end, where TMEM is freed.
//
// The base of a row's weights is the maximum when it was last moved, and moves
// only where a tile's sum of weights passes 2^15: no maximum is taken otherwise
// (half of the arithmetic that plain scores need). O is rescaled by its softmax
// threads then, seldom after the first tile, so there is no correction warp. Keys
// go from the last to the first: a bias by distance then only falls. The last key
// tile's rows behind the keys are zeros. Key tiles whose documents no row of the
// CTA can have are left out.
#pragma once

#include "kv_careful.cuh"
#include "kv_maps.h"
#include "kv_token.cuh"
#include "rope_tma.cuh"

namespace rope_gb300 {

constexpr int kTileThreads = kKvTileThreads;
constexpr int kTileRows = 128;
constexpr int kTileBring = 128;        // bringing threads
constexpr int kTileListed = 4096;      // key tiles of a CTA whose documents are looked at

template <bool FP8, int HD>
struct TileCfg {
  static constexpr int NT = HD <= 128 ? 2 : 1;
  static constexpr int N = HD <= 128 ? 128 : 64;
  static constexpr int SLABS = HD / 64;
  static constexpr int kQ = NT * kTileRows * HD * 2;
  static constexpr int kStage = N * HD * 2;  // of K, and of V
  static constexpr int kInfo = N * 4 + 128;  // documents, N/16 key scales, N/16 value scales
  static constexpr int kTail = 4 * kInfo + 2 * kTileListed / 8 + NT * kTileRows * 4 + 256;
  static constexpr int kSmem = 1024 + kQ + 4 * kStage + kTail;
};

struct TileBars {
  uint64_t k_full[2], k_free[2], v_full[2], v_free[2], s_full[2], p_full[2], o_full[2], info[4], q_full, drain;
};

__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tc_fence_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// One lane of a converged warp, always the same one.
__device__ __forceinline__ bool tc_elect() {
  uint32_t on;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(on));
  return on != 0;
}

// Matrix descriptor of a 128-byte-swizzled operand: the low word holds the
// shared address and the distance `lead` between 64-element slabs (read
// MN-major; ignored K-major), both / 16, the high word that groups of 8 rows are
// 1024 bytes apart, the version and the swizzle. Only the low word changes.
__device__ __forceinline__ uint32_t tc_desc(uint32_t a, uint32_t lead) { return ((a & 0x3ffffu) >> 4) | (lead >> 4) << 16; }
constexpr uint32_t kDescHigh = (1024 >> 4) | 1u << 14 | 2u << 29;

// D (TMEM) (+)= A (shared memory) B (shared memory); low words of descriptors
__device__ __forceinline__ void tc_mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "mov.b64 x, {%1, %5};\n\tmov.b64 y, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(add), "n"(kDescHigh)
      : "memory");
}
// D (TMEM) (+)= A (TMEM) B (shared memory)
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 y;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "mov.b64 y, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(add), "n"(kDescHigh)
      : "memory");
}

// Instruction descriptor: float32 accumulator, 16-bit operands, M = 128.
__device__ __forceinline__ uint32_t tc_idesc(bool bf16, int n, bool b_mn_major) {
  return 1u << 4 | (bf16 ? 1u << 7 | 1u << 10 : 0u) | (b_mn_major ? 1u << 16 : 0u) | (uint32_t)(n >> 3) << 17 |
         (uint32_t)(128 >> 4) << 24;
}

#define KV_R8(a, i) "=r"(a[i]), "=r"(a[i + 1]), "=r"(a[i + 2]), "=r"(a[i + 3]), "=r"(a[i + 4]), "=r"(a[i + 5]), "=r"(a[i + 6]), "=r"(a[i + 7])
#define KV_W8(a, i) "r"(a[i]), "r"(a[i + 1]), "r"(a[i + 2]), "r"(a[i + 3]), "r"(a[i + 4]), "r"(a[i + 5]), "r"(a[i + 6]), "r"(a[i + 7])

// 32 columns of this thread's TMEM lane (not complete before tc_wait_ld).
__device__ __forceinline__ void tc_ld32(uint32_t* r, uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : KV_R8(r, 0), KV_R8(r, 8), KV_R8(r, 16), KV_R8(r, 24)
      : "r"(addr));
}
__device__ __forceinline__ void tc_st32(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,"
      "%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::KV_W8(r, 0),
      KV_W8(r, 8), KV_W8(r, 16), KV_W8(r, 24), "r"(addr)
      : "memory");
}
// Waits for this thread's loads; the registers pass through, so that no use of
// them moves ahead of the wait.
#define KV_RW8(a, i) "+r"(a[i]), "+r"(a[i + 1]), "+r"(a[i + 2]), "+r"(a[i + 3]), "+r"(a[i + 4]), "+r"(a[i + 5]), "+r"(a[i + 6]), "+r"(a[i + 7])
__device__ __forceinline__ void tc_wait_ld32(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" : KV_RW8(r, 0), KV_RW8(r, 8), KV_RW8(r, 16), KV_RW8(r, 24)::"memory");
}
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 16 columns, waited for; and back.
__device__ __forceinline__ void tc_ld16(uint32_t* r, uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : KV_R8(r, 0), KV_R8(r, 8)
      : "r"(addr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" : KV_RW8(r, 0), KV_RW8(r, 8)::"memory");
}
__device__ __forceinline__ void tc_st16(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::KV_W8(r, 0),
      KV_W8(r, 8), "r"(addr)
      : "memory");
}

// Byte offset of 16-byte piece `piece` (8 elements) of row `row` in an operand
// of `rows` rows: slabs of 8 pieces, swizzled by the row.
__device__ __forceinline__ uint32_t tile_at(int rows, int row, int piece) {
  return (uint32_t)((piece >> 3) * rows * 128 + row * 128 + (((piece & 7) ^ (row & 7)) << 4));
}

// The key tiles of a CTA, from the last to the first: all of [0, count), or
// those that `need` names and those behind what it can name.
struct TileList {
  const uint32_t* need;
  int count;
  bool listed;
  __device__ __forceinline__ int next(int t) const {  // the one before t (count: the last), or -1
    --t;
    if (!listed) return t;
    while (t >= 0 && t < kTileListed) {
      const uint32_t w = need[t >> 5] << (31 - (t & 31));
      if (w) return t - __clz(w);
      t = (t & ~31) - 1;
    }
    return t;
  }
};

__device__ __forceinline__ void tile_tma(uint32_t dst, const CUtensorMap* map, int x, int row, int plane, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::
          "r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(row), "r"(plane), "r"(bar)
      : "memory");
}

// What a softmax thread knows of its row, and the tile it is at.
struct TileRow {
  float unit;                   // of a bfloat16 Q row over 8-bit keys, see kv_row_shift
  float mult, slope, cap2;      // score factor; bias and cap in log2
  bool ahead;                   // some key of the tile is ahead of some row of the warp
  float dist;                   // the row's position less the tile's first key
  int limit;                    // columns of the tile below this are not ahead of it
  int doc;
  bool part, look;              // some column is hidden: by position, by document
  const int4* docs;             // of the tile
  const float* ks;              // of each 16 columns
};

// N raw scores of a row from TMEM; over 8-bit caches times what the codes of each 16
// columns and the query row stand for.
template <bool FP8, int N>
__device__ __forceinline__ void tile_load(float (&x)[N], uint32_t ts, const TileRow& r, bool raw) {
  uint32_t c[N];
#pragma unroll
  for (int i = 0; i < N; i += 32) tc_ld32(c + i, ts + i);
#pragma unroll
  for (int i = 0; i < N; i += 32) tc_wait_ld32(c + i);
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = __uint_as_float(c[i]);
  if (FP8 && raw) {
#pragma unroll
    for (int h = 0; h < N / 16; ++h) {
      // to q.k first: queries may be as small as keys are large
      const float f = fminf(r.ks[h] * r.unit, FLT_MAX);
#pragma unroll
      for (int k = 16 * h; k < 16 * h + 16; k += 2) {
        const float2 y = __fmul2_rn(make_float2(x[k], x[k + 1]), make_float2(f, f));
        x[k] = y.x, x[k + 1] = y.y;
      }
    }
  }
}

// Whether all of a warp's raw scores have |y| <= 0.4: then the cap is a polynomial.
// The bounds of mult keep the polynomial's powers normal numbers.
template <int N>
__device__ __forceinline__ bool tile_small(const float (&x)[N], const TileRow& r) {
  float a0 = 0.0f, a1 = 0.0f;
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    a0 = fmaxf(a0, fmaxf(fabsf(x[i]), fabsf(x[i + 1])));
    a1 = fmaxf(a1, fmaxf(fabsf(x[i + 2]), fabsf(x[i + 3])));
  }
  return __all_sync(0xffffffffu, fmaxf(a0, a1) * r.mult <= 2.0f * kTanhEnd * kLog2e && r.mult > 1e-5f && r.mult < 1e4f);
}

// Other scores, and those of tiles with hidden keys, are capped where they lie in
// TMEM, 32 columns at a time: in registers, code for N columns that is seldom reached
// cost the common path 10 % of 8-bit capped prompts.
template <bool FP8, int N>
__device__ __forceinline__ void tile_cap(uint32_t ts, const TileRow& r) {
#pragma unroll 1
  for (int q = 0; q < N; q += 32) {
    uint32_t c[32];
    tc_ld32(c, ts + q);
    tc_wait_ld32(c);
#pragma unroll
    for (int k = 0; k < 32; k += 2) {
      float2 y = make_float2(__uint_as_float(c[k]), __uint_as_float(c[k + 1]));
      if constexpr (FP8) {
        const float f = fminf(r.ks[q / 16 + k / 16] * r.unit, FLT_MAX);
        y = __fmul2_rn(y, make_float2(f, f));
      }
      y = kv_tanh_of(__fmul2_rn(y, make_float2(r.mult, r.mult)));
      y = __fmul2_rn(y, make_float2(r.cap2, r.cap2));
      c[k] = __float_as_uint(y.x), c[k + 1] = __float_as_uint(y.y);
    }
    tc_st32(ts + q, c);
  }
  tc_wait_st();
}

// BIAS: scores get their bias, raw ones their factor first. Hidden ones become -inf.
template <bool BIAS, int N>
__device__ __forceinline__ void tile_scores(float (&x)[N], const TileRow& r, bool raw) {
  if constexpr (BIAS) {
    if (raw) {
#pragma unroll
      for (int i = 0; i < N; i += 2) {
        const float2 y = __fmul2_rn(make_float2(x[i], x[i + 1]), make_float2(r.mult, r.mult));
        x[i] = y.x, x[i + 1] = y.y;
      }
    }
    if (r.ahead) {  // some key is ahead of its query (a prefix)
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] = fmaf(-r.slope, fabsf(r.dist - (float)i), x[i]);
    } else {  // -slope * (dist - i)
      const float2 at = make_float2(-r.slope * r.dist, -r.slope * r.dist);
      const float2 sl = make_float2(r.slope, r.slope);
#pragma unroll
      for (int i = 0; i < N; i += 2) {
        const float2 y = __fadd2_rn(make_float2(x[i], x[i + 1]), __ffma2_rn(sl, make_float2((float)i, (float)(i + 1)), at));
        x[i] = y.x, x[i + 1] = y.y;
      }
    }
  }
  if (r.part) {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = i < r.limit ? x[i] : -CUDART_INF_F;
  }
  if (r.look) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const int4 d = r.docs[i / 4];
      x[i] = d.x == r.doc ? x[i] : -CUDART_INF_F;
      x[i + 1] = d.y == r.doc ? x[i + 1] : -CUDART_INF_F;
      x[i + 2] = d.z == r.doc ? x[i + 2] : -CUDART_INF_F;
      x[i + 3] = d.w == r.doc ? x[i + 3] : -CUDART_INF_F;
    }
  }
}

template <int N>
__device__ __forceinline__ float tile_max(const float (&x)[N]) {
  float m[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
  for (int i = 4; i + 8 <= N; i += 8) {
#pragma unroll
    for (int k = 0; k < 4; ++k) m[k] = fmaxf(m[k], fmaxf(x[i + k], x[i + 4 + k]));
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) m[k] = fmaxf(m[k], x[N - 4 + k]);
  return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}

// Weights 2^(score - base), written to TMEM at `ts` as 16-bit values (times
// vs[16-column block] / vref over 8-bit caches); their sum.
// MODE 0: score = x * mult; 1: capped by kv_tanh_of's polynomial, mult = scale / cap;
// 2: x itself.
template <bool FP8, bool BF, int MODE, int N>
__device__ __forceinline__ float tile_weights(const float (&x)[N], uint32_t ts, const TileRow& r, float mult, float nbase,
                                              const float* vs, float vref) {
  const float vinv = FP8 ? __uint_as_float((254u << 23) - __float_as_uint(vref)) : 1.0f;  // 2^127 for vref = 0
  float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
  float2 k0, k1, k2, k3;  // cap * tanh(mult * x) = x (k0 + x^2 (k1 + x^2 (k2 + x^2 k3)))
  if constexpr (MODE == 1) {
    const float u = mult * mult, v = r.cap2 * mult;
    k0 = make_float2(v, v);
    k1 = make_float2(v * u * kTanh1, v * u * kTanh1);
    k2 = make_float2(v * u * u * kTanh2, v * u * u * kTanh2);
    k3 = make_float2(v * u * u * u * kTanh3, v * u * u * u * kTanh3);
  }
  const float2 mul = make_float2(mult, mult), nb = make_float2(nbase, nbase);
#pragma unroll
  for (int q = 0; q < N / 32; ++q) {
    uint32_t w[16];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float2 fv = make_float2(1.0f, 1.0f);
      // at most the reference: a larger one is of a block that the row does not see
      if constexpr (FP8) fv.x = fv.y = fminf(vs[2 * q + h], vref) * vinv;
#pragma unroll
      for (int k = 0; k < 16; k += 2) {
        const int i = 32 * q + 16 * h + k;
        float2 y = make_float2(x[i], x[i + 1]);
        if constexpr (MODE == 0) {
          y = __ffma2_rn(y, mul, nb);
        } else if constexpr (MODE == 2) {
          y = __fadd2_rn(y, nb);
        } else {
          const float2 z = __fmul2_rn(y, y);
          y = __ffma2_rn(y, __ffma2_rn(z, __ffma2_rn(z, __ffma2_rn(z, k3, k2), k1), k0), nb);
        }
        float2 e = make_float2(kv_exp2(y.x), kv_exp2(y.y));
        sum[h] = __fadd2_rn(sum[h], e);
        if constexpr (FP8) e = __fmul2_rn(e, fv);
        w[8 * h + k / 2] = kv_pack2<BF>(e.x, e.y);
      }
    }
    tc_st16(ts + 16 * q, w);
  }
  return (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
}

// KIND: what the scores may hold besides q.k. Each kind's instance has less code,
// which shows in these unrolled rows: without one for plain scores, 2 x 2048
// float16 tokens took 152 us for 140 (a row of documents 142 for 129), without
// the biased one 3 x 1531 tokens 59.5 us for 55.7. An instance for capped scores
// alone did not: the compiler spilled there (61 -> 81 us).
template <class T, bool FP8, int HD, int KIND>
__global__ void __launch_bounds__(kTileThreads, 1)
    kv_tile_kernel_t(const KvParams p, const __grid_constant__ KvTileMaps maps) {
  using C = TileCfg<FP8, HD>;
  using bits = typename Elem<T>::bits;
  constexpr bool BF = !FP8 && kIsBf16<T>;
  constexpr int NT = C::NT, N = C::N, NB = N / 16;
  extern __shared__ uint8_t kv_tiles[];
  __shared__ TileBars bars;
  __shared__ uint32_t s_tmem;
  __shared__ int s_qdoc[2];
  uint8_t* base = kv_tiles + ((1024 - (kv_smem(kv_tiles) & 1023)) & 1023);
  const uint32_t sq = kv_smem(base), sk = sq + C::kQ, sv = sk + 2 * C::kStage;
  uint8_t* info = base + C::kQ + 4 * C::kStage;
  uint32_t* need = reinterpret_cast<uint32_t*>(info + 4 * C::kInfo);
  uint32_t* mixed = need + kTileListed / 32;
  float* undo = reinterpret_cast<float*>(mixed + kTileListed / 32);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  auto bar = [&](uint64_t* b) { return kv_smem(b); };

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(&bars.k_full[i]), kTileBring);
      mbar_init(bar(&bars.v_full[i]), kTileBring);
      mbar_init(bar(&bars.k_free[i]), 1);
      mbar_init(bar(&bars.v_free[i]), 1);
      mbar_init(bar(&bars.s_full[i]), 1);
      mbar_init(bar(&bars.p_full[i]), kTileRows);
      mbar_init(bar(&bars.o_full[i]), 1);
    }
    for (int i = 0; i < 4; ++i) mbar_init(bar(&bars.info[i]), kTileBring);
    mbar_init(bar(&bars.q_full), NT * kTileRows);
    mbar_init(bar(&bars.drain), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    s_qdoc[0] = 0x7fffffff;
    s_qdoc[1] = (int)0x80000000;
  }
  if (!FP8 && tid == 256) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&maps.k)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&maps.v)) : "memory");
  }
  if (warp == 12) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(kv_smem(&s_tmem)), "n"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  pdl_launch_dependents();
  pdl_wait();

  const int kvh = blockIdx.x / p.splits, split = blockIdx.x % p.splits;
  const int b = blockIdx.y;
  const int64_t rows0 = (int64_t)(gridDim.z - 1 - blockIdx.z) * (NT * kTileRows);  // the longest rows first
  const KvSeq seq = kv_seq(p, b);
  if (blockIdx.x == 0 && blockIdx.z == 0 && tid == 0) kv_flag_rows(p, seq);
  const int nrows = p.R - rows0 < NT * kTileRows ? (int)(p.R - rows0) : NT * kTileRows;  // at least 1
  const int live_tiles = nrows > kTileRows ? NT : 1;
  const int64_t tok0 = rows0 / p.G;  // token and head of row r: see tok_of, row_at
  const uint32_t rem0 = (uint32_t)(rows0 - tok0 * p.G), G = (uint32_t)p.G;
  auto tok_of = [&](int r) { return tok0 + (rem0 + (uint32_t)r) / G; };
  auto row_at = [&](int r) {
    const uint32_t d = (rem0 + (uint32_t)r) / G, h = rem0 + (uint32_t)r - d * G;
    return (((int64_t)b * p.S + tok0 + d) * p.Nq + (int64_t)kvh * p.G + h) * p.H;
  };
  int64_t end = kv_limit(seq, seq.past + tok_of(nrows - 1));
  if (end < 0) end = 0;
  int64_t lo64, hi64;
  kv_split(end, p.splits, split, N, &lo64, &hi64);
  const int lo = (int)lo64, hi = (int)hi64;
  const int64_t plane = (int64_t)b * p.Nkv + kvh;
  const int32_t* docs = p.docs ? p.docs + (int64_t)b * p.max_len : nullptr;
  TileList list{need, (hi - lo + N - 1) / N, docs != nullptr};
  if (docs) {
    // which key tiles hold a document of some row, and which need a look at each key
    for (int i = tid; i < 2 * kTileListed / 32; i += kTileThreads) need[i] = 0;
    __syncthreads();
    int dmin = 0x7fffffff, dmax = (int)0x80000000;
    for (int64_t t = tok0 + tid; t <= tok_of(nrows - 1); t += kTileThreads) {
      int32_t d;
      if (kv_document(p, b, seq.past + t, &d)) dmin = d < dmin ? d : dmin, dmax = d > dmax ? d : dmax;
    }
    dmin = __reduce_min_sync(0xffffffffu, dmin);
    dmax = __reduce_max_sync(0xffffffffu, dmax);
    if (lane == 0 && dmin <= dmax) {
      atomicMin(&s_qdoc[0], dmin);
      atomicMax(&s_qdoc[1], dmax);
    }
    __syncthreads();
    dmin = s_qdoc[0];
    dmax = s_qdoc[1];
    const int look = list.count < kTileListed ? list.count : kTileListed;
    for (int t0 = warp * 4; t0 < look; t0 += kTileThreads / 32 * 4) {
      int kmin[4], kmax[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        kmin[u] = 0x7fffffff, kmax[u] = (int)0x80000000;
#pragma unroll
        for (int i = 0; i < N / 32; ++i) {
          const int j = lo + (t0 + u) * N + i * 32 + lane;
          if (j < hi) {
            const int d = __ldg(docs + j);
            kmin[u] = d < kmin[u] ? d : kmin[u], kmax[u] = d > kmax[u] ? d : kmax[u];
          }
        }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int a = __reduce_min_sync(0xffffffffu, kmin[u]), z = __reduce_max_sync(0xffffffffu, kmax[u]);
        const int t = t0 + u;
        if (lane == 0 && t < look && a <= dmax && z >= dmin) {
          atomicOr(&need[t >> 5], 1u << (t & 31));
          if (a != z || dmin != dmax || a != dmin) atomicOr(&mixed[t >> 5], 1u << (t & 31));
        }
      }
    }
  }
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = s_tmem;
  const int first = list.next(list.count);
  // 512 threads x 128 registers, dealt out again: see kKvTileRegisters
  bool ok = true;

  if (warp < 8) {
    // ------------------------------------------------------------------ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
    const int t = warp >> 2;
    const bool live = tid < nrows;  // row rows0 + tid: TMEM lane tid % 128 of row tile t
    const int64_t row = rows0 + tid;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // 32 lanes of TMEM a warp
    // Q to shared memory, 16 bytes at a time
    if (t >= NT) {  // no second row tile
    } else if constexpr (FP8 && kIsBf16<T>) {
      constexpr int LANES = HD <= 128 ? 16 : 32, PER = 32 / LANES, ROUNDS = 32 / PER;
      const int sub = lane / LANES, piece = lane % LANES;
#pragma unroll 1
      for (int i0 = 0; i0 < ROUNDS; i0 += 8) {
        uint4 w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int r = warp * 32 + (i0 + i) * PER + sub;
          w[i] = make_uint4(0, 0, 0, 0);
          if (r < nrows && piece * 8 < p.H)
            w[i] = __ldg(reinterpret_cast<const uint4*>(static_cast<const bits*>(p.q) + row_at(r) + piece * 8));
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int r = warp * 32 + (i0 + i) * PER + sub;
          uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
          float amax = 0.0f;
#pragma unroll
          for (int k = 0; k < 4; ++k)
            amax = fmaxf(amax, fmaxf(fabsf(Elem<T>::tof((bits)x[k])), fabsf(Elem<T>::tof((bits)(x[k] >> 16)))));
#pragma unroll
          for (int o = LANES / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
          float f;
          const float u = kv_row_shift(amax, &f);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            x[k] = kv_pack2<false>(Elem<T>::tof((bits)x[k]) * f, Elem<T>::tof((bits)(x[k] >> 16)) * f);
          if (piece == 0) undo[r] = u;
          if (piece * 8 < HD)
            *reinterpret_cast<uint4*>(base + t * (kTileRows * HD * 2) + tile_at(kTileRows, r % kTileRows, piece)) =
                make_uint4(x[0], x[1], x[2], x[3]);
        }
      }
      __syncwarp();  // a warp brings its own 32 rows: undo[] stays within it
    } else {
      // a lane keeps its piece of the row and goes from row to row of the (S, Nq) plane
      constexpr int PPR = HD / 8, RS = PPR < 32 ? 32 / PPR : 1;
      const int piece = lane % PPR;
      int r = warp * 32 + lane / PPR;
      uint32_t h = (rem0 + (uint32_t)r) % G;
      const bits* src = static_cast<const bits*>(p.q) + row_at(r) + piece * 8;
      const uint32_t dst = sq + t * (kTileRows * HD * 2);
#pragma unroll 4
      for (int i = 0; i < 32 / RS; ++i, r += RS) {
        const bool on = r < nrows && piece * 8 < p.H;
        kv_cp<16>(dst + tile_at(kTileRows, r % kTileRows, piece), on ? src : static_cast<const bits*>(p.q), on);
        src += (int64_t)RS * p.H;
        for (h += RS; h >= G; h -= G) src += (int64_t)(p.Nq - p.G) * p.H;
      }
      kv_cp_commit();
      kv_cp_wait<0>();
    }
    if (t < NT) {
      tc_fence_smem();
      mbar_arrive(bar(&bars.q_full));
    }

    const int64_t pos = seq.past + tok_of(live ? tid : nrows - 1);
    int lim = 0;
    TileRow tr;
    tr.doc = 0;
    {
      int64_t k = live ? kv_limit(seq, pos) : 0;
      if (docs && live && !kv_document(p, b, pos, &tr.doc)) k = 0;
      lim = k > 0 ? (int)k : 0;
    }
    const int full = __reduce_min_sync(0xffffffffu, live ? lim : 0x7fffffff);
    const int first_pos = __reduce_min_sync(0xffffffffu, pos > 0x7fffffff ? 0x7fffffff : (int)pos);
    tr.slope = 0.0f;
    if (p.slopes && live) tr.slope = __ldg(p.slopes + kvh * p.G + (rem0 + tid) % G) * kLog2e;
    const bool capped = KIND == kKvAnyScore && p.cap > 0.0f;
    const float mult = capped ? 2.0f * kLog2e * p.over : p.scale * kLog2e;
    tr.unit = FP8 && kIsBf16<T> ? undo[tid % (NT * kTileRows)] : 1.0f;
    tr.mult = mult;
    tr.cap2 = p.cap * kLog2e;
    const bool general = KIND == kKvBiased || (KIND == kKvAnyScore && (p.slopes || !(p.scale > 0.0f)));
    float m = live ? -CUDART_INF_F : 0.0f, l = 0.0f, vref = 0.0f;  // rows behind the last never move the base
    if (t < live_tiles) {
      int step = 0;
      for (int tile = first; tile >= 0; ++step) {
        const int j0 = lo + tile * N;
        const int buf = NT == 2 ? t : step & 1;
        const uint32_t par = (NT == 2 ? step : step >> 1) & 1;
        const uint32_t ts = tmem + lanes + (NT == 2 ? t * 128 : buf * N);
        const uint32_t to = tmem + lanes + 256 + (NT == 2 ? t * 128 : 0);
        const uint8_t* in = info + (step & 3) * C::kInfo;
        tr.dist = (float)(pos - j0);
        tr.limit = lim - j0;
        tr.part = j0 + N > full;
        tr.ahead = j0 + N > first_pos;
        tr.look = docs && (tile >= kTileListed || (mixed[tile >> 5] >> (tile & 31)) & 1u);
        tr.docs = reinterpret_cast<const int4*>(in);
        tr.ks = reinterpret_cast<const float*>(in + N * 4);
        const float* vs = tr.ks + NB;
        ok = mbar_wait(bar(&bars.s_full[buf]), par);
        if (FP8 || docs) ok = ok && mbar_wait(bar(&bars.info[step & 3]), (step >> 2) & 1);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        tc_after();
        float x[N];
        tile_load<FP8, N>(x, ts, tr, true);
        bool done = general;  // x holds scores in log2, not raw ones
        const bool masked = tr.part || tr.look;
        if (capped && (general || masked || !tile_small(x, tr))) {
          // (an infinite product is at an end of the cap from here on: -inf means hidden)
          tile_cap<FP8, N>(ts, tr);
          tile_load<FP8, N>(x, ts, tr, false);
          done = true;
        }
        if (general)
          tile_scores<true, N>(x, tr, !capped);
        else
          tile_scores<false, N>(x, tr, true);
        bool grown = false;
        float vmax = 0.0f;
        if constexpr (FP8) {
#pragma unroll
          for (int i = 0; i < NB; ++i) vmax = fmaxf(vmax, vs[i]);
          grown = __any_sync(0xffffffffu, vmax > vref);
          if (grown && masked) {  // what counts are the blocks that the row sees something of
            vmax = 0.0f;
#pragma unroll
            for (int i = 0; i < NB; ++i) {
              float top = x[16 * i];
#pragma unroll
              for (int k = 1; k < 16; ++k) top = fmaxf(top, x[16 * i + k]);
              if (top != -CUDART_INF_F) vmax = fmaxf(vmax, vs[i]);
            }
          }
        }
        auto weights = [&]() {
          const float nb = m == -CUDART_INF_F ? 0.0f : -m;
          if (done) return tile_weights<FP8, BF, 2, N>(x, ts, tr, 1.0f, nb, vs, vref);
          if (!capped) return tile_weights<FP8, BF, 0, N>(x, ts, tr, mult, nb, vs, vref);
          return tile_weights<FP8, BF, 1, N>(x, ts, tr, mult * (0.5f / kLog2e), nb, vs, vref);
        };
        // Weights by the base so far, where every row has one; only where a row's sum
        // says that one may be too large (2^15 fits float16) is the maximum taken, the
        // base moved and the tile's weights formed again.
        bool move = __any_sync(0xffffffffu, m == -CUDART_INF_F) || grown;
        float sum = 0.0f;
        if (!move) {
          sum = weights();
          move = __any_sync(0xffffffffu, !(sum <= 32768.0f));
        }
        if (move) {
          const float top = tile_max(x);
          float mx = top * (done ? 1.0f : mult);
          if (capped && !done) mx = kv_tanh_of(mx) * tr.cap2;
          const float mn = fmaxf(m, mx);
          float a = mn == -CUDART_INF_F ? 1.0f : kv_exp2(m - mn);
          m = mn;
          l *= a;
          if constexpr (FP8) {
            if (vmax > vref) {
              a *= vref * __uint_as_float((254u << 23) - __float_as_uint(vmax));  // old / new, powers of two
              vref = vmax;
            }
          }
          if (step > 0 && __any_sync(0xffffffffu, a != 1.0f)) {
            if constexpr (NT == 1) {  // here S runs ahead of P V
              ok = mbar_wait(bar(&bars.o_full[1]), (step - 1) & 1);
              ok = __all_sync(0xffffffffu, ok);
              if (!ok) break;
              tc_after();
            }
#pragma unroll 1
            for (int i = 0; i < HD; i += 16) {
              uint32_t o[16];
              tc_ld16(o, to + i);
#pragma unroll
              for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * a);
              tc_st16(to + i, o);
            }
          }
          sum = weights();
        }
        l += sum;
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        tc_before();
        mbar_arrive(bar(&bars.p_full[buf]));
        tile = list.next(tile);
      }
      // ---------------------------------------------------------------- output
      if (ok && first >= 0) {
        ok = mbar_wait(bar(&bars.o_full[NT == 2 ? t : 0]), 0);
        ok = __all_sync(0xffffffffu, ok);
        tc_after();
      }
      if (ok) {
        const uint32_t to = tmem + lanes + 256 + (NT == 2 ? t * 128 : 0);
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        const float f = (p.splits > 1 ? 1.0f : inv) * (FP8 ? vref : 1.0f);
        const bool empty = m == -CUDART_INF_F && l == 0.0f;  // nothing seen (TMEM may never have been written)
        const int64_t at = (plane * p.splits + split) * p.R + row;
        bits* dst = static_cast<bits*>(p.out) + row_at(live ? tid : 0);
        bool odd = false;
        if (live && p.splits > 1) p.ws_ml[at] = make_float2(m, l);
        constexpr int OC = HD < 128 ? HD : 128;  // columns at once
#pragma unroll 1
        for (int i0 = 0; i0 < HD; i0 += OC) {
          uint32_t all[OC];
#pragma unroll
          for (int i = 0; i < OC; i += 32) tc_ld32(all + i, to + i0 + i);
#pragma unroll
          for (int i = 0; i < OC; i += 32) tc_wait_ld32(all + i);
#pragma unroll
          for (int i1 = 0; i1 < OC; i1 += 32) {
            const int i = i0 + i1;
            const uint32_t* o = all + i1;
            float y[32];
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              y[k] = empty ? 0.0f : __uint_as_float(o[k]) * f;
              odd |= !(fabsf(y[k]) < CUDART_INF_F) && i + k < p.H;
            }
            if (!live) continue;
#pragma unroll
            for (int k = 0; k < 32; k += 8) {
              if (i + k >= p.H) continue;
              if (p.splits > 1) {
                float* part = p.ws_o + at * p.H + i + k;
                *reinterpret_cast<float4*>(part) = make_float4(y[k], y[k + 1], y[k + 2], y[k + 3]);
                *reinterpret_cast<float4*>(part + 4) = make_float4(y[k + 4], y[k + 5], y[k + 6], y[k + 7]);
              } else {
                VecT<T, 8> v;
#pragma unroll
                for (int q = 0; q < 8; ++q) v.v[q] = Elem<T>::fromf(y[k + q]);
                *reinterpret_cast<VecT<T, 8>*>(dst + i + k) = v;
              }
            }
        }
          }
        // An infinity or a NaN may have come from a value that the row does not see
        uint32_t again = __ballot_sync(0xffffffffu, odd && live);
        if (again && !docs) {
          bool found = false;  // in a value that some row of the warp does not see and its key tile holds
          const int upto = hi < lo + list.count * N ? hi : lo + list.count * N;
          const int from = full > lo ? full : lo;
          for (int64_t e = (plane * p.max_len + from) * p.H + lane; e < (plane * p.max_len + upto) * p.H; e += 32) {
            if constexpr (FP8)
              found |= (static_cast<const uint8_t*>(p.v)[e] & 127) == 127;
            else
              found |= !(fabsf(Elem<T>::tof(static_cast<const bits*>(p.v)[e])) < CUDART_INF_F);
          }
          if (!__any_sync(0xffffffffu, found)) again = 0;
        }
        __syncwarp();
        while (again) {
          const int r = __ffs(again) - 1;
          again &= again - 1;
          const int64_t w = (plane * p.splits + split) * p.R + rows0 + (warp * 32 + r);
          kv_careful_row<T, FP8>(p, seq, b, kvh, rows0 + (warp * 32 + r), lo64, hi64,
                                 p.splits > 1 ? p.ws_o + w * p.H : nullptr, p.ws_ml + w, lane);
        }
      }
    }
  } else if (warp >= 12) {
    // ------------------------------------------------------------------ MMA
    asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    if (warp == 12 && first >= 0) {
      // The whole warp walks the steps, so that what an MMA takes stays in uniform
      // registers; one lane issues.
      const uint32_t iqk = tc_idesc(BF, N, false), ipv = tc_idesc(BF, HD, true);
      const int steps = (p.H + 15) / 16;
      const uint32_t dq = tc_desc(sq, 16), dk = tc_desc(sk, 16), dv = tc_desc(sv, N * 128);
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      auto wait = [&](uint64_t* w, int parity) {
        ok = ok && mbar_wait(bar(w), parity);
        ok = __all_sync(0xffffffffu, ok);
      };
      auto commit = [&](uint64_t* w) {
        if (tc_elect()) tc_commit(bar(w));
      };
      auto qk = [&](int t, int stage, uint32_t d) {
        const uint32_t a = dq + t * (kTileRows * HD * 2 / 16), c = dk + stage * (C::kStage / 16);
        if (tc_elect()) {
#pragma unroll
          for (int k = 0; k < HD / 16; ++k)
            if (k < steps)
              tc_mma_ss(d, a + ((k >> 2) * (kTileRows * 128) + (k & 3) * 32) / 16,
                        c + ((k >> 2) * (N * 128) + (k & 3) * 32) / 16, iqk, k > 0);
        }
      };
      auto pv = [&](uint32_t d, uint32_t a, int stage, bool add) {
        const uint32_t c = dv + stage * (C::kStage / 16);
        if (tc_elect()) {
#pragma unroll
          for (int k = 0; k < N / 16; ++k)
            tc_mma_ts(d, a + k * 8, c + k * (2048 / 16), ipv, k > 0 ? 1u : (uint32_t)add);
        }
      };
      int step = 0, tile = first;
      wait(&bars.q_full, 0);
      wait(&bars.k_full[0], 0);
      tc_after();
      if (ok) {
        for (int t = 0; t < live_tiles; ++t) {
          qk(t, 0, tm + t * 128);
          commit(&bars.s_full[t]);
        }
        commit(&bars.k_free[0]);
      }
      while (ok && tile >= 0) {
        const int after = list.next(tile);
        const bool more = after >= 0;
        const int st = step & 1, sn = st ^ 1;
        if constexpr (NT == 2) {
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (t >= live_tiles) break;
            wait(&bars.p_full[t], step & 1);
            if (t == 0) wait(&bars.v_full[st], (step >> 1) & 1);
            if (!ok) break;
            tc_after();
            pv(tm + 256 + t * 128, tm + t * 128, st, step > 0);
            if (t == live_tiles - 1) commit(&bars.v_free[st]);
            if (more) {
              if (t == 0) wait(&bars.k_full[sn], ((step + 1) >> 1) & 1);
              if (!ok) break;
              tc_after();
              qk(t, sn, tm + t * 128);
              commit(&bars.s_full[t]);
              if (t == live_tiles - 1) commit(&bars.k_free[sn]);
            } else {
              commit(&bars.o_full[t]);
            }
          }
        } else {
          if (more) {
            wait(&bars.k_full[sn], ((step + 1) >> 1) & 1);
            if (!ok) break;
            tc_after();
            qk(0, sn, tm + sn * N);
            commit(&bars.s_full[sn]);
            commit(&bars.k_free[sn]);
          }
          wait(&bars.p_full[st], (step >> 1) & 1);
          wait(&bars.v_full[st], (step >> 1) & 1);
          if (!ok) break;
          tc_after();
          pv(tm + 256, tm + st * N, st, step > 0);
          commit(&bars.v_free[st]);
          commit(&bars.o_full[1]);
          if (!more) commit(&bars.o_full[0]);
        }
        tile = after;
        ++step;
      }
      if (!ok) {  // let what was issued end before TMEM and shared memory go
        commit(&bars.drain);
        mbar_wait(bar(&bars.drain), 0);
      }
    }
  } else if (warp >= 8) {
    // ------------------------------------------------------------------ K and V
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    const int me = tid - 256;
    constexpr int PPR = HD / 8;              // 16-byte pieces of a row in shared memory
    const int HB = p.H * (FP8 ? 1 : 2);      // bytes of a cache row
    const uint8_t* kb = static_cast<const uint8_t*>(p.k) + plane * p.max_len * HB;
    const uint8_t* vb = static_cast<const uint8_t*>(p.v) + plane * p.max_len * HB;
    auto put_info = [&](int j0, int step) {
      if (!FP8 && !docs) return;
      uint8_t* in = info + (step & 3) * C::kInfo;
      if (docs)
        for (int i = me; i < N; i += kTileBring)
          reinterpret_cast<int32_t*>(in)[i] = j0 + i < hi ? __ldg(docs + j0 + i) : 0;
      if (FP8 && me < 2 * NB) {
        const int blk = me % NB;
        const float* s = me < NB ? p.ks : p.vs;
        float f = j0 + blk * 16 < hi ? __ldg(s + plane * p.nblk + j0 / kKvBlock + blk) : 0.0f;
        if (!(f >= 0.0f && f < CUDART_INF_F)) f = 0.0f;  // of a block that no row sees
        reinterpret_cast<float*>(in + N * 4)[me] = f;
      }
      mbar_arrive(bar(&bars.info[step & 3]));
    };
    if constexpr (!FP8) {
      auto bring = [&](uint32_t dst, const uint8_t* src, const CUtensorMap* map, int j0, uint32_t full) {
        if (p.tma && j0 + N <= hi) {
          if (me == 0) {
            mbar_arrive_expect_tx(full, C::kStage);
#pragma unroll
            for (int q = 0; q < C::SLABS; ++q) tile_tma(dst + q * (N * 128), map, q * 64, j0, (int)plane, full);
          } else {
            mbar_arrive(full);
          }
          return;
        }
        for (int i = me; i < N * PPR; i += kTileBring) {
          const int r = i / PPR, piece = i % PPR;
          const bool on = j0 + r < hi && piece * 16 < HB;
          kv_cp<16>(dst + tile_at(N, r, piece), src + (on ? (int64_t)(j0 + r) * HB + piece * 16 : 0), on);
        }
        kv_cp_commit();
        kv_cp_wait<0>();
        tc_fence_smem();
        mbar_arrive(full);
      };
      int step = 0, nk = 0, nv = 0;  // tiles of K and of V whose loads have begun
      for (int tile = first; tile >= 0; tile = list.next(tile), ++step) {
        const int st = step & 1, j0 = lo + tile * N;
        if (step >= 2) ok = mbar_wait(bar(&bars.k_free[st]), ((step >> 1) - 1) & 1);
        if (!__all_sync(0xffffffffu, ok)) break;
        put_info(j0, step);
        bring(sk + st * C::kStage, kb, &maps.k, j0, bar(&bars.k_full[st]));
        ++nk;
        if (step >= 2) ok = mbar_wait(bar(&bars.v_free[st]), ((step >> 1) - 1) & 1);
        if (!__all_sync(0xffffffffu, ok)) break;
        bring(sv + st * C::kStage, vb, &maps.v, j0, bar(&bars.v_full[st]));
        ++nv;
      }
      if (!__all_sync(0xffffffffu, ok)) {  // what TMA still brings has to land before shared memory goes
        ok = false;
        for (int i = nk - 2; i < nk; ++i)
          if (i >= 0) mbar_wait(bar(&bars.k_full[i & 1]), (i >> 1) & 1);
        for (int i = nv - 2; i < nv; ++i)
          if (i >= 0) mbar_wait(bar(&bars.v_full[i & 1]), (i >> 1) & 1);
      }
    } else {
      // a 16-byte piece of codes becomes two 16-byte pieces of float16
      // (the rows of a thread are a multiple of 8 apart, so their swizzle is the same)
      constexpr int CPR = HD / 16, RS = kTileBring / CPR, PER = N / RS;
      const int r0 = me / CPR, piece = me % CPR;
      const bool in_row = piece * 16 < HB;
      // of 8 lanes that share a row of two slabs, half store their second piece first:
      // their pieces then lie in different banks
      const bool turn = HD >= 128 && (piece & 4);
      const uint32_t at0 = tile_at(N, r0, 2 * piece + turn), at1 = tile_at(N, r0, 2 * piece + !turn);
      uint4 a[PER], c[PER];
      auto load = [&](uint4 (&x)[PER], const uint8_t* src, int j0) {
        const uint8_t* from = src + (int64_t)(j0 + r0) * HB + piece * 16;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          x[i] = make_uint4(0, 0, 0, 0);
          if (in_row && j0 + r0 + i * RS < hi) x[i] = __ldg(reinterpret_cast<const uint4*>(from + (int64_t)i * RS * HB));
        }
      };
      auto store = [&](const uint4 (&x)[PER], uint8_t* dst) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          const uint32_t u0 = turn ? x[i].z : x[i].x, u1 = turn ? x[i].w : x[i].y;
          const uint32_t u2 = turn ? x[i].x : x[i].z, u3 = turn ? x[i].y : x[i].w;
          *reinterpret_cast<uint4*>(dst + at0 + i * RS * 128) =
              make_uint4(kv_codes2(u0), kv_codes2_high(u0), kv_codes2(u1), kv_codes2_high(u1));
          *reinterpret_cast<uint4*>(dst + at1 + i * RS * 128) =
              make_uint4(kv_codes2(u2), kv_codes2_high(u2), kv_codes2(u3), kv_codes2_high(u3));
        }
      };
      uint8_t* pk = base + C::kQ;
      uint8_t* pv8 = pk + 2 * C::kStage;
      int step = 0, tile = first;
      if (tile >= 0) load(a, kb, lo + tile * N);
      while (tile >= 0) {
        const int st = step & 1, j0 = lo + tile * N;
        const int after = list.next(tile);
        load(c, vb, j0);
        if (step >= 2) ok = mbar_wait(bar(&bars.k_free[st]), ((step >> 1) - 1) & 1);
        if (!__all_sync(0xffffffffu, ok)) break;
        put_info(j0, step);
        store(a, pk + st * C::kStage);
        tc_fence_smem();
        mbar_arrive(bar(&bars.k_full[st]));
        if (after >= 0) load(a, kb, lo + after * N);
        if (step >= 2) ok = mbar_wait(bar(&bars.v_free[st]), ((step >> 1) - 1) & 1);
        if (!__all_sync(0xffffffffu, ok)) break;
        store(c, pv8 + st * C::kStage);
        tc_fence_smem();
        mbar_arrive(bar(&bars.v_full[st]));
        tile = after;
        ++step;
      }
    }
  }
  if (!ok && p.status) atomicOr(p.status, 2);
  tc_before();
  __syncthreads();
  if (warp == 12)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(512) : "memory");
}

template <class T, bool FP8, int HD>
KvTileKernel kv_tile_of(int kind) {
  const void* fn = kind == kKvPlain    ? (const void*)kv_tile_kernel_t<T, FP8, HD, kKvPlain>
                   : kind == kKvBiased ? (const void*)kv_tile_kernel_t<T, FP8, HD, kKvBiased>
                                       : (const void*)kv_tile_kernel_t<T, FP8, HD, kKvAnyScore>;
  return {fn, TileCfg<FP8, HD>::kSmem};
}

template <class T, bool FP8>
KvTileKernel kv_tile_pick(int H, int kind) {
  if (H <= 64) return kv_tile_of<T, FP8, 64>(kind);
  if (H <= 128) return kv_tile_of<T, FP8, 128>(kind);
  return kv_tile_of<T, FP8, 256>(kind);
}

}  // namespace rope_gb300
