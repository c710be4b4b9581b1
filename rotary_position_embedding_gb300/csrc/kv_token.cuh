// Attention over a key/value cache for few rows (single tokens, short drafts):
// R = S * G rows of a (b, kvh), 8 or 16 of them a CTA, 16-bit T.
//
// Every cached byte is used once per 8 or 16 rows, so the cache's bandwidth is
// the bound and the arithmetic has to stay out of its way. Both products run
// on mma.m16n8k16 with the keys on the 16-row side, so that a group of up to 8
// query heads fills the 8-column side:
//   S^T = K Q^T   (16 tokens x 8 rows),   O^T += V^T P^T   (16 dims x 8 rows).
// A warp walks units of 16 tokens by itself: no barrier until its keys are done.
//
// Loads. A warp copies a unit's K and V, 16 rows and so 16 * H elements side by
// side, with cp.async into a ring of its own in shared memory, in the order of
// memory (64-byte pieces of 8 rows at once reached 5.0 TB/s). __syncwarp is all the
// synchronisation there is, and the bytes in flight do not depend on registers.
// Any order of the head's dimensions serves S as long as K and Q share it, and
// any order serves O as long as the output undoes it; the orders are chosen so
// that a lane reads 16 bytes at a time without bank conflicts:
//   K: lane (g = lane / 4, c = lane % 4) takes tokens g and g + 8, bytes
//      q * 64 + c * 16 .. + 15 of the row for each q;
//   V: tokens 2c, 2c + 1, 2c + 8, 2c + 9, dims v * 8 * VD + g * VD .. + VD - 1;
//      two tokens' words are interleaved in registers into V^T fragments.
// 8-bit caches: codes become float16 exactly on the way into the fragments; the
// key scale of a unit (a block of 16 rows has one) multiplies its scores, the
// value scale its weights, relative to the largest that the row has seen so far (a
// power of two, so nothing is rounded; rows of one CTA may see different blocks).
// Q is float16 too, for bfloat16 after scaling each row by a power of two; the
// scores undo it.
//
// Softmax: the running maximum moves only where a score passes it by 8 (in
// log2), so weights stay below 2^8 (exact in float32, far from float16's end) and
// the common unit costs one vote. P^T fragments come from S^T by movmatrix.
//
// Measured: 64 sequences of 1 to 8190 bfloat16 keys (8 heads of 128, 32 query heads)
// 214 us with the joining, 5.0 TB/s; 256 of 1 to 4096 keys in 8 bits 225 us, 4.8 TB/s;
// one of 131001 keys in 8 bits 68.5 us. The copy rate's floors are 158, 159 and 40 us.
// Head sizes between run padded, and copy piece by piece: 64 sequences of up to 8190
// bfloat16 keys, 8 heads of 64 114 us, 80 167, 96 172, 112 188, 128 205, 160 534, 192
// 543, 256 454 (8 bits: 93, 140, 141, 143, 132, 278, 280, 254).
//
// A value that no row sees is zeroed before the product. Where one that only
// some rows see is not finite, its zero weight in the others would make a NaN
// of it: the CTA then does its rows over again one by one (kv_careful_row).
#pragma once

#include <cfloat>

#include "kv_careful.cuh"

namespace rope_gb300 {

constexpr int kTokWarps = kKvTokenThreads / 32;

template <class T>
constexpr bool kIsBf16 = false;
template <>
constexpr bool kIsBf16<__nv_bfloat16> = true;

__device__ __forceinline__ float kv_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float kv_rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// tanh(y) from h = 2 log2(e) y, to 2^-20 of its value: an absolute error would grow
// with the cap. From |y| = 0.4 on 1 - 2 / (1 + e^(2y)), off by at most 4 * 2^-22 of
// the result; below, where the difference loses the result's leading bits, the
// polynomial y (1 + z (c1 + z (c2 + z c3))), z = y^2, of the smallest largest
// relative error over [0, 0.4], 1.2e-7.
constexpr float kTanhEnd = 0.4f, kTanh1 = -0.333318830f, kTanh2 = 0.132776290f, kTanh3 = -0.0477942079f;
__device__ __forceinline__ float kv_tanh_of(float h) {
  const float y = h * (0.5f / kLog2e), z = y * y;
  const float p = fmaf(y * z, fmaf(z, fmaf(z, kTanh3, kTanh2), kTanh1), y);
  const float t = fmaf(-2.0f, kv_rcp(1.0f + kv_exp2(h)), 1.0f);
  return fabsf(y) < kTanhEnd ? p : t;
}
__device__ __forceinline__ float2 kv_tanh_of(float2 h) {
  constexpr float k = 0.5f / kLog2e;
  const float2 y = __fmul2_rn(h, make_float2(k, k)), z = __fmul2_rn(y, y);
  float2 p = __ffma2_rn(z, make_float2(kTanh3, kTanh3), make_float2(kTanh2, kTanh2));
  p = __ffma2_rn(z, p, make_float2(kTanh1, kTanh1));
  p = __ffma2_rn(__fmul2_rn(y, z), p, y);
  const float2 e = __fadd2_rn(make_float2(kv_exp2(h.x), kv_exp2(h.y)), make_float2(1.0f, 1.0f));
  const float2 t = __ffma2_rn(make_float2(kv_rcp(e.x), kv_rcp(e.y)), make_float2(-2.0f, -2.0f), make_float2(1.0f, 1.0f));
  return make_float2(fabsf(y.x) < kTanhEnd ? p.x : t.x, fabsf(y.y) < kTanhEnd ? p.y : t.y);
}

// 1 / s for s = 2^e, -126 <= e <= 126, exactly; 0 and 2^127 become each other.
__device__ __forceinline__ float kv_pow2_over(float s) { return __uint_as_float((254u << 23) - __float_as_uint(s)); }

template <bool BF16>
__device__ __forceinline__ void kv_mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
  if constexpr (BF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t kv_transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Two e4m3 codes (the low 16 bits) to float16x2, exactly.
__device__ __forceinline__ uint32_t kv_codes2(uint32_t two) {
  uint32_t y;
  asm("{.reg .b16 l, h; mov.b32 {l, h}, %1; cvt.rn.f16x2.e4m3x2 %0, l;}" : "=r"(y) : "r"(two));
  return y;
}
__device__ __forceinline__ uint32_t kv_codes2_high(uint32_t two) {
  uint32_t y;
  asm("{.reg .b16 l, h; mov.b32 {l, h}, %1; cvt.rn.f16x2.e4m3x2 %0, h;}" : "=r"(y) : "r"(two));
  return y;
}

template <bool BF16>
__device__ __forceinline__ uint32_t kv_pack2(float lo, float hi) {
  uint32_t y;
  if constexpr (BF16)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(y) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(y) : "f"(hi), "f"(lo));
  return y;
}

// Whether either 16-bit half of x is an infinity or a NaN.
template <bool BF16>
__device__ __forceinline__ bool kv_odd2(uint32_t x) {
  constexpr uint32_t E = BF16 ? 0x7f80u : 0x7c00u;
  return (x & E) == E || ((x >> 16) & E) == E;
}

// Whether one of four e4m3 codes is NaN (all bits but the sign set).
__device__ __forceinline__ bool kv_nan4(uint32_t x) { return ((((x & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u)) != 0; }

// A row of bfloat16 values as float16: scaled by the power of two that brings
// its largest magnitude to 2^8..2^9. Returns what undoes it. `amax` is the
// row's; rows that are 0 or not finite stay unscaled.
__device__ __forceinline__ float kv_row_shift(float amax, float* factor) {
  const int e = (int)(__float_as_uint(amax) >> 23);  // biased exponent of amax >= 0
  *factor = 1.0f;
  if (e == 0 || e >= 255) return 1.0f;
  int s = 127 + 8 - e;  // factor 2^s
  if (s > 120) s = 120;
  if (s < -120) s = -120;
  *factor = __uint_as_float((uint32_t)(127 + s) << 23);
  return __uint_as_float((uint32_t)(127 - s) << 23);
}

// Work is dealt out in units of 64 keys (16 a warp) of one problem (b, kvh, tile
// of rows). With p.deal CTAs, CTA i takes the units [i T / n, (i + 1) T / n) of all T
// in the order of the problems, whatever the sequences' lengths: a problem that
// one CTA has whole goes to the output, the others' parts to the workspace (2
// slots a CTA: its first segment's, its last one's), with a word on the problem that
// the CTA begins and leaves unfinished, for kv_join_kernel. Without (no workspace,
// or more sequences than fit) a CTA takes one problem. Equal splits of ragged
// sequences left some SMs with 1.25 times the mean's work.
//
// Few problems of caches that are not long (p.cluster CTAs a problem, a cluster):
// each CTA takes its share of the problem's units, and the parts meet in the
// CTAs' shared memory, so there is one launch and no workspace.
constexpr int kTokUnit = 16 * kTokWarps;

__device__ __forceinline__ void kv_cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address in CTA `rank` of the cluster of what is at `at` in this one.
__device__ __forceinline__ uint32_t kv_cluster_at(uint32_t at, int rank) {
  uint32_t y;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(y) : "r"(at), "r"(rank));
  return y;
}
__device__ __forceinline__ float4 kv_cluster_ld4(uint32_t at) {
  float4 y;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(y.x), "=f"(y.y), "=f"(y.z), "=f"(y.w) : "r"(at) : "memory");
  return y;
}
__device__ __forceinline__ float2 kv_cluster_ld2(uint32_t at) {
  float2 y;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(y.x), "=f"(y.y) : "r"(at) : "memory");
  return y;
}

struct TokenPlan {
  const int32_t* before;  // units of one problem of the sequences before b, for each b, and of all
  int total;              // units of all problems, below 2^31
  __device__ __forceinline__ int first(const KvParams& p, int cta) const {
    return (int)((uint64_t)(uint32_t)cta * (uint32_t)total / (uint32_t)p.deal);
  }
  __device__ __forceinline__ int owner(const KvParams& p, int unit) const {
    return (int)((((uint64_t)(uint32_t)unit + 1) * (uint32_t)p.deal - 1) / (uint32_t)total);
  }
};

__device__ __forceinline__ int token_end(const KvParams& p, const KvSeq& seq, int last_row) {
  const int64_t e = kv_limit(seq, seq.past + kv_div(last_row, p.by_g));
  return e > 0 ? (int)e : 0;
}

// Units of a problem of sequence b: at least one, so that its output is written.
__device__ __forceinline__ int token_units(const KvParams& p, int b) {
  const int u = (token_end(p, kv_seq(p, b), (int)p.R - 1) + kTokUnit - 1) / kTokUnit;
  return u > 0 ? u : 1;
}

// The units before each sequence, in shared memory (kKvDealMost + 1 values); all
// kKvTokenThreads threads come here.
__device__ __forceinline__ TokenPlan token_plan(const KvParams& p, int32_t* before, int32_t* warp_sum) {
  constexpr int PER = kKvDealMost / kKvTokenThreads;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int u[PER], sum = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int b = tid * PER + i;
    u[i] = b < p.B ? token_units(p, b) : 0;
    sum += u[i];
  }
  int pre = sum;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const int x = __shfl_up_sync(0xffffffffu, pre, o);
    if (lane >= o) pre += x;
  }
  if (lane == 31) warp_sum[warp] = pre;
  __syncthreads();
  int at = pre - sum;
  for (int w = 0; w < warp; ++w) at += warp_sum[w];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (tid * PER + i <= p.B) before[tid * PER + i] = at;
    at += u[i];
  }
  if (tid == kKvTokenThreads - 1 && p.B == kKvDealMost) before[p.B] = at;
  __syncthreads();
  TokenPlan plan;
  plan.before = before;
  plan.total = before[p.B] * p.Nkv * p.tiles;
  return plan;
}

template <class T, bool FP8, int HD, int NB>
struct TokenCfg {
  static constexpr int ES = FP8 ? 1 : 2;
  static constexpr int KQ = HD * ES / 64;               // 16-byte pieces of K per lane and token
  static constexpr int VD = FP8 ? (HD >= 128 ? 16 : 8) : 8;  // dims of a V piece
  static constexpr int VB = VD * ES;                    // bytes of a V piece
  static constexpr int VQ = HD / (8 * VD);              // V pieces per lane and token
  // Byte offset of 16-byte piece `piece` of token `row` in a stage's K, and of VB-byte
  // piece in its V: 32 lanes' pieces side by side, turned so that neither the
  // copies (pieces of one row) nor the reads (a lane's own) meet in a bank.
  static __device__ __forceinline__ int k_at(int row, int piece) {
    const int q = piece >> 2, lane = (row & 7) * 4 + (piece & 3);
    return ((row >> 3) * KQ + q) * 512 + ((lane ^ ((q & 1) << 2)) << 4);
  }
  static __device__ __forceinline__ int v_at(int row, int piece) {
    const int v = piece >> 3, g = piece & 7, c = (row & 7) >> 1, t = (row & 1) + 2 * (row >> 3);
    return ((t * VQ + v) * 32 + g * 4 + (c ^ ((g >> 1) & 3))) * VB;
  }
  static constexpr int kK = 2 * KQ * 512;
  static constexpr int kV = 4 * VQ * 32 * VB;
  static constexpr int kStage = kK + kV + 128;          // and 16 documents, 2 scales
  // Two stages, and more warps rather than deeper rings: 64 sequences of 2 to 8191
  // bfloat16 keys, 8 heads of 128, 212 us with 2 stages and 3 CTAs an SM, 235 with 3
  // and 2; 256 sequences of 1 to 4096 keys in 8 bits 232 us with 2 and 4, 239 with 3
  // and 4, 268 with 5 and 2.
  static constexpr int kStages = 2;
  static constexpr int kCtas = HD > 128 || NB > 1 ? 1 : FP8 ? 4 : 3;  // on an SM, at least
  static constexpr int kMerge = kTokWarps * NB * 8 * (HD + 4) * 4;
  static constexpr int kRing = kStage * kStages * kTokWarps;
  static constexpr int kSmem = kRing > kMerge ? kRing : kMerge;
  // 228 KB an SM; a CTA holds about 4.5 KB statically, and 1 KB is reserved for it
  static_assert(kv_token_ctas(FP8, HD, NB > 1) / 152 * (kSmem + 5632) <= 228 * 1024, "CTAs that are resident");
};

template <class T, bool FP8, int HD, int NB>
__global__ void __launch_bounds__(kKvTokenThreads, TokenCfg<T, FP8, HD, NB>::kCtas) kv_token_kernel_t(const KvParams p) {
  using C = TokenCfg<T, FP8, HD, NB>;
  using bits = typename Elem<T>::bits;
  constexpr bool BF = !FP8 && kIsBf16<T>;  // type of the matrix operands
  constexpr int OT = HD / 16;                                   // 16-dim tiles of O^T
  extern __shared__ __align__(128) uint8_t kv_ring[];
  __shared__ float s_m[kTokWarps][NB * 8], s_l[kTokWarps][NB * 8];
  __shared__ int32_t s_before[kKvDealMost + 1], s_sum[kTokWarps];
  __shared__ float2 s_part[NB * 8];  // statistics of this CTA's part for its cluster
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, c = lane & 3;
  pdl_launch_dependents();
  pdl_wait();
  uint8_t* const ring = kv_ring + warp * (C::kStage * C::kStages);
  TokenPlan plan;
  int at_unit = 0, last_unit = 0;
  const bool dealt = p.deal > 0;
  const int ranks = p.cluster, rank = ranks > 1 ? (int)blockIdx.x % ranks : 0;
  constexpr int LD = HD + 4;  // of a row of O in shared memory
  float* const so = reinterpret_cast<float*>(kv_ring);
  if (dealt) {
    plan = token_plan(p, s_before, s_sum);
    at_unit = plan.first(p, blockIdx.x);
    last_unit = plan.first(p, blockIdx.x + 1);
    if (at_unit >= last_unit) {
      // no units: nothing begins here, and nothing of this CTA's counts where a
      // problem's CTAs lie on both sides of it
      if (tid == 0) p.ws_join[blockIdx.x] = make_int4(0, 0, 0, 0);
      if (tid < NB * 8) p.ws_ml[2 * (int64_t)blockIdx.x * (NB * 8) + tid] = make_float2(-CUDART_INF_F, 0.0f);
      return;
    }
  }
  const int rows_all = (int)p.R;
  bool again = true;
  for (int segment = 0; again; ++segment) {
    // the next problem of this CTA, and its units
    int b, kvh, rows0, u0 = 0, u1 = -1;
    bool whole_problem = true;
    if (dealt) {
      const int problems = p.Nkv * p.tiles;  // of a sequence
      int x = 0, y = p.B;                    // the sequence of at_unit: before[x] <= . < before[x + 1]
      while (y - x > 1) {
        const int mid = (x + y) >> 1;
        if (plan.before[mid] * problems <= at_unit)
          x = mid;
        else
          y = mid;
      }
      b = x;
      const int units = plan.before[b + 1] - plan.before[b];
      const int in = at_unit - plan.before[b] * problems;
      const int problem = (int)((uint32_t)in / (uint32_t)units);
      u0 = in - problem * units;
      u1 = u0 + (last_unit - at_unit) < units ? u0 + (last_unit - at_unit) : units;
      whole_problem = u0 == 0 && u1 == units;
      kvh = kv_div(problem, p.by_tiles);
      rows0 = (problem - kvh * p.tiles) * (NB * 8);
      at_unit += u1 - u0;
      again = at_unit < last_unit;
      // the one problem that may begin in this CTA and go on in others: kv_join_kernel_t's
      if (!again && tid == 0) {
        // (`parts` further CTAs, and which of this one's slots holds the first part)
        const bool open = u0 == 0 && u1 < units;  // a problem that began before is another CTA's
        const int parts = open ? plan.owner(p, at_unit - u1 + units - 1) - (int)blockIdx.x : 0;
        p.ws_join[blockIdx.x] = make_int4(b, kvh, rows0, 2 * parts + (segment > 0 ? 1 : 0));
      }
    } else {
      const int problem = ranks > 1 ? (int)blockIdx.x / ranks : (int)blockIdx.x;
      kvh = kv_div(problem, p.by_tiles);
      rows0 = (problem - kvh * p.tiles) * (NB * 8);
      b = (int)blockIdx.z + segment * (int)gridDim.z;
      again = b + (int)gridDim.z < p.B;
    }
    const KvSeq seq = kv_seq(p, b);
    if (kvh == 0 && rows0 == 0 && u0 == 0 && tid == 0) kv_flag_rows(p, seq);
    const int end = token_end(p, seq, (rows0 + NB * 8 < rows_all ? rows0 + NB * 8 : rows_all) - 1);
    if (ranks > 1) {
      const int units = (end + kTokUnit - 1) / kTokUnit;
      u0 = (int)((int64_t)units * rank / ranks);
      u1 = (int)((int64_t)units * (rank + 1) / ranks);
      whole_problem = false;
    }
    int lo = u0 * kTokUnit < end ? u0 * kTokUnit : end;
    int hi = u1 < 0 || u1 * kTokUnit > end ? end : u1 * kTokUnit;
    const int64_t plane = (int64_t)b * p.Nkv + kvh;
    // where a part of a problem goes
    const int64_t slot = 2 * (int64_t)blockIdx.x + (segment > 0 ? 1 : 0);
    float* const part_o = whole_problem ? nullptr : ranks > 1 ? so : p.ws_o + slot * (NB * 8) * p.H;
    float2* const part_ml = whole_problem ? nullptr : ranks > 1 ? s_part : p.ws_ml + slot * (NB * 8);
    const int part_ld = ranks > 1 ? LD : p.H;
    const int HB = p.H * C::ES;  // bytes of a cache row
    const uint8_t* kbase = static_cast<const uint8_t*>(p.k) + plane * p.max_len * HB;
    const uint8_t* vbase = static_cast<const uint8_t*>(p.v) + plane * p.max_len * HB;
    const int32_t* dbase = p.docs ? p.docs + (int64_t)b * p.max_len : nullptr;

    // A unit's K and V are 16 whole rows each, copied in the order of memory; the
    // pieces land where kk() and vv() look for them.
    auto copy_unit = [&](int j0, int stage) {
      const uint32_t at = kv_smem(ring + stage * C::kStage);
      constexpr int FB = HD * C::ES, KP = FB / 16, VP = FB / C::VB;  // bytes and pieces of a row
      const bool whole_unit = HB == FB && j0 + 16 <= hi;              // constant offsets, no zeros
      const uint8_t* ks = kbase + (int64_t)j0 * FB + lane * 16;
      const uint8_t* vs = vbase + (int64_t)j0 * FB + lane * C::VB;
      if (whole_unit) {
#pragma unroll
        for (int i = 0; i < KP / 2; ++i)
          kv_cp<16>(at + C::k_at((i * 32 + lane) / KP, (i * 32 + lane) % KP), ks + i * 512);
#pragma unroll
        for (int i = 0; i < VP / 2; ++i)
          kv_cp<C::VB>(at + C::kK + C::v_at((i * 32 + lane) / VP, (i * 32 + lane) % VP), vs + i * 32 * C::VB);
      } else {
#pragma unroll 1
        for (int i = 0; i < KP / 2; ++i) {
          const int row = (i * 32 + lane) / KP, piece = (i * 32 + lane) % KP;
          const bool on = j0 + row < hi && piece * 16 < HB;
          kv_cp<16>(at + C::k_at(row, piece), on ? kbase + (int64_t)(j0 + row) * HB + piece * 16 : kbase + (int64_t)lo * HB,
                    on);
        }
#pragma unroll 1
        for (int i = 0; i < VP / 2; ++i) {
          const int row = (i * 32 + lane) / VP, piece = (i * 32 + lane) % VP;
          const bool on = j0 + row < hi && piece * C::VB < HB;
          kv_cp<C::VB>(at + C::kK + C::v_at(row, piece),
                       on ? vbase + (int64_t)(j0 + row) * HB + piece * C::VB : vbase + (int64_t)lo * HB, on);
        }
      }
      const uint32_t meta = at + C::kK + C::kV;
      if (dbase && lane < 16) kv_cp<4>(meta + lane * 4, dbase + (j0 + lane < hi ? j0 + lane : lo), j0 + lane < hi);
      if (FP8 && lane >= 16 && lane < 18)
        kv_cp<4>(meta + lane * 4, (lane == 16 ? p.ks : p.vs) + plane * p.nblk + j0 / kKvBlock, j0 < hi);
    };
    auto row_of = [&](int r) {  // element offset of a row of Q or of the output
      const int tok = kv_div(r, p.by_g);
      return (((int64_t)b * p.S + tok) * p.Nq + (int64_t)kvh * p.G + (r - tok * p.G)) * p.H;
    };
    // Q fragments: row g of each column tile, in the order of K's pieces. Their
    // loads go out first, then the copies of the first units.
    constexpr int QP = FP8 ? 2 * C::KQ : C::KQ;  // 8-element pieces of Q a lane
    uint4 raw[NB][QP];
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      const int r = rows0 + n * 8 + g;
      const bits* src = static_cast<const bits*>(p.q) + (r < rows_all ? row_of(r) : 0);
#pragma unroll
      for (int q = 0; q < QP; ++q) {
        const int d = FP8 ? (q >> 1) * 64 + c * 16 + (q & 1) * 8 : q * 32 + c * 8;
        raw[n][q] = make_uint4(0, 0, 0, 0);
        if (r < rows_all && d < p.H) raw[n][q] = __ldg(reinterpret_cast<const uint4*>(src + d));
      }
    }
    const int first = lo + warp * 16, step = 16 * kTokWarps;
#pragma unroll 1
    for (int s = 0; s < C::kStages - 1; ++s) {
      if (first + s * step < hi) copy_unit(first + s * step, s);
      kv_cp_commit();
    }
    uint32_t qf[NB][HD / 16][2];
    float undo[NB];
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      undo[n] = 1.0f;
      if constexpr (FP8 && kIsBf16<T>) {  // bfloat16 rows become float16 after scaling by a power of two
        float amax = 0.0f, f;
#pragma unroll
        for (int q = 0; q < QP; ++q) {
          const uint32_t w[4] = {raw[n][q].x, raw[n][q].y, raw[n][q].z, raw[n][q].w};
#pragma unroll
          for (int i = 0; i < 4; ++i)
            amax = fmaxf(amax, fmaxf(fabsf(Elem<T>::tof((bits)w[i])), fabsf(Elem<T>::tof((bits)(w[i] >> 16)))));
        }
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        undo[n] = kv_row_shift(amax, &f);
#pragma unroll
        for (int q = 0; q < QP; ++q) {
          uint32_t w[4] = {raw[n][q].x, raw[n][q].y, raw[n][q].z, raw[n][q].w};
#pragma unroll
          for (int i = 0; i < 4; ++i)
            w[i] = kv_pack2<false>(Elem<T>::tof((bits)w[i]) * f, Elem<T>::tof((bits)(w[i] >> 16)) * f);
          raw[n][q] = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
#pragma unroll
      for (int q = 0; q < QP; ++q) {
        qf[n][2 * q][0] = raw[n][q].x, qf[n][2 * q][1] = raw[n][q].y;
        qf[n][2 * q + 1][0] = raw[n][q].z, qf[n][2 * q + 1][1] = raw[n][q].w;
      }
    }

    // the rows whose scores this lane holds: 2c and 2c + 1 of each column tile
    float unit[NB][2], slope[NB][2], m[NB][2], l[NB][2];  // unit: of bfloat16 Q rows, see kv_row_shift
    int64_t pos[NB][2];
    int lim[NB][2], doc[NB][2];
    const float c1 = p.cap > 0.0f ? 2.0f * kLog2e * p.over : p.scale * kLog2e;
    const float c2 = p.cap * kLog2e;
    int full = 0x7fffffff;  // keys below this are seen by every row
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = rows0 + n * 8 + 2 * c + e;
        const bool live = r < rows_all;
        const int tok = live ? kv_div(r, p.by_g) : 0;
        unit[n][e] = __shfl_sync(0xffffffffu, undo[n], 4 * (2 * c + e));
        pos[n][e] = seq.past + tok;
        int64_t k = live ? kv_limit(seq, pos[n][e]) : 0;
        doc[n][e] = 0;
        if (p.docs && live && !kv_document(p, b, pos[n][e], &doc[n][e])) k = 0;
        lim[n][e] = k > 0 ? (int)k : 0;
        slope[n][e] = p.slopes && live ? __ldg(p.slopes + kvh * p.G + (r - tok * p.G)) * kLog2e : 0.0f;
        if (live && lim[n][e] < full) full = lim[n][e];
        m[n][e] = -CUDART_INF_F;
        l[n][e] = 0.0f;
      }
#pragma unroll
    for (int o = 1; o <= 2; o *= 2) {
      const int x = __shfl_xor_sync(0xffffffffu, full, o);
      full = x < full ? x : full;
    }
    float acc[OT][NB][4];
#pragma unroll
    for (int t = 0; t < OT; ++t)
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[t][n][i] = 0.0f;
    float vinv[NB][2];  // one over the row's largest value scale so far, in whose units O is held
#pragma unroll
    for (int n = 0; n < NB; ++n) vinv[n][0] = vinv[n][1] = 0x1p127f;  // 0: none seen
    bool odd = false;   // an infinity or a NaN in a value that not every row sees

    int stage = 0, next = C::kStages - 1;
    for (int j0 = first; j0 < hi; j0 += step) {
      kv_cp_wait<C::kStages - 2>();
      __syncwarp();  // a lane's pieces were copied by others
      // the unit before this one is done with: its stage is filled while this one is worked on
      if (j0 + (C::kStages - 1) * step < hi) copy_unit(j0 + (C::kStages - 1) * step, next);
      kv_cp_commit();
      const uint8_t* const at = ring + stage * C::kStage;
      const uint8_t* const meta = at + C::kK + C::kV;
      float s[NB][4], s2[NB][4];  // two sums: half as long a chain of dependent products
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[n][i] = s2[n][i] = 0.0f;
#pragma unroll
      for (int q = 0; q < C::KQ; ++q) {
        const uint4 x = *reinterpret_cast<const uint4*>(at + C::k_at(g, 4 * q + c));
        const uint4 y = *reinterpret_cast<const uint4*>(at + C::k_at(g + 8, 4 * q + c));
        if constexpr (!FP8) {
#pragma unroll
          for (int n = 0; n < NB; ++n) {
            kv_mma<BF>(s[n], x.x, y.x, x.y, y.y, qf[n][2 * q][0], qf[n][2 * q][1]);
            kv_mma<BF>(s2[n], x.z, y.z, x.w, y.w, qf[n][2 * q + 1][0], qf[n][2 * q + 1][1]);
          }
        } else {
          const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t a0 = kv_codes2(xs[i]), a2 = kv_codes2_high(xs[i]);
            const uint32_t a1 = kv_codes2(ys[i]), a3 = kv_codes2_high(ys[i]);
#pragma unroll
            for (int n = 0; n < NB; ++n)
              kv_mma<false>(i & 1 ? s2[n] : s[n], a0, a1, a2, a3, qf[n][4 * q + i][0], qf[n][4 * q + i][1]);
          }
        }
      }
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[n][i] += s2[n][i];
      float ks = 1.0f, vs = 1.0f;
      if constexpr (FP8) {
        ks = reinterpret_cast<const float*>(meta)[16];
        vs = reinterpret_cast<const float*>(meta)[17];
      }
      const bool whole = !dbase && j0 + 16 <= full;  // uniform over the warp
      uint32_t any0 = 0xffffffffu, any1 = 0xffffffffu;
      int d0 = 0, d1 = 0;
      if (dbase) d0 = reinterpret_cast<const int*>(meta)[g], d1 = reinterpret_cast<const int*>(meta)[g + 8];
      bool seen0 = false, seen1 = false;
      bool moved = false;
      uint32_t larger = 0;  // rows whose value scale grows here
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x = s[n][e], y = s[n][2 + e];
          if constexpr (FP8) {  // to q.k first: queries may be as small as keys are large
            const float f = kIsBf16<T> ? fminf(unit[n][e] * ks, FLT_MAX) : ks;
            x *= f, y *= f;
          }
          x *= c1, y *= c1;
          if (p.cap > 0.0f) {
            x = kv_tanh_of(x) * c2;
            y = kv_tanh_of(y) * c2;
          }
          if (p.slopes) {
            const float dist = (float)(pos[n][e] - j0 - g);
            x = fmaf(-slope[n][e], fabsf(dist), x);
            y = fmaf(-slope[n][e], fabsf(dist - 8.0f), y);
          }
          if (!whole) {
            const bool a = j0 + g < lim[n][e] && (!dbase || d0 == doc[n][e]);
            const bool d = j0 + g + 8 < lim[n][e] && (!dbase || d1 == doc[n][e]);
            x = a ? x : -CUDART_INF_F;
            y = d ? y : -CUDART_INF_F;
            seen0 |= a;
            seen1 |= d;
            if (FP8 && (__ballot_sync(0xffffffffu, a || d) >> c & 0x11111111u) && vs * vinv[n][e] > 1.0f) larger |= 1u << (2 * n + e);
          } else if (FP8 && vs * vinv[n][e] > 1.0f) {
            larger |= 1u << (2 * n + e);
          }
          s[n][e] = x;
          s[n][2 + e] = y;
          moved |= fmaxf(x, y) > m[n][e] + 8.0f;
        }
      if (!whole) {
        any0 = __ballot_sync(0xffffffffu, seen0);
        any1 = __ballot_sync(0xffffffffu, seen1);
      }
      if (any0 | any1) {  // a unit that no row sees is left out
        if (__any_sync(0xffffffffu, moved || larger)) {
#pragma unroll
          for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float x = fmaxf(s[n][e], s[n][2 + e]);
#pragma unroll
              for (int o = 4; o <= 16; o *= 2) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
              x = fmaxf(m[n][e], x);
              const float a = x == -CUDART_INF_F ? 1.0f : kv_exp2(m[n][e] - x);
              m[n][e] = x;
              l[n][e] *= a;
              float f = a;
              if (FP8 && (larger >> (2 * n + e) & 1u)) {
                const float inv = kv_pow2_over(vs);
                f *= kv_pow2_over(vinv[n][e]) * inv;  // old / new
                vinv[n][e] = inv;
              }
#pragma unroll
              for (int t = 0; t < OT; ++t) {
                acc[t][n][e] *= f;
                acc[t][n][2 + e] *= f;
              }
            }
        }
        uint32_t pf[NB][2];
#pragma unroll
        for (int n = 0; n < NB; ++n) {
          float w[4];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float base = m[n][e] == -CUDART_INF_F ? 0.0f : m[n][e];
            w[e] = kv_exp2(s[n][e] - base);
            w[2 + e] = kv_exp2(s[n][2 + e] - base);
            l[n][e] += w[e] + w[2 + e];
            if constexpr (FP8) {  // (a scale above the row's is of a unit that it does not see)
              const float fp = fminf(vs * vinv[n][e], 1.0f);
              w[e] *= fp;
              w[2 + e] *= fp;
            }
          }
          pf[n][0] = kv_transpose8(kv_pack2<BF>(w[0], w[1]));
          pf[n][1] = kv_transpose8(kv_pack2<BF>(w[2], w[3]));
        }
        // tokens 2c, 2c + 1, 2c + 8, 2c + 9: whether some row sees them
        const bool on[4] = {((any0 >> (8 * c)) & 15u) != 0, ((any0 >> (8 * c + 4)) & 15u) != 0,
                            ((any1 >> (8 * c)) & 15u) != 0, ((any1 >> (8 * c + 4)) & 15u) != 0};
#pragma unroll
        for (int v = 0; v < C::VQ; ++v) {
          uint32_t x[4][C::VB / 4];
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            const uint8_t* a = at + C::kK + C::v_at(2 * c + (t & 1) + 8 * (t >> 1), 8 * v + g);
            if constexpr (C::VB == 16) {
              const uint4 y = *reinterpret_cast<const uint4*>(a);
              x[t][0] = y.x, x[t][1] = y.y, x[t][2] = y.z, x[t][3] = y.w;
            } else {
              const uint2 y = *reinterpret_cast<const uint2*>(a);
              x[t][0] = y.x, x[t][1] = y.y;
            }
            if (!whole && !on[t]) {
#pragma unroll
              for (int w = 0; w < C::VB / 4; ++w) x[t][w] = 0u;
            }
            if (!whole && p.S > 1) {
#pragma unroll
              for (int w = 0; w < C::VB / 4; ++w) odd |= FP8 ? kv_nan4(x[t][w]) : kv_odd2<BF>(x[t][w]);
            }
          }
#pragma unroll
          for (int w = 0; w < C::VB / 4; ++w) {
            if constexpr (!FP8) {  // word w: dims 2w, 2w + 1 of the piece
              const uint32_t a[4] = {__byte_perm(x[0][w], x[1][w], 0x5410), __byte_perm(x[0][w], x[1][w], 0x7632),
                                     __byte_perm(x[2][w], x[3][w], 0x5410), __byte_perm(x[2][w], x[3][w], 0x7632)};
              #pragma unroll
              for (int n = 0; n < NB; ++n) kv_mma<BF>(acc[v * 4 + w][n], a[0], a[1], a[2], a[3], pf[n][0], pf[n][1]);
            } else {  // word w: dims 4w .. 4w + 3
              const uint32_t p01 = __byte_perm(x[0][w], x[1][w], 0x5140), p23 = __byte_perm(x[0][w], x[1][w], 0x7362);
              const uint32_t r01 = __byte_perm(x[2][w], x[3][w], 0x5140), r23 = __byte_perm(x[2][w], x[3][w], 0x7362);
              const uint32_t a[4] = {kv_codes2(p01), kv_codes2_high(p01), kv_codes2(r01), kv_codes2_high(r01)};
              const uint32_t d[4] = {kv_codes2(p23), kv_codes2_high(p23), kv_codes2(r23), kv_codes2_high(r23)};
              const int t = v * (C::VD / 2) + 2 * w;
#pragma unroll
              for (int n = 0; n < NB; ++n) {
                kv_mma<BF>(acc[t][n], a[0], a[1], a[2], a[3], pf[n][0], pf[n][1]);
                kv_mma<BF>(acc[t + 1][n], d[0], d[1], d[2], d[3], pf[n][0], pf[n][1]);
              }
            }
          }
        }
      }
      stage = stage + 1 == C::kStages ? 0 : stage + 1;
      next = next + 1 == C::kStages ? 0 : next + 1;
    }
    kv_cp_wait<0>();

    if (__syncthreads_or(odd)) {
#pragma unroll 1
      for (int r = warp; r < NB * 8; r += kTokWarps)
        if (rows0 + r < rows_all)
          kv_careful_row<T, FP8>(p, seq, b, kvh, rows0 + r, lo, hi, part_o ? part_o + r * part_ld : nullptr,
                                 part_ml + r, lane);
    } else {
    // join the warps: their O (in units of 1) and statistics meet in shared memory
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float sum = l[n][e];
#pragma unroll
        for (int o = 4; o <= 16; o *= 2) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        const int r = n * 8 + 2 * c + e;
        if (g == 0) s_m[warp][r] = m[n][e], s_l[warp][r] = sum;
        float* o = so + (warp * NB * 8 + r) * LD;
        const float f = FP8 ? kv_pow2_over(vinv[n][e]) : 1.0f;
#pragma unroll
        for (int t = 0; t < OT; ++t) {
          // tile t: dims piece(t / (VD / 2)) + g * VD + 2 * (t % (VD / 2)) and the next
          const int d = (t / (C::VD / 2)) * 8 * C::VD + g * C::VD + 2 * (t % (C::VD / 2));
          o[d] = acc[t][n][e] * f;
          o[d + 1] = acc[t][n][2 + e] * f;
        }
      }
    __syncthreads();
    for (int i = tid; i < NB * 8 * (HD / 4); i += kKvTokenThreads) {
      const int r = i / (HD / 4), d = (i % (HD / 4)) * 4;
      const int row = rows0 + r;
      if (row >= rows_all || d >= p.H) continue;
      float M = s_m[0][r];
#pragma unroll
      for (int w = 1; w < kTokWarps; ++w) M = fmaxf(M, s_m[w][r]);
      float L = 0.0f, o0 = 0.0f, o1 = 0.0f, o2 = 0.0f, o3 = 0.0f;
#pragma unroll
      for (int w = 0; w < kTokWarps; ++w) {
        const float lw = s_l[w][r];
        if (s_m[w][r] == -CUDART_INF_F && lw == 0.0f) continue;
        const float f = kv_exp2(s_m[w][r] - (M == -CUDART_INF_F ? 0.0f : M));
        const float4 x = *reinterpret_cast<const float4*>(so + (w * NB * 8 + r) * LD + d);
        L = fmaf(lw, f, L);
        o0 = fmaf(x.x, f, o0), o1 = fmaf(x.y, f, o1), o2 = fmaf(x.z, f, o2), o3 = fmaf(x.w, f, o3);
      }
      if (part_o) {
        if (d == 0) part_ml[r] = make_float2(M, L);
        *reinterpret_cast<float4*>(part_o + r * part_ld + d) = make_float4(o0, o1, o2, o3);
      } else {
        const float inv = L == 0.0f ? 0.0f : 1.0f / L;
        VecT<T, 4> y;
        y.v[0] = Elem<T>::fromf(o0 * inv), y.v[1] = Elem<T>::fromf(o1 * inv);
        y.v[2] = Elem<T>::fromf(o2 * inv), y.v[3] = Elem<T>::fromf(o3 * inv);
        *reinterpret_cast<VecT<T, 4>*>(static_cast<bits*>(p.out) + row_of(row) + d) = y;
      }
    }
    }
    if (ranks > 1) {
      // the cluster's parts: each thread takes four dims of a row from all of them
      kv_cluster_sync();
      for (int i = rank * kKvTokenThreads + tid; i < NB * 8 * (HD / 4); i += ranks * kKvTokenThreads) {
        const int r = i / (HD / 4), d = (i % (HD / 4)) * 4;
        const int row = rows0 + r;
        if (row >= rows_all || d >= p.H) continue;
        const uint32_t at_ml = kv_smem(s_part + r), at_o = kv_smem(so + r * LD + d);
        float M = -CUDART_INF_F;
        for (int n = 0; n < ranks; ++n) M = fmaxf(M, kv_cluster_ld2(kv_cluster_at(at_ml, n)).x);
        const float base = M == -CUDART_INF_F ? 0.0f : M;
        float L = 0.0f, o0 = 0.0f, o1 = 0.0f, o2 = 0.0f, o3 = 0.0f;
        for (int n = 0; n < ranks; ++n) {
          const float2 ml = kv_cluster_ld2(kv_cluster_at(at_ml, n));
          const float4 x = kv_cluster_ld4(kv_cluster_at(at_o, n));
          if (ml.x == -CUDART_INF_F && ml.y == 0.0f) continue;
          const float f = kv_exp2(ml.x - base);
          L = fmaf(ml.y, f, L);
          o0 = fmaf(x.x, f, o0), o1 = fmaf(x.y, f, o1), o2 = fmaf(x.z, f, o2), o3 = fmaf(x.w, f, o3);
        }
        const float inv = L == 0.0f ? 0.0f : 1.0f / L;
        VecT<T, 4> y;
        y.v[0] = Elem<T>::fromf(o0 * inv), y.v[1] = Elem<T>::fromf(o1 * inv);
        y.v[2] = Elem<T>::fromf(o2 * inv), y.v[3] = Elem<T>::fromf(o3 * inv);
        *reinterpret_cast<VecT<T, 4>*>(static_cast<bits*>(p.out) + row_of(row) + d) = y;
      }
      kv_cluster_sync();  // no CTA leaves before its part has been read
    }
    __syncthreads();
  }
}

// Joins the parts of the problems that kv_token_kernel_t dealt to several CTAs.
// CTA (x, y): the problem that begins in CTA x there and goes on in others, if
// there is one; its rows y, y + gridDim.y, ..; with more than 8 parts the four
// warps share a row, else each takes rows of its own.
template <class T>
__global__ void __launch_bounds__(kKvTokenThreads) kv_join_kernel_t(const KvParams p) {
  using bits = typename Elem<T>::bits;
  __shared__ float s_o[kTokWarps][kKvMaxHead], s_l[kTokWarps];
  pdl_wait();  // it lets nothing start early: the next call's CTAs would take places unevenly
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int4 what = p.ws_join[blockIdx.x];  // b, kvh, first row, 2 * further CTAs + slot
  if (what.w < 2) return;
  const int b = what.x, kvh = what.y, rows0 = what.z, parts = (what.w >> 1) + 1, c0 = blockIdx.x;
  // Part 0 is the last segment of CTA c0, the others the first segments of theirs.
  const bool shared_row = parts > 8;
  const int rows = (int)p.R - rows0 < p.rt ? (int)p.R - rows0 : p.rt;
  const int dr = shared_row ? gridDim.y : gridDim.y * kTokWarps;
  const int n0 = shared_row ? warp : 0, dn = shared_row ? kTokWarps : 1;
  auto slot_of = [&](int n) -> int64_t { return 2 * (int64_t)(c0 + n) + (n == 0 ? what.w & 1 : 0); };
  for (int r = shared_row ? (int)blockIdx.y : (int)blockIdx.y * kTokWarps + warp; r < rows; r += dr) {
    float M = -CUDART_INF_F;
    for (int n = lane; n < parts; n += 32) {
      M = fmaxf(M, p.ws_ml[slot_of(n) * p.rt + r].x);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    const float base = M == -CUDART_INF_F ? 0.0f : M;
    float L = 0.0f, acc[kKvMaxHead / 32];
#pragma unroll
    for (int j = 0; j < kKvMaxHead / 32; ++j) acc[j] = 0.0f;
#pragma unroll 8
    for (int n = n0; n < parts; n += dn) {
      const int64_t s = slot_of(n);
      const float2 ml = p.ws_ml[s * p.rt + r];
      const float* o = p.ws_o + (s * p.rt + r) * p.H;
      const float f = exp2f(ml.x - base);
      L = fmaf(ml.y, f, L);
#pragma unroll
      for (int j = 0; j < kKvMaxHead / 128; ++j)
        if (lane * 4 + 128 * j < p.H) {
          float4 x = *reinterpret_cast<const float4*>(o + lane * 4 + 128 * j);
          if (f == 0.0f) x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);  // never written where a CTA had no units
          acc[4 * j] = fmaf(x.x, f, acc[4 * j]);
          acc[4 * j + 1] = fmaf(x.y, f, acc[4 * j + 1]);
          acc[4 * j + 2] = fmaf(x.z, f, acc[4 * j + 2]);
          acc[4 * j + 3] = fmaf(x.w, f, acc[4 * j + 3]);
        }
    }
    const int row = rows0 + r, tok = kv_div(row, p.by_g);
    bits* y = static_cast<bits*>(p.out) + (((int64_t)b * p.S + tok) * p.Nq + (int64_t)kvh * p.G + (row - tok * p.G)) * p.H;
    if (shared_row) {
      __syncthreads();  // the previous row's sums have been read
#pragma unroll
      for (int j = 0; j < kKvMaxHead / 128; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (lane * 4 + 128 * j < p.H) s_o[warp][lane * 4 + 128 * j + i] = acc[4 * j + i];
      if (lane == 0) s_l[warp] = L;
      __syncthreads();
      L = (s_l[0] + s_l[1]) + (s_l[2] + s_l[3]);
      const float inv = L == 0.0f ? 0.0f : 1.0f / L;
      for (int d = threadIdx.x; d < p.H; d += kKvTokenThreads)
        y[d] = Elem<T>::fromf(((s_o[0][d] + s_o[1][d]) + (s_o[2][d] + s_o[3][d])) * inv);
    } else {
      const float inv = L == 0.0f ? 0.0f : 1.0f / L;
#pragma unroll
      for (int j = 0; j < kKvMaxHead / 128; ++j)
        if (lane * 4 + 128 * j < p.H) {
          VecT<T, 4> v;
#pragma unroll
          for (int i = 0; i < 4; ++i) v.v[i] = Elem<T>::fromf(acc[4 * j + i] * inv);
          *reinterpret_cast<VecT<T, 4>*>(y + lane * 4 + 128 * j) = v;
        }
    }
  }
}

}  // namespace rope_gb300
