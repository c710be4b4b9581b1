// Attention over a paged cache for few rows (single tokens, short drafts): up to 16
// rows n * G of a (b, kvh), 16-bit T.
//
// Every cached byte is used once for 8 or 16 rows, so the pages' bandwidth is the
// bound: 64 single bfloat16 tokens over 1 to 8190 keys of 8 heads of 128, 167 us, 6.4
// TB/s; 256 over up to 2000, 173 us, 6.1; 8 over up to 8190, 30 us. One token over 778 keys
// takes 7.5 us, over 30000 29: there the start, the joining and a second launch count. Two warps bring units of 64 keys into a ring by TMA, box by box (a box:
// the rows of a unit that lie in one page, 64 elements wide), and run ahead of the
// four that compute, across problems too: nothing that those do between two
// problems (queries, joining, output) leaves the memory idle while the ring is
// filling. 96 KB of ring and two CTAs an SM; 192 KB and one above H = 128.
//
// Both products run on mma.m16n8k16 with the keys on the 16-row side, so that a
// group of up to 8 query heads fills the 8-column side:
//   S^T = K Q^T   (16 keys x 8 rows),   O^T += V^T P^T   (16 dims x 8 rows);
// a warp takes 16 keys of each unit. K and V lie in shared memory as TMA's 128-byte
// swizzle leaves them: ldmatrix reads both without bank conflicts, V transposed.
// P^T fragments come from S^T by movmatrix. Softmax: the running maximum moves only
// where a score passes it by 8 (in log2), so weights stay below 2^8 and the common
// unit costs one vote.
//
// Weights are rounded to T, the product's type, and their sum is of the unrounded ones: in
// bfloat16 outputs are off by 1.9e-3 where one rounding at the end gives 1.7e-3, in float16
// by 2.6e-4 for 2.1e-4.
//
// A value that no row sees is zeroed before the product. Where one that only some
// rows see is not finite, its zero weight in the others would make a NaN of it: the
// rows are then done over again one by one (paged_careful_row).
//
// Dealing. CTA i takes the part [i W / n, (i + 1) W / n) of the problems' weight W (their
// units, and what each costs beside) in the order of the problems (sequence, head): a
// problem that one CTA has whole goes to the output, the others' parts to the workspace (2
// slots a CTA: its first segment's, its last one's), with a word on the problem that the
// CTA begins and leaves unfinished, for paged_join_kernel_t. Without (no workspace, or more than
// kKvDealMost sequences) a CTA takes one problem. Few problems of caches that are not
// long: a cluster of CTAs each, whose parts meet in shared memory, so there is one
// launch and no workspace.
#pragma once

#include "kv_token.cuh"
#include "paged_careful.cuh"
#include "paged_maps.h"
#include "rope_tma.cuh"

namespace rope_gb300 {

constexpr int kPagedWarps = 4;                   // that compute
static_assert(kPagedUnit == 16 * kPagedWarps, "keys of a unit");

template <int HD, int NB>
struct PagedTokenCfg {
  static constexpr int SLABS = HD / 64;
  static constexpr int kHalf = SLABS * kPagedUnit * 128;  // bytes of K, and of V, in a stage
  static constexpr int kStage = 2 * kHalf;
  static constexpr int kStages = HD <= 64 ? 6 : 3;
  static constexpr int kCtas = HD <= 128 ? 2 : 1;  // on an SM
  static constexpr int kParts = NB * HD / 64;      // passes in which the warps' outputs meet
  static constexpr int kCols = HD / kParts;        // dims of a pass
  static constexpr int kMerge = kPagedWarps * NB * 8 * (kCols + 4) * 4;
  static constexpr int kRing = kStage * kStages;
  static constexpr int kSmem = 1024 + kRing + kMerge;
  static constexpr int kClusterPart = NB * 8 * (HD + 4) * 4;  // more, in clusters
  // 228 KB an SM; a CTA holds about 5 KB statically, and 1 KB is reserved for it
  static_assert(kCtas * (kSmem + 6144) <= 228 * 1024, "CTAs that are resident");
  static_assert(kSmem + kClusterPart + 5120 <= 227 * 1024, "a CTA of a cluster fits");
};

__device__ __forceinline__ void paged_tma(uint32_t dst, const CUtensorMap* map, int x, int row, int kvh, int page,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::
          "r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(row), "r"(kvh), "r"(page), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void paged_ldsm(uint32_t (&a)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ void paged_ldsm_t(uint32_t (&a)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3])
               : "r"(at)
               : "memory");
}

// Barrier of the computing warps.
__device__ __forceinline__ void paged_sync() { asm volatile("barrier.cta.sync 1, 128;" ::: "memory"); }
__device__ __forceinline__ bool paged_sync_or(bool x) {
  uint32_t y;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, 1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(y)
      : "r"((uint32_t)x)
      : "memory");
  return y != 0;
}

// What a problem weighs beside its units: queries, joining, output. Without it the CTA that
// had the shortest sequences' problems ended 15 to 40 us behind the others: 64 sequences of
// up to 8190 keys with 2 to 4 new tokens 204 us, 176 so.
template <int NB>
constexpr int kPagedTokenOver = NB == 1 ? 3 : 5;

struct PagedDeal {
  const int32_t* before;  // weight of one problem of the sequences before b, for each b, and of all
  int total;              // weight of all problems, below 2^31
  int ctas;               // that it is dealt to
  __device__ __forceinline__ int first(int cta) const {
    return cta < ctas ? (int)((uint64_t)(uint32_t)cta * (uint32_t)total / (uint32_t)ctas) : total;
  }
  __device__ __forceinline__ int owner(int unit) const {
    return (int)((((uint64_t)(uint32_t)unit + 1) * (uint32_t)ctas - 1) / (uint32_t)total);
  }
};

// The weight before each sequence, in shared memory; all threads come here. (Sequences side
// by side to threads side by side: 8 of them one after the other took a thread 3 us, one 1.5.)
template <int NB>
__device__ __forceinline__ PagedDeal paged_deal(const PagedParams& p, int32_t* before, int32_t* warp_sum,
                                                PagedTimes* times) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int WARPS = kPagedTokenThreads / 32;
  PagedTimes t = {0, 0};
  int upto = 0;  // the weight of the sequences before b0
  for (int b0 = 0; b0 < p.s.B; b0 += kPagedTokenThreads) {
    const int b = b0 + tid;
    int u = 0;
    if (b < p.s.B) {
      const PagedSeq q = paged_seq(p.s, b);
      if (paged_few(p, q)) u = paged_span(p, q).units() + kPagedTokenOver<NB>;
      if (p.shared) paged_time(p, q, &t);
    }
    int pre = u;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int x = __shfl_up_sync(0xffffffffu, pre, o);
      if (lane >= o) pre += x;
    }
    if (lane == 31) warp_sum[warp] = pre;
    __syncthreads();
    int at = upto + pre - u;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      const int x = warp_sum[w];
      if (w < warp) at += x;
      upto += x;
    }
    if (b < p.s.B) before[b] = at;
    __syncthreads();  // the sums have been read
  }
  if (tid == 0) before[p.s.B] = upto;
  if (p.shared) paged_times(t, times + warp);
  __syncthreads();
  PagedDeal d;
  d.before = before;
  d.total = upto * p.Nkv;
  d.ctas = p.deal;
  if (p.shared) {  // those of the SMs that the other kernel leaves
    d.ctas = p.deal * (152 - paged_shares<WARPS>(times)) / 152;
    if (d.ctas < 1) d.ctas = 1;
  }
  return d;
}

// The problems of a CTA, one after the other, and its units of each.
template <int NB>
struct PagedWork {
  int at, last;      // weight left (dealt)
  int b, kvh, u0, u1;
  PagedSeq seq;
  PagedSpan span;
  bool whole;        // all of the problem
  __device__ __forceinline__ bool next(const PagedParams& p, const PagedDeal& d, int segment) {
    if (p.deal > 0) {
      if (at >= last) return false;
      int x = 0, y = p.s.B;  // the sequence of `at`: before[x] <= . < before[y]
      while (y - x > 1) {
        const int mid = (x + y) >> 1;
        if (d.before[mid] * p.Nkv <= at)
          x = mid;
        else
          y = mid;
      }
      // a problem's weight: kPagedTokenOver of nothing, then a unit each
      constexpr int OVER = kPagedTokenOver<NB>;
      const int weight = d.before[x + 1] - d.before[x];
      int in = at - d.before[x] * p.Nkv;
      b = x;
      kvh = (int)((uint32_t)in / (uint32_t)weight);
      in -= kvh * weight;
      if (in < OVER) {
        at += OVER - in;
        in = OVER;
        if (at >= last) return false;
      }
      u0 = in - OVER;
      u1 = u0 + (last - at) < weight - OVER ? u0 + (last - at) : weight - OVER;
      whole = u0 == 0 && u1 == weight - OVER;
      at += u1 - u0;
      seq = paged_seq(p.s, b);
      span = paged_span(p, seq);
      return true;
    }
    if (segment > 0) return false;
    const int ranks = p.cluster > 1 ? p.cluster : 1;
    const int problem = (int)blockIdx.x / ranks, rank = (int)blockIdx.x - problem * ranks;
    b = problem / p.Nkv;
    kvh = problem - b * p.Nkv;
    seq = paged_seq(p.s, b);
    span = paged_span(p, seq);
    const int units = paged_few(p, seq) ? span.units() : 0;
    u0 = (int)((int64_t)units * rank / ranks);
    u1 = (int)((int64_t)units * (rank + 1) / ranks);
    whole = ranks == 1;
    return units > 0;
  }
};

template <class T, int HD, int NB>
__global__ void __launch_bounds__(kPagedTokenThreads, PagedTokenCfg<HD, NB>::kCtas)
    paged_token_kernel_t(const PagedParams p, const __grid_constant__ PagedMaps maps) {
  using C = PagedTokenCfg<HD, NB>;
  using bits = typename Elem<T>::bits;
  constexpr bool BF = kIsBf16<T>;
  constexpr int KB = HD / 16;  // 16-dim blocks
  extern __shared__ uint8_t paged_smem[];
  __shared__ float s_m[kPagedWarps][NB * 8], s_l[kPagedWarps][NB * 8];
  __shared__ int32_t s_before[kKvDealMost + 1], s_sum[kPagedTokenThreads / 32];
  __shared__ float2 s_part[NB * 8];
  __shared__ uint64_t s_full[C::kStages], s_empty[C::kStages];
  __shared__ PagedTimes s_times[kPagedTokenThreads / 32];
  const uint32_t ring = (kv_smem(paged_smem) + 1023u) & ~1023u;
  float* const merge = reinterpret_cast<float*>(paged_smem + (ring - kv_smem(paged_smem)) + C::kRing);
  float* const part_smem = merge + C::kMerge / 4;  // in clusters
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(kv_smem(&s_full[i]), 2);
      mbar_init(kv_smem(&s_empty[i]), kPagedWarps);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (tid == kPagedWarps * 32) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&maps.k)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&maps.v)) : "memory");
  }
  pdl_launch_dependents();
  // Beside paged_tile_kernel_t, which begins after all that came before and lets this
  // kernel start then, its end is waited for at this one's.
  if (!p.shared)
    pdl_wait();
  else
    __syncthreads();
  PagedDeal deal;
  deal.before = s_before;
  deal.total = deal.ctas = 0;
  PagedWork<NB> work;
  work.at = work.last = 0;
  if (p.deal > 0) {
    deal = paged_deal<NB>(p, s_before, s_sum, s_times);
    if (deal.total > 0) {
      work.at = deal.first(blockIdx.x);
      work.last = deal.first(blockIdx.x + 1);
    }
    // so far nothing begins here that goes on elsewhere, and nothing of this CTA's counts
    // where a problem's CTAs lie on both sides of it
    if (tid == 0) p.ws_join[blockIdx.x] = make_int4(0, 0, 0, 0);
    if (work.at >= work.last && tid < NB * 8)
      p.ws_ml[2 * (int64_t)blockIdx.x * (NB * 8) + tid] = make_float2(-CUDART_INF_F, 0.0f);
  } else {
    __syncthreads();
  }
  // every sequence's lengths are looked at once
  if (p.s.status)
    for (int64_t b = (int64_t)blockIdx.x * kPagedTokenThreads + tid; b < p.s.B; b += (int64_t)gridDim.x * kPagedTokenThreads)
      paged_flag_seq(p.s, (int)b, paged_seq(p.s, (int)b));
  const int ranks = p.cluster > 1 ? p.cluster : 1;
  bool ok = true;

  if (warp >= kPagedWarps) {
    // ------------------------------------------------------------ K, V: a warp each
    const bool is_k = warp == kPagedWarps;
    const CUtensorMap* const map = is_k ? &maps.k : &maps.v;
    const uint32_t half = ring + (is_k ? 0 : C::kHalf);
    const int chunks = kPagedUnit / p.chunk;         // boxes of a slab in a unit
    const int mine = lane & (chunks - 1), slab = lane / chunks;  // this lane's rows and slab, or unit of a batch
    int it = 0;
    bool bad = false;
    for (int segment = 0; ok && work.next(p, deal, segment); ++segment) {
      const int base = work.span.lo + mine * p.chunk;
      const int end = work.span.end;
      const int32_t* table = p.s.table + (int64_t)work.b * p.s.max_pages;
      const int seen = paged_first(p, work.seq.past);  // keys before this are nobody's
      // The table's entries of `batch` units at a time, a lane each, and those of the batch
      // behind it on their way: a load that was waited for at each unit (1000 clocks) kept an
      // SM below 42 GB/s.
      auto entry = [&](int u) {
        const int j = base + u * kPagedUnit;
        return u < work.u1 && j < end && j + p.chunk > seen ? __ldg(table + kv_div(j, p.s.by_ps)) : -1;
      };
      const int batch = 32 / chunks;
      int pages = entry(work.u0 + slab), pages_next = entry(work.u0 + batch + slab);
      for (int u = work.u0, in = 0; u < work.u1; ++u, ++it, ++in) {
        if (in == batch) {
          in = 0;
          pages = pages_next;
          pages_next = entry(u + batch + slab);
        }
        const int page = __shfl_sync(0xffffffffu, pages, in * chunks + mine);
        const int st = it % C::kStages;
        if (it >= C::kStages) ok = mbar_wait(kv_smem(&s_empty[st]), (it / C::kStages - 1) & 1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const uint32_t full = kv_smem(&s_full[st]);
        // rows behind the keys are not copied: what lies there is nobody's
        const int live = (end - (work.span.lo + u * kPagedUnit) + p.chunk - 1) / p.chunk;
        if (lane == 0)
          mbar_arrive_expect_tx(full, (uint32_t)(live < 0 ? 0 : live < chunks ? live : chunks) * C::SLABS * p.chunk * 128);
        __syncwarp();
        const int j = base + u * kPagedUnit;
        if (slab < C::SLABS && j < end) {
          const bool in_pool = (uint32_t)page < (uint32_t)p.s.pages;
          bad |= !in_pool && j + p.chunk > seen;
          // (in a page that does not exist TMA fills in zeros)
          paged_tma(half + st * C::kStage + slab * (kPagedUnit * 128) + mine * p.chunk * 128, map, slab * 64,
                    j - kv_div(j, p.s.by_ps) * p.s.ps, work.kvh, in_pool ? page : -1, full);
        }
      }
    }
    if (bad && p.s.status) atomicOr(p.s.status, 4);
    if (!ok) {  // what is on its way has to land before shared memory goes
      for (int i = it - C::kStages < 0 ? 0 : it - C::kStages; i < it; ++i)
        mbar_wait(kv_smem(&s_full[i % C::kStages]), (i / C::kStages) & 1);
    }
  } else {
    const int g = lane >> 2, c = lane & 3;
    // ldmatrix: this lane's row and 16-byte piece of a 16 x 16 block, swizzled
    const int krow = (lane & 7) + (lane >> 3 & 1) * 8, vrow = (lane & 7) + (lane >> 4) * 8;
    const uint32_t kat = (uint32_t)(warp * 16 + krow) * 128, kx = (uint32_t)((lane >> 4) ^ (lane & 7));
    const uint32_t vat = (uint32_t)(warp * 16 + vrow) * 128 + C::kHalf, vx = (uint32_t)((lane >> 3 & 1) ^ (lane & 7));
    int it = 0;
    for (int segment = 0; ok && work.next(p, deal, segment); ++segment) {
      const int b = work.b, kvh = work.kvh;
      const PagedSeq& seq = work.seq;
      const int rows_all = seq.n * p.G;
      const int end = work.span.end;
      // the one problem that begins in this CTA and goes on in others: paged_join_kernel_t's
      if (p.deal > 0 && work.u0 == 0 && !work.whole && tid == 0) {
        const int parts = deal.owner(work.at - work.u1 + work.span.units() - 1) - (int)blockIdx.x;
        p.ws_join[blockIdx.x] = make_int4(b, kvh, 0, 2 * parts + (segment > 0 ? 1 : 0));
      }
      const int64_t slot = 2 * (int64_t)blockIdx.x + (segment > 0 ? 1 : 0);
      const int part_ld = ranks > 1 ? HD + 4 : p.H;
      float* const part_o = work.whole ? nullptr : ranks > 1 ? part_smem : p.ws_o + slot * (NB * 8) * p.H;
      float2* const part_ml = work.whole ? nullptr : ranks > 1 ? s_part : p.ws_ml + slot * (NB * 8);
      auto row_of = [&](int r) {
        const int tok = kv_div(r, p.by_g);
        return ((seq.t0 + tok) * p.Nq + (int64_t)kvh * p.G + (r - tok * p.G)) * p.H;
      };
      uint32_t qf[NB][KB][2];
#pragma unroll
      for (int n = 0; n < NB; ++n) {
        const int r = n * 8 + g;
        const bits* src = static_cast<const bits*>(p.q) + (r < rows_all ? row_of(r) : 0);
#pragma unroll
        for (int k = 0; k < KB; ++k)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int d = k * 16 + h * 8 + 2 * c;
            qf[n][k][h] = 0;
            if (r < rows_all && d < p.H) qf[n][k][h] = __ldg(reinterpret_cast<const uint32_t*>(src + d));
          }
      }
      // the rows whose scores this lane holds: 2c and 2c + 1 of each column tile
      float slope[NB][2], m[NB][2], l[NB][2];
      int pos[NB][2], lim[NB][2], from[NB][2];
      uint64_t word[NB][2];
      const float c1 = p.cap > 0.0f ? 2.0f * kLog2e * p.over : p.scale * kLog2e;
      const float c2 = p.cap * kLog2e;
      int full = 0x7fffffff, below = 0;  // keys in [below, full) are seen by every row
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = n * 8 + 2 * c + e;
          const bool live = r < rows_all;
          const int tok = live ? kv_div(r, p.by_g) : 0;
          pos[n][e] = seq.past + tok;
          lim[n][e] = live ? paged_limit(p, seq, pos[n][e]) : 0;
          from[n][e] = paged_first(p, pos[n][e]);
          word[n][e] = p.masks && live ? (uint64_t)__ldg(p.masks + seq.t0 + tok) : ~0ull;
          slope[n][e] = p.slopes && live ? __ldg(p.slopes + kvh * p.G + (r - tok * p.G)) * kLog2e : 0.0f;
          if (live) {
            const int f = p.masks && seq.past < lim[n][e] ? seq.past : lim[n][e];
            full = f < full ? f : full;
            below = from[n][e] > below ? from[n][e] : below;
          }
          m[n][e] = -CUDART_INF_F;
          l[n][e] = 0.0f;
        }
#pragma unroll
      for (int o = 1; o <= 2; o *= 2) {
        const int x = __shfl_xor_sync(0xffffffffu, full, o), y = __shfl_xor_sync(0xffffffffu, below, o);
        full = x < full ? x : full;
        below = y > below ? y : below;
      }
      float acc[KB][NB][4];
#pragma unroll
      for (int t = 0; t < KB; ++t)
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[t][n][i] = 0.0f;
      bool odd = false;  // an infinity or a NaN in a value that not every row sees

      // The products of a unit's keys with Q, two sums: half as long a chain of dependent ones.
      auto scores = [&](int stage, float (&s)[NB][4]) {
        const uint32_t at = ring + stage * C::kStage;
        float t[NB][4];
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[n][i] = t[n][i] = 0.0f;
#pragma unroll
        for (int k = 0; k < KB; ++k) {
          uint32_t a[4];
          paged_ldsm(a, at + kat + (k >> 2) * (kPagedUnit * 128) + ((((2 * k) & 7) ^ kx) << 4));
#pragma unroll
          for (int n = 0; n < NB; ++n) kv_mma<BF>(k & 1 ? t[n] : s[n], a[0], a[1], a[2], a[3], qf[n][k][0], qf[n][k][1]);
        }
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[n][i] += t[n][i];
      };
      for (int u = work.u0; u < work.u1; ++u, ++it) {
        const int st = it % C::kStages;
        const int j0 = work.span.lo + u * kPagedUnit + warp * 16;
        ok = mbar_wait(kv_smem(&s_full[st]), (it / C::kStages) & 1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (j0 < end) {
          const uint32_t at = ring + st * C::kStage;
          float s[NB][4];
          scores(st, s);
          const bool whole = j0 >= below && j0 + 16 <= full;  // uniform over the warp
          uint32_t any0 = 0xffffffffu, any1 = 0xffffffffu;
          bool seen0 = false, seen1 = false, moved = false;
#pragma unroll
          for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float x = s[n][e] * c1, y = s[n][2 + e] * c1;
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
                auto see = [&](int j) {
                  bool on = j >= from[n][e] && j < lim[n][e];
                  if (p.masks && j >= seq.past) on = on && j - seq.past < 64 && (word[n][e] >> (j - seq.past) & 1);
                  return on;
                };
                const bool a = see(j0 + g), d = see(j0 + g + 8);
                x = a ? x : -CUDART_INF_F;
                y = d ? y : -CUDART_INF_F;
                seen0 |= a;
                seen1 |= d;
              }
              s[n][e] = x;
              s[n][2 + e] = y;
              moved |= fmaxf(x, y) > m[n][e] + 8.0f;
            }
          if (!whole) {
            any0 = __ballot_sync(0xffffffffu, seen0);
            any1 = __ballot_sync(0xffffffffu, seen1);
          }
          if (any0 | any1) {  // keys that no row sees are left out
            if (__any_sync(0xffffffffu, moved)) {
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
#pragma unroll
                  for (int t = 0; t < KB; ++t) {
                    acc[t][n][e] *= a;
                    acc[t][n][2 + e] *= a;
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
              }
              pf[n][0] = kv_transpose8(kv_pack2<BF>(w[0], w[1]));
              pf[n][1] = kv_transpose8(kv_pack2<BF>(w[2], w[3]));
            }
            // keys 2c, 2c + 1 (low, high half) and 2c + 8, 2c + 9: whether some row sees them
            const uint32_t on0 = ((any0 >> (8 * c)) & 15u ? 0xffffu : 0u) | ((any0 >> (8 * c + 4)) & 15u ? 0xffff0000u : 0u);
            const uint32_t on1 = ((any1 >> (8 * c)) & 15u ? 0xffffu : 0u) | ((any1 >> (8 * c + 4)) & 15u ? 0xffff0000u : 0u);
#pragma unroll
            for (int t = 0; t < KB; ++t) {
              uint32_t a[4];
              paged_ldsm_t(a, at + vat + (t >> 2) * (kPagedUnit * 128) + ((((2 * t) & 7) ^ vx) << 4));
              if (!whole) {
                a[0] &= on0, a[1] &= on0, a[2] &= on1, a[3] &= on1;
                if (seq.n > 1) odd |= kv_odd2<BF>(a[0]) || kv_odd2<BF>(a[1]) || kv_odd2<BF>(a[2]) || kv_odd2<BF>(a[3]);
              }
#pragma unroll
              for (int n = 0; n < NB; ++n) kv_mma<BF>(acc[t][n], a[0], a[1], a[2], a[3], pf[n][0], pf[n][1]);
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(kv_smem(&s_empty[st]));
      }
      if (paged_sync_or(!ok)) {
        ok = false;
        break;
      }
      const int lo = work.span.lo + work.u0 * kPagedUnit;
      const int hi = work.span.lo + work.u1 * kPagedUnit < end ? work.span.lo + work.u1 * kPagedUnit : end;
      if (paged_sync_or(odd)) {
#pragma unroll 1
        for (int r = warp; r < rows_all; r += kPagedWarps)
          paged_careful_row<T>(p, seq, b, kvh, r, lo, hi, part_o ? part_o + r * part_ld : nullptr, 4, part_ml + r,
                              lane);
      } else {
        // join the warps: their O and statistics meet in shared memory, some dims at a time
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float sum = l[n][e];
#pragma unroll
            for (int o = 4; o <= 16; o *= 2) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (g == 0) s_m[warp][n * 8 + 2 * c + e] = m[n][e], s_l[warp][n * 8 + 2 * c + e] = sum;
          }
        constexpr int LD = C::kCols + 4, PT = C::kCols / 16;
#pragma unroll
        for (int part = 0; part < C::kParts; ++part) {
#pragma unroll
          for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float* o = merge + (warp * NB * 8 + n * 8 + 2 * c + e) * LD;
#pragma unroll
              for (int t = 0; t < PT; ++t) {
                o[t * 16 + g] = acc[part * PT + t][n][e];
                o[t * 16 + g + 8] = acc[part * PT + t][n][2 + e];
              }
            }
          paged_sync();
          for (int i = tid; i < NB * 8 * (C::kCols / 4); i += kPagedWarps * 32) {
            const int r = i / (C::kCols / 4), in = (i % (C::kCols / 4)) * 4, d = part * C::kCols + in;
            if (r >= rows_all || d >= p.H) continue;
            float M = s_m[0][r];
#pragma unroll
            for (int w = 1; w < kPagedWarps; ++w) M = fmaxf(M, s_m[w][r]);
            float L = 0.0f, o0 = 0.0f, o1 = 0.0f, o2 = 0.0f, o3 = 0.0f;
#pragma unroll
            for (int w = 0; w < kPagedWarps; ++w) {
              const float lw = s_l[w][r];
              if (s_m[w][r] == -CUDART_INF_F && lw == 0.0f) continue;
              const float f = kv_exp2(s_m[w][r] - (M == -CUDART_INF_F ? 0.0f : M));
              const float4 x = *reinterpret_cast<const float4*>(merge + (w * NB * 8 + r) * LD + in);
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
              *reinterpret_cast<VecT<T, 4>*>(static_cast<bits*>(p.out) + row_of(r) + d) = y;
            }
          }
          paged_sync();
        }
      }
    }
  }
  if (!ok && p.s.status) atomicOr(p.s.status, 2);
  if (ranks > 1) {
    // the cluster's parts: each thread takes four dims of a row from all of them
    const int problem = (int)blockIdx.x / ranks, rank = (int)blockIdx.x - problem * ranks;
    const int b = problem / p.Nkv, kvh = problem - b * p.Nkv;
    const PagedSeq seq = paged_seq(p.s, b);
    const int rows_all = paged_few(p, seq) ? seq.n * p.G : 0;
    constexpr int LD = HD + 4;
    __syncthreads();
    kv_cluster_sync();
    for (int i = rank * kPagedTokenThreads + tid; i < rows_all * (HD / 4); i += ranks * kPagedTokenThreads) {
      const int r = i / (HD / 4), d = (i % (HD / 4)) * 4;
      if (d >= p.H) continue;
      const uint32_t at_ml = kv_smem(s_part + r), at_o = kv_smem(part_smem + r * LD + d);
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
      const int tok = kv_div(r, p.by_g);
      const int64_t at = ((seq.t0 + tok) * p.Nq + (int64_t)kvh * p.G + (r - tok * p.G)) * p.H;
      *reinterpret_cast<VecT<T, 4>*>(static_cast<bits*>(p.out) + at + d) = y;
    }
    kv_cluster_sync();  // no CTA leaves before its part has been read
  }
  if (p.shared && blockIdx.x == 0) pdl_wait();  // this kernel does not end before the other
}

// Loads that stay where they stand, ahead of what decides whether they count. Each value
// is read once, so L1 is passed by.
__device__ __forceinline__ float4 paged_load4(const float4* at) {
  float4 x;
  asm volatile("ld.global.cg.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w) : "l"(at) : "memory");
  return x;
}
__device__ __forceinline__ float2 paged_load2(const float2* at) {
  float2 x;
  asm volatile("ld.global.cg.v2.f32 {%0, %1}, [%2];" : "=f"(x.x), "=f"(x.y) : "l"(at) : "memory");
  return x;
}

// A lane's dims (4 lane + 128 j) of row r from the parts n0, n0 + dn, .. of a problem: its
// last segment's in CTA c0 (slot `last`), the first segments' of the CTAs behind. The loads of
// 8 parts are in flight together, what they count beside them.
__device__ __forceinline__ void paged_join_row(const PagedParams& p, int c0, int last, int parts, int n0, int dn, int r,
                                               int lane, float* M, float* L, float4 (&acc)[kKvMaxHead / 128]) {
  constexpr int NV = kKvMaxHead / 128, DEEP = 8;
  float top = -CUDART_INF_F, sum = 0.0f;
#pragma unroll
  for (int j = 0; j < NV; ++j) acc[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int n1 = n0; n1 < parts; n1 += DEEP * dn) {
    float2 ml[DEEP];
    float4 o[DEEP][NV];
#pragma unroll
    for (int k = 0; k < DEEP; ++k) {
      const int n = n1 + k * dn;
      ml[k] = make_float2(-CUDART_INF_F, 0.0f);
#pragma unroll
      for (int j = 0; j < NV; ++j) o[k][j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (n < parts) {
        const int at = (2 * (c0 + n) + (n == 0 ? last : 0)) * p.rt + r;
        ml[k] = paged_load2(p.ws_ml + at);
#pragma unroll
        for (int j = 0; j < NV; ++j)
          if (lane * 4 + 128 * j < p.H)
            o[k][j] = paged_load4(reinterpret_cast<const float4*>(p.ws_o + at * p.H) + lane + 32 * j);
      }
    }
    float m = top;
#pragma unroll
    for (int k = 0; k < DEEP; ++k) m = fmaxf(m, ml[k].x);
    const float base = m == -CUDART_INF_F ? 0.0f : m, a = exp2f(top - base);
    top = m;
    sum *= a;
#pragma unroll
    for (int j = 0; j < NV; ++j) acc[j].x *= a, acc[j].y *= a, acc[j].z *= a, acc[j].w *= a;
#pragma unroll
    for (int k = 0; k < DEEP; ++k) {
      const float f = exp2f(ml[k].x - base);
      sum = fmaf(ml[k].y, f, sum);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        // a CTA that had no units wrote nothing
        if (ml[k].x == -CUDART_INF_F && ml[k].y == 0.0f) o[k][j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        acc[j].x = fmaf(o[k][j].x, f, acc[j].x);
        acc[j].y = fmaf(o[k][j].y, f, acc[j].y);
        acc[j].z = fmaf(o[k][j].z, f, acc[j].z);
        acc[j].w = fmaf(o[k][j].w, f, acc[j].w);
      }
    }
  }
  *M = top;
  *L = sum;
}

// Joins the parts of the problems that paged_token_kernel_t dealt to several CTAs.
// CTA (x, y): the problem that begins in CTA x there and goes on in others, if there
// is one; its rows y, y + gridDim.y, ... Each warp takes rows of its own, or, where a
// problem has more than 8 parts and each row a CTA, all four share it (8 sequences of up to
// 8190 keys, 10 parts: all sharing one row after the other 38 us for the call, 30 so).
template <class T>
__global__ void __launch_bounds__(kKvTokenThreads) paged_join_kernel_t(const PagedParams p) {
  using bits = typename Elem<T>::bits;
  constexpr int NV = kKvMaxHead / 128;
  __shared__ float4 s_o[kTokWarps][kKvMaxHead / 4];
  __shared__ float s_l[kTokWarps], s_m[kTokWarps];
  // It lets nothing start early: the next call's CTAs would take places unevenly. Behind
  // paged_tile_join_kernel_t, which begins after all parts are there, that one's end is
  // waited for at this one's.
  if (!p.shared)
    pdl_wait();
  else if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x < 32)
    pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int4 what = p.ws_join[blockIdx.x];  // b, kvh, -, 2 * further CTAs + slot
  if (what.w < 2) return;
  const int b = what.x, kvh = what.y, parts = (what.w >> 1) + 1, c0 = blockIdx.x, last = what.w & 1;
  const bool shared_row = parts > 8 && gridDim.y > 1;
  const PagedSeq seq = paged_seq(p.s, b);
  const int rows = seq.n * p.G;
  const int dr = shared_row ? gridDim.y : gridDim.y * kTokWarps;
  for (int r = shared_row ? (int)blockIdx.y : (int)blockIdx.y * kTokWarps + warp; r < rows; r += dr) {
    float M, L;
    float4 acc[NV];
    paged_join_row(p, c0, last, parts, shared_row ? warp : 0, shared_row ? kTokWarps : 1, r, lane, &M, &L, acc);
    if (shared_row) {
      __syncthreads();  // the previous row's sums have been read
#pragma unroll
      for (int j = 0; j < NV; ++j) s_o[warp][lane + 32 * j] = acc[j];
      if (lane == 0) s_m[warp] = M, s_l[warp] = L;
      __syncthreads();
      if (warp > 0) continue;
      float top = s_m[0];
#pragma unroll
      for (int w = 1; w < kTokWarps; ++w) top = fmaxf(top, s_m[w]);
      const float base = top == -CUDART_INF_F ? 0.0f : top;
      L = 0.0f;
#pragma unroll
      for (int j = 0; j < NV; ++j) acc[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int w = 0; w < kTokWarps; ++w) {
        const float f = exp2f(s_m[w] - base);
        L = fmaf(s_l[w], f, L);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          const float4 x = s_o[w][lane + 32 * j];
          acc[j].x = fmaf(x.x, f, acc[j].x);
          acc[j].y = fmaf(x.y, f, acc[j].y);
          acc[j].z = fmaf(x.z, f, acc[j].z);
          acc[j].w = fmaf(x.w, f, acc[j].w);
        }
      }
    }
    const int tok = kv_div(r, p.by_g);
    bits* y = static_cast<bits*>(p.out) + ((seq.t0 + tok) * p.Nq + (int64_t)kvh * p.G + (r - tok * p.G)) * p.H;
    const float inv = L == 0.0f ? 0.0f : 1.0f / L;
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (lane * 4 + 128 * j < p.H) {
        VecT<T, 4> v;
        v.v[0] = Elem<T>::fromf(acc[j].x * inv);
        v.v[1] = Elem<T>::fromf(acc[j].y * inv);
        v.v[2] = Elem<T>::fromf(acc[j].z * inv);
        v.v[3] = Elem<T>::fromf(acc[j].w * inv);
        *reinterpret_cast<VecT<T, 4>*>(y + lane * 4 + 128 * j) = v;
      }
  }
}

}  // namespace rope_gb300
