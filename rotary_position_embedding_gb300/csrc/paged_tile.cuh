// Attention over a paged cache for many rows (prompts, chunks, draft trees): tcgen05.
//
// What is done with a key tile is what kv_tile_kernel_t (kv_tile.cuh) does: two tiles
// of 128 rows take turns on the tensor cores, S and O in TMEM, P = 2^(x - m) by the
// threads that own the rows, the base moved only where a tile's weights ask for it.
//
// One CTA an SM stays for the whole call. The work is the key tiles of all items (up to
// ROWS rows of a sequence, whole tokens) and heads, and CTA i takes the part [i W / n, (i +
// 1) W / n) of their weight W, an item's being its key tiles and over_item for its beginning
// and its output: sequences of any lengths, few long ones and many short ones, even out, and
// nothing is split where it need not be. An item that one CTA has whole goes to the
// output, the others' parts to the workspace (2 slots a CTA), where
// paged_tile_join_kernel_t adds them up. The roles run through a CTA's segments
// without meeting: while the last tile of one is with the softmax threads and its
// output is on its way, K, V and Q of the next come in and its first products run.
//   Warps (12): 0-3 and 4-7 softmax and output of row tile 0 and 1, a thread a row; 8 and 9
//   bring K and V by TMA in boxes (the rows of a key tile that lie in one page x 64
//   elements), a lane a box, the next tile's pages looked up a step ahead; 10 brings Q as
//   soon as the last product of the segment before has read its own; 11 issues every MMA.
// V's rows behind the last key have to be zeros (their weights are, and 0 * NaN is not):
// boxes of such rows are asked for in a page that does not exist, and the box that holds
// the last key is brought in boxes of 8 rows and of one (all rows one by one, for K too,
// a segment began 4 us later with pages of 64). What K has there only hidden scores get.
// A row sees keys from its window on; of a draft tree's new keys those whose bit its
// mask holds. Only key tiles that some row does not see whole are looked at key by key,
// as bits of four words.
// Outputs leave in rows of 128 bytes, turned among 8 lanes by shuffles (a thread's own
// row, 16 bytes of 32 rows at a time, took 3 us an item); parts lie in the workspace with
// the same 4 dims of all rows side by side.
// Bound by the tensor cores for long prompts (8192 bfloat16 tokens, 32/8 heads of 128: 372 to
// 382 us, 1440 to 1476 Tflop/s); caps by the tanh between the products (2.5 us a key tile for 1.57); short
// calls by what comes before the first product (6.5 us: lengths, items, table, K) and by
// joining (one tree of 60 drafts behind 8000 keys 22 us, 32 trees over up to 4096 keys 79;
// 5 prompts of 100 to 1531 tokens that see 512 keys 35).
//
// Weights are rounded to T, as the product with V takes them, and their sum is of the
// unrounded ones: outputs are off by 1.9e-3 to 2.2e-3 in bfloat16 where one rounding at the
// end gives 1.65e-3, by 2.7e-4 in float16 for 2.1e-4. (Two products, of the weights and of
// what rounding took from them, would be half as many again as Q K and P V.)
//
// Without a workspace, or with more than kPagedItems items, a CTA takes one item and looks
// the lengths over for itself: 700 sequences of 33 tokens over 200 keys 289 us, 800 497.
#pragma once

#include "kv_tile.cuh"
#include "paged_token.cuh"

namespace rope_gb300 {

constexpr int kPagedTileThreads = kPagedTileBlock;

struct PagedTileBars {
  uint64_t k_full[2], k_free[2], v_full[2], v_free[2], s_full[2], p_full[2], o_full[2], q_full, q_free, drain;
};

// An item: tokens [tok0, tok0 + ntok) of sequence b, which are the batch's [g0, ..) and at
// rows [pos0, ..). Its keys are [start, end), start at the beginning of a key tile.
struct alignas(16) PagedItem {
  int b, tok0, start, end;
  int g0, ntok, pos0, total;  // total: rows of the sequence
  __device__ __forceinline__ PagedSeq seq() const {
    PagedSeq q;
    q.t0 = g0 - tok0;
    q.n = tok0 + ntok;
    q.past = pos0 - tok0;
    q.total = total;
    return q;
  }
};
__device__ __forceinline__ PagedItem paged_item(const PagedParams& p, const PagedSeq& q, int b, int tile, int keys) {
  PagedItem it;
  it.b = b;
  it.tok0 = tile * p.tpi;
  it.ntok = q.n - it.tok0 < p.tpi ? q.n - it.tok0 : p.tpi;
  it.g0 = (int)q.t0 + it.tok0;
  it.pos0 = q.past + it.tok0;
  it.total = q.total;
  it.start = paged_first(p, it.pos0) / keys * keys;
  it.end = paged_limit(p, q, it.pos0 + it.ntok - 1);
  return it;
}
// Its key tiles; one where there are no keys, so that its output is written.
__device__ __forceinline__ int paged_item_tiles(const PagedItem& it, int keys) {
  return it.end > it.start ? (it.end - it.start + keys - 1) / keys : 1;
}

// An inclusive sum over the CTA's threads, and the sum of all.
__device__ __forceinline__ int paged_scan(int n, int* s_sum, int* all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const int x = __shfl_up_sync(0xffffffffu, n, o);
    if (lane >= o) n += x;
  }
  __syncthreads();  // the sums before have been read
  if (lane == 31) s_sum[warp] = n;
  __syncthreads();
  int a = 0;
#pragma unroll
  for (int w = 0; w < kPagedTileThreads / 32; ++w) {
    const int x = s_sum[w];
    if (w < warp) n += x;
    a += x;
  }
  *all = a;
  return n;
}

// The items of the batch and the weight of one head of those before each, in shared
// memory; their number. Not dealt: only item number `only`, or none. With p.shared none
// where the CTA is beyond this kernel's share, `ctas`. All threads come here, and the
// tables hold when it returns.
__device__ __forceinline__ int paged_items(const PagedParams& p, int only, int keys, PagedItem* items, int32_t* before,
                                           int* s_sum, PagedTimes* times, uint32_t* ctas) {
  const int tid = threadIdx.x;
  int count = 0;
  PagedTimes t_all = {0, 0};
  for (int b0 = 0; b0 < p.s.B; b0 += kPagedTileThreads) {
    const int b = b0 + tid;
    PagedSeq q;
    int n = 0, all;
    if (b < p.s.B) {
      q = paged_seq(p.s, b);
      if (!(p.mixed && paged_few(p, q))) n = (q.n + p.tpi - 1) / p.tpi;
      if (p.shared) paged_time(p, q, &t_all);
    }
    const int first = paged_scan(n, s_sum, &all) - n + count;
    if (p.deal > 0) {
      if (b < p.s.B) before[b] = first;  // for now; there are at least as many items planned as sequences
    } else if (only >= first && only < first + n) {
      items[0] = paged_item(p, q, b, first + n - 1 - only, keys);  // the longest rows first
    }
    count += all;
    if (p.deal == 0 && only < count) break;  // the same for all threads
  }
  if (p.shared) paged_times(t_all, times + (tid >> 5));
  __syncthreads();
  *ctas = (uint32_t)p.deal;
  if (p.shared) {
    const uint32_t n = (uint32_t)paged_shares<kPagedTileThreads / 32>(times);
    *ctas = n < 1 ? 1 : n < *ctas ? n : *ctas;
    if (blockIdx.x >= *ctas) return 0;
  }
  if (p.deal == 0) return only < count ? 1 : 0;
  if (count > p.items) count = p.items;  // more than planned for only where query_starts does not ascend
  // Items of one length lie side by side; they are strewn (i -> i s mod count, s a prime
  // above count / 2 or coprime to it), so that each CTA has some of every kind: a prompt's
  // shortest items, each of masked tiles alone, cost more than they weigh.
  static_assert(kPagedItems == 2 * kPagedTileThreads, "two items a thread");
  const uint32_t n389 = 389u % (uint32_t)(count > 0 ? count : 1), n241 = 241u % (uint32_t)(count > 0 ? count : 1);
  auto far = [&](uint32_t r) { return r < count - r ? r : count - r; };
  const uint32_t s = count % 389 == 0 || (count % 241 != 0 && far(n241) > far(n389)) ? 241u : 389u;
  PagedItem mine[2];
  int n[2] = {0, 0}, sum;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint32_t i = 2 * tid + k;
    if (i >= (uint32_t)count) continue;
    const int at = (int)(i * s % (uint32_t)count);
    int x = 0, y = p.s.B;  // its sequence
    while (y - x > 1) {
      const int mid = (x + y) >> 1;
      if (before[mid] <= at)
        x = mid;
      else
        y = mid;
    }
    mine[k] = paged_item(p, paged_seq(p.s, x), x, at - before[x], keys);
    n[k] = paged_item_tiles(mine[k], keys) + p.over_item;
  }
  const int first = paged_scan(n[0] + n[1], s_sum, &sum) - n[0] - n[1];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int i = 2 * tid + k;
    if (i >= count) continue;
    items[i] = mine[k];
    before[i] = first + (k > 0 ? n[0] : 0);
  }
  if (tid == 0) before[count] = sum;
  __syncthreads();
  return count;
}

// The weight dealt out: CTA i has [first(i), first(i + 1)).
struct PagedTileShares {
  uint32_t per, more;  // each has `per`, the first `more` of them one more
  __device__ __forceinline__ void set(uint32_t total, uint32_t ctas) {
    per = total / ctas;
    more = total - per * ctas;
  }
  __device__ __forceinline__ uint32_t first(uint32_t cta) const { return cta * per + (cta < more ? cta : more); }
  __device__ __forceinline__ uint32_t owner(uint32_t at) const {
    const uint32_t upto = more * (per + 1);
    return at < upto ? at / (per + 1) : more + (at - upto) / per;
  }
};

// The beginning of an item and head, or the end of the last, that is nearest to `at`.
__device__ __forceinline__ int paged_nearest(const PagedParams& p, int at, const int32_t* before, int count) {
  if (count == 0) return 0;
  int x = 0, y = count;
  while (y - x > 1) {
    const int mid = (x + y) >> 1;
    if (before[mid] * p.Nkv <= at)
      x = mid;
    else
      y = mid;
  }
  const int weight = before[x + 1] - before[x], in = at - before[x] * p.Nkv;
  return at - in + (int)((uint32_t)(2 * in + weight) / (uint32_t)(2 * weight)) * weight;
}

// The segments of a CTA, one after the other: key tiles [u0, u1) of an item and head.
struct PagedTileWork {
  int at, last;     // weight left
  int item, kvh, u0, u1;
  bool whole;       // all of the item
  __device__ __forceinline__ bool next(const PagedParams& p, const int32_t* before, int count) {
    if (at >= last) return false;
    if (p.deal == 0) {
      item = 0;
      kvh = (int)(blockIdx.x % (uint32_t)p.Nkv);
      u0 = 0;
      u1 = last;
      whole = true;
      at = last;
      return true;
    }
    int x = 0, y = count;
    while (y - x > 1) {
      const int mid = (x + y) >> 1;
      if (before[mid] * p.Nkv <= at)
        x = mid;
      else
        y = mid;
    }
    // an item's weight: p.over_item of nothing, then a tile each
    int weight = before[x + 1] - before[x], in = at - before[x] * p.Nkv;
    kvh = (int)((uint32_t)in / (uint32_t)weight);
    in -= kvh * weight;
    if (in < p.over_item) {
      at += p.over_item - in;
      in = p.over_item;
      if (at >= last) return false;
    }
    item = x;
    const int tiles = weight - p.over_item;
    u0 = in - p.over_item;
    u1 = u0 + (last - at) < tiles ? u0 + (last - at) : tiles;
    whole = u0 == 0 && u1 == tiles;
    at += u1 - u0;
    return true;
  }
};

// 8 pieces of 16 bytes of each of 8 lanes, turned: piece j of lane i becomes piece i of lane j.
__device__ __forceinline__ void paged_turn(uint4 (&v)[8], int lane) {
#pragma unroll
  for (int s = 1; s < 8; s *= 2) {
    const bool high = lane & s;
#pragma unroll
    for (int a = 0; a < 8; ++a) {
      if (a & s) continue;
      uint4 x = high ? v[a] : v[a | s];
      x.x = __shfl_xor_sync(0xffffffffu, x.x, s);
      x.y = __shfl_xor_sync(0xffffffffu, x.y, s);
      x.z = __shfl_xor_sync(0xffffffffu, x.z, s);
      x.w = __shfl_xor_sync(0xffffffffu, x.w, s);
      if (high)
        v[a] = x;
      else
        v[a | s] = x;
    }
  }
}

// tile_cap where tile_small holds: the polynomial alone, as tile_weights forms it. (Every
// item has a tile or two with hidden keys, and all of tile_cap's tanh made them 9 us for 3.)
template <int N>
__device__ __forceinline__ void paged_cap_small(uint32_t ts, const TileRow& r) {
  const float mult = r.mult * (0.5f / kLog2e), u = mult * mult, v = r.cap2 * mult;
  const float2 k0 = make_float2(v, v), k1 = make_float2(v * u * kTanh1, v * u * kTanh1);
  const float2 k2 = make_float2(v * u * u * kTanh2, v * u * u * kTanh2);
  const float2 k3 = make_float2(v * u * u * u * kTanh3, v * u * u * u * kTanh3);
#pragma unroll 1
  for (int q = 0; q < N; q += 32) {
    uint32_t c[32];
    tc_ld32(c, ts + q);
    tc_wait_ld32(c);
#pragma unroll
    for (int k = 0; k < 32; k += 2) {
      float2 y = make_float2(__uint_as_float(c[k]), __uint_as_float(c[k + 1]));
      const float2 z = __fmul2_rn(y, y);
      y = __fmul2_rn(y, __ffma2_rn(z, __ffma2_rn(z, __ffma2_rn(z, k3, k2), k1), k0));
      c[k] = __float_as_uint(y.x), c[k + 1] = __float_as_uint(y.y);
    }
    tc_st32(ts + q, c);
  }
  tc_wait_st();
}

// Scores of the tile at j0 that the row does not see become -inf.
template <int N>
__device__ __forceinline__ void paged_hide(float (&x)[N], int j0, int from, int lim, bool masks, int past, uint64_t word) {
#pragma unroll
  for (int w = 0; w < N / 32; ++w) {
    const int at = j0 + 32 * w;
    auto below = [](int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; };  // n bits
    uint32_t on = below(lim - at) & ~below(from - at);
    if (masks) {
      const int off = past - at;  // the first new key's column
      const uint32_t bits = off <= -64 ? 0u : off <= 0 ? (uint32_t)(word >> -off) : off >= 32 ? 0u : (uint32_t)(word << off);
      on &= bits | below(off);
    }
#pragma unroll
    for (int i = 0; i < 32; ++i) x[32 * w + i] = on >> i & 1u ? x[32 * w + i] : -CUDART_INF_F;
  }
}

template <class T, int HD, int KIND>
__global__ void __launch_bounds__(kPagedTileThreads, 1)
    paged_tile_kernel_t(const PagedParams p, const __grid_constant__ PagedTileMaps maps) {
  using C = TileCfg<false, HD>;
  using bits = typename Elem<T>::bits;
  constexpr bool BF = kIsBf16<T>;
  constexpr int NT = C::NT, N = C::N, ROWS = NT * kTileRows;
  extern __shared__ uint8_t kv_tiles[];
  __shared__ PagedTileBars bars;
  __shared__ uint32_t s_tmem;
  __shared__ int s_sum[kPagedTileThreads / 32];
  __shared__ PagedTimes s_times[kPagedTileThreads / 32];
  __shared__ int s_ends[kPagedTileCtas + 1];
  uint8_t* base = kv_tiles + ((1024 - (kv_smem(kv_tiles) & 1023)) & 1023);
  const uint32_t sq = kv_smem(base), sk = sq + C::kQ, sv = sk + 2 * C::kStage;
  PagedItem* const items = reinterpret_cast<PagedItem*>(base + C::kQ + 4 * C::kStage);
  int32_t* const before = reinterpret_cast<int32_t*>(items + kPagedItems);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  auto bar = [&](uint64_t* b) { return kv_smem(b); };

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(&bars.k_full[i]), 1);
      mbar_init(bar(&bars.v_full[i]), 1);
      mbar_init(bar(&bars.k_free[i]), 1);
      mbar_init(bar(&bars.v_free[i]), 1);
      mbar_init(bar(&bars.s_full[i]), 1);
      mbar_init(bar(&bars.p_full[i]), kTileRows);
      mbar_init(bar(&bars.o_full[i]), 1);
    }
    mbar_init(bar(&bars.q_full), 1);
    mbar_init(bar(&bars.q_free), 1);
    mbar_init(bar(&bars.drain), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 8 && lane < 5)
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&maps) + lane * sizeof(CUtensorMap)) : "memory");
  if (warp == 11) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(kv_smem(&s_tmem)), "n"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  // rows of Q that no token fills: nobody's, but numbers
  const int q_rows = p.tpi * p.G;
  for (int i = tid; i < (ROWS - q_rows) * (HD / 8); i += kPagedTileThreads) {
    const int r = q_rows + i / (HD / 8), piece = i % (HD / 8);
    *reinterpret_cast<uint4*>(base + tile_at(ROWS, r, piece)) = make_uint4(0, 0, 0, 0);
  }
  tc_fence_smem();
  if (!p.shared) pdl_launch_dependents();
  pdl_wait();
  if (p.shared) pdl_launch_dependents();  // paged_token_kernel_t does not wait for what came before
  __syncthreads();

  tc_before();
  uint32_t ctas;  // that the work is dealt to
  const int count = paged_items(p, (int)(blockIdx.x / (uint32_t)p.Nkv), N, items, before, s_sum, s_times, &ctas);
  tc_after();
  const uint32_t tmem = s_tmem;
  if (p.shared && blockIdx.x >= ctas) {  // an SM of the other kernel's
    if (tid == 0) p.ws_join[blockIdx.x] = make_int4(0, 0, 0, 0);
    if (warp == 11)
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(512) : "memory");
    return;
  }
  PagedTileWork work;
  work.at = work.last = 0;
  PagedTileShares shares;
  if (p.deal > 0) {
    shares.set(count > 0 ? (uint32_t)before[count] * (uint32_t)p.Nkv : 0u, ctas);  // below 2^31
    // Whole items, if that costs less than joining: each CTA's ends moved to the nearest
    // item's. 288 items of 6 key tiles on 152 SMs 43.5 us split, 37 so.
    const int cta = tid <= (int)ctas ? tid : (int)ctas;
    s_ends[cta] = paged_nearest(p, (int)shares.first((uint32_t)cta), before, count);
    __syncthreads();
    const int load = s_ends[cta < (int)ctas ? cta + 1 : cta] - s_ends[cta];
    const bool split = __syncthreads_or(load > (int)shares.per + p.over_join) && !p.entire;
    if (blockIdx.x < ctas) {
      work.at = split ? (int)shares.first(blockIdx.x) : s_ends[blockIdx.x];
      work.last = split ? (int)shares.first(blockIdx.x + 1) : s_ends[blockIdx.x + 1];
    }
    // so far nothing begins here that goes on elsewhere, and nothing of this CTA's counts
    // where an item's CTAs lie on both sides of it
    if (!p.entire && tid == 0) p.ws_join[blockIdx.x] = make_int4(0, 0, 0, 0);
    if (!p.entire && work.at >= work.last && tid < ROWS) p.ws_ml[2 * (int64_t)blockIdx.x * ROWS + tid] = make_float2(-CUDART_INF_F, 0.0f);
  } else if (count > 0) {
    work.last = paged_item_tiles(items[0], N);
  }
  // every sequence's lengths are looked at once, where the other kernel has not
  if (p.s.status && !p.mixed)
    for (int64_t i = (int64_t)blockIdx.x * kPagedTileThreads + tid; i < p.s.B; i += (int64_t)gridDim.x * kPagedTileThreads)
      paged_flag_seq(p.s, (int)i, paged_seq(p.s, (int)i));
  // keys of a segment, and its key tiles
  auto keys_of = [&](const PagedItem& it, int& lo, int& hi) {
    lo = it.start + work.u0 * N;
    hi = it.start + work.u1 * N < it.end ? it.start + work.u1 * N : it.end;
    return hi > lo ? (hi - lo + N - 1) / N : 0;
  };
  // 384 threads x 168 registers, dealt out again: see kPagedTileRegisters
  bool ok = true;

  if (warp < 8) {
    // ------------------------------------------------------------------ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const int t = warp >> 2;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // 32 lanes of TMEM a warp
    const uint32_t to = tmem + lanes + 256 + (NT == 2 ? t * 128 : 0);
    const bool capped = KIND == kKvAnyScore && p.cap > 0.0f;
    const float mult = capped ? 2.0f * kLog2e * p.over : p.scale * kLog2e;
    const bool general = KIND == kKvBiased || (KIND == kKvAnyScore && (p.slopes || !(p.scale > 0.0f)));
    TileRow tr;
    tr.doc = 0;
    tr.part = tr.look = tr.ahead = false;
    tr.unit = 1.0f;
    tr.mult = mult;
    tr.cap2 = p.cap * kLog2e;
    int done_steps = 0, done_segments = 0;  // of this row tile
    for (int segment = 0; ok && t < NT && work.next(p, before, count); ++segment) {
      const PagedItem& it = items[work.item];
      int lo, hi;
      const int steps = keys_of(it, lo, hi);
      const int nrows = it.ntok * p.G;
      const int kvh = work.kvh;
      const bool whole = work.whole;
      // the one item that begins in this CTA and goes on in others: paged_tile_join_kernel_t's
      if (tid == 0 && work.u0 == 0 && !whole) {
        const uint32_t its_last = (uint32_t)(work.at - work.u1 + paged_item_tiles(it, N) - 1);
        const int parts = (int)shares.owner(its_last) - (int)blockIdx.x;
        p.ws_join[blockIdx.x] = make_int4(it.g0, kvh, nrows, 2 * parts + (segment > 0 ? 1 : 0));
      }
      if (t * kTileRows >= nrows) continue;
      const bool live = tid < nrows;  // row tid of the item: TMEM lane tid % 128 of row tile t
      const int past = it.pos0 - it.tok0;
      const int tok = kv_div(live ? tid : nrows - 1, p.by_g), head = (live ? tid : nrows - 1) - tok * p.G;
      const int pos = it.pos0 + tok;
      int lim = 0;
      if (live) lim = p.masks || pos >= it.total ? it.total : pos < 0 ? 0 : pos + 1;
      const int from = paged_first(p, pos);
      const uint64_t word = p.masks && live ? (uint64_t)__ldg(p.masks + it.g0 + tok) : ~0ull;
      // keys in [below, full) are seen by every row of the warp
      const int full = __reduce_min_sync(0xffffffffu, !live ? 0x7fffffff : p.masks && past < lim ? past : lim);
      const int below = __reduce_max_sync(0xffffffffu, live ? from : 0);
      tr.slope = 0.0f;
      if (p.slopes && live) tr.slope = __ldg(p.slopes + kvh * p.G + head) * kLog2e;
      // Rows behind the last (lim is 0) hold what TMA found there, tokens of other sequences or
      // of nobody: they have no say in what the warp does. Whose say it was is asked only where
      // somebody had one (asked at every key tile: 1 to 3 % of a prompt).
      float m = live ? -CUDART_INF_F : 0.0f, l = 0.0f;
      for (int step = 0; step < steps; ++step, ++done_steps) {
        const int j0 = lo + (steps - 1 - step) * N;
        const int buf = NT == 2 ? t : done_steps & 1;
        const uint32_t par = (NT == 2 ? done_steps : done_steps >> 1) & 1;
        const uint32_t ts = tmem + lanes + (NT == 2 ? t * 128 : buf * N);
        tr.dist = (float)(pos - j0);
        const bool masked = j0 + N > full || j0 < below;
        ok = mbar_wait(bar(&bars.s_full[buf]), par);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        tc_after();
        float x[N];
        tile_load<false, N>(x, ts, tr, true);
        bool done = general;  // x holds scores in log2, not raw ones
        const bool small = capped && tile_small<true>(x, tr, lim > 0);
        if (capped && (general || masked || !small)) {
          // (an infinite product is at an end of the cap from here on: -inf means hidden)
          if (small)
            paged_cap_small<N>(ts, tr);
          else
            tile_cap<false, N>(ts, tr);
          tile_load<false, N>(x, ts, tr, false);
          done = true;
        }
        if (general) tile_scores<true, N>(x, tr, !capped);
        if (masked) paged_hide<N>(x, j0, from, lim, p.masks != nullptr, past, word);
        auto weights = [&]() {
          const float nb = m == -CUDART_INF_F ? 0.0f : -m;
          if (done) return tile_weights<false, BF, 2, N>(x, ts, tr, 1.0f, nb, nullptr, 1.0f);
          if (!capped) return tile_weights<false, BF, 0, N>(x, ts, tr, mult, nb, nullptr, 1.0f);
          return tile_weights<false, BF, 1, N>(x, ts, tr, mult * (0.5f / kLog2e), nb, nullptr, 1.0f);
        };
        // Weights by the base so far, where every row has one; only where a row's sum
        // says that one may be too large (2^15 fits float16) is the maximum taken, the
        // base moved and the tile's weights formed again.
        bool move = __any_sync(0xffffffffu, m == -CUDART_INF_F);
        float sum = 0.0f;
        if (!move) {
          sum = weights();
          move = __any_sync(0xffffffffu, !(sum <= 32768.0f));
          if (move) move = __any_sync(0xffffffffu, lim > 0 && !(sum <= 32768.0f));
        }
        if (move) {
          const float top = tile_max(x);
          float mx = top * (done ? 1.0f : mult);
          if (capped && !done) mx = kv_tanh_of(mx) * tr.cap2;
          const float mn = fmaxf(m, mx);
          float a = mn == -CUDART_INF_F ? 1.0f : kv_exp2(m - mn);
          m = mn;
          l *= a;
          if (step > 0 && __any_sync(0xffffffffu, a != 1.0f)) {
            if constexpr (NT == 1) {  // here S runs ahead of P V
              ok = mbar_wait(bar(&bars.o_full[1]), (done_steps - 1) & 1);
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
      }
      // ---------------------------------------------------------------- output
      if (ok && steps > 0) {
        ok = mbar_wait(bar(&bars.o_full[NT == 2 ? t : 0]), done_segments & 1);
        ok = __all_sync(0xffffffffu, ok);
        tc_after();
        ++done_segments;
      }
      if (ok) {
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        const float f = whole ? inv : 1.0f;
        const bool empty = m == -CUDART_INF_F && l == 0.0f;  // nothing seen (TMEM may never have been written)
        const int64_t slot = 2 * (int64_t)blockIdx.x + (segment > 0 ? 1 : 0);
        float4* const part = reinterpret_cast<float4*>(p.ws_o) + slot * (p.H / 4) * ROWS + tid;
        bits* const out = static_cast<bits*>(p.out) + ((int64_t)it.g0 * p.Nq + (int64_t)kvh * p.G) * p.H;
        const int at = live ? (tok * p.Nq + head) * p.H : -1;  // of the row, from `out` on
        float2 sums = make_float2(0.0f, 0.0f);  // of 0 times each output: NaN where one is not finite
        const float2 f2 = make_float2(f, f), zero2 = make_float2(0.0f, 0.0f);
        if (live && !whole) p.ws_ml[slot * ROWS + tid] = make_float2(m, l);
#pragma unroll 1
        for (int i0 = 0; i0 < HD; i0 += 64) {
          uint32_t o[64];
          tc_ld32(o, to + i0);
          tc_ld32(o + 32, to + i0 + 32);
          tc_wait_ld32(o);
          tc_wait_ld32(o + 32);
          float y[64];
#pragma unroll
          for (int k = 0; k < 64; k += 2) {
            const float2 z = __fmul2_rn(make_float2(__uint_as_float(o[k]), __uint_as_float(o[k + 1])), f2);
            y[k] = empty ? 0.0f : z.x;
            y[k + 1] = empty ? 0.0f : z.y;
            sums = __ffma2_rn(make_float2(y[k], y[k + 1]), zero2, sums);
          }
          if (!whole) {
#pragma unroll
            for (int k = 0; k < 64; k += 4)
              if (live && i0 + k < p.H) part[(int64_t)((i0 + k) / 4) * ROWS] = make_float4(y[k], y[k + 1], y[k + 2], y[k + 3]);
          } else {
            uint4 v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
              v[k] = make_uint4(kv_pack2<BF>(y[8 * k], y[8 * k + 1]), kv_pack2<BF>(y[8 * k + 2], y[8 * k + 3]),
                                kv_pack2<BF>(y[8 * k + 4], y[8 * k + 5]), kv_pack2<BF>(y[8 * k + 6], y[8 * k + 7]));
            paged_turn(v, lane);
            const int d = i0 + 8 * (lane & 7);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const int to_row = __shfl_sync(0xffffffffu, at, (lane & ~7) | k);
              if (to_row >= 0 && d < p.H) *reinterpret_cast<uint4*>(out + to_row + d) = v[k];
            }
          }
        }
        // An infinity or a NaN may have come from a value that the row does not see
        uint32_t again = __ballot_sync(0xffffffffu, live && !(sums.x == 0.0f && sums.y == 0.0f));
        if (again) {
          bool found = false;  // in a value that some row of the warp does not see and its key tile holds
          auto look = [&](int from_key, int to_key) {
            for (int j = from_key; j < to_key; ++j) {
              const int64_t e = paged_row(p.s, it.b, kvh, j, p.H);
              for (int d = lane; d < p.H; d += 32)
                found |= e >= 0 && !(fabsf(Elem<T>::tof(static_cast<const bits*>(p.v)[e + d])) < CUDART_INF_F);
            }
          };
          look(lo, below < hi ? below : hi);
          look(full > lo ? full : lo, hi);
          if (!__any_sync(0xffffffffu, found)) again = 0;
        }
        __syncwarp();
        while (again) {
          const int r = __ffs(again) - 1;
          again &= again - 1;
          const int row = warp * 32 + r;
          paged_careful_row<T>(p, it.seq(), it.b, kvh, (int64_t)it.tok0 * p.G + row, lo, hi,
                               whole ? nullptr : p.ws_o + (slot * (p.H / 4) * ROWS + row) * 4, 4 * ROWS,
                               p.ws_ml + slot * ROWS + row, lane);
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp == 11) {
      // ---------------------------------------------------------------- MMA
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
        const uint32_t a = dq + t * (kTileRows * 128 / 16), c = dk + stage * (C::kStage / 16);
        if (tc_elect()) {
#pragma unroll
          for (int k = 0; k < HD / 16; ++k)
            if (k < steps)
              tc_mma_ss(d, a + ((k >> 2) * (ROWS * 128) + (k & 3) * 32) / 16,
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
      int gs = 0, c0 = 0, c1 = 0, segments = 0;  // key tiles; of each row tile; segments with any
      while (ok && work.next(p, before, count)) {
        const PagedItem& it = items[work.item];
        int lo, hi;
        const int n = keys_of(it, lo, hi);
        if (n == 0) continue;
        const int live_tiles = NT == 2 && it.ntok * p.G > kTileRows ? 2 : 1;
        wait(&bars.q_full, segments & 1);
        wait(&bars.k_full[gs & 1], (gs >> 1) & 1);
        if (!ok) break;
        ++segments;
        tc_after();
        for (int t = 0; t < live_tiles; ++t) {
          const int buf = NT == 2 ? t : c0 & 1;
          qk(t, gs & 1, tm + (NT == 2 ? t * 128 : buf * N));
          commit(&bars.s_full[buf]);
        }
        commit(&bars.k_free[gs & 1]);
        if (n == 1) commit(&bars.q_free);
        for (int step = 0; ok && step < n; ++step, ++gs) {
          const bool more = step + 1 < n;
          const int st = gs & 1, sn = st ^ 1;
          if constexpr (NT == 2) {
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              if (t >= live_tiles) break;
              wait(&bars.p_full[t], (t == 0 ? c0 : c1) & 1);
              if (t == 0) wait(&bars.v_full[st], (gs >> 1) & 1);
              if (!ok) break;
              tc_after();
              pv(tm + 256 + t * 128, tm + t * 128, st, step > 0);
              if (t == live_tiles - 1) commit(&bars.v_free[st]);
              if (more) {
                if (t == 0) wait(&bars.k_full[sn], ((gs + 1) >> 1) & 1);
                if (!ok) break;
                tc_after();
                qk(t, sn, tm + t * 128);
                commit(&bars.s_full[t]);
                if (t == live_tiles - 1) {
                  commit(&bars.k_free[sn]);
                  if (step + 2 == n) commit(&bars.q_free);
                }
              } else {
                commit(&bars.o_full[t]);
              }
              if (t == 0)
                ++c0;
              else
                ++c1;
            }
          } else {
            if (more) {
              wait(&bars.k_full[sn], ((gs + 1) >> 1) & 1);
              if (!ok) break;
              tc_after();
              qk(0, sn, tm + ((c0 + 1) & 1) * N);
              commit(&bars.s_full[(c0 + 1) & 1]);
              commit(&bars.k_free[sn]);
              if (step + 2 == n) commit(&bars.q_free);
            }
            wait(&bars.p_full[c0 & 1], (c0 >> 1) & 1);
            wait(&bars.v_full[st], (gs >> 1) & 1);
            if (!ok) break;
            tc_after();
            pv(tm + 256, tm + (c0 & 1) * N, st, step > 0);
            commit(&bars.v_free[st]);
            commit(&bars.o_full[1]);
            if (!more) commit(&bars.o_full[0]);
            ++c0;
          }
        }
      }
      if (!ok) {  // let what was issued end before TMEM and shared memory go
        commit(&bars.drain);
        mbar_wait(bar(&bars.drain), 0);
      }
    } else if (warp == 10) {
      // ---------------------------------------------------------------- Q
      int segments = 0;
      while (ok && work.next(p, before, count)) {
        const PagedItem& it = items[work.item];
        int lo, hi;
        if (keys_of(it, lo, hi) == 0) continue;
        if (segments > 0) ok = mbar_wait(bar(&bars.q_free), (segments - 1) & 1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        ++segments;
        if (lane == 0) mbar_arrive_expect_tx(bar(&bars.q_full), C::SLABS * q_rows * 128);
        __syncwarp();
        if (lane < C::SLABS)
          tile_tma(sq + lane * (ROWS * 128), &maps.q, lane * 64, work.kvh * p.G, it.g0, bar(&bars.q_full));
      }
      // what is on its way has to land before shared memory goes
      if (segments > 0 && !ok) mbar_wait(bar(&bars.q_full), (segments - 1) & 1);
    } else {
      // ---------------------------------------------------------------- K (warp 8) and V
      const bool is_k = warp == 8;
      uint64_t* const full = is_k ? bars.k_full : bars.v_full;
      uint64_t* const free_ = is_k ? bars.k_free : bars.v_free;
      const CUtensorMap* const map = is_k ? &maps.k : &maps.v;
      const uint32_t stage0 = is_k ? sk : sv;
      // a box: p.chunk rows (of one page) x 64 elements; this lane's rows and slab of a tile
      const int chunks = N / p.chunk;
      const int my_row = (lane & (chunks - 1)) * p.chunk, my_slab = lane / chunks;
      bool bad = false;
      int gs = 0;  // key tiles
      while (ok && work.next(p, before, count)) {
        const PagedItem& it = items[work.item];
        int lo, hi;
        const int n = keys_of(it, lo, hi);
        if (n == 0) continue;
        const int kvh = work.kvh, seen = paged_first(p, it.pos0);  // keys before `seen` are nobody's
        const int32_t* table = p.s.table + (int64_t)it.b * p.s.max_pages;
        // The table's entry for key j, looked at a tile later; -1 for keys that nobody sees,
        // as for pages outside the pool: TMA fills in zeros.
        auto entry = [&](int j, int upto) {
          return j < hi && upto > seen && j >= lo ? __ldg(table + kv_div(j, p.s.by_ps)) : -1;
        };
        auto bring = [&](const CUtensorMap* m, uint32_t dst, int slab, int j, int upto, int page, uint32_t done) {
          const bool in_pool = (uint32_t)page < (uint32_t)p.s.pages;
          bad |= !in_pool && j < hi && upto > seen;
          paged_tma(dst, m, slab * 64, j - kv_div(j, p.s.by_ps) * p.s.ps, kvh, in_pool ? page : -1, done);
        };
        auto box_entry = [&](int j0) { return entry(j0 + my_row, j0 + my_row + p.chunk); };
        int page = box_entry(lo + (n - 1) * N);
        for (int tile = n - 1; tile >= 0; --tile, ++gs) {
          const int st = gs & 1, j0 = lo + tile * N;
          const int page_after = box_entry(j0 - N);
          if (gs >= 2) ok = mbar_wait(bar(&free_[st]), ((gs >> 1) - 1) & 1);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          const uint32_t dst = stage0 + st * C::kStage, done = bar(&full[st]);
          if (lane == 0) mbar_arrive_expect_tx(done, C::kStage);
          __syncwarp();
          // the box of V that holds the last key and rows behind it
          const int cut = !is_k && hi < j0 + N ? (hi - j0) & ~(p.chunk - 1) : N;
          const bool cut_box = cut < N && cut + j0 < hi;
          if (my_slab < C::SLABS && !(cut_box && my_row == cut))
            bring(map, dst + my_slab * (N * 128) + my_row * 128, my_slab, j0 + my_row, j0 + my_row + p.chunk, page, done);
          if (cut_box) {
            const int cut_page = entry(j0 + cut, j0 + cut + p.chunk);
            // 8 rows at a time, those with the last key one by one; zeros behind it
            const int eights = p.chunk / 8 - 1, copies = eights + 8, last8 = (hi - j0) & ~7;
            for (int i = lane; i < copies * C::SLABS; i += 32) {
              const int slab = i / copies, n8 = i - slab * copies;
              const bool one = n8 >= eights;
              int r = one ? last8 + n8 - eights : cut + 8 * n8;
              if (!one && r >= last8) r += 8;  // (where hi ends a box of 8, the one behind goes row by row)
              const int j = j0 + r, upto = j + (one ? 1 : 8);
              bring(one ? &maps.v_row : &maps.v_eight, dst + slab * (N * 128) + r * 128, slab, j, upto,
                    j < hi && upto > seen ? cut_page : -1, done);
            }
          }
          page = page_after;
        }
      }
      if (bad && p.s.status) atomicOr(p.s.status, 4);
      if (!ok)  // what is on its way has to land before shared memory goes
        for (int i = gs - 2; i < gs; ++i)
          if (i >= 0) mbar_wait(bar(&full[i & 1]), (i >> 1) & 1);
    }
  }
  if (!ok && p.s.status) atomicOr(p.s.status, 2);
  tc_before();
  __syncthreads();
  if (warp == 11)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(512) : "memory");
}

// 4 dims of `RW` rows of one item, kRows apart, from its parts: slots c0 * 2 + (what.w & 1)
// and the first ones of the CTAs behind. The loads of 8 / RW parts of all rows are in flight
// together, what they count beside them.
template <class T, int RW>
__device__ __forceinline__ void paged_tile_join_rows(const PagedParams& p, const int4& what, int c0, int first_row,
                                                     int apart, int piece, int rows) {
  constexpr int DEEP = 8 / RW;
  const int parts = (what.w >> 1) + 1, pieces = p.H / 4;
  const float4* const from = reinterpret_cast<const float4*>(p.ws_o) + piece * rows;
  float M[RW], L[RW];
  float4 acc[RW];
#pragma unroll
  for (int i = 0; i < RW; ++i) M[i] = -CUDART_INF_F, L[i] = 0.0f, acc[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int n0 = 0; n0 < parts; n0 += DEEP) {
    float4 o[DEEP][RW];
    float2 ml[DEEP][RW];
#pragma unroll
    for (int k = 0; k < DEEP; ++k) {
      const int n = n0 + k;
      // (offsets are below 2 kPagedTileCtas slots of 256 rows x 64 pieces, 2^23)
      const uint32_t slot = 2 * (c0 + n) + (n == 0 ? what.w & 1 : 0);
#pragma unroll
      for (int i = 0; i < RW; ++i) {
        const int r = first_row + i * apart;
        ml[k][i] = make_float2(-CUDART_INF_F, 0.0f);
        o[k][i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (n < parts && r < what.z) {
          ml[k][i] = paged_load2(p.ws_ml + (slot * rows + r));
          o[k][i] = paged_load4(from + (slot * pieces * rows + r));
        }
      }
    }
#pragma unroll
    for (int i = 0; i < RW; ++i) {
      float m = M[i];
#pragma unroll
      for (int k = 0; k < DEEP; ++k) m = fmaxf(m, ml[k][i].x);
      const float base = m == -CUDART_INF_F ? 0.0f : m, a = exp2f(M[i] - base);
      M[i] = m;
      L[i] *= a;
      acc[i].x *= a, acc[i].y *= a, acc[i].z *= a, acc[i].w *= a;
#pragma unroll
      for (int k = 0; k < DEEP; ++k) {
        const float f = exp2f(ml[k][i].x - base);
        if (f == 0.0f) o[k][i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);  // where a CTA had no part it wrote nothing
        L[i] = fmaf(ml[k][i].y, f, L[i]);
        acc[i].x = fmaf(o[k][i].x, f, acc[i].x);
        acc[i].y = fmaf(o[k][i].y, f, acc[i].y);
        acc[i].z = fmaf(o[k][i].z, f, acc[i].z);
        acc[i].w = fmaf(o[k][i].w, f, acc[i].w);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < RW; ++i) {
    const int r = first_row + i * apart;
    if (r >= what.z) continue;
    const float inv = L[i] == 0.0f ? 0.0f : 1.0f / L[i];
    const int tok = kv_div(r, p.by_g);
    VecT<T, 4> v;
    v.v[0] = Elem<T>::fromf(acc[i].x * inv);
    v.v[1] = Elem<T>::fromf(acc[i].y * inv);
    v.v[2] = Elem<T>::fromf(acc[i].z * inv);
    v.v[3] = Elem<T>::fromf(acc[i].w * inv);
    *reinterpret_cast<VecT<T, 4>*>(static_cast<typename Elem<T>::bits*>(p.out) +
                                   (((int64_t)what.x + tok) * p.Nq + (int64_t)what.y * p.G + (r - tok * p.G)) * p.H +
                                   4 * piece) = v;
  }
}

// Joins the parts of the items that paged_tile_kernel_t dealt to several CTAs. The rows of
// all such items, a group at a time, go around the CTAs, which are as many as are resident
// (one for each CTA dealt to and 16 rows, most of them with nothing to join, came in waves:
// one tree of 60 drafts behind 8000 keys 29 us, 22 so; 32 trees 83 and 79);
// a thread has 4 dims of a row, or of 2 or 4 rows where there are few parts.
template <class T, int HD>
__global__ void __launch_bounds__(kPagedJoinThreads, kPagedJoinCtas) paged_tile_join_kernel_t(const PagedParams p, int rows) {
  constexpr int PIECES = HD / 4, kRows = kPagedJoinThreads / PIECES;
  __shared__ int4 s_what[kPagedTileCtas];
  __shared__ int s_first[kPagedTileCtas + 1], s_cta[kPagedTileCtas], s_count[2][kPagedJoinThreads / 32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  auto side_by_side = [](const int4& what) { return what.w < 4 ? 4 : what.w < 8 ? 2 : 1; };  // rows of a thread
  pdl_wait();
  pdl_launch_dependents();
  // the items that have parts, and the groups of rows before each
  int4 what = make_int4(0, 0, 0, 0);  // first token, kvh, rows, 2 * further CTAs + slot
  if (tid < p.deal) what = p.ws_join[tid];
  const int group = kRows * side_by_side(what), mine = what.w < 2 ? 0 : (what.z + group - 1) / group;
  int upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const int x = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += x;
  }
  const uint32_t some = __ballot_sync(0xffffffffu, mine > 0);
  if (lane == 31) s_count[0][warp] = upto, s_count[1][warp] = __popc(some);
  __syncthreads();
  int before = upto - mine, at = __popc(some & ((1u << lane) - 1u)), total = 0, count = 0;
#pragma unroll
  for (int w = 0; w < kPagedJoinThreads / 32; ++w) {
    if (w < warp) before += s_count[0][w], at += s_count[1][w];
    total += s_count[0][w], count += s_count[1][w];
  }
  if (mine > 0) s_what[at] = what, s_first[at] = before, s_cta[at] = tid;
  __syncthreads();
  const int r0 = tid % kRows, piece = tid / kRows;
  if (piece >= p.H / 4) return;
  for (int w = blockIdx.x; w < total; w += gridDim.x) {
    int x = 0, y = count;
    while (y - x > 1) {
      const int mid = (x + y) >> 1;
      if (s_first[mid] <= w)
        x = mid;
      else
        y = mid;
    }
    what = s_what[x];
    const int n = side_by_side(what), row = (w - s_first[x]) * kRows * n + r0;
    if (n == 4)
      paged_tile_join_rows<T, 4>(p, what, s_cta[x], row, kRows, piece, rows);
    else if (n == 2)
      paged_tile_join_rows<T, 2>(p, what, s_cta[x], row, kRows, piece, rows);
    else
      paged_tile_join_rows<T, 1>(p, what, s_cta[x], row, kRows, piece, rows);
  }
}

template <class T, int HD>
PagedTileKernel paged_tile_of(int kind) {
  using C = TileCfg<false, HD>;
  const void* fn = kind == kKvPlain    ? (const void*)paged_tile_kernel_t<T, HD, kKvPlain>
                   : kind == kKvBiased ? (const void*)paged_tile_kernel_t<T, HD, kKvBiased>
                                       : (const void*)paged_tile_kernel_t<T, HD, kKvAnyScore>;
  return {fn, (const void*)paged_tile_join_kernel_t<T, HD>, 1024 + C::kQ + 4 * C::kStage + kPagedItems * (sizeof(PagedItem) + 4) + 16};
}

template <class T>
PagedTileKernel paged_tile_pick(int H, int kind) {
  if (H <= 64) return paged_tile_of<T, 64>(kind);
  if (H <= 128) return paged_tile_of<T, 128>(kind);
  return paged_tile_of<T, 256>(kind);
}

}  // namespace rope_gb300
