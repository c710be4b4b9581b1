// Attention over a paged cache for many rows (prompts, chunks, draft trees): tcgen05.
//
// What is done with a key tile is what kv_tile_kernel_t (kv_tile.cuh) does: two tiles
// of 128 rows take turns on the tensor cores, S and O in TMEM, P = 2^(x - m) by the
// threads that own the rows, the base moved only where a tile's weights ask for it.
//
// One CTA an SM stays for the whole call. The work is the key tiles of all items (a
// sequence's tile of rows) and heads, and CTA i takes the key tiles [i U / n, (i + 1) U / n)
// of all U: sequences of any lengths, few long ones and many short ones, even out, and
// nothing is split where it need not be. An item that one CTA has whole goes to the
// output, the others' parts to the workspace (2 slots a CTA), where
// paged_tile_join_kernel_t adds them up. The roles run through a CTA's segments
// without meeting: while the last tile of one is with the softmax threads and its
// output is on its way, K, V and Q of the next come in and its first products run.
//   Warps (16): 0-3 and 4-7 softmax and output of row tile 0 and 1; 8-11 bring K and V,
//   by TMA in boxes (the rows of a key tile that lie in one page x 64 elements), one
//   thread a box, each with the next tile's page looked up a step ahead; the tile that
//   holds the last key by cp.async, rows behind it zeros; 12 issues every MMA; 13-15
//   bring Q as soon as the last product of the segment before has read its own.
// A row sees keys from its window on; of a draft tree's new keys those whose bit its
// mask holds. Only key tiles that some row does not see whole are looked at key by key,
// as bits of four words.
// Bound by the tensor cores for prompts; trees, whose rows are two tiles or less, by the
// softmax between the products of a key tile.
//
// Without a workspace, or with more than kPagedItems items, a CTA takes one item.
#pragma once

#include "kv_tile.cuh"
#include "paged_token.cuh"

namespace rope_gb300 {

constexpr int kPagedQThreads = 96;  // that bring Q

struct PagedTileBars {
  uint64_t k_full[2], k_free[2], v_full[2], v_free[2], s_full[2], p_full[2], o_full[2], q_full, q_free, drain;
};

// The key tiles' range of an item: keys [start, end), start at the beginning of a tile.
// Its units are those tiles, at least one, so that its output is written.
__device__ __forceinline__ int4 paged_item(const PagedParams& p, const PagedSeq& q, int b, int tile, int rows, int keys) {
  const int64_t rows0 = (int64_t)tile * rows, R = (int64_t)q.n * p.G;
  const int64_t last = rows0 + rows < R ? rows0 + rows : R;
  int4 it;
  it.x = b;
  it.y = tile;
  it.z = paged_first(p, q.past + rows0 / p.G) / keys * keys;
  it.w = paged_limit(p, q, q.past + (last - 1) / p.G);
  return it;
}
__device__ __forceinline__ int paged_item_units(int4 it, int keys) { return it.w > it.z ? (it.w - it.z + keys - 1) / keys : 1; }

// Tiles of rows of sequence b that are this kernel's.
__device__ __forceinline__ int paged_tiles(const PagedParams& p, const PagedSeq& q, int rows) {
  const int64_t R = (int64_t)q.n * p.G;
  return p.mixed && R <= p.mixed ? 0 : (int)((R + rows - 1) / rows);
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
  for (int w = 0; w < kTileThreads / 32; ++w) {
    const int x = s_sum[w];
    if (w < warp) n += x;
    a += x;
  }
  *all = a;
  return n;
}

// The items of the batch and the units of one head of those before each, in shared
// memory; their number. Not dealt: only item number `only`, or none. All threads come
// here, and the tables hold when it returns.
__device__ __forceinline__ int paged_items(const PagedParams& p, int only, int rows, int keys, int4* items, int32_t* before,
                                           int* s_sum) {
  const int tid = threadIdx.x;
  int count = 0;
  for (int b0 = 0; b0 < p.s.B; b0 += kTileThreads) {
    const int b = b0 + tid;
    PagedSeq q;
    int n = 0, all;
    if (b < p.s.B) {
      q = paged_seq(p.s, b);
      n = paged_tiles(p, q, rows);
    }
    const int first = paged_scan(n, s_sum, &all) - n + count;
    if (p.deal > 0) {
      // (more than planned for only where query_starts does not ascend)
      for (int t = 0; t < n && first + t < kPagedItems; ++t) items[first + t] = make_int4(b, t, 0, 0);
    } else if (only >= first && only < first + n) {
      items[0] = paged_item(p, q, b, first + n - 1 - only, rows, keys);  // the longest rows first
      before[0] = 0;
      before[1] = paged_item_units(items[0], keys);
    }
    count += all;
    if (p.deal == 0 && only < count) break;  // the same for all threads
  }
  __syncthreads();
  if (p.deal == 0) return only < count ? 1 : 0;
  if (count > kPagedItems) count = kPagedItems;
  int sum = 0;
  for (int i0 = 0; i0 < count; i0 += kTileThreads) {
    const int i = i0 + tid;
    int n = 0, all;
    if (i < count) {
      const int4 it = items[i];
      items[i] = paged_item(p, paged_seq(p.s, it.x), it.x, it.y, rows, keys);
      n = paged_item_units(items[i], keys);
    }
    const int upto = paged_scan(n, s_sum, &all) + sum;
    if (i < count) before[i] = upto - n;
    sum += all;
  }
  if (tid == 0) before[count] = sum;
  __syncthreads();
  return count;
}

// The segments of a CTA, one after the other.
struct PagedTileWork {
  int at, last;     // units left
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
    item = x;
    const int units = before[x + 1] - before[x], in = at - before[x] * p.Nkv;
    kvh = (int)((uint32_t)in / (uint32_t)units);
    u0 = in - kvh * units;
    u1 = u0 + (last - at) < units ? u0 + (last - at) : units;
    whole = u0 == 0 && u1 == units;
    at += u1 - u0;
    return true;
  }
};

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
__global__ void __launch_bounds__(kTileThreads, 1)
    paged_tile_kernel_t(const PagedParams p, const __grid_constant__ PagedMaps maps) {
  using C = TileCfg<false, HD>;
  using bits = typename Elem<T>::bits;
  constexpr bool BF = kIsBf16<T>;
  constexpr int NT = C::NT, N = C::N, ROWS = NT * kTileRows;
  extern __shared__ uint8_t kv_tiles[];
  __shared__ PagedTileBars bars;
  __shared__ uint32_t s_tmem;
  __shared__ int s_sum[kTileThreads / 32];
  uint8_t* base = kv_tiles + ((1024 - (kv_smem(kv_tiles) & 1023)) & 1023);
  const uint32_t sq = kv_smem(base), sk = sq + C::kQ, sv = sk + 2 * C::kStage;
  int4* const items = reinterpret_cast<int4*>(base + C::kQ + 4 * C::kStage);
  int32_t* const before = reinterpret_cast<int32_t*>(items + kPagedItems);
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
    mbar_init(bar(&bars.q_full), kPagedQThreads);
    mbar_init(bar(&bars.q_free), 1);
    mbar_init(bar(&bars.drain), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (tid == 256) {
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

  tc_before();
  const int count = paged_items(p, (int)(blockIdx.x / (uint32_t)p.Nkv), ROWS, N, items, before, s_sum);
  tc_after();
  const uint32_t tmem = s_tmem;
  PagedTileWork work;
  work.at = work.last = 0;
  if (count > 0) {
    const uint32_t total = (uint32_t)before[count] * (p.deal > 0 ? p.Nkv : 1);  // below 2^31
    work.last = (int)total;
    if (p.deal > 0) {
      work.at = (int)((uint64_t)blockIdx.x * total / (uint32_t)p.deal);
      work.last = (int)((uint64_t)(blockIdx.x + 1) * total / (uint32_t)p.deal);
    }
  }
  if (p.deal > 0 && work.at >= work.last && tid < ROWS) {
    // no units: nothing begins here, and nothing of this CTA's counts where an item's
    // CTAs lie on both sides of it
    if (tid == 0) p.ws_join[blockIdx.x] = make_int4(0, 0, 0, 0);
    p.ws_ml[2 * (int64_t)blockIdx.x * ROWS + tid] = make_float2(-CUDART_INF_F, 0.0f);
  }
  // every sequence's lengths are looked at once, where the other kernel has not
  if (p.s.status && !p.mixed)
    for (int64_t i = (int64_t)blockIdx.x * kTileThreads + tid; i < p.s.B; i += (int64_t)gridDim.x * kTileThreads)
      paged_flag_seq(p.s, (int)i, paged_seq(p.s, (int)i));
  // keys of a segment
  auto keys_of = [&](const int4& it, int& lo, int& hi) {
    lo = it.z + work.u0 * N;
    hi = it.z + work.u1 * N < it.w ? it.z + work.u1 * N : it.w;
    return hi > lo ? (hi - lo + N - 1) / N : 0;  // key tiles
  };
  auto rows_of = [&](const PagedSeq& seq, const int4& it) {
    const int64_t left = (int64_t)seq.n * p.G - (int64_t)it.y * ROWS;
    return left < ROWS ? (int)left : ROWS;  // at least 1
  };
  // 512 threads x 128 registers, dealt out again: see kKvTileRegisters
  bool ok = true;

  if (warp < 8) {
    // ------------------------------------------------------------------ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
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
      const int4 it = items[work.item];
      const PagedSeq seq = paged_seq(p.s, it.x);
      int lo, hi;
      const int steps = keys_of(it, lo, hi);
      const int nrows = rows_of(seq, it);
      // the one item that may begin in this CTA and go on in others: paged_tile_join_kernel_t's
      if (p.deal > 0 && work.at >= work.last && tid == 0) {
        const bool open = work.u0 == 0 && !work.whole;  // an item that began before is another CTA's
        const uint32_t total = (uint32_t)before[count] * p.Nkv;
        const int upto = work.at - work.u1 + paged_item_units(it, N);  // its last unit, and one
        const int parts =
            open ? (int)(((uint64_t)(uint32_t)upto * (uint32_t)p.deal - 1) / total) - (int)blockIdx.x : 0;
        p.ws_join[blockIdx.x] = make_int4(it.x, work.kvh, it.y, 2 * parts + (segment > 0 ? 1 : 0));
      }
      if (t * kTileRows >= nrows) continue;
      const bool live = tid < nrows;  // row tid of the item: TMEM lane tid % 128 of row tile t
      const int kvh = work.kvh;
      const bool whole = work.whole;
      const int64_t row = (int64_t)it.y * ROWS + (live ? tid : nrows - 1);
      const int64_t tok = row / p.G;
      const int head = (int)(row - tok * p.G);
      const int64_t pos = seq.past + tok;
      const int lim = live ? paged_limit(p, seq, pos) : 0, from = paged_first(p, pos);
      const uint64_t word = p.masks && live ? (uint64_t)__ldg(p.masks + seq.t0 + tok) : ~0ull;
      // keys in [below, full) are seen by every row of the warp
      const int full = __reduce_min_sync(0xffffffffu, !live ? 0x7fffffff : p.masks && seq.past < lim ? seq.past : lim);
      const int below = __reduce_max_sync(0xffffffffu, live ? from : 0);
      tr.slope = 0.0f;
      if (p.slopes && live) tr.slope = __ldg(p.slopes + kvh * p.G + head) * kLog2e;
      float m = live ? -CUDART_INF_F : 0.0f, l = 0.0f;  // rows behind the last never move the base
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
        if (capped && (general || masked || !tile_small(x, tr))) {
          // (an infinite product is at an end of the cap from here on: -inf means hidden)
          tile_cap<false, N>(ts, tr);
          tile_load<false, N>(x, ts, tr, false);
          done = true;
        }
        if (general) tile_scores<true, N>(x, tr, !capped);
        if (masked) paged_hide<N>(x, j0, from, lim, p.masks != nullptr, seq.past, word);
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
        const int64_t slot = (2 * (int64_t)blockIdx.x + (segment > 0 ? 1 : 0)) * ROWS;
        bits* dst = static_cast<bits*>(p.out) + ((seq.t0 + tok) * p.Nq + (int64_t)kvh * p.G + head) * p.H;
        bool odd = false;
        if (live && !whole) p.ws_ml[slot + tid] = make_float2(m, l);
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
              if (!whole) {
                float* part = p.ws_o + (slot + tid) * p.H + i + k;
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
        if (again) {
          bool found = false;  // in a value that some row of the warp does not see and its key tile holds
          auto look = [&](int from_key, int to_key) {
            for (int j = from_key; j < to_key; ++j) {
              const int64_t e = paged_row(p.s, it.x, kvh, j, p.H);
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
          const int64_t w = slot + warp * 32 + r;
          paged_careful_row<T>(p, seq, it.x, kvh, (int64_t)it.y * ROWS + (warp * 32 + r), lo, hi,
                               whole ? nullptr : p.ws_o + w * p.H, p.ws_ml + w, lane);
        }
      }
    }
  } else if (warp >= 12) {
    // ------------------------------------------------------------------ MMA
    asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    if (warp == 12) {
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
      int gs = 0, c0 = 0, c1 = 0, segments = 0;  // key tiles; of each row tile; segments with any
      while (ok && work.next(p, before, count)) {
        const int4 it = items[work.item];
        int lo, hi;
        const int n = keys_of(it, lo, hi);
        if (n == 0) continue;
        const int live_tiles = NT == 2 && rows_of(paged_seq(p.s, it.x), it) > kTileRows ? 2 : 1;
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
    } else {
      // ---------------------------------------------------------------- Q
      const int me = tid - 13 * 32;
      constexpr int PPR = HD / 8;  // 16-byte pieces of a row
      int segments = 0;
      while (ok && work.next(p, before, count)) {
        const int4 it = items[work.item];
        int lo, hi;
        if (keys_of(it, lo, hi) == 0) continue;
        const PagedSeq seq = paged_seq(p.s, it.x);
        const int nrows = rows_of(seq, it);
        const int64_t tok0 = (int64_t)it.y * ROWS / p.G;
        const int rem0 = (int)((int64_t)it.y * ROWS - tok0 * p.G);
        const bits* q0 = static_cast<const bits*>(p.q) + ((seq.t0 + tok0) * p.Nq + (int64_t)work.kvh * p.G) * p.H;
        if (segments > 0) ok = mbar_wait(bar(&bars.q_free), (segments - 1) & 1);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        ++segments;
        const int upto = nrows > kTileRows ? ROWS : kTileRows;
#pragma unroll 8
        for (int i = me; i < upto * PPR; i += kPagedQThreads) {
          const int r = i / PPR, piece = i % PPR;
          const bool on = r < nrows && piece * 8 < p.H;
          const int d = kv_div(rem0 + r, p.by_g);  // token from tok0 on; head rem0 + r - d G
          const int64_t at = (int64_t)d * p.Nq * p.H + (int64_t)(rem0 + r - d * p.G) * p.H + piece * 8;
          kv_cp<16>(sq + (r / kTileRows) * (kTileRows * HD * 2) + tile_at(kTileRows, r % kTileRows, piece),
                    on ? q0 + at : static_cast<const bits*>(p.q), on);
        }
        kv_cp_commit();
        kv_cp_wait<0>();
        tc_fence_smem();
        mbar_arrive(bar(&bars.q_full));
      }
    }
  } else if (warp >= 8) {
    // ------------------------------------------------------------------ K and V
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    const int me = tid - 256;
    constexpr int PPR = HD / 8;              // 16-byte pieces of a row in shared memory
    // a box: p.chunk rows (of one page) x 64 elements; this thread's rows and slab of a tile
    const int chunks = N / p.chunk, boxes = chunks * C::SLABS;
    const int my_row = (me & (chunks - 1)) * p.chunk, my_slab = me / chunks;
    bool bad = false;
    int gs = 0, nk = 0, nv = 0;  // key tiles; those of K and of V whose loads have begun
    while (ok && work.next(p, before, count)) {
      const int4 it = items[work.item];
      int lo, hi;
      const int n = keys_of(it, lo, hi);
      if (n == 0) continue;
      const int b = it.x, kvh = work.kvh;
      const PagedSeq seq = paged_seq(p.s, b);
      const int seen = paged_first(p, seq.past + (int64_t)it.y * ROWS / p.G);  // keys before this are nobody's
      const int32_t* table = p.s.table + (int64_t)b * p.s.max_pages;
      // (row in the page, page) of this thread's box of the tile at j0; -1: zeros
      auto box_of = [&](int j0) {
        const int j = j0 + my_row;
        int2 at = make_int2(0, -1);
        if (me >= boxes || j0 < lo || j0 + N > hi || j + p.chunk <= seen) return at;
        const int i = kv_div(j, p.s.by_ps);
        at.x = j - i * p.s.ps;
        at.y = __ldg(table + i);
        if ((uint32_t)at.y >= (uint32_t)p.s.pages) bad = true, at.y = -1;
        return at;
      };
      auto bring = [&](uint32_t dst, const void* src, const CUtensorMap* map, int j0, int2 box, uint32_t full) {
        if (j0 + N <= hi) {
          if (me == 0)
            mbar_arrive_expect_tx(full, C::kStage);
          else
            mbar_arrive(full);
          if (me < boxes)
            paged_tma(dst + my_slab * (N * 128) + my_row * 128, map, my_slab * 64, box.x, kvh, box.y, full);
          return;
        }
        // the last tile: rows behind the keys have to be zeros
#pragma unroll 4
        for (int i = me; i < N * PPR; i += kTileBring) {
          const int r = i / PPR, piece = i % PPR;
          int64_t at = -1;
          if (j0 + r < hi && j0 + r >= seen && piece * 8 < p.H) {
            at = paged_row(p.s, b, kvh, j0 + r, p.H);
            bad |= at < 0;
          }
          kv_cp<16>(dst + tile_at(N, r, piece), static_cast<const bits*>(src) + (at >= 0 ? at + piece * 8 : 0), at >= 0);
        }
        kv_cp_commit();
        kv_cp_wait<0>();
        tc_fence_smem();
        mbar_arrive(full);
      };
      int2 box = box_of(lo + (n - 1) * N);
      for (int tile = n - 1; tile >= 0; --tile, ++gs) {
        const int st = gs & 1, j0 = lo + tile * N;
        const int2 after = box_of(j0 - N);
        if (gs >= 2) ok = mbar_wait(bar(&bars.k_free[st]), ((gs >> 1) - 1) & 1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        bring(sk + st * C::kStage, p.k, &maps.k, j0, box, bar(&bars.k_full[st]));
        ++nk;
        if (gs >= 2) ok = mbar_wait(bar(&bars.v_free[st]), ((gs >> 1) - 1) & 1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        bring(sv + st * C::kStage, p.v, &maps.v, j0, box, bar(&bars.v_full[st]));
        ++nv;
        box = after;
      }
    }
    if (bad && p.s.status) atomicOr(p.s.status, 4);
    if (!ok) {  // what TMA still brings has to land before shared memory goes
      for (int i = nk - 2; i < nk; ++i)
        if (i >= 0) mbar_wait(bar(&bars.k_full[i & 1]), (i >> 1) & 1);
      for (int i = nv - 2; i < nv; ++i)
        if (i >= 0) mbar_wait(bar(&bars.v_full[i & 1]), (i >> 1) & 1);
    }
  }
  if (!ok && p.s.status) atomicOr(p.s.status, 2);
  tc_before();
  __syncthreads();
  if (warp == 12)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(512) : "memory");
}

// Joins the parts of the items that paged_tile_kernel_t dealt to several CTAs. CTA (x,
// y): the item that begins in CTA x there and goes on in others, if there is one; a warp
// a row, rows 4 y + warp, + 4 gridDim.y, ... `rows`: of a slot.
template <class T>
__global__ void __launch_bounds__(kKvTokenThreads) paged_tile_join_kernel_t(const PagedParams p, int rows) {
  using bits = typename Elem<T>::bits;
  pdl_wait();  // it lets nothing start early: the next call's CTAs would take places unevenly
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int4 what = p.ws_join[blockIdx.x];  // b, kvh, tile of rows, 2 * further CTAs + slot
  if (what.w < 2) return;
  const int kvh = what.y, parts = (what.w >> 1) + 1, c0 = blockIdx.x;
  const PagedSeq seq = paged_seq(p.s, what.x);
  const int64_t row0 = (int64_t)what.z * rows, left = (int64_t)seq.n * p.G - row0;
  const int n_rows = left < rows ? (int)left : rows;
  // Part 0 is the last segment of CTA c0, the others the first segments of theirs.
  auto slot_of = [&](int n) -> int64_t { return 2 * (int64_t)(c0 + n) + (n == 0 ? what.w & 1 : 0); };
  for (int r = (int)blockIdx.y * kTokWarps + warp; r < n_rows; r += gridDim.y * kTokWarps) {
    float M = -CUDART_INF_F;
    for (int n = lane; n < parts; n += 32) M = fmaxf(M, p.ws_ml[slot_of(n) * rows + r].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    const float base = M == -CUDART_INF_F ? 0.0f : M;
    float L = 0.0f, acc[kKvMaxHead / 32];
#pragma unroll
    for (int j = 0; j < kKvMaxHead / 32; ++j) acc[j] = 0.0f;
#pragma unroll 4
    for (int n = 0; n < parts; ++n) {
      const int64_t s = slot_of(n) * rows + r;
      const float2 ml = p.ws_ml[s];
      const float* o = p.ws_o + s * p.H;
      const float f = exp2f(ml.x - base);
      L = fmaf(ml.y, f, L);
#pragma unroll
      for (int j = 0; j < kKvMaxHead / 128; ++j)
        if (lane * 4 + 128 * j < p.H) {
          float4 x = *reinterpret_cast<const float4*>(o + lane * 4 + 128 * j);
          if (ml.x == -CUDART_INF_F && ml.y == 0.0f) x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);  // never written where a CTA had no units
          acc[4 * j] = fmaf(x.x, f, acc[4 * j]);
          acc[4 * j + 1] = fmaf(x.y, f, acc[4 * j + 1]);
          acc[4 * j + 2] = fmaf(x.z, f, acc[4 * j + 2]);
          acc[4 * j + 3] = fmaf(x.w, f, acc[4 * j + 3]);
        }
    }
    const int64_t row = row0 + r, tok = row / p.G;
    bits* y = static_cast<bits*>(p.out) + ((seq.t0 + tok) * p.Nq + (int64_t)kvh * p.G + (row - tok * p.G)) * p.H;
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

template <class T, int HD>
PagedTileKernel paged_tile_of(int kind) {
  using C = TileCfg<false, HD>;
  const void* fn = kind == kKvPlain    ? (const void*)paged_tile_kernel_t<T, HD, kKvPlain>
                   : kind == kKvBiased ? (const void*)paged_tile_kernel_t<T, HD, kKvBiased>
                                       : (const void*)paged_tile_kernel_t<T, HD, kKvAnyScore>;
  return {fn, (const void*)paged_tile_join_kernel_t<T>, 1024 + C::kQ + 4 * C::kStage + kPagedItems * 20 + 16};
}

template <class T>
PagedTileKernel paged_tile_pick(int H, int kind) {
  if (H <= 64) return paged_tile_of<T, 64>(kind);
  if (H <= 128) return paged_tile_of<T, 128>(kind);
  return paged_tile_of<T, 256>(kind);
}

}  // namespace rope_gb300
