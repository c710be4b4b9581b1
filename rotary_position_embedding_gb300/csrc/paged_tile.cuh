// Attention over a paged cache for many rows (prompts, chunks, draft trees): tcgen05.
//
// The kernel is kv_tile_kernel_t (kv_tile.cuh) for 16-bit caches, step for step: two
// tiles of 128 rows take turns on the tensor cores, S and O in TMEM, P = 2^(x - m) by
// the threads that own the rows, the base moved only where a tile's weights ask for
// it. What differs:
//   - a CTA finds its sequence and rows from query_starts;
//   - K and V come in boxes, the rows of a key tile that lie in one page x 64 elements,
//     one thread a box (16 boxes of 16 rows at H = 128), each with the next tile's page
//     looked up a step ahead;
//   - a row sees keys from its window on; of a draft tree's new keys those whose bit its
//     mask holds. Only key tiles that some row does not see whole are looked at key by
//     key, as bits of four words.
// Bound by the tensor cores for prompts; trees, whose rows are one tile or less, by the
// pages' bandwidth.
#pragma once

#include "kv_tile.cuh"
#include "paged_token.cuh"

namespace rope_gb300 {

// The sequence and tile of rows that are number `item` among those of the batch, in
// s_item (s_item[0] is -1 before, and stays so where there are fewer). All threads come
// here. The longest rows of a sequence go first.
__device__ __forceinline__ void paged_tile_item(const PagedParams& p, int item, int rows, int* s_sum, int* s_item) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int before = 0;  // items of the sequences behind us
  for (int b0 = 0; b0 < p.s.B; b0 += kTileThreads) {
    const int b = b0 + tid;
    int n = 0;
    if (b < p.s.B) {
      const int64_t R = (int64_t)paged_seq(p.s, b).n * p.G;
      if (!(p.mixed && R <= kPagedFewRows)) n = (int)((R + rows - 1) / rows);
    }
    int upto = n;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int x = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += x;
    }
    __syncthreads();  // the sums before have been read
    if (lane == 31) s_sum[warp] = upto;
    __syncthreads();
    int all = 0;
    for (int w = 0; w < kTileThreads / 32; ++w) {
      if (w < warp) upto += s_sum[w];
      all += s_sum[w];
    }
    upto += before;
    if (n > 0 && item < upto && item >= upto - n) {
      s_item[0] = b;
      s_item[1] = upto - 1 - item;
    }
    before += all;
    if (item < before) break;  // the same for all threads
  }
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
__global__ void __launch_bounds__(kTileThreads, 1)
    paged_tile_kernel_t(const PagedParams p, const __grid_constant__ PagedMaps maps) {
  using C = TileCfg<false, HD>;
  using bits = typename Elem<T>::bits;
  constexpr bool BF = kIsBf16<T>;
  constexpr int NT = C::NT, N = C::N;
  extern __shared__ uint8_t kv_tiles[];
  __shared__ TileBars bars;
  __shared__ uint32_t s_tmem;
  __shared__ int s_sum[kTileThreads / 32], s_item[2];
  uint8_t* base = kv_tiles + ((1024 - (kv_smem(kv_tiles) & 1023)) & 1023);
  const uint32_t sq = kv_smem(base), sk = sq + C::kQ, sv = sk + 2 * C::kStage;
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
    mbar_init(bar(&bars.q_full), NT * kTileRows);
    mbar_init(bar(&bars.drain), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    s_item[0] = -1;
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

  // this CTA's sequence, rows, head and split of the keys
  const int per = p.Nkv * p.splits, item = (int)blockIdx.x / per, in = (int)blockIdx.x - item * per;
  const int kvh = in / p.splits, split = in - kvh * p.splits;
  if (p.s.starts) {
    paged_tile_item(p, item, NT * kTileRows, s_sum, s_item);
  } else if (tid == 0) {
    s_item[0] = item % p.s.B;
    s_item[1] = p.tiles - 1 - item / p.s.B;  // the longest rows first
  }
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = s_tmem;
  const int b = s_item[0];
  // every sequence's lengths are looked at once, where the other kernel has not
  if (p.s.status && !p.mixed)
    for (int64_t i = (int64_t)blockIdx.x * kTileThreads + tid; i < p.s.B; i += (int64_t)gridDim.x * kTileThreads)
      paged_flag_seq(p.s, (int)i, paged_seq(p.s, (int)i));
  const PagedSeq seq = paged_seq(p.s, b < 0 ? 0 : b);
  const int64_t R = (int64_t)seq.n * p.G, rows0 = b < 0 ? 0 : (int64_t)s_item[1] * (NT * kTileRows);
  if (b < 0 || rows0 >= R) {  // more CTAs than tiles of rows (the same for all threads)
    if (warp == 12)
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(512) : "memory");
    return;
  }
  const int nrows = R - rows0 < NT * kTileRows ? (int)(R - rows0) : NT * kTileRows;  // at least 1
  const int live_tiles = nrows > kTileRows ? NT : 1;
  const int64_t tok0 = rows0 / p.G;  // token and head of row r: see tok_of, row_at
  const uint32_t rem0 = (uint32_t)(rows0 - tok0 * p.G), G = (uint32_t)p.G;
  auto tok_of = [&](int r) { return tok0 + (rem0 + (uint32_t)r) / G; };
  auto row_at = [&](int r) {
    const uint32_t d = (rem0 + (uint32_t)r) / G, h = rem0 + (uint32_t)r - d * G;
    return ((seq.t0 + tok0 + d) * p.Nq + (int64_t)kvh * p.G + h) * p.H;
  };
  // the keys that some row sees, from the start of a key tile on, and this split's
  const int seen = paged_first(p, seq.past + tok0), start = seen / N * N;
  const int end = paged_limit(p, seq, seq.past + tok_of(nrows - 1));
  int64_t lo64, hi64;
  kv_split(end > start ? end - start : 0, p.splits, split, N, &lo64, &hi64);
  const int lo = start + (int)lo64, hi = start + (int)hi64;
  const int first = (hi - lo + N - 1) / N - 1;  // key tiles go from the last to the first
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
    if (t < NT) {
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
    const int lim = live ? paged_limit(p, seq, pos) : 0, from = paged_first(p, pos);
    const uint64_t word = p.masks && live ? (uint64_t)__ldg(p.masks + seq.t0 + tok_of(tid)) : ~0ull;
    TileRow tr;
    tr.doc = 0;
    tr.part = tr.look = tr.ahead = false;
    // keys in [below, full) are seen by every row of the warp
    const int full = __reduce_min_sync(0xffffffffu, !live ? 0x7fffffff : p.masks && seq.past < lim ? seq.past : lim);
    const int below = __reduce_max_sync(0xffffffffu, live ? from : 0);
    tr.slope = 0.0f;
    if (p.slopes && live) tr.slope = __ldg(p.slopes + kvh * p.G + (rem0 + tid) % G) * kLog2e;
    const bool capped = KIND == kKvAnyScore && p.cap > 0.0f;
    const float mult = capped ? 2.0f * kLog2e * p.over : p.scale * kLog2e;
    tr.unit = 1.0f;
    tr.mult = mult;
    tr.cap2 = p.cap * kLog2e;
    const bool general = KIND == kKvBiased || (KIND == kKvAnyScore && (p.slopes || !(p.scale > 0.0f)));
    float m = live ? -CUDART_INF_F : 0.0f, l = 0.0f;  // rows behind the last never move the base
    if (t < live_tiles) {
      int step = 0;
      for (int tile = first; tile >= 0; --tile, ++step) {
        const int j0 = lo + tile * N;
        const int buf = NT == 2 ? t : step & 1;
        const uint32_t par = (NT == 2 ? step : step >> 1) & 1;
        const uint32_t ts = tmem + lanes + (NT == 2 ? t * 128 : buf * N);
        const uint32_t to = tmem + lanes + 256 + (NT == 2 ? t * 128 : 0);
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
        const float f = p.splits > 1 ? 1.0f : inv;
        const bool empty = m == -CUDART_INF_F && l == 0.0f;  // nothing seen (TMEM may never have been written)
        const int64_t at = ((int64_t)kvh * p.splits + split) * p.s.T * p.G + seq.t0 * p.G + row;
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
        if (again) {
          bool found = false;  // in a value that some row of the warp does not see and its key tile holds
          auto look = [&](int from_key, int to_key) {
            for (int j = from_key; j < to_key; ++j) {
              const int64_t e = paged_row(p.s, b, kvh, j, p.H);
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
          const int64_t w = ((int64_t)kvh * p.splits + split) * p.s.T * p.G + seq.t0 * p.G + rows0 + (warp * 32 + r);
          paged_careful_row<T>(p, seq, b, kvh, rows0 + (warp * 32 + r), lo, hi, p.splits > 1 ? p.ws_o + w * p.H : nullptr,
                               p.ws_ml + w, lane);
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
        const bool more = tile > 0;
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
        --tile;
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
    // a box: p.chunk rows (of one page) x 64 elements; this thread's rows and slab of a tile
    const int chunks = N / p.chunk, boxes = chunks * C::SLABS;
    const int my_row = (me & (chunks - 1)) * p.chunk, my_slab = me / chunks;
    const int32_t* table = p.s.table + (int64_t)b * p.s.max_pages;
    bool bad = false;
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
    int step = 0, nk = 0, nv = 0;  // tiles of K and of V whose loads have begun
    int2 box = box_of(lo + first * N);
    for (int tile = first; tile >= 0; --tile, ++step) {
      const int st = step & 1, j0 = lo + tile * N;
      const int2 after = box_of(j0 - N);
      if (step >= 2) ok = mbar_wait(bar(&bars.k_free[st]), ((step >> 1) - 1) & 1);
      if (!__all_sync(0xffffffffu, ok)) break;
      bring(sk + st * C::kStage, p.k, &maps.k, j0, box, bar(&bars.k_full[st]));
      ++nk;
      if (step >= 2) ok = mbar_wait(bar(&bars.v_free[st]), ((step >> 1) - 1) & 1);
      if (!__all_sync(0xffffffffu, ok)) break;
      bring(sv + st * C::kStage, p.v, &maps.v, j0, box, bar(&bars.v_full[st]));
      ++nv;
      box = after;
    }
    if (bad && p.s.status) atomicOr(p.s.status, 4);
    if (!__all_sync(0xffffffffu, ok)) {  // what TMA still brings has to land before shared memory goes
      ok = false;
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

template <class T, int HD>
KvTileKernel paged_tile_of(int kind) {
  const void* fn = kind == kKvPlain    ? (const void*)paged_tile_kernel_t<T, HD, kKvPlain>
                   : kind == kKvBiased ? (const void*)paged_tile_kernel_t<T, HD, kKvBiased>
                                       : (const void*)paged_tile_kernel_t<T, HD, kKvAnyScore>;
  return {fn, TileCfg<false, HD>::kSmem};
}

template <class T>
KvTileKernel paged_tile_pick(int H, int kind) {
  if (H <= 64) return paged_tile_of<T, 64>(kind);
  if (H <= 128) return paged_tile_of<T, 128>(kind);
  return paged_tile_of<T, 256>(kind);
}

}  // namespace rope_gb300
