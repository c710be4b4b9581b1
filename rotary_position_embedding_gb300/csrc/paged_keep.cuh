// Accepted drafts move up: rows past + kept[b, i] of sequence b to past + i, in K
// and V, for every key/value head.
//
// A thread has one unit of a row of one (b, K or V, kvh) and takes its rows in
// order, kBatch at a time, all loads before all stores. As kept ascends, kept[i] >=
// i: what a batch overwrites lies before every row that a later one reads. Threads
// share nothing, so nothing is waited for. Bound by the latency of three dependent
// loads (length, index, page) and of the rows behind them.
#pragma once

#include "paged_common.cuh"

namespace rope_gb300 {

template <class V>
__global__ void __launch_bounds__(kPagedKeepThreads) paged_keep_kernel_t(const PagedKeepParams p) {
  constexpr int kBatch = 8;
  pdl_launch_dependents();
  pdl_wait();
  const int64_t per = 2 * (int64_t)p.Nkv * p.units;  // threads of a sequence
  const int64_t all = per * p.s.B;
  for (int64_t w = (int64_t)blockIdx.x * kPagedKeepThreads + threadIdx.x; w < all;
       w += (int64_t)gridDim.x * kPagedKeepThreads) {
    const int b = (int)(w / per);
    const int64_t r = w - b * per;
    const int plane = (int)(r / p.units);
    const int64_t u = r - plane * p.units;
    const int kvh = plane >> 1;
    V* pages = static_cast<V*>(plane & 1 ? p.v : p.k);
    const int64_t past = __ldg(p.s.past + b);
    const int n = __ldg(p.kept_lens + b);
    const int32_t* kept = p.kept + (int64_t)b * p.width;
    // the sequence stays as it is unless every row is there and the indices ascend
    bool ok = n >= 0 && n <= p.width && past >= 0;
    int before = -1;
    for (int i = 0; i < n && ok; ++i) {
      const int x = __ldg(kept + i);
      ok = x > before && past + x < p.s.rows;
      before = x;
    }
    for (int i = 0; i < n && ok; ++i) {
      const int x = __ldg(kept + i);
      ok = x == i || (paged_page(p.s, b, (int)past + x) >= 0 && paged_page(p.s, b, (int)past + i) >= 0);
    }
    if (!ok) {
      if (r == 0 && p.s.status) atomicOr(p.s.status, 4);
      continue;
    }
    for (int i0 = 0; i0 < n; i0 += kBatch) {
      V x[kBatch];
      int64_t to[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        to[i] = -1;
        if (i0 + i >= n) continue;
        const int from = __ldg(kept + i0 + i);
        if (from == i0 + i) continue;
        to[i] = paged_row(p.s, b, kvh, (int)past + i0 + i, (int)p.units) + u;
        x[i] = pages[paged_row(p.s, b, kvh, (int)past + from, (int)p.units) + u];
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        if (to[i] >= 0) pages[to[i]] = x[i];
    }
  }
}

}  // namespace rope_gb300
