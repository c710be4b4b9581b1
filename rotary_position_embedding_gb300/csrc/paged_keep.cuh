// Accepted drafts move up: rows past + kept[b, i] of sequence b to past + i, in K and
// V, for every key/value head.
//
// A warp has one (b, K or V, kvh). It looks the path over, a lane an index, and then
// moves kKeepBatch rows for each group of lanes that shares a row, all loads before all
// stores. As kept ascends, kept[i] >= i: what a batch overwrites lies before every row
// that a later one reads. Warps share nothing, so nothing is waited for. Bound by the
// latency of four dependent loads (length, index, page, row): a thread that walked its
// path by itself took 18 us for 40 rows, this 5.5 (paths of 1 to 7 rows of 64 sequences 3.4).
#pragma once

#include "paged_common.cuh"

namespace rope_gb300 {

constexpr int kKeepBatch = 16;

template <class V>
__global__ void __launch_bounds__(kPagedKeepThreads) paged_keep_kernel_t(const PagedKeepParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, warps = kPagedKeepThreads / 32;
  const int64_t planes = 2 * (int64_t)p.Nkv, all = planes * p.s.B;
  const int per = p.lanes, at_row = lane / per, at_unit = lane & (per - 1), rows = 32 / per;  // lanes of a row; rows at a time
  for (int64_t w = (int64_t)blockIdx.x * warps + threadIdx.x / 32; w < all; w += (int64_t)gridDim.x * warps) {
    const int b = (int)(w / planes), plane = (int)(w - b * planes), kvh = plane >> 1;
    V* pages = static_cast<V*>(plane & 1 ? p.v : p.k);
    const int64_t past = __ldg(p.s.past + b);
    const int n = __ldg(p.kept_lens + b);
    const int32_t* kept = p.kept + (int64_t)b * p.width;
    // the sequence stays as it is unless every row is there, those that have their place already
    // among them, and the indices ascend
    bool ok = n >= 0 && n <= p.width && (n == 0 || past >= 0);
    int before = -1;
    for (int i0 = 0; ok && i0 < n; i0 += 32) {
      const int i = i0 + lane;
      const int x = i < n ? __ldg(kept + i) : 0x7fffffff;
      int left = __shfl_up_sync(0xffffffffu, x, 1);
      if (lane == 0) left = before;
      before = __shfl_sync(0xffffffffu, x, 31);
      bool mine = true;
      if (i < n) {
        mine = x > left && past + x < p.s.rows;
        if (mine) mine = paged_page(p.s, b, (int)past + x) >= 0 && (x == i || paged_page(p.s, b, (int)past + i) >= 0);
      }
      ok = __all_sync(0xffffffffu, mine);
    }
    if (!ok) {
      if (plane == 0 && lane == 0 && p.s.status) atomicOr(p.s.status, 4);
      continue;
    }
    for (int64_t u0 = 0; u0 < p.units; u0 += per) {
      const int64_t u = u0 + at_unit;
      for (int i0 = 0; i0 < n; i0 += kKeepBatch * rows) {
        V x[kKeepBatch];
        int64_t to[kKeepBatch];
#pragma unroll
        for (int k = 0; k < kKeepBatch; ++k) {
          const int i = i0 + k * rows + at_row;
          to[k] = -1;
          if (i >= n || u >= p.units) continue;
          const int from = __ldg(kept + i);
          if (from == i) continue;
          to[k] = paged_row(p.s, b, kvh, (int)past + i, (int)p.units) + u;
          x[k] = pages[paged_row(p.s, b, kvh, (int)past + from, (int)p.units) + u];
        }
        __syncwarp();  // other lanes' loads too come before these stores
#pragma unroll
        for (int k = 0; k < kKeepBatch; ++k)
          if (to[k] >= 0) pages[to[k]] = x[k];
        __syncwarp();
      }
    }
  }
}

}  // namespace rope_gb300
