// Shared by the kernels over paged caches: which tokens a sequence has, where its
// rows lie, and which keys a row sees.
//
// Sequence b has the tokens [t0, t0 + n); token t0 + s is at row i = past[b] + s,
// and total = past[b] + n, at most the rows of its page table. Key j is visible to
// it if 0 <= j < total and
//   j <= i and (no window or j > i - window), or with masks
//   j < past[b], or bit j - past[b] (below 64) of the token's mask is set.
// A page outside the pool holds zeros for a reader and takes nothing.
#pragma once

#include "kv_common.cuh"
#include "paged_internal.h"

namespace rope_gb300 {

struct PagedSeq {
  int64_t t0;      // its first token
  int n;           // new tokens (0 where there are more than the call allows)
  int past;        // clipped to [-2^30, 2^30]
  int total;       // rows that exist, within [0, rows]
};

__device__ __forceinline__ PagedSeq paged_seq(const PagedBatch& s, int b) {
  PagedSeq q;
  int64_t a, e;
  if (s.starts) {
    a = __ldg(s.starts + b);
    e = __ldg(s.starts + b + 1);
    a = a < 0 ? 0 : a > s.T ? s.T : a;
    e = e < a ? a : e > s.T ? s.T : e;
  } else {
    a = s.S * b;
    e = a + s.S;
  }
  q.t0 = a;
  q.n = e - a > s.most ? 0 : (int)(e - a);
  int p = __ldg(s.past + b);
  constexpr int kFar = 1 << 30;
  q.past = p < -kFar ? -kFar : p > kFar ? kFar : p;
  const int64_t t = (int64_t)q.past + q.n;
  q.total = t < 0 ? 0 : t > s.rows ? (int)s.rows : (int)t;
  return q;
}

// Once for each sequence: rows outside its page table, or more tokens than allowed.
__device__ __forceinline__ void paged_flag_seq(const PagedBatch& s, int b, const PagedSeq& q) {
  if (!s.status) return;
  const int64_t n = s.starts ? (int64_t)__ldg(s.starts + b + 1) - __ldg(s.starts + b) : s.S;
  if (n > s.most || (q.n > 0 && (q.past < 0 || (int64_t)q.past + q.n > s.rows))) atomicOr(s.status, 4);
}

// The page of row j, 0 <= j < rows, or -1.
__device__ __forceinline__ int paged_page(const PagedBatch& s, int b, int j) {
  const int page = __ldg(s.table + (int64_t)b * s.max_pages + kv_div(j, s.by_ps));
  return (uint32_t)page < (uint32_t)s.pages ? page : -1;
}

// Element offset of row j of (b, kvh) in the pages, or -1.
__device__ __forceinline__ int64_t paged_row(const PagedBatch& s, int b, int kvh, int j, int H) {
  const int i = kv_div(j, s.by_ps);
  const int page = __ldg(s.table + (int64_t)b * s.max_pages + i);
  if ((uint32_t)page >= (uint32_t)s.pages) return -1;
  return page * s.page_stride + ((int64_t)kvh * s.ps + (j - i * s.ps)) * H;
}

// The sequence of token t, and true if it has one. Where each sequence before it
// has one token it is t itself, which is looked at first: a decode step's tokens
// need no search.
__device__ __forceinline__ bool paged_find(const PagedBatch& s, int64_t t, int* b) {
  if (!s.starts) {
    *b = (int)(t / s.S);
    return true;
  }
  int x = 0, y = s.B;  // starts[x] <= t < starts[y], if t is some sequence's
  if (t < s.B && __ldg(s.starts + t) == t) x = (int)t;
  if (x < s.B && __ldg(s.starts + x + 1) > t) y = x + 1;
  while (y - x > 1) {
    const int mid = (x + y) >> 1;
    if (__ldg(s.starts + mid) <= t)
      x = mid;
    else
      y = mid;
  }
  *b = x;
  return __ldg(s.starts + x) <= t && t < __ldg(s.starts + x + 1);
}

// Keys that the token at row i can see lie in [first, limit).
__device__ __forceinline__ int paged_limit(const PagedParams& p, const PagedSeq& q, int64_t i) {
  if (i < 0) return 0;
  const int64_t l = p.masks ? q.total : i + 1;
  return l < q.total ? (int)l : q.total;
}
__device__ __forceinline__ int paged_first(const PagedParams& p, int64_t i) {
  const int64_t f = p.window > 0 ? i - p.window + 1 : 0;
  return f <= 0 ? 0 : f < (1 << 30) ? (int)f : 1 << 30;
}

}  // namespace rope_gb300
