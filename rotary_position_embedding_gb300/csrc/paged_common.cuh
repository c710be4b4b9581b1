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

// The tokens [a, e) of sequence b: starts count as clipped to [0, T].
__device__ __forceinline__ void paged_tokens(const PagedBatch& s, int b, int64_t& a, int64_t& e) {
  if (s.starts) {
    a = __ldg(s.starts + b);
    e = __ldg(s.starts + b + 1);
    a = a < 0 ? 0 : a > s.T ? s.T : a;
    e = e < a ? a : e > s.T ? s.T : e;
  } else {
    a = s.S * b;
    e = a + s.S;
  }
}

__device__ __forceinline__ PagedSeq paged_seq(const PagedBatch& s, int b) {
  PagedSeq q;
  int64_t a, e;
  paged_tokens(s, b, a, e);
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
  int64_t a, e;
  paged_tokens(s, b, a, e);
  if (e - a > s.most || (q.n > 0 && (q.past < 0 || (int64_t)q.past + q.n > s.rows))) atomicOr(s.status, 4);
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

// Which of sequence b's tokens `t` is, one of them: attention counts from the clipped start too.
__device__ __forceinline__ int64_t paged_nth(const PagedBatch& s, int b, int64_t t) {
  if (!s.starts) return t - s.S * b;
  const int64_t a = __ldg(s.starts + b);
  return t - (a < 0 ? 0 : a);
}

// Keys that the token at row i can see lie in [first, limit).
__device__ __forceinline__ int paged_limit(const PagedParams& p, const PagedSeq& q, int64_t i) {
  if (i < 0 && !p.masks) return 0;
  const int64_t l = p.masks ? q.total : i + 1;
  return l < q.total ? (int)l : q.total;
}
__device__ __forceinline__ int paged_first(const PagedParams& p, int64_t i) {
  const int64_t f = p.window > 0 ? i - p.window + 1 : 0;
  return f <= 0 ? 0 : f < (1 << 30) ? (int)f : 1 << 30;
}

// Keys [lo, end) of a sequence for the kernel for few rows, lo at the start of a unit; a
// unit where there are none, so that its output is written.
constexpr int kPagedUnit = 64;  // keys of a unit
struct PagedSpan {
  int lo, end;
  __device__ __forceinline__ int units() const { return end > lo ? (end - lo + kPagedUnit - 1) / kPagedUnit : 1; }
};
__device__ __forceinline__ PagedSpan paged_span(const PagedParams& p, const PagedSeq& q) {
  PagedSpan s;
  s.lo = paged_first(p, q.past) / kPagedUnit * kPagedUnit;
  s.end = paged_limit(p, q, (int64_t)q.past + q.n - 1);
  return s;
}
// Whether a sequence is the kernel's for few rows.
__device__ __forceinline__ bool paged_few(const PagedParams& p, const PagedSeq& q) {
  return q.n > 0 && (int64_t)q.n * p.G <= (p.mixed ? p.mixed : kPagedFewRows);
}

// A mixed batch: prompts are bound by the tensor cores, single tokens by the memory, so
// paged_tile_kernel_t and paged_token_kernel_t run at a time, the first on `n` SMs, the
// second on the others: about 100 of them take what the memory gives (62 GB/s an SM).
// Both work n out of the lengths in whole numbers, each sequence's time (ns of an SM)
// added up in any order. The weights are what divided mixed batches best (12 of them, heads
// of 64 to 256, capped or not; 4 ns a dim in place of 104 + 2.8 a dim: 4 to 8 % slower where
// scores are not capped, the same where they are). A mixed step of a capped prompt of 2048 tokens and 95 single
// tokens over up to 4000 keys: one after the other 255 us, so 175.
struct PagedTimes {
  unsigned long long tile, token;
};
__device__ __forceinline__ void paged_time(const PagedParams& p, const PagedSeq& q, PagedTimes* t) {
  if (q.n == 0) return;
  if (paged_few(p, q)) {
    t->token += (unsigned long long)paged_span(p, q).units() * (104u + (unsigned)p.H * 28u / 10u);
  } else {
    const int keys = p.H <= 128 ? 128 : 64, step = p.H <= 64 ? 1400 : p.H <= 128 ? 1600 : 1000;
    int64_t span = (int64_t)q.past + q.n / 2;
    if (p.window > 0 && span > p.window + p.tpi) span = p.window + p.tpi;
    if (span < 0) span = 0;
    const int64_t items = (q.n + p.tpi - 1) / p.tpi;
    t->tile += (unsigned long long)(items * (span / keys + 1 + p.over_item)) * (unsigned)(p.cap > 0.0f ? step + 650 : step);
  }
}
// The times of a warp's threads, added up, to the warp's own place; paged_shares adds up
// those of all warps. (96 threads' atomics on one place and a quotient of doubles took both
// kernels 6 us.)
__device__ __forceinline__ void paged_times(PagedTimes t, PagedTimes* of_warp) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    t.tile += __shfl_xor_sync(0xffffffffu, t.tile, o);
    t.token += __shfl_xor_sync(0xffffffffu, t.token, o);
  }
  if ((threadIdx.x & 31) == 0) *of_warp = t;
}
template <int WARPS>
__device__ __forceinline__ int paged_shares(const PagedTimes* of_warp) {
  PagedTimes t = {0, 0};
#pragma unroll
  for (int w = 0; w < WARPS; ++w) t.tile += of_warp[w].tile, t.token += of_warp[w].token;
  const unsigned long long all = t.tile + t.token;  // below 2^50
  if (t.tile == 0) return 0;
  int n = (int)((2 * 152 * t.tile + all) / (2 * all));
  if (n < 1) n = 1;
  return t.token > 0 && n > 151 ? 151 : n > 152 ? 152 : n;
}

}  // namespace rope_gb300
