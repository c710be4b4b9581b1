// Shared by the attention kernels over a key/value cache: which keys a row
// sees, and the score's arithmetic.
//
// For row r = (token s, query head h) of sequence b, with i = past[b] + s and
// total = past[b] + S clipped to [0, max_len], key j is visible if
//   0 <= j < total,  j <= i or j < prefix[b],  docs[b, j] == docs[b, i],
// and its score is
//   x = c(q.k * scale) - slope[h] * |i - j|,  c(y) = cap * tanh(y / cap) or y.
// The kernels hold x * log2(e), so a weight is one exp2. A row that sees no key,
// or whose largest score is -inf, is 0.
#pragma once

#include <cuda_fp8.h>
#include <math_constants.h>

#include "kv_internal.h"
#include "rope_kernels.cuh"

namespace rope_gb300 {

constexpr float kLog2e = 1.4426950408889634f;

// n / d for 0 <= n < 2^31 by the multiplier and shift of KvDiv.
__device__ __forceinline__ int kv_div(int n, const KvDiv& d) { return (int)(((uint64_t)(uint32_t)n * d.m) >> d.shift); }

struct KvSeq {
  int64_t past, total, prefix;  // prefix clipped to [0, total]
};

__device__ __forceinline__ KvSeq kv_seq(const KvParams& p, int b) {
  KvSeq q;
  q.past = __ldg(p.past + b);
  int64_t t = q.past + p.S;
  if (t > p.max_len) t = p.max_len;
  if (t < 0) t = 0;
  q.total = t;
  int64_t x = p.prefix ? (int64_t)__ldg(p.prefix + b) : 0;
  if (x < 0) x = 0;
  if (x > t) x = t;
  q.prefix = x;
  return q;
}

// Keys [0, limit) are what a query at position i may see before documents.
__device__ __forceinline__ int64_t kv_limit(const KvSeq& q, int64_t i) {
  int64_t l = i + 1 > q.prefix ? i + 1 : q.prefix;
  return l < q.total ? l : q.total;
}

// A query outside the cache has no document: with documents it sees nothing.
__device__ __forceinline__ bool kv_document(const KvParams& p, int b, int64_t i, int32_t* id) {
  if (i < 0 || i >= p.max_len) return false;
  *id = __ldg(p.docs + (int64_t)b * p.max_len + i);
  return true;
}

// Keys of split `n` of `splits`: [lo, hi) within [0, end), a multiple of `unit`
// keys each but the last.
__device__ __forceinline__ void kv_split(int64_t end, int splits, int n, int unit, int64_t* lo, int64_t* hi) {
  int64_t per = (end + splits - 1) / splits;
  per = (per + unit - 1) / unit * unit;
  *lo = per * n < end ? per * n : end;
  *hi = *lo + per < end ? *lo + per : end;
}

__device__ __forceinline__ void kv_flag_rows(const KvParams& p, const KvSeq& q) {
  if (p.status && (q.past < 0 || q.past + p.S > p.max_len)) atomicOr(p.status, 4);
}

__device__ __forceinline__ float2 kv_fp8x2(uint16_t two) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3);
  return __half22float2(__half2(h));
}

__device__ __forceinline__ uint32_t kv_smem(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

// 16 (or 8) bytes global -> shared.
template <int BYTES>
__device__ __forceinline__ void kv_cp(uint32_t dst, const void* src) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES) : "memory");
}

// 16 (or 8, 4) bytes global -> shared; zeros where `on` is false.
template <int BYTES>
__device__ __forceinline__ void kv_cp(uint32_t dst, const void* src, bool on) {
  const int n = on ? BYTES : 0;
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(BYTES), "r"(n) : "memory");
}
__device__ __forceinline__ void kv_cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void kv_cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

}  // namespace rope_gb300
