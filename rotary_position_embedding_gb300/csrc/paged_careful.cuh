// One row of attention over a paged cache by one warp, key by key on CUDA cores:
// taken where a matrix product over a tile would carry an infinity or a NaN of a
// value into a row that does not see it (0 * NaN). Rare, so plain: lanes share the
// head's dimensions, the keys that the row does not see are never read.
#pragma once

#include "paged_common.cuh"

namespace rope_gb300 {

// Row `row` of (b, kvh) over the keys [lo, hi): the output, or with `part_o` (H
// values, each 4 of them part_ld apart) a partial one and its (maximum, sum) at `part_ml`.
template <class T>
__device__ __noinline__ void paged_careful_row(const PagedParams& p, const PagedSeq& seq, int b, int kvh, int64_t row,
                                               int lo, int hi, float* part_o, int part_ld, float2* part_ml,
                                               int lane) {
  using bits = typename Elem<T>::bits;
  constexpr int ND = kKvMaxHead / 32;
  const int64_t tok = row / p.G;
  const int64_t at_row = ((seq.t0 + tok) * p.Nq + (int64_t)kvh * p.G + row % p.G) * p.H;
  const int64_t pos = seq.past + tok;
  const int first = paged_first(p, pos), lim = paged_limit(p, seq, pos);
  if (lo < first) lo = first;
  if (hi > lim) hi = lim;
  const uint64_t word = p.masks ? (uint64_t)__ldg(p.masks + seq.t0 + tok) : ~0ull;
  const float slope = p.slopes ? __ldg(p.slopes + kvh * p.G + row % p.G) * kLog2e : 0.0f;
  const float c1 = p.cap > 0.0f ? p.over : p.scale * kLog2e;
  const float c2 = p.cap * kLog2e;
  float q[ND], o[ND], m = -CUDART_INF_F, l = 0.0f;
#pragma unroll
  for (int i = 0; i < ND; ++i) {
    const int d = lane + 32 * i;
    q[i] = d < p.H ? Elem<T>::tof(static_cast<const bits*>(p.q)[at_row + d]) : 0.0f;
    o[i] = 0.0f;
  }
  for (int j = lo; j < hi; ++j) {
    if (p.masks && j >= seq.past && (j - seq.past >= 64 || !(word >> (j - seq.past) & 1))) continue;
    const int64_t at = paged_row(p.s, b, kvh, j, p.H);
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < ND; ++i) {
      const int d = lane + 32 * i;
      if (d < p.H && at >= 0) s = fmaf(q[i], Elem<T>::tof(static_cast<const bits*>(p.k)[at + d]), s);
    }
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
    float x = s * c1;
    if (p.cap > 0.0f) x = tanhf(x) * c2;
    x = fmaf(-slope, (float)(pos > j ? pos - j : j - pos), x);
    const float mn = fmaxf(m, x);
    const float base = mn == -CUDART_INF_F ? 0.0f : mn;
    const float a = exp2f(m - base), w = exp2f(x - base);
    m = mn;
    l = fmaf(l, a, w);
#pragma unroll
    for (int i = 0; i < ND; ++i) {
      const int d = lane + 32 * i;
      o[i] *= a;
      if (d < p.H && w != 0.0f && at >= 0) o[i] = fmaf(w, Elem<T>::tof(static_cast<const bits*>(p.v)[at + d]), o[i]);
    }
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  if (part_o && lane == 0) *part_ml = make_float2(m, l);
#pragma unroll
  for (int i = 0; i < ND; ++i) {
    const int d = lane + 32 * i;
    if (d >= p.H) continue;
    if (part_o)
      part_o[(d >> 2) * part_ld + (d & 3)] = o[i];
    else
      static_cast<bits*>(p.out)[at_row + d] = Elem<T>::fromf(o[i] * inv);
  }
}

}  // namespace rope_gb300
