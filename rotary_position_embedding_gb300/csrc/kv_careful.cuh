// One row of attention by one warp, key by key on CUDA cores: taken where a
// matrix product over a tile would carry an infinity or a NaN of a value into a
// row that does not see it (0 * NaN). Rare, so plain: lanes share the head's
// dimensions, the keys that the row does not see are never read.
#pragma once

#include "kv_common.cuh"

namespace rope_gb300 {

// Row `row` of (b, kvh) over the keys [lo, hi): the output, or with `part_o` (H
// values) a partial one and its (maximum, sum) at `part_ml`.
template <class T, bool FP8>
__device__ __noinline__ void kv_careful_row(const KvParams& p, const KvSeq& seq, int b, int kvh, int64_t row,
                                            int64_t lo, int64_t hi, float* part_o, float2* part_ml, int lane) {
  using bits = typename Elem<T>::bits;
  constexpr int ND = kKvMaxHead / 32;
  const int64_t plane = (int64_t)b * p.Nkv + kvh;
  const int64_t at_row = (((int64_t)b * p.S + row / p.G) * p.Nq + (int64_t)kvh * p.G + row % p.G) * p.H;
  const int64_t pos = seq.past + row / p.G;
  int64_t lim = kv_limit(seq, pos);
  int32_t doc = 0;
  if (p.docs && !kv_document(p, b, pos, &doc)) lim = 0;
  if (hi < lim) lim = hi;
  const float slope = p.slopes ? __ldg(p.slopes + kvh * p.G + row % p.G) * kLog2e : 0.0f;
  const float c1 = p.cap > 0.0f ? p.over : p.scale * kLog2e;
  const float c2 = p.cap * kLog2e;
  auto value = [&](const void* base, const float* scales, int64_t j, int d) -> float {
    const int64_t e = (plane * p.max_len + j) * p.H + d;
    if constexpr (FP8)
      return kv_fp8x2(static_cast<const uint8_t*>(base)[e]).x * __ldg(scales + plane * p.nblk + j / kKvBlock);
    else
      return Elem<T>::tof(static_cast<const bits*>(base)[e]);
  };
  float q[ND], o[ND], m = -CUDART_INF_F, l = 0.0f;
#pragma unroll
  for (int i = 0; i < ND; ++i) {
    const int d = lane + 32 * i;
    q[i] = d < p.H ? Elem<T>::tof(static_cast<const bits*>(p.q)[at_row + d]) : 0.0f;
    o[i] = 0.0f;
  }
  for (int64_t j = lo; j < lim; ++j) {
    if (p.docs && __ldg(p.docs + (int64_t)b * p.max_len + j) != doc) continue;
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < ND; ++i) {
      const int d = lane + 32 * i;
      if (d < p.H) s = fmaf(q[i], value(p.k, p.ks, j, d), s);
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
      if (d < p.H && w != 0.0f) o[i] = fmaf(w, value(p.v, p.vs, j, d), o[i]);
    }
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  if (part_o && lane == 0) *part_ml = make_float2(m, l);
#pragma unroll
  for (int i = 0; i < ND; ++i) {
    const int d = lane + 32 * i;
    if (d >= p.H) continue;
    if (part_o)
      part_o[d] = o[i];
    else
      static_cast<bits*>(p.out)[at_row + d] = Elem<T>::fromf(o[i] * inv);
  }
}

}  // namespace rope_gb300
