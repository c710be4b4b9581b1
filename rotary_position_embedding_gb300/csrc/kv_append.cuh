// Q and K rotation with the append of K and V to 8-bit caches.
//
// Every Q and K head goes through the arithmetic of rope_qkv.cuh (the same
// functions, so the same bits): optional RMS norm, rotation, one rounding to T.
// What differs is where K and V go: each value of a new row is rounded to e4m3
// (4 exponent and 3 mantissa bits, largest 448, nearest even) after division
// by the scale of its block of 16 cache rows of one head. A scale is the
// smallest power of two by which the block's largest magnitude fits 448:
//   scale = 2^ceil(log2(amax / 448)).
// A power of two loses nothing over a free scale (an 8-bit float keeps its
// relative precision over 2^15), makes code * scale exact, and makes the
// rescaling of a block exact but for subnormal codes: when an append ends up in
// a block that already holds older rows, the scale only grows, and the codes
// of the older rows are rounded again by the ratio old / new.
//
// Bound by memory: (Nq + 2 Nkv) * H values of T in, Nq * H of T and 2 * Nkv * H
// bytes out per token. Measured: 4 x 2048 bfloat16 tokens of 32/8 heads of 128 with
// QK-Norm 64 us against 27 at the copy rate (latency: 80 registers leave a third
// of the warps); 256 single float16 tokens 3.7 us.
#pragma once

#include <cuda_fp8.h>

#include <type_traits>

#include "kv_common.cuh"
#include "rope_packed.cuh"
#include "rope_qkv.cuh"

namespace rope_gb300 {

// Exponent of the scale of a block without any finite non-zero value.
constexpr int kKvTinyExp = -120;

// 2^ceil(log2(amax / 448)) for a finite amax >= 0: 448 = 0.875 * 2^9, so a
// significand (of 1..2) up to 1.75 fits at exponent - 8.
__device__ __forceinline__ float kv_scale_of(float amax) {
  const uint32_t u = __float_as_uint(amax);
  int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  if (e < kKvTinyExp) e = kKvTinyExp;  // subnormal amax included
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

// The reciprocal of a power of two 2^e, -126 <= e <= 126, exactly.
__device__ __forceinline__ float kv_pow2_inverse(float s) {
  return __uint_as_float((254u << 23) - __float_as_uint(s));
}

__device__ __forceinline__ uint8_t kv_code(float x) {
  return (uint8_t)__nv_cvt_float_to_fp8(x, __NV_SATFINITE, __NV_E4M3);
}

__device__ __forceinline__ float kv_value(uint8_t c) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)c, __NV_E4M3)));
}

// Magnitude for a block's maximum: infinities and NaN do not count (an
// infinity is stored as +-448 * scale, NaN as NaN).
__device__ __forceinline__ float kv_magnitude(float x) {
  const float a = fabsf(x);
  return a < INFINITY ? a : 0.0f;
}

// The largest magnitude that counts among V values. 16-bit values two at a time;
// where that meets an infinity, one by one (a maximum of two drops a NaN).
template <class T, int V>
__device__ __forceinline__ float kv_amax(const VecT<T, V>& x) {
  float m = 0.0f;
  if constexpr (V == 8) {
    Unit8<T> u;
    __builtin_memcpy(&u, &x, 16);
    const auto w = __hmax2(__hmax2(__habs2(u.w[0]), __habs2(u.w[1])), __hmax2(__habs2(u.w[2]), __habs2(u.w[3])));
    const float2 f = P2<T>::tof(w);
    m = fmaxf(f.x, f.y);
    if (m < INFINITY) return m;  // NaN in every place: falls through to 0
    m = 0.0f;
  }
#pragma unroll
  for (int j = 0; j < V; ++j) m = fmaxf(m, kv_magnitude(Elem<T>::tof(x.v[j])));
  return m;
}

template <int V>
struct CodeWord;
template <>
struct CodeWord<8> {
  using t = uint2;
};
template <>
struct CodeWord<4> {
  using t = uint32_t;
};
template <>
struct CodeWord<1> {
  using t = uint8_t;
};

// V codes at once; `dst` is aligned to V bytes.
template <class T, int V>
__device__ __forceinline__ void kv_store_codes(uint8_t* dst, const VecT<T, V>& x, float inv) {
  uint8_t c[V];
  if constexpr (V % 2 == 0) {
#pragma unroll
    for (int j = 0; j < V; j += 2) {
      const __nv_fp8x2_storage_t two = __nv_cvt_float2_to_fp8x2(
          make_float2(Elem<T>::tof(x.v[j]) * inv, Elem<T>::tof(x.v[j + 1]) * inv), __NV_SATFINITE, __NV_E4M3);
      c[j] = (uint8_t)(two & 0xff);
      c[j + 1] = (uint8_t)(two >> 8);
    }
  } else {
    c[0] = kv_code(Elem<T>::tof(x.v[0]) * inv);
  }
  typename CodeWord<V>::t w;
  __builtin_memcpy(&w, c, V);
  *reinterpret_cast<typename CodeWord<V>::t*>(dst) = w;
}

// One unit of a Q or K row: normalised by r and the weights (NORM), then rotated
// where `rotates`. 16-bit data takes the packed forms, which round as the scalar
// ones do.
template <class T, int V, bool INTER, bool NORM>
__device__ __forceinline__ void kv_finish(VecT<T, V>& xa, VecT<T, V>& xb, float r, const VecT<T, V>& wa,
                                          const VecT<T, V>& wb, bool rotates, const VecT<T, V>& c,
                                          const VecT<T, V>& sn) {
  if constexpr (V == 8) {
    Unit8<T> ua, ub, va, vb;
    __builtin_memcpy(&ua, &xa, 16);
    __builtin_memcpy(&ub, &xb, 16);
    if constexpr (NORM) {
      float2 fa[4], fb[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) fa[q] = P2<T>::tof(ua.w[q]), fb[q] = P2<T>::tof(ub.w[q]);
      __builtin_memcpy(&va, &wa, 16);
      __builtin_memcpy(&vb, &wb, 16);
      ua = norm8p<T>(fa, r, va);
      ub = norm8p<T>(fb, r, vb);
    }
    if (rotates) {
      float2 cf[4], sf[4];
      unpack_coef8<T>(c, cf);
      unpack_coef8<T>(sn, sf);
      rotate8p<T, INTER>(ua, ub, cf, sf, va, vb);
      ua = va;
      ub = vb;
    }
    __builtin_memcpy(&xa, &ua, 16);
    __builtin_memcpy(&xb, &ub, 16);
  } else {
    if constexpr (NORM) {
      xa = norm_weight<T, V>(xa, r, wa);
      xb = norm_weight<T, V>(xb, r, wb);
    }
    if (rotates) {
      VecT<T, V> ya, yb;
      rotate_unit<T, V, INTER>(xa, xb, c, sn, ya, yb);
      xa = ya;
      xb = yb;
    }
  }
}

// One unit of a K or V row, from memory to its final T values. With NORM the lanes
// of a K row add up its squares: every one of them comes here together.
template <class T, int V, bool INTER, bool NORM>
__device__ __forceinline__ void kv_row_unit(const KvAppendParams& p, const typename Elem<T>::bits* xr, int k, bool key,
                                            bool valid, int64_t crow, unsigned gmask, VecT<T, V>& xa, VecT<T, V>& xb,
                                            int& oa, int& ob) {
  using VT = VecT<T, V>;
  using bits = typename Elem<T>::bits;
  const bool has = k < p.U, tail = k >= p.nP;
  oa = ob = 0;
  if (tail)
    oa = p.rd + (k - p.nP) * V;
  else
    unit_offsets<V, INTER>(k, p.h, oa, ob);
  VT c{}, sn{}, wa{}, wb{};
  xa = xb = VT{};
  const bool rotates = key && valid && has && !tail;
  if (has) {
    xa = ld_stream(reinterpret_cast<const VT*>(xr + oa));
    if (!tail) xb = ld_stream(reinterpret_cast<const VT*>(xr + ob));
    if (rotates) {
      c = ld_shared_ro(reinterpret_cast<const VT*>(static_cast<const bits*>(p.cos) + crow + k * V));
      sn = ld_shared_ro(reinterpret_cast<const VT*>(static_cast<const bits*>(p.sin) + crow + k * V));
    }
    if (NORM && key) {
      wa = ld_shared_ro(reinterpret_cast<const VT*>(static_cast<const bits*>(p.kw) + oa));
      if (!tail) wb = ld_shared_ro(reinterpret_cast<const VT*>(static_cast<const bits*>(p.kw) + ob));
    }
  }
  if (!key) return;
  float r = 0.0f;
  if (NORM) {
    float ss = sum_squares<T, V>(xa) + sum_squares<T, V>(xb);
    for (int o = p.lanes >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(gmask, ss, o);
    r = 1.0f / sqrtf(ss / (float)p.H + p.eps);
  }
  if (has) kv_finish<T, V, INTER, NORM>(xa, xb, r, wa, wb, rotates, c, sn);
}

// Q: `lanes` threads take one unit each of kKvAppendHeads heads of a token, which
// share position, coefficients and weights; every load goes out before the first
// value is used.
template <class T, int V, bool INTER, bool NORM>
__device__ __forceinline__ void kv_append_q(const KvAppendParams& p, int item, int k, unsigned gmask) {
  using VT = VecT<T, V>;
  using bits = typename Elem<T>::bits;
  constexpr int HPT = kKvAppendHeads;
  const bool live = item < p.q_items;  // uniform over the lanes of a row
  const int tok = live ? kv_div(item, p.by_q) : 0, hd = live ? (item - tok * p.q_groups) * HPT : 0;
  const int b = kv_div(tok, p.by_s), s = tok - b * (int)p.S;
  const int n = p.Nq - hd < HPT ? p.Nq - hd : HPT;
  const bool tail = k >= p.nP, has = live && k < p.U;
  int oa = 0, ob = 0;
  if (tail)
    oa = p.rd + (k - p.nP) * V;
  else
    unit_offsets<V, INTER>(k, p.h, oa, ob);
  const bits* xr =
      static_cast<const bits*>(p.q) + ((int64_t)tok * (p.packed ? p.Nq + 2 * p.Nkv : p.Nq) + hd) * p.H;
  VT xa[HPT], xb[HPT];
#pragma unroll
  for (int i = 0; i < HPT; ++i) {
    xa[i] = xb[i] = VT{};
    if (has && i < n) {
      xa[i] = ld_stream(reinterpret_cast<const VT*>(xr + i * p.H + oa));
      if (!tail) xb[i] = ld_stream(reinterpret_cast<const VT*>(xr + i * p.H + ob));
    }
  }
  const int64_t row = (int64_t)__ldg(p.past + b) + s;
  const int64_t pp = p.pos ? __ldg(p.pos + tok) : row;
  const bool valid = (uint64_t)pp < (uint64_t)p.cache_rows;
  if (live && hd == 0 && k == 0 && p.status) {
    const int f = (valid ? 0 : 1) | (row >= 0 && row < p.max_len ? 0 : 4);
    if (f) atomicOr(p.status, f);
  }
  VT c{}, sn{}, wa{}, wb{};
  const bool rotates = has && valid && !tail;
  if (rotates) {
    const int64_t crow = pp * p.h + k * V;
    c = ld_shared_ro(reinterpret_cast<const VT*>(static_cast<const bits*>(p.cos) + crow));
    sn = ld_shared_ro(reinterpret_cast<const VT*>(static_cast<const bits*>(p.sin) + crow));
  }
  if (NORM && has) {
    wa = ld_shared_ro(reinterpret_cast<const VT*>(static_cast<const bits*>(p.qw) + oa));
    if (!tail) wb = ld_shared_ro(reinterpret_cast<const VT*>(static_cast<const bits*>(p.qw) + ob));
  }
  float ss[HPT];
  if (NORM) {
#pragma unroll
    for (int i = 0; i < HPT; ++i) ss[i] = sum_squares<T, V>(xa[i]) + sum_squares<T, V>(xb[i]);
    for (int o = p.lanes >> 1; o > 0; o >>= 1) {
#pragma unroll
      for (int i = 0; i < HPT; ++i) ss[i] += __shfl_xor_sync(gmask, ss[i], o);
    }
  }
  bits* yr = static_cast<bits*>(p.q_out) + ((int64_t)tok * p.Nq + hd) * p.H;
#pragma unroll
  for (int i = 0; i < HPT; ++i) {
    if (!has || i >= n) break;
    const float r = NORM ? 1.0f / sqrtf(ss[i] / (float)p.H + p.eps) : 0.0f;
    kv_finish<T, V, INTER, NORM>(xa[i], xb[i], r, wa, wb, rotates, c, sn);
    st_stream(reinterpret_cast<VT*>(yr + i * p.H + oa), xa[i]);
    if (!tail) st_stream(reinterpret_cast<VT*>(yr + i * p.H + ob), xb[i]);
  }
}

// The largest value over a group: within a warp, or over group / 32 warps
// through `s` (every thread of the CTA comes here).
__device__ __forceinline__ float kv_group_max(float x, int group, int gi, float* s) {
  for (int o = (group < 32 ? group : 32) >> 1; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  if (group > 32) {
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = x;
    __syncthreads();
    const int w0 = gi * (group >> 5);
    for (int w = 0; w < (group >> 5); ++w) x = fmaxf(x, s[w0 + w]);
  }
  return x;
}

// Rounds the codes of `n` bytes of older rows again by `ratio`.
__device__ __forceinline__ void kv_rescale(uint8_t* held, int64_t n, float ratio, int t, int group, bool wide) {
  if (wide) {
    for (int64_t i = t * 16; i < n; i += (int64_t)group * 16) {
      const uint4 w = *reinterpret_cast<const uint4*>(held + i);
      uint8_t c[16];
      __builtin_memcpy(c, &w, 16);
#pragma unroll
      for (int j = 0; j < 16; ++j) c[j] = kv_code(kv_value(c[j]) * ratio);
      uint4 y;
      __builtin_memcpy(&y, c, 16);
      *reinterpret_cast<uint4*>(held + i) = y;
    }
  } else {
    for (int64_t i = t; i < n; i += group) held[i] = kv_code(kv_value(held[i]) * ratio);
  }
}

// A CTA's threads are groups of lanes * rows (a power of two). The first kv_ctas
// CTAs take blocks of 16 cache rows, a group the K and the V block of a (b, head)
// together, `rows` new rows at a time; the others take Q, `lanes` threads two
// heads of a token. Blocks go first: they do more.
// FAST: a block's new rows and a row's units are no more than the threads.
// Two heads a thread and four CTAs an SM (three for the norm on bfloat16, whose
// registers spill at four): 4 x 2048 tokens, 32 query and 8 key/value heads of
// 128: 46 us in float16, 55 us (float16) and 64 us (bfloat16) with the norm; with
// four heads a thread 54, 63 and 82 us. 256 single tokens: 3.7 us.
template <class T, int V, bool INTER, bool NORM, bool FAST>
__global__ void __launch_bounds__(kKvAppendThreads, NORM && std::is_same<T, __nv_bfloat16>::value ? 3 : 4)
    kv_append_kernel_t(const KvAppendParams p) {
  using VT = VecT<T, V>;
  using bits = typename Elem<T>::bits;
  __shared__ float s_max[2][kKvAppendThreads / 32];
  pdl_launch_dependents();
  pdl_wait();
  const int tid = threadIdx.x;
  const unsigned lane = tid & 31u;
  const unsigned gmask =
      p.lanes >= 32 ? 0xffffffffu : (((1u << p.lanes) - 1u) << (lane & ~(unsigned)(p.lanes - 1)));
  if ((int)blockIdx.x >= p.kv_ctas) {
    const int gi = tid / p.lanes, k0 = tid - gi * p.lanes;
    const int item = ((int)blockIdx.x - p.kv_ctas) * (kKvAppendThreads / p.lanes) + gi;
    // heads of more units than lanes: again for each `lanes` units (never with NORM)
    for (int k = k0; k < p.U || (NORM && k == k0); k += p.lanes) kv_append_q<T, V, INTER, NORM>(p, item, k, gmask);
    return;
  }
  const int group = p.lanes * p.rows;
  const int gi = tid / group, t = tid - gi * group;
  const int slot = t / p.lanes, k0 = t - slot * p.lanes;
  const int64_t nall = (int64_t)p.Nq + 2 * p.Nkv;
  const int task = (int)blockIdx.x * (kKvAppendThreads / group) + gi;
  // `work` is uniform over a group
  bool work = task < p.kv_tasks;
  const int plane = work ? kv_div(task, p.by_blocks) : 0, nb = work ? task - plane * (int)p.blocks : 0;
  const int b = kv_div(plane, p.by_kv), hd = plane - b * p.Nkv;
  const int64_t past = __ldg(p.past + b);
  const int64_t blk = (past > 0 ? past : 0) / kKvBlock + nb;
  int64_t r0 = blk * kKvBlock > past ? blk * kKvBlock : past, r1 = (blk + 1) * kKvBlock;
  if (past + p.S < r1) r1 = past + p.S;
  if (p.max_len < r1) r1 = p.max_len;
  if (r0 < 0) r0 = 0;
  work = work && r0 < r1;
  const bits* src[2];  // K, V
  int64_t sstride;
  if (p.packed) {
    src[0] = static_cast<const bits*>(p.q) + (p.Nq + hd) * p.H;
    src[1] = src[0] + p.Nkv * p.H;
    sstride = nall * p.H;
  } else {
    src[0] = static_cast<const bits*>(p.k) + hd * p.H;
    src[1] = static_cast<const bits*>(p.v) + hd * p.H;
    sstride = (int64_t)p.Nkv * p.H;
  }
  const bool older = work && blk * kKvBlock < past;
  const int64_t at = plane * p.nblk + blk, row0 = plane * p.max_len;
  const float was[2] = {older ? p.k_scale[at] : 0.0f, older ? p.v_scale[at] : 0.0f};
  // The first unit of a thread stays in its registers between the maximum and
  // the store; what follows it (more rows or units than threads) is formed twice.
  VT ya0[2] = {}, yb0[2] = {};
  int oa0 = 0, ob0 = 0;
  auto form = [&](int kind, int64_t row, int k, VT& ya, VT& yb, int& oa, int& ob) {
    const int64_t tok = b * p.S + (row - past);
    bool valid = false;
    int64_t pp = 0;
    if (kind == 0) {
      pp = p.pos ? __ldg(p.pos + tok) : row;
      valid = (uint64_t)pp < (uint64_t)p.cache_rows;
    }
    kv_row_unit<T, V, INTER, NORM>(p, src[kind] + tok * sstride, k, kind == 0, valid, pp * p.h, gmask, ya, yb, oa, ob);
  };
  auto norm_lane = [&](int k) { return NORM && k == k0; };  // every lane of a row joins its sum
  float amax[2] = {0.0f, 0.0f};
  if constexpr (FAST) {
    if (work && r0 + slot < r1) {
#pragma unroll
      for (int i = 1; i >= 0; --i) {  // V first: its loads wait for nothing
        form(i, r0 + slot, k0, ya0[i], yb0[i], oa0, ob0);
        amax[i] = fmaxf(kv_amax<T, V>(ya0[i]), kv_amax<T, V>(yb0[i]));
      }
    }
  } else if (work) {
    for (int64_t row = r0 + slot; row < r1; row += p.rows)
      for (int k = k0; k < p.U || norm_lane(k); k += p.lanes) {
        VT ya[2] = {}, yb[2] = {};
        int oa, ob;
#pragma unroll
        for (int i = 1; i >= 0; --i) {
          form(i, row, k, ya[i], yb[i], oa, ob);
          amax[i] = fmaxf(amax[i], fmaxf(kv_amax<T, V>(ya[i]), kv_amax<T, V>(yb[i])));
        }
        if (row == r0 + slot && k == k0) {
          ya0[0] = ya[0], ya0[1] = ya[1], yb0[0] = yb[0], yb0[1] = yb[1];
          oa0 = oa, ob0 = ob;
        }
      }
  }
  amax[0] = kv_group_max(amax[0], group, gi, s_max[0]);
  amax[1] = kv_group_max(amax[1], group, gi, s_max[1]);
  if (!work) return;  // no barrier below
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float scale = kv_scale_of(amax[i]);
    if (older && was[i] > scale) scale = was[i];
    const float inv = kv_pow2_inverse(scale);
    uint8_t* cache = (i ? p.v_cache : p.k_cache) + row0 * p.H;
    if constexpr (FAST) {
      if (r0 + slot < r1 && k0 < p.U) {
        uint8_t* dst = cache + (r0 + slot) * p.H;
        kv_store_codes<T, V>(dst + oa0, ya0[i], inv);
        if (k0 < p.nP) kv_store_codes<T, V>(dst + ob0, yb0[i], inv);
      }
    } else {
      for (int64_t row = r0 + slot; row < r1; row += p.rows)
        for (int k = k0; k < p.U || norm_lane(k); k += p.lanes) {
          VT ya = ya0[i], yb = yb0[i];
          int oa = oa0, ob = ob0;
          if (!(row == r0 + slot && k == k0)) form(i, row, k, ya, yb, oa, ob);
          if (k >= p.U) continue;
          uint8_t* dst = cache + row * p.H;
          kv_store_codes<T, V>(dst + oa, ya, inv);
          if (k < p.nP) kv_store_codes<T, V>(dst + ob, yb, inv);
        }
    }
    if (older && was[i] < scale)
      kv_rescale(cache + blk * kKvBlock * p.H, (past - blk * kKvBlock) * p.H, was[i] * inv, t, group, p.wide);
    // `was` was read by every thread before the maximum's exchange
    if (t == 0) (i ? p.v_scale : p.k_scale)[at] = scale;
  }
}

}  // namespace rope_gb300
