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
// bytes out per token.
#pragma once

#include <cuda_fp8.h>

#include "kv_internal.h"
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

template <class T, int V>
__device__ __forceinline__ float kv_amax(const VecT<T, V>& x) {
  float m = 0.0f;
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

// One unit of a Q or K row: loaded, normalised (NORM: the row's lanes add up
// its squares; every lane of the row comes here together) and rotated. `xr` is
// null for lanes without a row (they only take part in the sum).
template <class T, int V, bool INTER, bool NORM>
__device__ __forceinline__ void kv_row_unit(const KvAppendParams& p, const typename Elem<T>::bits* xr, int k,
                                            bool rotates, const void* weight, bool valid, int64_t crow,
                                            unsigned gmask, VecT<T, V>& ya, VecT<T, V>& yb, int& oa, int& ob) {
  using VT = VecT<T, V>;
  using bits = typename Elem<T>::bits;
  const bool has = xr && k < p.U;
  const bool tail = k >= p.nP;
  oa = ob = 0;
  if (tail)
    oa = p.rd + (k - p.nP) * V;
  else
    unit_offsets<V, INTER>(k, p.h, oa, ob);
  VT xa{}, xb{}, c{}, sn{};
  if (has) {
    xa = ld_stream(reinterpret_cast<const VT*>(xr + oa));
    if (!tail) {
      xb = ld_stream(reinterpret_cast<const VT*>(xr + ob));
      if (rotates && valid) {
        c = ld_shared_ro(reinterpret_cast<const VT*>(static_cast<const bits*>(p.cos) + crow + k * V));
        sn = ld_shared_ro(reinterpret_cast<const VT*>(static_cast<const bits*>(p.sin) + crow + k * V));
      }
    }
  }
  if (NORM && rotates) {
    float ss = sum_squares<T, V>(xa) + sum_squares<T, V>(xb);
    for (int o = p.lanes >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(gmask, ss, o);
    if (has) {
      const float r = 1.0f / sqrtf(ss / (float)p.H + p.eps);
      const bits* w = static_cast<const bits*>(weight);
      xa = norm_weight<T, V>(xa, r, ld_shared_ro(reinterpret_cast<const VT*>(w + oa)));
      if (!tail) xb = norm_weight<T, V>(xb, r, ld_shared_ro(reinterpret_cast<const VT*>(w + ob)));
    }
  }
  ya = xa;
  yb = xb;
  if (has && !tail && rotates && valid) rotate_unit<T, V, INTER>(xa, xb, c, sn, ya, yb);
}

// A group of lanes * rows threads (a power of two) takes one task at a time:
// `rows` consecutive Q rows, or one block of 16 rows of a K or V cache, `rows`
// new rows at a time. Task order: K and V blocks first (they do more), then Q.
template <class T, int V, bool INTER, bool NORM>
__global__ void __launch_bounds__(kKvAppendThreads) kv_append_kernel_t(const KvAppendParams p) {
  using VT = VecT<T, V>;
  using bits = typename Elem<T>::bits;
  __shared__ float s_max[kKvAppendThreads / 32];
  pdl_launch_dependents();
  pdl_wait();
  const int group = p.lanes * p.rows;
  const int per_cta = kKvAppendThreads / group;
  const int tid = threadIdx.x;
  const int gi = tid / group, t = tid - gi * group;
  const int slot = t / p.lanes, k0 = t - slot * p.lanes;
  const unsigned lane = tid & 31u;
  const unsigned gmask =
      p.lanes >= 32 ? 0xffffffffu : (((1u << p.lanes) - 1u) << (lane & ~(unsigned)(p.lanes - 1)));
  const int64_t tasks = p.kv_tasks + p.q_tasks;
  const int64_t nall = (int64_t)p.Nq + 2 * p.Nkv;
  // every thread of a CTA makes the same number of rounds (barriers below)
  for (int64_t base = (int64_t)blockIdx.x * per_cta; base < tasks; base += (int64_t)gridDim.x * per_cta) {
    const int64_t task = base + gi;
    const bool is_kv = task < p.kv_tasks;
    const bool is_q = !is_kv && task < tasks;
    if (is_q) {
      const int64_t r = (task - p.kv_tasks) * p.rows + slot;
      const bool live = r < p.B * p.S * p.Nq;
      const int64_t tok = live ? r / p.Nq : 0, hd = live ? r - tok * p.Nq : 0;
      const int64_t b = tok / p.S, s = tok - b * p.S;
      const int64_t row = (int64_t)__ldg(p.past + b) + s;
      const int64_t pp = p.pos ? __ldg(p.pos + tok) : row;
      const bool valid = (uint64_t)pp < (uint64_t)p.cache_rows;
      if (live && hd == 0 && k0 == 0 && p.status) {
        const int f = (valid ? 0 : 1) | (row >= 0 && row < p.max_len ? 0 : 4);
        if (f) atomicOr(p.status, f);
      }
      const bits* xr = nullptr;
      if (live) xr = static_cast<const bits*>(p.q) + (p.packed ? (tok * nall + hd) : r) * p.H;
      bits* yr = static_cast<bits*>(p.q_out) + r * p.H;
      for (int k = k0; k < p.U || (NORM && k == k0); k += p.lanes) {
        VT ya, yb;
        int oa, ob;
        kv_row_unit<T, V, INTER, NORM>(p, xr, k, true, p.qw, valid, pp * p.h, gmask, ya, yb, oa, ob);
        if (live && k < p.U) {
          st_stream(reinterpret_cast<VT*>(yr + oa), ya);
          if (k < p.nP) st_stream(reinterpret_cast<VT*>(yr + ob), yb);
        }
      }
    }
    // K and V blocks. `work` is uniform over a group.
    bool work = false, is_k = false;
    int64_t b = 0, hd = 0, blk = 0, past = 0, r0 = 0, r1 = 0;
    if (is_kv) {
      int64_t i = task;
      is_k = (i & 1) == 0;
      i >>= 1;
      const int64_t nb = i % p.blocks;
      i /= p.blocks;
      hd = i % p.Nkv;
      b = i / p.Nkv;
      past = __ldg(p.past + b);
      blk = (past > 0 ? past : 0) / kKvBlock + nb;
      r0 = blk * kKvBlock > past ? blk * kKvBlock : past;
      r1 = (blk + 1) * kKvBlock;
      if (past + p.S < r1) r1 = past + p.S;
      if (p.max_len < r1) r1 = p.max_len;
      if (r0 < 0) r0 = 0;
      work = r0 < r1;
    }
    const int64_t plane = b * p.Nkv + hd;
    const bits* src = nullptr;
    int64_t sstride = 0;
    if (work) {
      if (p.packed) {
        src = static_cast<const bits*>(p.q) + (p.Nq + (is_k ? 0 : p.Nkv) + hd) * p.H;
        sstride = nall * p.H;
      } else {
        src = static_cast<const bits*>(is_k ? p.k : p.v) + hd * p.H;
        sstride = (int64_t)p.Nkv * p.H;
      }
    }
    float* scales = (is_k ? p.k_scale : p.v_scale) + plane * p.nblk + blk;
    uint8_t* cache = (is_k ? p.k_cache : p.v_cache) + plane * p.max_len * p.H;
    const bool older = work && blk * kKvBlock < past;
    const float was = older ? *scales : 0.0f;
    // The first unit of a thread stays in its registers between the maximum and
    // the store; what follows it (more rows or units than threads) is formed twice.
    VT ya0{}, yb0{};
    int oa0 = 0, ob0 = 0;
    float amax = 0.0f;
    auto form = [&](int64_t row, int k, VT& ya, VT& yb, int& oa, int& ob) {
      const int64_t tok = b * p.S + (row - past);
      bool valid = false;
      int64_t pp = 0;
      if (is_k) {
        pp = p.pos ? __ldg(p.pos + tok) : row;
        valid = (uint64_t)pp < (uint64_t)p.cache_rows;
      }
      kv_row_unit<T, V, INTER, NORM>(p, src + tok * sstride, k, is_k, p.kw, valid, pp * p.h, gmask, ya, yb, oa, ob);
    };
    auto norm_lane = [&](int k) { return NORM && k == k0; };  // every lane of a row joins its sum
    if (work) {
      for (int64_t row = r0 + slot; row < r1; row += p.rows)
        for (int k = k0; k < p.U || norm_lane(k); k += p.lanes) {
          VT ya{}, yb{};
          int oa, ob;
          form(row, k, ya, yb, oa, ob);
          amax = fmaxf(amax, fmaxf(kv_amax<T, V>(ya), kv_amax<T, V>(yb)));
          if (row == r0 + slot && k == k0) ya0 = ya, yb0 = yb, oa0 = oa, ob0 = ob;
        }
    }
    for (int o = (group < 32 ? group : 32) >> 1; o > 0; o >>= 1)
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if (group > 32) {
      __syncthreads();  // the previous round's values have been read
      if (lane == 0) s_max[tid >> 5] = amax;
      __syncthreads();
      const int w0 = gi * (group >> 5);
      for (int w = 0; w < (group >> 5); ++w) amax = fmaxf(amax, s_max[w0 + w]);
    }
    if (!work) continue;  // uniform over the group; no barrier below
    float scale = kv_scale_of(amax);
    if (older && was > scale) scale = was;
    const float inv = kv_pow2_inverse(scale);
    for (int64_t row = r0 + slot; row < r1; row += p.rows)
      for (int k = k0; k < p.U || norm_lane(k); k += p.lanes) {
        VT ya = ya0, yb = yb0;
        int oa = oa0, ob = ob0;
        if (!(row == r0 + slot && k == k0)) form(row, k, ya, yb, oa, ob);
        if (k >= p.U) continue;
        uint8_t* dst = cache + row * p.H;
        kv_store_codes<T, V>(dst + oa, ya, inv);
        if (k < p.nP) kv_store_codes<T, V>(dst + ob, yb, inv);
      }
    if (older && was < scale) {
      const float ratio = was * inv;
      uint8_t* held = cache + blk * kKvBlock * p.H;
      const int64_t n = (past - blk * kKvBlock) * p.H;
      if (p.wide) {
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
    if (t == 0) *scales = scale;  // `was` was read by every thread before the maximum's exchange
  }
}

}  // namespace rope_gb300
