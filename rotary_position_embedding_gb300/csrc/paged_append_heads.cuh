// Q and K rotation (and the optional QK-RMSNorm) with the append of K and V to caches
// held in pages, several heads a thread, on the 128-bit path.
//
// As rope_qkv_heads_kernel (rope_qkv_heads.cuh), whose arithmetic and bits these are: a
// thread owns unit k of HPT heads of one role (Q, K or V) and goes from token to token;
// it issues the loads of all its heads first (2 * HPT of 16 bytes), and what depends on
// the token (its sequence, row, page, position, coefficients) is looked up meanwhile.
// Bound by the memory: 8222 bfloat16 tokens of 32/8 heads of 128 in 7 ragged sequences
// 34.8 us, 5.8 TB/s; with the norm 41.7 us (float32 69 us, 5.8 TB/s), where 190
// instructions a unit of 16 values stand beside the loads.
#pragma once

#include "paged_append.cuh"

namespace rope_gb300 {

// Two 16-bit values in a word.
template <class T>
struct Words;
template <>
struct Words<__half> {
  static __device__ __forceinline__ float2 tof(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }
  static __device__ __forceinline__ uint32_t fromf(float2 f) {
    const __half2 h = __float22half2_rn(f);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  static __device__ __forceinline__ uint32_t mul(uint32_t a, uint32_t b) {
    const __half2 h = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  static __device__ __forceinline__ uint32_t of(const uint4& x, int q) { return q == 0 ? x.x : q == 1 ? x.y : q == 2 ? x.z : x.w; }
};
template <>
struct Words<__nv_bfloat16> {
  static __device__ __forceinline__ float2 tof(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
  static __device__ __forceinline__ uint32_t fromf(float2 f) {
    const __nv_bfloat162 h = __float22bfloat162_rn(f);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  static __device__ __forceinline__ uint32_t mul(uint32_t a, uint32_t b) {
    const __nv_bfloat162 h =
        __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  static __device__ __forceinline__ uint32_t of(const uint4& x, int q) { return q == 0 ? x.x : q == 1 ? x.y : q == 2 ? x.z : x.w; }
};

// 1 / sqrt(mean + eps) of head j. The lanes of a head hold the same sums: each works out
// one head's and they exchange them (a root and two quotients are 60 instructions).
template <int HPT>
__device__ __forceinline__ float paged_head_r(const PagedAppendParams& p, const float (&ss)[HPT], int j, int k, unsigned gmask) {
  auto r = [&](float s) { return __frcp_rn(sqrtf(__fdiv_rn(s, p.width) + p.eps)); };
  if (p.U < HPT) return r(ss[j]);
  float mine = ss[0];
#pragma unroll
  for (int i = 1; i < HPT; ++i) mine = (k & (HPT - 1)) == i ? ss[i] : mine;
  return __shfl_sync(gmask, r(mine), (threadIdx.x & 31 & ~(unsigned)(p.U - 1)) | j);
}

template <class T, bool INTER, bool NORM, int HPT>
__global__ void __maxnreg__(NORM ? 80 : 64) paged_append_heads_kernel_t(const PagedAppendParams p) {
  constexpr int V = 16 / (int)sizeof(typename Elem<T>::bits);
  using VT = VecT<T, V>;
  using bits = typename Elem<T>::bits;
  // a unit in registers: 4 words (as 8 values of 16 bits the compiler gave each its own
  // register: 103 of them, and the norm took 76 us)
  using RT = uint4;
  const int U = p.U, per_tok = p.groups * U;
  const int slot = threadIdx.x / per_tok, in = threadIdx.x - slot * per_tok;
  const int grp = in / U, k = in - grp * U;
  pdl_launch_dependents();
  pdl_wait();
  if (slot >= p.tokens) return;  // a whole token: no group of heads is split
  const int gq = (p.Nq + HPT - 1) / HPT, gk = (p.Nkv + HPT - 1) / HPT;
  const int role = grp < gq ? 0 : grp < gq + gk ? 1 : 2;
  const int hd0 = (role == 0 ? grp : role == 1 ? grp - gq : grp - gq - gk) * HPT;
  const int of_role = role == 0 ? p.Nq : p.Nkv;
  const int nh = of_role - hd0 < HPT ? of_role - hd0 : HPT;  // a role's last group may be short
  const int64_t H = p.H;
  const bits* src;
  int64_t sstride;
  if (p.packed) {
    src = static_cast<const bits*>(p.q) + (int64_t)(role == 0 ? hd0 : role == 1 ? p.Nq + hd0 : p.Nq + p.Nkv + hd0) * H;
    sstride = (int64_t)(p.Nq + 2 * p.Nkv) * H;
  } else {
    src = static_cast<const bits*>(role == 0 ? p.q : role == 1 ? p.k : p.v) + hd0 * H;
    sstride = of_role * H;
  }
  const int64_t dhead = role == 0 ? H : (int64_t)p.s.ps * H;  // between heads where they go
  const bool pair = k < p.nP, rotates = role != 2, first = role == 0 && hd0 == 0 && k == 0;
  int oa = 0, ob = 0;
  if (pair)
    unit_offsets<V, INTER>(k, p.h, oa, ob);
  else
    oa = p.rd + (k - p.nP) * V;
  const RT zero = make_uint4(0, 0, 0, 0);
  auto load = [](const bits* at) { return __ldcs(reinterpret_cast<const RT*>(at)); };
  auto load_ro = [](const bits* at) { return __ldg(reinterpret_cast<const RT*>(at)); };
  auto as_unit = [](const RT& x) {
    VT v;
    __builtin_memcpy(&v, &x, 16);
    return v;
  };
  RT wa = zero, wb = zero;
  unsigned gmask = 0u;
  if (NORM) {
    const unsigned lane = threadIdx.x & 31u;
    gmask = U >= 32 ? 0xffffffffu : ((1u << U) - 1u) << (lane & ~(unsigned)(U - 1));
    if (rotates) {
      const bits* w = static_cast<const bits*>(role == 0 ? p.qw : p.kw);
      wa = load_ro(w + oa);
      if (pair) wb = load_ro(w + ob);
    }
  }
  for (int64_t tok = (int64_t)blockIdx.x * p.tokens + slot; tok < p.s.T; tok += (int64_t)gridDim.x * p.tokens) {
    const bits* xr = src + tok * sstride;
    RT xa[HPT], xb[HPT];
#pragma unroll
    for (int j = 0; j < HPT; ++j) {  // a short group reads its last head again
      const bits* xj = xr + (j < nh ? j : nh - 1) * H;
      xa[j] = load(xj + oa);
      xb[j] = zero;
      if (pair) xb[j] = load(xj + ob);
    }
    int b;
    if (!paged_find(p.s, tok, &b)) continue;  // the same for a token's threads
    const int64_t row = (int64_t)__ldg(p.s.past + b) + paged_nth(p.s, b, tok);
    bool valid = false;
    RT c = zero, sn = zero;
    if (rotates) {
      const int64_t pp = p.pos ? __ldg(p.pos + tok) : row;
      valid = (uint64_t)pp < (uint64_t)p.cache_rows;
      if (!valid && first) flag_oor(p.s.status);
      if (valid && pair) {
        c = load_ro(static_cast<const bits*>(p.cos) + pp * p.h + k * V);
        sn = load_ro(static_cast<const bits*>(p.sin) + pp * p.h + k * V);
      }
    }
    bits* yr;
    if (role == 0) {
      yr = static_cast<bits*>(p.q_out) + (tok * p.Nq + hd0) * H;
    } else {
      const int64_t at = row >= 0 && row < p.s.rows ? paged_row(p.s, b, hd0, (int)row, (int)H) : -1;
      if (at < 0) {  // the same for a group's threads
        if (role == 1 && hd0 == 0 && k == 0) flag_cache_row(p.s.status);
        continue;
      }
      yr = static_cast<bits*>(role == 1 ? p.k_pages : p.v_pages) + at;
    }
    if constexpr (NORM && sizeof(bits) == 2) {
      // 16-bit data in 32-bit words, two values at a time, which rounds as the scalar form
      if (rotates) {
        using W = Words<T>;
        float ss[HPT];
#pragma unroll
        for (int j = 0; j < HPT; ++j) {
          float sa = 0.f, sb = 0.f;  // sum_squares' order
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float2 fa = W::tof(W::of(xa[j], q)), fb = W::tof(W::of(xb[j], q));
            sa = __fmaf_rn(fa.x, fa.x, sa);
            sa = __fmaf_rn(fa.y, fa.y, sa);
            sb = __fmaf_rn(fb.x, fb.x, sb);
            sb = __fmaf_rn(fb.y, fb.y, sb);
          }
          ss[j] = sa + sb;
        }
        // (the words, not their 32 values, are what is kept meanwhile)
#pragma unroll
        for (int j = 0; j < HPT; ++j)
          asm volatile("" : "+r"(xa[j].x), "+r"(xa[j].y), "+r"(xa[j].z), "+r"(xa[j].w), "+r"(xb[j].x), "+r"(xb[j].y),
                       "+r"(xb[j].z), "+r"(xb[j].w));
        for (int o = U >> 1; o > 0; o >>= 1) {
#pragma unroll
          for (int j = 0; j < HPT; ++j) ss[j] += __shfl_xor_sync(gmask, ss[j], o);
        }
#pragma unroll
        for (int j = 0; j < HPT; ++j) {
          const float r = paged_head_r<HPT>(p, ss, j, k, gmask);  // (every lane: it takes a shuffle)
          if (j >= nh) continue;
          const float2 r2 = make_float2(r, r);
          uint32_t za[4], zb[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            za[q] = W::mul(W::fromf(__fmul2_rn(W::tof(W::of(xa[j], q)), r2)), W::of(wa, q));
            zb[q] = W::mul(W::fromf(__fmul2_rn(W::tof(W::of(xb[j], q)), r2)), W::of(wb, q));
          }
          if (pair && valid) {
            uint32_t ya[4], yb[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const float2 cf = W::tof(W::of(c, q)), sf = W::tof(W::of(sn, q)), ns = make_float2(-sf.x, -sf.y);
              if (!INTER) {
                const float2 x0 = W::tof(za[q]), x1 = W::tof(zb[q]);
                ya[q] = W::fromf(__ffma2_rn(x0, cf, __fmul2_rn(x1, ns)));
                yb[q] = W::fromf(__ffma2_rn(x1, cf, __fmul2_rn(x0, sf)));
              } else {  // words 2q and 2q + 1 of a||b hold pairs 2q and 2q + 1
                const float2 f0 = W::tof(q < 2 ? za[2 * q] : zb[2 * q - 4]), f1 = W::tof(q < 2 ? za[2 * q + 1] : zb[2 * q - 3]);
                const float2 x0 = make_float2(f0.x, f1.x), x1 = make_float2(f0.y, f1.y);
                const float2 y0 = __ffma2_rn(x0, cf, __fmul2_rn(x1, ns)), y1 = __ffma2_rn(x1, cf, __fmul2_rn(x0, sf));
                (q < 2 ? ya[2 * q] : yb[2 * q - 4]) = W::fromf(make_float2(y0.x, y1.x));
                (q < 2 ? ya[2 * q + 1] : yb[2 * q - 3]) = W::fromf(make_float2(y0.y, y1.y));
              }
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) za[q] = ya[q], zb[q] = yb[q];
          }
          bits* yj = yr + j * dhead;
          __stcs(reinterpret_cast<uint4*>(yj + oa), make_uint4(za[0], za[1], za[2], za[3]));
          if (pair) __stcs(reinterpret_cast<uint4*>(yj + ob), make_uint4(zb[0], zb[1], zb[2], zb[3]));
        }
        continue;
      }
    }
    if constexpr (NORM && sizeof(bits) != 2) {
      if (rotates) {
        float ss[HPT];
#pragma unroll
        for (int j = 0; j < HPT; ++j) ss[j] = sum_squares<T, V>(as_unit(xa[j])) + sum_squares<T, V>(as_unit(xb[j]));
        for (int o = U >> 1; o > 0; o >>= 1) {
#pragma unroll
          for (int j = 0; j < HPT; ++j) ss[j] += __shfl_xor_sync(gmask, ss[j], o);
        }
        auto r_of = [&](int j) { return paged_head_r<HPT>(p, ss, j, k, gmask); };
#pragma unroll
        for (int j = 0; j < HPT; ++j) {
          const float r = r_of(j);
          const VT za = norm_weight<T, V>(as_unit(xa[j]), r, as_unit(wa)), zb = norm_weight<T, V>(as_unit(xb[j]), r, as_unit(wb));
          __builtin_memcpy(&xa[j], &za, 16);
          if (pair) __builtin_memcpy(&xb[j], &zb, 16);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < HPT; ++j) {
      if (j >= nh) break;
      bits* yj = yr + j * dhead;
      if (pair && valid) {
        VT ya, yb;
        rotate_unit<T, V, INTER>(as_unit(xa[j]), as_unit(xb[j]), as_unit(c), as_unit(sn), ya, yb);
        st_stream(reinterpret_cast<VT*>(yj + oa), ya);
        st_stream(reinterpret_cast<VT*>(yj + ob), yb);
      } else {  // V, a tail unit or an out-of-range position: copied through
        __stcs(reinterpret_cast<RT*>(yj + oa), xa[j]);
        if (pair) __stcs(reinterpret_cast<RT*>(yj + ob), xb[j]);
      }
    }
  }
}

}  // namespace rope_gb300
