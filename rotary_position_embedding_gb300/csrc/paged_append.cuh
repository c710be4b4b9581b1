// Q and K rotation (and the optional QK-RMSNorm) with the append of K and V to
// caches held in pages.
//
// Every head is computed as rope_qkv_kernel (rope_qkv.cuh) computes it, with its
// bits; the row that a token's K and V go to is looked up in the page table.
#pragma once

#include "paged_common.cuh"
#include "rope_qkv.cuh"

namespace rope_gb300 {

// A group of p.lanes threads takes one head row of a token: every storage type,
// head size and alignment.
template <class T, int V, bool INTER, bool NORM>
__global__ void __launch_bounds__(kPagedAppendThreads) paged_append_kernel_t(const PagedAppendParams p) {
  using VT = VecT<T, V>;
  using bits = typename Elem<T>::bits;
  pdl_launch_dependents();
  pdl_wait();
  const int lanes = p.lanes, k0 = threadIdx.x & (lanes - 1);
  const int per = kPagedAppendThreads / lanes;
  const unsigned lane = threadIdx.x & 31u;
  const unsigned mask = lanes == 32 ? 0xffffffffu : ((1u << lanes) - 1u) << (lane & ~(unsigned)(lanes - 1));
  const int N = p.Nq + 2 * p.Nkv;
  const int64_t H = p.H, all = p.s.T * N;
  for (int64_t w = (int64_t)blockIdx.x * per + threadIdx.x / lanes; w < all; w += (int64_t)gridDim.x * per) {
    const int64_t tok = w / N;
    const int n = (int)(w - tok * N);
    const int role = n < p.Nq ? 0 : n < p.Nq + p.Nkv ? 1 : 2;  // Q, K, V
    const int hd = role == 0 ? n : role == 1 ? n - p.Nq : n - p.Nq - p.Nkv;
    int b;
    if (!paged_find(p.s, tok, &b)) continue;  // the same for the group
    const int64_t row = (int64_t)__ldg(p.s.past + b) + paged_nth(p.s, b, tok);
    const bits* x = p.packed ? static_cast<const bits*>(p.q) + (tok * N + n) * H
                             : static_cast<const bits*>(role == 0 ? p.q : role == 1 ? p.k : p.v) +
                                   (tok * (role == 0 ? p.Nq : p.Nkv) + hd) * H;
    bits* y = nullptr;
    if (role == 0) {
      y = static_cast<bits*>(p.q_out) + (tok * p.Nq + hd) * H;
    } else {
      const int64_t at = row >= 0 && row < p.s.rows ? paged_row(p.s, b, hd, (int)row, (int)H) : -1;
      if (at >= 0) y = static_cast<bits*>(role == 1 ? p.k_pages : p.v_pages) + at;
      if (!y && role == 1 && hd == 0 && k0 == 0) flag_cache_row(p.s.status);
    }
    if (!y) continue;
    const int64_t pp = role == 2 ? -1 : p.pos ? __ldg(p.pos + tok) : row;
    const bool valid = (uint64_t)pp < (uint64_t)p.cache_rows;
    if (!valid && n == 0 && k0 == 0) flag_oor(p.s.status);
    const bits* cosr = static_cast<const bits*>(p.cos) + pp * p.h;
    const bits* sinr = static_cast<const bits*>(p.sin) + pp * p.h;
    const bits* wt = static_cast<const bits*>(role == 0 ? p.qw : p.kw);
    auto place = [&](int k, int& oa, int& ob) {
      if (k < p.nP)
        unit_offsets<V, INTER>(k, p.h, oa, ob);
      else
        oa = p.rd + (k - p.nP) * V;
    };
    float r = 1.0f;
    if (NORM && role != 2) {
      float ss = 0.0f;
      for (int k = k0; k < p.U; k += lanes) {
        int oa, ob;
        place(k, oa, ob);
        float u = sum_squares<T, V>(ld_shared_ro(reinterpret_cast<const VT*>(x + oa)));
        if (k < p.nP) u += sum_squares<T, V>(ld_shared_ro(reinterpret_cast<const VT*>(x + ob)));
        ss += u;
      }
      for (int o = lanes >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(mask, ss, o);
      r = 1.0f / sqrtf(ss / (float)H + p.eps);
    }
    for (int k = k0; k < p.U; k += lanes) {
      int oa, ob;
      place(k, oa, ob);
      const bool pair = k < p.nP;
      VT a = ld_shared_ro(reinterpret_cast<const VT*>(x + oa)), c{};
      if (pair) c = ld_shared_ro(reinterpret_cast<const VT*>(x + ob));
      if (NORM && role != 2) {
        a = norm_weight<T, V>(a, r, ld_shared_ro(reinterpret_cast<const VT*>(wt + oa)));
        if (pair) c = norm_weight<T, V>(c, r, ld_shared_ro(reinterpret_cast<const VT*>(wt + ob)));
      }
      if (pair && valid) {
        VT ya, yb;
        rotate_unit<T, V, INTER>(a, c, ld_shared_ro(reinterpret_cast<const VT*>(cosr + k * V)),
                                 ld_shared_ro(reinterpret_cast<const VT*>(sinr + k * V)), ya, yb);
        a = ya, c = yb;
      }
      st_stream(reinterpret_cast<VT*>(y + oa), a);
      if (pair) st_stream(reinterpret_cast<VT*>(y + ob), c);
    }
  }
}

}  // namespace rope_gb300
