// Attention over a key/value cache on CUDA cores: every storage type, head
// size, alignment and mask; float32 keeps 32-bit products throughout.
//
// A CTA takes 64 rows of one (b, kvh), or 16 where there are no more, and walks
// its keys 64 at a time: scores (4 x 4 or 1 x 4 a thread), the running maximum
// and sum of each row (held by the 16 threads that share the row), then
// O = O * alpha + P V with 4 or 1 rows x 4 * NJ columns of O in each thread's
// registers. The tiles are float32 in shared memory, so every product is a
// 32-bit FMA, and a row's weights stay within the warp that formed them. Bound
// by the FMA pipes: 4 x 4 products for 12 shared-memory wavefronts (2 x 2 on
// tiles of 32 x 32, each loaded when it was needed, took 60 us for 2 x 301 tokens
// of 8 heads, where these take 33).
// K of the next tile is on its way during the softmax and P V, V during Q K^T
// (cp.async where nothing has to be converted).
#pragma once

#include <type_traits>

#include "kv_common.cuh"

namespace rope_gb300 {

constexpr int kSimpleCols = 64, kSimpleP = kSimpleCols + 4;

// 4 consecutive values of T, or of codes, as float32.
template <class T, bool FP8>
__device__ __forceinline__ float4 simple_load4(const void* src, int64_t at, float scale) {
  if constexpr (FP8) {
    const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(src) + at));
    const float2 a = kv_fp8x2((uint16_t)w), b = kv_fp8x2((uint16_t)(w >> 16));
    return make_float4(a.x * scale, a.y * scale, b.x * scale, b.y * scale);
  } else {
    using VT = VecT<T, 4>;
    const VT v = ld_shared_ro(reinterpret_cast<const VT*>(static_cast<const typename Elem<T>::bits*>(src) + at));
    return make_float4(Elem<T>::tof(v.v[0]), Elem<T>::tof(v.v[1]), Elem<T>::tof(v.v[2]), Elem<T>::tof(v.v[3]));
  }
}
template <class T, bool FP8>
__device__ __forceinline__ float simple_load1(const void* src, int64_t at, float scale) {
  if constexpr (FP8)
    return kv_fp8x2(static_cast<const uint8_t*>(src)[at]).x * scale;
  else
    return Elem<T>::tof(static_cast<const typename Elem<T>::bits*>(src)[at]);
}

// NJ: 4 * NJ columns of O a thread, 16 threads a row: H <= 64 * NJ. RA: 16 * RA rows a CTA.
template <class T, bool FP8, int NJ, int RA>
__global__ void __launch_bounds__(kKvSimpleThreads, NJ < 4 ? 2 : 1) kv_simple_kernel_t(const KvParams p) {
  using bits = typename Elem<T>::bits;
  constexpr int ROWS = 16 * RA, WARPS = kKvSimpleThreads / 32;
  constexpr bool kCopied = !FP8 && sizeof(T) == 4;  // nothing to convert
  extern __shared__ float smem[];
  const int H = p.H, HP = (H + 3) / 4 * 4 + 4;
  float* sq = smem;                    // [ROWS][HP]
  float* sk = sq + ROWS * HP;          // [64][HP]
  float* sv = sk + kSimpleCols * HP;   // [64][HP]
  float* sp = sv + kSimpleCols * HP;   // [ROWS][kSimpleP]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int tx = tid & 15, ty = tid >> 4;
  // where a thread's pieces of a tile lie: LPR lanes a row
  constexpr int LPR = NJ == 1 ? 16 : 32, RPW = 32 / LPR;
  const int piece_row = warp * RPW + lane / LPR, piece_dim = lane % LPR * 4;
  // what(row, dim): 4 values at a time
  auto each_piece = [&](int rows, auto&& what) {
#pragma unroll 4
    for (int c = piece_row; c < rows; c += WARPS * RPW)
      for (int d = piece_dim; d < H; d += LPR * 4) what(c, d);
  };
  // rows j0 .. j0 + 63 of a cache; zeros from row n on
  auto bring = [&](float* dst, const void* src, const float* scales, int64_t plane, int64_t j0, int n) {
    const int64_t at = (plane * p.max_len + j0) * H;
    auto scale = [&](int c) { return FP8 && c < n ? __ldg(scales + plane * p.nblk + (j0 + c) / kKvBlock) : 1.0f; };
    if (p.vec) {
      each_piece(kSimpleCols, [&](int c, int d) {
        if constexpr (kCopied) {
          const float* from = static_cast<const float*>(src);
          kv_cp<16>(kv_smem(dst + c * HP + d), c < n ? from + at + (int64_t)c * H + d : from, c < n);
        } else {
          *reinterpret_cast<float4*>(dst + c * HP + d) =
              c < n ? simple_load4<T, FP8>(src, at + (int64_t)c * H + d, scale(c)) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        }
      });
    } else {
      for (int c = warp; c < kSimpleCols; c += WARPS) {
        const float f = scale(c);
        for (int d = lane; d < H; d += 32) dst[c * HP + d] = c < n ? simple_load1<T, FP8>(src, at + (int64_t)c * H + d, f) : 0.0f;
      }
    }
    kv_cp_commit();
  };
  // whether what this thread brought is finite
  auto finite = [&](const float* dst) {
    bool fin = true;
    if (p.vec) {
      each_piece(kSimpleCols, [&](int c, int d) {
        const float4 f = *reinterpret_cast<const float4*>(dst + c * HP + d);
        fin &= isfinite(f.x) && isfinite(f.y) && isfinite(f.z) && isfinite(f.w);
      });
    } else {
      for (int c = warp; c < kSimpleCols; c += WARPS)
        for (int d = lane; d < H; d += 32) fin &= isfinite(dst[c * HP + d]);
    }
    return fin;
  };
  pdl_launch_dependents();
  pdl_wait();
  const int64_t tile = blockIdx.x / p.splits;
  const int split = blockIdx.x % p.splits;
  const int kvh = blockIdx.y;
  const int64_t r0 = tile * ROWS;
  // token and head of row r0 + r, for r < 64: one 64-bit division
  const int64_t tok0 = r0 / p.G;
  const uint32_t G = (uint32_t)p.G, rem0 = (uint32_t)(r0 - tok0 * p.G);
  const int nrows = p.R - r0 < ROWS ? (int)(p.R - r0) : ROWS;
  auto tok_of = [&](int r) { return tok0 + (rem0 + (uint32_t)r) / G; };
  auto row_at = [&](int b, int r) {
    const uint32_t t = (rem0 + (uint32_t)r) / G, h = rem0 + (uint32_t)r - t * G;
    return (((int64_t)b * p.S + tok0 + t) * p.Nq + (int64_t)kvh * p.G + h) * H;
  };
  for (int b = blockIdx.z; b < p.B; b += gridDim.z) {
    const KvSeq seq = kv_seq(p, b);
    if (blockIdx.x == 0 && kvh == 0 && tid == 0) kv_flag_rows(p, seq);
    int64_t end = kv_limit(seq, seq.past + tok_of(nrows - 1));  // no row of the tile sees more
    if (end < 0) end = 0;
    int64_t lo, hi;
    kv_split(end, p.splits, split, kSimpleCols, &lo, &hi);
    const int64_t plane = (int64_t)b * p.Nkv + kvh;
    auto width = [&](int64_t j0) { return hi - j0 < kSimpleCols ? (int)(hi - j0) : kSimpleCols; };
    __syncthreads();  // the sequence before has been read
    if (p.vec) {
      const float4 zero = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      each_piece(ROWS, [&](int r, int d) {
        const int64_t at = row_at(b, r) + d;
        if constexpr (sizeof(T) == 4)
          kv_cp<16>(kv_smem(sq + r * HP + d), static_cast<const float*>(p.q) + (r < nrows ? at : 0), r < nrows);
        else
          *reinterpret_cast<float4*>(sq + r * HP + d) = r < nrows ? simple_load4<T, false>(p.q, at, 1.0f) : zero;
      });
    } else {
      for (int r = warp; r < ROWS; r += WARPS) {
        const int64_t at = row_at(b, r);
        for (int d = lane; d < H; d += 32) sq[r * HP + d] = r < nrows ? simple_load1<T, false>(p.q, at + d, 1.0f) : 0.0f;
      }
    }
    if (lo < hi) {  // Q and K are waited for together
      bring(sk, p.k, p.ks, plane, lo, width(lo));
      bring(sv, p.v, p.vs, plane, lo, width(lo));
    } else {
      kv_cp_commit();
      kv_cp_wait<0>();
    }
    // the rows of this thread: ty + 16 a
    int64_t pos[RA], lim[RA];
    float slope[RA], m[RA], l[RA];
    int32_t doc[RA];
    float4 acc[RA][NJ];
#pragma unroll
    for (int a = 0; a < RA; ++a) {
      const int r = ty + 16 * a;
      const bool live = r < nrows;
      pos[a] = seq.past + tok_of(live ? r : nrows - 1);
      lim[a] = live ? kv_limit(seq, pos[a]) : 0;
      slope[a] = p.slopes ? __ldg(p.slopes + kvh * p.G + (rem0 + (uint32_t)(live ? r : 0)) % G) * kLog2e : 0.0f;
      doc[a] = 0;
      if (p.docs && live && !kv_document(p, b, pos[a], &doc[a])) lim[a] = 0;
      m[a] = -CUDART_INF_F;
      l[a] = 0.0f;
#pragma unroll
      for (int j = 0; j < NJ; ++j) acc[a][j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
    const float c1 = p.cap > 0.0f ? p.over : p.scale * kLog2e;
    const float c2 = p.cap * kLog2e;
    const int32_t* docs = p.docs ? p.docs + (int64_t)b * p.max_len : nullptr;
    for (int64_t j0 = lo; j0 < hi; j0 += kSimpleCols) {
      const int n = width(j0);
      const bool more = j0 + kSimpleCols < hi;
      kv_cp_wait<1>();  // K; V may still be on its way
      __syncthreads();
      float s[RA][4];
#pragma unroll
      for (int a = 0; a < RA; ++a)
#pragma unroll
        for (int c = 0; c < 4; ++c) s[a][c] = 0.0f;
      const float* qr = sq + ty * HP;
      const float* kr = sk + tx * HP;
      int d = 0;
#pragma unroll 2
      for (; d + 4 <= H; d += 4) {
        float4 k4[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) k4[c] = *reinterpret_cast<const float4*>(kr + 16 * c * HP + d);
#pragma unroll
        for (int a = 0; a < RA; ++a) {
          const float4 q = *reinterpret_cast<const float4*>(qr + 16 * a * HP + d);
#pragma unroll
          for (int c = 0; c < 4; ++c)
            s[a][c] = fmaf(q.x, k4[c].x, fmaf(q.y, k4[c].y, fmaf(q.z, k4[c].z, fmaf(q.w, k4[c].w, s[a][c]))));
        }
      }
      for (; d < H; ++d)
#pragma unroll
        for (int a = 0; a < RA; ++a)
#pragma unroll
          for (int c = 0; c < 4; ++c) s[a][c] = fmaf(qr[16 * a * HP + d], kr[16 * c * HP + d], s[a][c]);
      int32_t kdoc[4] = {0, 0, 0, 0};
      if (docs) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (tx + 16 * c < n) kdoc[c] = __ldg(docs + j0 + tx + 16 * c);
      }
#pragma unroll
      for (int a = 0; a < RA; ++a) {
        const int64_t ahead = lim[a] - j0, far = pos[a] - j0;
        const int seen = ahead < 0 ? 0 : ahead < n ? (int)ahead : n;  // columns below this
        float mx = -CUDART_INF_F;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int col = tx + 16 * c;
          float y = s[a][c] * c1;
          if (p.cap > 0.0f) y = tanhf(y) * c2;
          if (p.slopes) {
            const int64_t dist = far - col;
            y = fmaf(-slope[a], (float)(dist < 0 ? -dist : dist), y);
          }
          s[a][c] = col < seen && kdoc[c] == doc[a] ? y : -CUDART_INF_F;
          mx = fmaxf(mx, s[a][c]);  // drops NaN: a NaN score shows in the sum
        }
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        const float mn = fmaxf(m[a], mx);
        const float base = mn == -CUDART_INF_F ? 0.0f : mn;
        const float alpha = exp2f(m[a] - base);
        float sum = 0.0f;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float w = exp2f(s[a][c] - base);
          sum += w;
          sp[(ty + 16 * a) * kSimpleP + tx + 16 * c] = w;
        }
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        l[a] = l[a] * alpha + sum;
        m[a] = mn;
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          acc[a][j].x *= alpha;
          acc[a][j].y *= alpha;
          acc[a][j].z *= alpha;
          acc[a][j].w *= alpha;
        }
      }
      kv_cp_wait<0>();
      const bool all_finite = __syncthreads_and(finite(sv));  // V is there, K has been read
      if (more) bring(sk, p.k, p.ks, plane, j0 + kSimpleCols, width(j0 + kSimpleCols));
      // rows from n on are zeros with weight zero
      auto add = [&](auto careful) {
        constexpr bool kCareful = decltype(careful)::value;
        auto fma4 = [&](float4& o, float w, const float4& v) {
          if (kCareful && w == 0.0f) return;  // a hidden key's weight is exactly 0, and its value is not touched
          o.x = fmaf(w, v.x, o.x);
          o.y = fmaf(w, v.y, o.y);
          o.z = fmaf(w, v.z, o.z);
          o.w = fmaf(w, v.w, o.w);
        };
        for (int c = 0; c < n; c += 4) {
          float4 w[RA];
#pragma unroll
          for (int a = 0; a < RA; ++a) w[a] = *reinterpret_cast<const float4*>(sp + (ty + 16 * a) * kSimpleP + c);
#pragma unroll
          for (int j = 0; j < NJ; ++j) {
            const int dd = tx * 4 + 64 * j;
            if (dd >= H) continue;
            const float* v = sv + c * HP + dd;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float4 x = *reinterpret_cast<const float4*>(v + k * HP);
#pragma unroll
              for (int a = 0; a < RA; ++a)
                fma4(acc[a][j], k == 0 ? w[a].x : k == 1 ? w[a].y : k == 2 ? w[a].z : w[a].w, x);
            }
          }
        }
      };
      if (all_finite)
        add(std::false_type{});
      else
        add(std::true_type{});
      __syncthreads();
      if (more) bring(sv, p.v, p.vs, plane, j0 + kSimpleCols, width(j0 + kSimpleCols));
    }
#pragma unroll
    for (int a = 0; a < RA; ++a) {
      const int r = ty + 16 * a;
      if (r >= nrows) continue;
      const int64_t at = (plane * p.splits + split) * p.R + r0 + r;
      if (p.splits > 1 && tx == 0) p.ws_ml[at] = make_float2(m[a], l[a]);
      const float inv = l[a] == 0.0f ? 0.0f : 1.0f / l[a];
      bits* o = static_cast<bits*>(p.out) + row_at(b, r);
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const int dd = tx * 4 + 64 * j;
        const float y[4] = {acc[a][j].x, acc[a][j].y, acc[a][j].z, acc[a][j].w};
        if (p.vec && dd < H) {
          if (p.splits > 1) {
            *reinterpret_cast<float4*>(p.ws_o + at * H + dd) = acc[a][j];
          } else {
            VecT<T, 4> v;
#pragma unroll
            for (int i = 0; i < 4; ++i) v.v[i] = Elem<T>::fromf(y[i] * inv);
            *reinterpret_cast<VecT<T, 4>*>(o + dd) = v;
          }
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (dd + i < H) {
              if (p.splits > 1)
                p.ws_o[at * H + dd + i] = y[i];
              else
                o[dd + i] = Elem<T>::fromf(y[i] * inv);
            }
        }
      }
    }
  }
}

// Joins the splits of a row: with M the largest maximum and w_n = 2^(m_n - M),
// o = sum w_n O_n / sum w_n l_n. A split that saw nothing has m = -inf, l = 0 and
// O = 0. Up to 8 splits a warp takes a row; above, the 4 warps of a CTA share
// one and meet in shared memory (76 splits of 32 rows: 74 us by one warp a row,
// whose loads wait for one another).
template <class T>
__global__ void __launch_bounds__(kKvCombineThreads) kv_combine_kernel_t(const KvParams p) {
  using bits = typename Elem<T>::bits;
  constexpr int W = kKvCombineThreads / 32;
  __shared__ float s_o[W][kKvMaxHead], s_l[W];
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool shared_row = p.splits > kKvCombineWarpSplits;
  const int64_t rows = (int64_t)p.B * p.Nkv * p.R;
  const int n0 = shared_row ? warp : 0, dn = shared_row ? W : 1;
  for (int64_t w = shared_row ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * W + warp; w < rows;
       w += (int64_t)gridDim.x * (shared_row ? 1 : W)) {
    const int64_t plane = w / p.R, row = w - plane * p.R;
    const int64_t b = plane / p.Nkv, kvh = plane - b * p.Nkv;
    const int64_t at = plane * p.splits * p.R + row;
    float M = -CUDART_INF_F;
    for (int n = lane; n < p.splits; n += 32) M = fmaxf(M, p.ws_ml[at + n * p.R].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    const float base = M == -CUDART_INF_F ? 0.0f : M;
    float L = 0.0f;
    float acc[kKvMaxHead / 32];
#pragma unroll
    for (int j = 0; j < kKvMaxHead / 32; ++j) acc[j] = 0.0f;
    const bool four = p.H % 4 == 0;  // lane: dims 4 lane + 128 j, or lane + 32 j
#pragma unroll 4
    for (int n = n0; n < p.splits; n += dn) {
      const float2 ml = p.ws_ml[at + n * p.R];
      const float* o = p.ws_o + (at + n * p.R) * p.H;
      const float f = exp2f(ml.x - base);
      L = fmaf(ml.y, f, L);
      if (four) {
#pragma unroll
        for (int j = 0; j < kKvMaxHead / 128; ++j)
          if (lane * 4 + 128 * j < p.H) {
            const float4 x = *reinterpret_cast<const float4*>(o + lane * 4 + 128 * j);
            acc[4 * j] = fmaf(x.x, f, acc[4 * j]);
            acc[4 * j + 1] = fmaf(x.y, f, acc[4 * j + 1]);
            acc[4 * j + 2] = fmaf(x.z, f, acc[4 * j + 2]);
            acc[4 * j + 3] = fmaf(x.w, f, acc[4 * j + 3]);
          }
      } else {
#pragma unroll
        for (int j = 0; j < kKvMaxHead / 32; ++j)
          if (lane + 32 * j < p.H) acc[j] = fmaf(o[lane + 32 * j], f, acc[j]);
      }
    }
    auto dim = [&](int j) { return four ? lane * 4 + 128 * (j / 4) + j % 4 : lane + 32 * j; };
    bits* y = static_cast<bits*>(p.out) + ((b * p.S + row / p.G) * p.Nq + kvh * p.G + row % p.G) * p.H;
    if (shared_row) {
      __syncthreads();  // the previous row's sums have been read
#pragma unroll
      for (int j = 0; j < kKvMaxHead / 32; ++j)
        if (dim(j) < p.H) s_o[warp][dim(j)] = acc[j];
      if (lane == 0) s_l[warp] = L;
      __syncthreads();
      L = 0.0f;
#pragma unroll
      for (int i = 0; i < W; ++i) L += s_l[i];
      const float inv = L == 0.0f ? 0.0f : 1.0f / L;
      for (int d = threadIdx.x; d < p.H; d += kKvCombineThreads) {
        float x = 0.0f;
#pragma unroll
        for (int i = 0; i < W; ++i) x += s_o[i][d];
        y[d] = Elem<T>::fromf(x * inv);
      }
    } else {
      const float inv = L == 0.0f ? 0.0f : 1.0f / L;
      if (four && p.vec) {
#pragma unroll
        for (int j = 0; j < kKvMaxHead / 128; ++j)
          if (lane * 4 + 128 * j < p.H) {
            VecT<T, 4> v;
#pragma unroll
            for (int i = 0; i < 4; ++i) v.v[i] = Elem<T>::fromf(acc[4 * j + i] * inv);
            *reinterpret_cast<VecT<T, 4>*>(y + lane * 4 + 128 * j) = v;
          }
      } else {
#pragma unroll
        for (int j = 0; j < kKvMaxHead / 32; ++j)
          if (dim(j) < p.H) y[dim(j)] = Elem<T>::fromf(acc[j] * inv);
      }
    }
  }
}

}  // namespace rope_gb300
