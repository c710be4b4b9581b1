// Attention over a key/value cache on CUDA cores: every storage type, head
// size, alignment and mask; float32 keeps 32-bit products throughout.
//
// A CTA takes 32 rows of one (b, kvh) and walks its keys 32 at a time: scores
// of a 32 x 32 tile (2 x 2 a thread), the running maximum and sum of each row
// (held by the 16 threads that share the row), then O = O * alpha + P V with
// 2 rows x H/16 columns of O in each thread's registers. The tiles are float32
// in shared memory, so every product is a 32-bit FMA.
#pragma once

#include "kv_common.cuh"

namespace rope_gb300 {

constexpr int kSimpleCols = 32;

// n consecutive elements of a row at `src` (scaled) to float32 at `dst`;
// the threads of a warp cooperate.
template <class T, bool FP8>
__device__ __forceinline__ void simple_load_row(float* dst, const void* src, int64_t off, int n, float scale,
                                                bool vec, int lane, bool& finite) {
  if constexpr (FP8) {
    const uint8_t* s = static_cast<const uint8_t*>(src) + off;
    if (vec) {
      for (int d = lane * 4; d < n; d += 128) {
        const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(s + d));
        const float2 a = kv_fp8x2((uint16_t)w), b = kv_fp8x2((uint16_t)(w >> 16));
        const float4 f = make_float4(a.x * scale, a.y * scale, b.x * scale, b.y * scale);
        *reinterpret_cast<float4*>(dst + d) = f;
        finite &= isfinite(f.x) && isfinite(f.y) && isfinite(f.z) && isfinite(f.w);
      }
    } else {
      for (int d = lane; d < n; d += 32) {
        const float x = kv_fp8x2(s[d]).x * scale;
        dst[d] = x;
        finite &= isfinite(x);
      }
    }
  } else {
    using bits = typename Elem<T>::bits;
    const bits* s = static_cast<const bits*>(src) + off;
    if (vec) {
      using VT = VecT<T, 4>;
      for (int d = lane * 4; d < n; d += 128) {
        const VT v = ld_shared_ro(reinterpret_cast<const VT*>(s + d));
        const float4 f = make_float4(Elem<T>::tof(v.v[0]), Elem<T>::tof(v.v[1]), Elem<T>::tof(v.v[2]),
                                     Elem<T>::tof(v.v[3]));
        *reinterpret_cast<float4*>(dst + d) = f;
        finite &= isfinite(f.x) && isfinite(f.y) && isfinite(f.z) && isfinite(f.w);
      }
    } else {
      for (int d = lane; d < n; d += 32) {
        const float x = Elem<T>::tof(s[d]);
        dst[d] = x;
        finite &= isfinite(x);
      }
    }
  }
}

// NJ: columns of O that a thread holds, 16 threads a row: H <= 16 * NJ.
template <class T, bool FP8, int NJ>
__device__ __forceinline__ void simple_body(const KvParams& p) {
  using bits = typename Elem<T>::bits;
  extern __shared__ float smem[];
  const int H = p.H, HP = (H + 3) / 4 * 4 + 4;
  float* sq = smem;                        // [32][HP]
  float* skv = sq + kKvSimpleRows * HP;    // [32][HP]
  float* sp = skv + kSimpleCols * HP;      // [32][33]
  __shared__ int32_t sdoc[kSimpleCols];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int tx = tid & 15, ty = tid >> 4;
  pdl_launch_dependents();
  pdl_wait();
  const int64_t tile = blockIdx.x / p.splits;
  const int split = blockIdx.x % p.splits;
  const int kvh = blockIdx.y;
  const int64_t r0 = tile * kKvSimpleRows;
  for (int b = blockIdx.z; b < p.B; b += gridDim.z) {
    const KvSeq seq = kv_seq(p, b);
    if (blockIdx.x == 0 && kvh == 0 && tid == 0) kv_flag_rows(p, seq);
    const int64_t rlast = (r0 + kKvSimpleRows < p.R ? r0 + kKvSimpleRows : p.R) - 1;
    int64_t end = kv_limit(seq, seq.past + rlast / p.G);  // no row of the tile sees more
    if (end < 0) end = 0;
    int64_t lo, hi;
    kv_split(end, p.splits, split, kSimpleCols, &lo, &hi);
    __syncthreads();
    for (int r = warp; r < kKvSimpleRows; r += kKvSimpleThreads / 32) {
      bool fin = true;
      const int64_t row = r0 + r;
      if (row < p.R)
        simple_load_row<T, false>(sq + r * HP, p.q,
                                  (((int64_t)b * p.S + row / p.G) * p.Nq + (int64_t)kvh * p.G + row % p.G) * H, H,
                                  1.0f, p.vec, lane, fin);
      else
        for (int d = lane; d < H; d += 32) sq[r * HP + d] = 0.0f;
    }
    // the two rows of this thread
    int64_t pos[2], lim[2];
    float slope[2], m[2], l[2];
    int32_t doc[2] = {0, 0};
    float acc[2][NJ];
#pragma unroll
    for (int a = 0; a < 2; ++a) {
      const int64_t row = r0 + ty + 16 * a;
      pos[a] = seq.past + (row < p.R ? row : p.R - 1) / p.G;
      lim[a] = row < p.R ? kv_limit(seq, pos[a]) : 0;
      slope[a] = p.slopes ? __ldg(p.slopes + kvh * p.G + (row < p.R ? row : 0) % p.G) * kLog2e : 0.0f;
      if (p.docs && row < p.R && !kv_document(p, b, pos[a], &doc[a])) lim[a] = 0;
      m[a] = -CUDART_INF_F;
      l[a] = 0.0f;
#pragma unroll
      for (int j = 0; j < NJ; ++j) acc[a][j] = 0.0f;
    }
    const int64_t plane = (int64_t)b * p.Nkv + kvh;
    const float c1 = p.cap > 0.0f ? p.scale / p.cap : p.scale * kLog2e;
    const float c2 = p.cap * kLog2e;
    for (int64_t j0 = lo; j0 < hi; j0 += kSimpleCols) {
      const int n = hi - j0 < kSimpleCols ? (int)(hi - j0) : kSimpleCols;
      __syncthreads();
      bool fin = true;
      for (int c = warp; c < n; c += kKvSimpleThreads / 32)
        simple_load_row<T, FP8>(skv + c * HP, p.k, (plane * p.max_len + j0 + c) * H, H,
                                FP8 ? __ldg(p.ks + plane * p.nblk + (j0 + c) / kKvBlock) : 1.0f, p.vec, lane, fin);
      if (p.docs && tid < n) sdoc[tid] = __ldg(p.docs + (int64_t)b * p.max_len + j0 + tid);
      __syncthreads();
      float s[2][2] = {{0.0f, 0.0f}, {0.0f, 0.0f}};
      const float* q0 = sq + ty * HP;
      const float* q1 = q0 + 16 * HP;
      const float* k0 = skv + tx * HP;
      const float* k1 = k0 + 16 * HP;
      int d = 0;
      for (; d + 4 <= H; d += 4) {
        const float4 a0 = *reinterpret_cast<const float4*>(q0 + d), a1 = *reinterpret_cast<const float4*>(q1 + d);
        const float4 b0 = *reinterpret_cast<const float4*>(k0 + d), b1 = *reinterpret_cast<const float4*>(k1 + d);
#define KV_DOT(S, A, B) S = fmaf(A.x, B.x, fmaf(A.y, B.y, fmaf(A.z, B.z, fmaf(A.w, B.w, S))))
        KV_DOT(s[0][0], a0, b0);
        KV_DOT(s[0][1], a0, b1);
        KV_DOT(s[1][0], a1, b0);
        KV_DOT(s[1][1], a1, b1);
#undef KV_DOT
      }
      for (; d < H; ++d) {
        s[0][0] = fmaf(q0[d], k0[d], s[0][0]);
        s[0][1] = fmaf(q0[d], k1[d], s[0][1]);
        s[1][0] = fmaf(q1[d], k0[d], s[1][0]);
        s[1][1] = fmaf(q1[d], k1[d], s[1][1]);
      }
      float alpha[2];
#pragma unroll
      for (int a = 0; a < 2; ++a) {
        float x[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int col = tx + 16 * c;
          const int64_t j = j0 + col;
          const int64_t dist = pos[a] > j ? pos[a] - j : j - pos[a];
          float y = s[a][c] * c1;
          if (p.cap > 0.0f) y = tanhf(y) * c2;
          y = fmaf(-slope[a], (float)dist, y);
          const bool seen = col < n && j < lim[a] && (!p.docs || sdoc[col] == doc[a]);
          x[c] = seen ? y : -CUDART_INF_F;
        }
        // fmaxf drops NaN, so a NaN score shows in the sum
        float mx = fmaxf(x[0], x[1]);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        const float mn = fmaxf(m[a], mx);
        const float base = mn == -CUDART_INF_F ? 0.0f : mn;
        alpha[a] = exp2f(m[a] - base);
        const float p0 = exp2f(x[0] - base), p1 = exp2f(x[1] - base);
        float sum = p0 + p1;
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        l[a] = l[a] * alpha[a] + sum;
        m[a] = mn;
        sp[(ty + 16 * a) * 33 + tx] = p0;
        sp[(ty + 16 * a) * 33 + tx + 16] = p1;
      }
      __syncthreads();
      fin = true;
      for (int c = warp; c < n; c += kKvSimpleThreads / 32)
        simple_load_row<T, FP8>(skv + c * HP, p.v, (plane * p.max_len + j0 + c) * H, H,
                                FP8 ? __ldg(p.vs + plane * p.nblk + (j0 + c) / kKvBlock) : 1.0f, p.vec, lane, fin);
      const bool all_finite = __syncthreads_and(fin);
#pragma unroll
      for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int j = 0; j < NJ; ++j) acc[a][j] *= alpha[a];
      for (int c = 0; c < n; ++c) {
        const float w0 = sp[ty * 33 + c], w1 = sp[(ty + 16) * 33 + c];
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          const int dd = tx + 16 * j;
          const float v = dd < H ? skv[c * HP + dd] : 0.0f;
          if (all_finite) {
            acc[0][j] = fmaf(w0, v, acc[0][j]);
            acc[1][j] = fmaf(w1, v, acc[1][j]);
          } else {  // a masked key's weight is exactly 0, and its value is not touched
            if (w0 != 0.0f) acc[0][j] = fmaf(w0, v, acc[0][j]);
            if (w1 != 0.0f) acc[1][j] = fmaf(w1, v, acc[1][j]);
          }
        }
      }
    }
#pragma unroll
    for (int a = 0; a < 2; ++a) {
      const int64_t row = r0 + ty + 16 * a;
      if (row >= p.R) continue;
      if (p.splits > 1) {
        const int64_t at = (plane * p.splits + split) * p.R + row;
        if (tx == 0) p.ws_ml[at] = make_float2(m[a], l[a]);
#pragma unroll
        for (int j = 0; j < NJ; ++j)
          if (tx + 16 * j < H) p.ws_o[at * H + tx + 16 * j] = acc[a][j];
      } else {
        const float inv = l[a] == 0.0f ? 0.0f : 1.0f / l[a];
        bits* o = static_cast<bits*>(p.out) +
                  (((int64_t)b * p.S + row / p.G) * p.Nq + (int64_t)kvh * p.G + row % p.G) * H;
#pragma unroll
        for (int j = 0; j < NJ; ++j)
          if (tx + 16 * j < H) o[tx + 16 * j] = Elem<T>::fromf(acc[a][j] * inv);
      }
    }
  }
}

template <class T, bool FP8>
__global__ void __launch_bounds__(kKvSimpleThreads) kv_simple_kernel_t(const KvParams p) {
  if (p.H <= 64)
    simple_body<T, FP8, 4>(p);
  else if (p.H <= 128)
    simple_body<T, FP8, 8>(p);
  else
    simple_body<T, FP8, 16>(p);
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
