// Host helpers shared by the C ABI layers of the cache operators (kv_api.cu,
// paged_api.cu): errors, checks of arguments, launches. Internal.
#pragma once

#include <cuda_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <initializer_list>
#include <map>
#include <mutex>
#include <set>
#include <tuple>
#include <utility>

#include "kv_internal.h"
#include "rope.h"
#include "rope_internal.h"

#define KV_TRY(expr)              \
  do {                            \
    rope_status _s = (expr);      \
    if (_s != ROPE_OK) return _s; \
  } while (0)

namespace rope_gb300 {

constexpr int kSms = 152;  // GB300
constexpr int64_t kMaxLen = 1 << 30;     // positions and offsets between them stay in 32 bits
constexpr int64_t kWorkspaceSlack = 16;  // aligns the part behind the partial outputs

inline rope_status fail(rope_status st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  set_last_error(buf);
  return st;
}

inline rope_status cuda_fail(cudaError_t e, const char* what) {
  return fail(ROPE_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline rope_status check_ptr(const void* p, const char* name, size_t align) {
  if (!p) return fail(ROPE_ERR_INVALID_ARG, "%s is NULL", name);
  if (!aligned(p, align)) return fail(ROPE_ERR_INVALID_ARG, "%s is not aligned to %zu bytes", name, align);
  return ROPE_OK;
}

inline rope_status check_optional(const void* p, const char* name, size_t align) {
  return p ? check_ptr(p, name, align) : ROPE_OK;
}

inline rope_status check_dtype(rope_dtype dt) {
  if (dt != ROPE_F32 && dt != ROPE_F16 && dt != ROPE_BF16)
    return fail(ROPE_ERR_UNSUPPORTED, "dtype %d: only float32 (0), float16 (1) and bfloat16 (2) are implemented",
                (int)dt);
  return ROPE_OK;
}

// The product of non-negative sizes stays below 2^62 (bytes of every tensor fit int64).
inline bool sizes_fit(std::initializer_list<int64_t> v) {
  int64_t n = 1;
  for (int64_t x : v) {
    if (x == 0) return true;
    if (n > ((int64_t)1 << 62) / x) return false;
    n *= x;
  }
  return true;
}

inline int pow2_at_least(int64_t n) {
  int p = 1;
  while (p < n) p *= 2;
  return p;
}

// (n * m) >> shift == n / d for 0 <= n < 2^31: m = ceil(2^(31 + l) / d), l = ceil(log2 d).
inline KvDiv div_of(int64_t d) {
  int l = 0;
  while (((int64_t)1 << l) < d) ++l;
  KvDiv r;
  r.m = (uint32_t)((((uint64_t)1 << (31 + l)) + (uint64_t)d - 1) / (uint64_t)d);
  r.shift = 31 + l;
  return r;
}

// A kernel with more than 48 KB of dynamic shared memory is allowed the
// device's most, once for each device.
inline std::mutex g_mu;
inline std::set<std::pair<int, const void*>> g_raised;

// `registers`: what a kernel that deals its registers out again has to be
// launched with (0: any).
inline rope_status allow_smem(const void* fn, size_t smem, int registers) {
  if (smem <= 48 * 1024) return ROPE_OK;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  std::lock_guard<std::mutex> lk(g_mu);
  if (g_raised.count(std::make_pair(dev, fn))) return ROPE_OK;
  int most = 0;
  e = cudaDeviceGetAttribute(&most, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaDeviceGetAttribute(shared memory opt-in)");
  cudaFuncAttributes fa;
  e = cudaFuncGetAttributes(&fa, fn);
  if (e != cudaSuccess) return cuda_fail(e, "cudaFuncGetAttributes");
  if (registers && fa.numRegs != registers)
    return fail(ROPE_ERR_UNSUPPORTED, "the kernel was built with %d registers a thread, not %d", fa.numRegs, registers);
  most -= (int)fa.sharedSizeBytes;  // what the kernel holds statically
  if (most < (int)smem) return fail(ROPE_ERR_UNSUPPORTED, "needs %zu bytes of shared memory", smem);
  e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
  if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(max dynamic shared memory)");
  try {
    g_raised.insert(std::make_pair(dev, fn));
  } catch (...) {  // no memory: asked for again by the next call
  }
  return ROPE_OK;
}

// CTAs of `threads` threads without dynamic shared memory that an SM holds, asked for once.
inline std::map<std::tuple<int, const void*, int>, int> g_resident;
inline rope_status resident_ctas(const void* fn, int threads, int* n) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  std::lock_guard<std::mutex> lk(g_mu);
  const auto key = std::make_tuple(dev, fn, threads);
  const auto held = g_resident.find(key);
  if (held != g_resident.end()) {
    *n = held->second;
    return ROPE_OK;
  }
  int b = 0;
  e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&b, fn, threads, 0);
  if (e != cudaSuccess) return cuda_fail(e, "cudaOccupancyMaxActiveBlocksPerMultiprocessor");
  *n = b < 1 ? 1 : b;
  try {
    g_resident.emplace(key, *n);
  } catch (...) {  // no memory: asked for again by the next call
  }
  return ROPE_OK;
}

// Launched as a programmatic dependent, as every kernel of the library.
inline rope_status launch(const void* fn, dim3 grid, int threads, size_t smem, rope_stream_t stream, void** args,
                   const char* what, int registers = 0, int cluster = 0) {
  KV_TRY(allow_smem(fn, smem, registers));
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = (cudaStream_t)stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelExC(&cfg, fn, args);
  if (e != cudaSuccess) return cuda_fail(e, what);
  return ROPE_OK;
}

}  // namespace rope_gb300
