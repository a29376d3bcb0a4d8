// Argument checks shared by the operators on dense tensors: alignment, strides
// and device of a [tokens][heads][head_dim] tensor.
#pragma once

#include <cuda_runtime.h>

#include "kvq_host.h"

#define KVQ_TRY(x)                       \
  do {                                   \
    const kvq_status st_ = (x);          \
    if (st_ != KVQ_OK) return st_;       \
  } while (0)

namespace kvq {

constexpr int64_t kMaxTokens = int64_t(1) << 30;  // positions and tile ends stay within 32 bits
constexpr int64_t kMaxTiles = (int64_t(1) << 31) - 1;

// A [tokens][heads][head_dim] tensor of esize-byte elements: strides in
// elements, 16-byte steps; those of a dimension of one entry are not looked at.
inline kvq_status check_tensor(const char* name, const void* ptr, int esize, int64_t tokens, int heads, int head_dim,
                               int64_t ts, int64_t hs) {
  if (!ptr || ((uintptr_t)ptr & 15u))
    return fail(KVQ_EINVAL, "%s must be a non-NULL 16-byte aligned device pointer", name);
  const int64_t step = 16 / esize;
  if ((tokens > 1 && (ts < head_dim || ts % step)) || (heads > 1 && (hs < head_dim || hs % step)))
    return fail(KVQ_EINVAL, "%s strides (token %lld, head %lld) must be multiples of %lld elements and at least head_dim",
                name, (long long)ts, (long long)hs, (long long)step);
  const int64_t most = (int64_t(1) << 40) / esize;
  if ((tokens > 1 && ts >= most) || (heads > 1 && hs >= most))
    return fail(KVQ_EUNSUPPORTED, "%s strides must be below 2^40 bytes", name);
  return KVQ_OK;
}

// As check_tensor, and no two of its rows may share memory.
inline kvq_status check_out_tensor(const char* name, const void* ptr, int esize, int64_t tokens, int heads,
                                   int head_dim, int64_t ts, int64_t hs) {
  KVQ_TRY(check_tensor(name, ptr, esize, tokens, heads, head_dim, ts, hs));
  if (tokens > 1 && heads > 1 && hs * (heads - 1) + head_dim > ts && ts * (tokens - 1) + head_dim > hs)
    return fail(KVQ_EINVAL, "%s strides (token %lld, head %lld) make its rows overlap", name, (long long)ts,
                (long long)hs);
  return KVQ_OK;
}

// Kernels launch on the current device: every tensor has to live there.
inline kvq_status check_on_device(const char* name, const void* ptr) {
  int cur = -1;
  cudaError_t e = cudaGetDevice(&cur);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  cudaPointerAttributes attr;
  e = cudaPointerGetAttributes(&attr, ptr);
  if (e != cudaSuccess) return cuda_fail(e, "cudaPointerGetAttributes");
  if (attr.type != cudaMemoryTypeDevice && attr.type != cudaMemoryTypeManaged)
    return fail(KVQ_EINVAL, "%s is not device memory", name);
  if (attr.type == cudaMemoryTypeDevice && attr.device != cur)
    return fail(KVQ_EINVAL, "the current device is %d but %s lives on device %d", cur, name, attr.device);
  return KVQ_OK;
}

inline kvq_status check_floats(const char* name, const void* ptr) {
  if (!ptr || ((uintptr_t)ptr & 3u)) return fail(KVQ_EINVAL, "%s must be a non-NULL 4-byte aligned device pointer", name);
  return check_on_device(name, ptr);
}

inline kvq_status sm_count(int* n) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(n, cudaDevAttrMultiProcessorCount, dev);
  return e == cudaSuccess ? KVQ_OK : cuda_fail(e, "cudaDeviceGetAttribute");
}

}  // namespace kvq
