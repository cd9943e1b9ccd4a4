// Host-side checks the draft-tree and cache entry points share (no device access but the
// pointer queries; nothing is launched).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace mtpattn {

inline bool ptr_aligned(const void* p, size_t a) {
  return reinterpret_cast<uintptr_t>(p) % a == 0;
}

// Whether two runs of 32-bit words have a word in common.
inline bool words_overlap(const void* a, int64_t n, const void* b, int64_t m) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + 4 * static_cast<uintptr_t>(m) && y < x + 4 * static_cast<uintptr_t>(n);
}

// The current device, or -1.
inline int current_device() {
  int device = -1;
  if (cudaGetDevice(&device) != cudaSuccess) {
    cudaGetLastError();
    return -1;
  }
  return device;
}

// A pointer the kernels may dereference: device (or managed) memory of `device`.
inline bool ptr_on_device(const void* ptr, int device) {
  cudaPointerAttributes attr;
  if (cudaPointerGetAttributes(&attr, ptr) != cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  return (attr.type == cudaMemoryTypeDevice || attr.type == cudaMemoryTypeManaged) &&
         attr.device == device;
}

template <int N>
inline bool all_on_device(const void* const (&ptrs)[N], int device) {
  for (const void* p : ptrs)
    if (!ptr_on_device(p, device)) return false;
  return true;
}

}  // namespace mtpattn
