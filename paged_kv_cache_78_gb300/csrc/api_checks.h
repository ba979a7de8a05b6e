// Argument checks that the C entry points share.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "pa.h"

namespace pa {

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline bool is_pow2(int x) { return x > 0 && (x & (x - 1)) == 0; }
inline int ilog2(int x) {
  int r = 0;
  while ((1 << r) < x) ++r;
  return r;
}
inline pa_status cuda_status(cudaError_t e) { return e == cudaSuccess ? PA_OK : PA_ERR_CUDA; }

inline bool dtype_ok(int32_t t) { return t == PA_BF16 || t == PA_FP32; }
inline int64_t elem_bytes(int32_t dtype) { return dtype == PA_BF16 ? 2 : 4; }

// Elements per row, and whether rows `stride` elements apart keep 16-byte
// alignment without overlapping.
inline bool stride_ok(int64_t stride, int64_t row, int32_t dtype) {
  return stride >= row && stride * elem_bytes(dtype) % 16 == 0;
}

// A buffer of a call, to tell whether two overlap.
struct Range {
  const void* p;
  int64_t bytes;
  bool written;
};
inline bool overlap(const Range& a, const Range& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x && y && a.bytes > 0 && b.bytes > 0 && x < y + (uint64_t)b.bytes &&
         y < x + (uint64_t)a.bytes;
}

// Whether a buffer that the call writes (they come first) overlaps another.
template <int N>
bool conflict(const Range (&buffers)[N]) {
  for (int i = 0; i < N && buffers[i].written; ++i)
    for (int j = i + 1; j < N; ++j)
      if (overlap(buffers[i], buffers[j])) return true;
  return false;
}

// `n` rows of `row` elements, `stride` apart.
inline int64_t rows_bytes(int64_t n, int64_t stride, int64_t row, int32_t dtype) {
  return ((n - 1) * stride + row) * elem_bytes(dtype);
}

}  // namespace pa
