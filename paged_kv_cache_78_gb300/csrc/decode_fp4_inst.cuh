// Launchers of the 4-bit decode: one translation unit per element type and head
// size keeps the build parallel.
#pragma once

#include <atomic>

#include "decode_fp4_kernel.cuh"
#include "pa_launch.h"

namespace pa {

template <typename T, int D, int H>
cudaError_t launch_decode_fp4_one(const Fp4DecodeParams& params, int num_sms,
                                  cudaStream_t stream) {
  using C = Fp4Config<T, D, H>;
  static std::atomic<bool> configured[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!configured[dev].load(std::memory_order_relaxed)) {
    e = cudaFuncSetAttribute(decode_fp4_kernel<T, D, H>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    configured[dev].store(true, std::memory_order_relaxed);
  }
  void* args[] = {const_cast<Fp4DecodeParams*>(&params)};
  return launch_overlapped((const void*)decode_fp4_kernel<T, D, H>, dim3((unsigned)num_sms),
                           dim3(C::kThreads), C::kSmem, stream, args);
}

template <typename T, int D>
cudaError_t launch_decode_fp4_heads(const Fp4DecodeParams& params, int num_sms,
                                    cudaStream_t stream) {
  constexpr int kMost = fp4_heads(D, 16);
  switch (fp4_heads(D, params.group)) {
    case 4: return launch_decode_fp4_one<T, D, 4>(params, num_sms, stream);
    case 8: return launch_decode_fp4_one<T, D, 8>(params, num_sms, stream);
    default: return launch_decode_fp4_one<T, D, kMost>(params, num_sms, stream);
  }
}

}  // namespace pa

#define PA_DEFINE_DECODE_FP4_UNIT(TYPE, TAG, D)                                          \
  namespace pa {                                                                         \
  cudaError_t launch_decode_fp4_##TAG##_d##D(const Fp4DecodeParams& params, int num_sms, \
                                             cudaStream_t stream) {                      \
    return launch_decode_fp4_heads<TYPE, D>(params, num_sms, stream);                    \
  }                                                                                      \
  }
