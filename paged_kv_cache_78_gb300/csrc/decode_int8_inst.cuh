// Launchers of the 8-bit decode: one translation unit per element type and head size keeps
// the build parallel.
#pragma once

#include <atomic>

#include "decode_int8_kernel.cuh"
#include "pa_launch.h"

namespace pa {

template <typename T, int D, int H, bool kWeights>
cudaError_t launch_decode_int8_one(const Int8DecodeParams& params, int num_sms,
                                   cudaStream_t stream) {
  using C = Int8Config<T, D, H, kWeights>;
  static std::atomic<bool> configured[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!configured[dev].load(std::memory_order_relaxed)) {
    e = cudaFuncSetAttribute(decode_int8_kernel<T, D, H, kWeights>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    configured[dev].store(true, std::memory_order_relaxed);
  }
  void* args[] = {const_cast<Int8DecodeParams*>(&params)};
  return launch_overlapped((const void*)decode_int8_kernel<T, D, H, kWeights>,
                           dim3((unsigned)num_sms), dim3(C::kThreads), C::kSmem, stream, args);
}

template <typename T, int D>
cudaError_t launch_decode_int8_heads(const Int8DecodeParams& p, int num_sms, cudaStream_t stream) {
  constexpr int kMost = int8_heads(D, 16);
  const bool weights = p.block_weights_out != nullptr;
  if (int8_heads(D, p.group) == 8)
    return weights ? launch_decode_int8_one<T, D, 8, true>(p, num_sms, stream)
                   : launch_decode_int8_one<T, D, 8, false>(p, num_sms, stream);
  return weights ? launch_decode_int8_one<T, D, kMost, true>(p, num_sms, stream)
                 : launch_decode_int8_one<T, D, kMost, false>(p, num_sms, stream);
}

}  // namespace pa

#define PA_DEFINE_DECODE_INT8_UNIT(TYPE, TAG, D)                                           \
  namespace pa {                                                                           \
  cudaError_t launch_decode_int8_##TAG##_d##D(const Int8DecodeParams& params, int num_sms, \
                                              cudaStream_t stream) {                       \
    return launch_decode_int8_heads<TYPE, D>(params, num_sms, stream);                     \
  }                                                                                        \
  }
