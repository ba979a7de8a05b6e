// Launchers of the 4-bit decode: one translation unit per head size keeps the
// build parallel.
#pragma once

#include <atomic>

#include "decode_fp4_kernel.cuh"
#include "pa_launch.h"

namespace pa {

template <typename T, int D, int NT>
cudaError_t launch_decode_fp4_one(const Fp4DecodeParams& params, int num_sms,
                                  cudaStream_t stream) {
  using C = Fp4Config<T, D, NT>;
  static std::atomic<bool> configured[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!configured[dev].load(std::memory_order_relaxed)) {
    e = cudaFuncSetAttribute(decode_fp4_kernel<T, D, NT>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    configured[dev].store(true, std::memory_order_relaxed);
  }
  void* args[] = {const_cast<Fp4DecodeParams*>(&params)};
  return launch_overlapped((const void*)decode_fp4_kernel<T, D, NT>, dim3((unsigned)num_sms),
                           dim3(C::kThreads), C::kSmem, stream, args);
}

}  // namespace pa

#define PA_DEFINE_DECODE_FP4_UNIT(D)                                                        \
  namespace pa {                                                                            \
  cudaError_t launch_decode_fp4_d##D(const Fp4DecodeParams& params, int dtype, int num_sms, \
                                     cudaStream_t stream) {                                 \
    constexpr int kTwo = fp4_head_tiles(D, 16);                                             \
    const bool two = fp4_head_tiles(D, params.group) == 2;                                  \
    if (dtype == PA_BF16)                                                                   \
      return two ? launch_decode_fp4_one<__nv_bfloat16, D, kTwo>(params, num_sms, stream)   \
                 : launch_decode_fp4_one<__nv_bfloat16, D, 1>(params, num_sms, stream);     \
    return two ? launch_decode_fp4_one<float, D, kTwo>(params, num_sms, stream)             \
               : launch_decode_fp4_one<float, D, 1>(params, num_sms, stream);               \
  }                                                                                         \
  }
