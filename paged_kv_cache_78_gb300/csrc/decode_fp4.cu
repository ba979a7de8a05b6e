// Dispatch of the 4-bit decode over element types and head sizes, and its workspace.
#include "decode_fp4.cuh"
#include "pa_launch.h"

namespace pa {

cudaError_t launch_decode_fp4_bf16_d64(const Fp4DecodeParams&, int num_sms, cudaStream_t);
cudaError_t launch_decode_fp4_bf16_d128(const Fp4DecodeParams&, int num_sms, cudaStream_t);
cudaError_t launch_decode_fp4_bf16_d256(const Fp4DecodeParams&, int num_sms, cudaStream_t);
cudaError_t launch_decode_fp4_f32_d64(const Fp4DecodeParams&, int num_sms, cudaStream_t);
cudaError_t launch_decode_fp4_f32_d128(const Fp4DecodeParams&, int num_sms, cudaStream_t);
cudaError_t launch_decode_fp4_f32_d256(const Fp4DecodeParams&, int num_sms, cudaStream_t);

namespace {

// Floats of one partial result at most, whatever the element type.
size_t partial_floats(int head_size, int group) {
  return fp4_partial_floats(fp4_unit_rows(fp4_heads(head_size, group), group), head_size, 2);
}

}  // namespace

// Header (the counters), a partial per warp (16 at most), four per CTA, the ended
// chains of every warp.
size_t decode_fp4_workspace_bytes(int head_size, int group, int num_sms) {
  return kFp4HeaderBytes + (size_t)num_sms * 4 *
                               ((16 + 4) * partial_floats(head_size, group) +
                                16 * fp4_chain_floats(head_size, fp4_heads(head_size, group)));
}

cudaError_t launch_decode_fp4(const Fp4DecodeParams& params, void* workspace, int dtype,
                              int num_sms, cudaStream_t stream) {
  Fp4DecodeParams p = params;
  p.counters = static_cast<unsigned int*>(workspace);
  p.warp_partials =
      reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kFp4HeaderBytes);
  p.cta_partials = p.warp_partials + (size_t)num_sms * 16 * partial_floats(p.head_size, p.group);
  p.chains = p.cta_partials + (size_t)num_sms * 4 * partial_floats(p.head_size, p.group);
  const bool half = dtype == PA_BF16;
  switch (p.head_size) {
    case 64:
      return half ? launch_decode_fp4_bf16_d64(p, num_sms, stream)
                  : launch_decode_fp4_f32_d64(p, num_sms, stream);
    case 128:
      return half ? launch_decode_fp4_bf16_d128(p, num_sms, stream)
                  : launch_decode_fp4_f32_d128(p, num_sms, stream);
    default:
      return half ? launch_decode_fp4_bf16_d256(p, num_sms, stream)
                  : launch_decode_fp4_f32_d256(p, num_sms, stream);
  }
}

}  // namespace pa
