// Host-side launchers shared by the C-ABI translation unit and the kernel
// translation units of the library.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "pa.h"

namespace pa {

struct DecodeParams;

// Device-side state of the current device: the error word's address and the
// SM count.
pa_status device_state(unsigned int** err, int* num_sms);

// Geometry checks of a 4-bit pool (PA_FP4), and the bytes of one block.
pa_status check_fp4_desc(const pa_cache_desc* desc);
int64_t fp4_block_bytes(const pa_cache_desc* desc);

// The same of an 8-bit pool (PA_INT8).
pa_status check_int8_desc(const pa_cache_desc* desc);
int64_t int8_block_bytes(const pa_cache_desc* desc);

// Half of a block as the block copies see it: its bytes, and the distance
// between the same halves of neighbouring blocks.
struct BlockGeometry {
  int64_t bytes;
  int64_t stride;
};

// Launch `kernel` with programmatic stream serialization: it may begin (and
// run the part before its grid_dependency_wait) while the previous kernel on
// the stream finishes.  `args` points at the kernel's arguments, in order.
inline cudaError_t launch_overlapped(const void* kernel, dim3 grid, dim3 block, size_t smem,
                                     cudaStream_t stream, void** args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelExC(&cfg, kernel, args);
}

cudaError_t launch_reshape_and_cache(void* cache, const void* key, const void* value,
                                     const int64_t* slot_mapping, int64_t num_tokens,
                                     int64_t num_slots, int row_bytes, int64_t plane_bytes,
                                     unsigned int* err, cudaStream_t stream);

// Block copies from src_cache to dst_cache (the same pool for copy-on-write).
// dst_half / src_half: the distance between the halves of a block.
cudaError_t launch_copy_blocks(void* dst_cache, const void* src_cache, const int64_t* pairs,
                               int num_pairs, int64_t dst_blocks, int64_t src_blocks,
                               BlockGeometry geometry, int64_t dst_half, int64_t src_half,
                               unsigned int* err, cudaStream_t stream);

// Byte copy by a kernel (device or page-locked host memory on either side).
cudaError_t launch_copy_bytes(void* dst, const void* src, int64_t bytes, int num_sms,
                              cudaStream_t stream);

// Decode launchers, one per element type.  `supported` is set to false (and
// nothing launched) when no kernel exists for (head_size, group).
cudaError_t launch_decode_bf16(int head_size, int group, dim3 grid, int smem_bytes,
                               cudaStream_t stream, const CUtensorMap& map,
                               const DecodeParams& params, bool* supported);
cudaError_t launch_decode_f32(int head_size, int group, dim3 grid, int smem_bytes,
                              cudaStream_t stream, const CUtensorMap& map,
                              const DecodeParams& params, bool* supported);

// Tensor-core decode (bf16, head size 64 or 128, group <= 16).
cudaError_t launch_decode_tc(int head_size, int num_sms, int smem_bytes, cudaStream_t stream,
                             const CUtensorMap& kv_map, const CUtensorMap& q_map,
                             const DecodeParams& params, bool* supported);

// Shared-prefix decode (bf16, head size 64 or 128): grid = (stage ranges,
// KV heads, chunks).  shared_stage_slots / shared_smem_bytes give its stage
// ring and dynamic shared memory.
struct SharedParams;
int shared_stage_slots(int head_size);
int shared_smem_bytes(int head_size);
cudaError_t launch_decode_shared(int head_size, dim3 grid, int smem_bytes, cudaStream_t stream,
                                 const CUtensorMap& kv_map, const SharedParams& params,
                                 bool* supported);

// Log-sum-exp reduce of split-KV partials.  A row's partial count comes from
// counts[row / group] when counts is given (balanced split), else from its
// sequence length and partition_tokens.
cudaError_t launch_lse_reduce(int dtype, int head_size, void* out, const float* part_o,
                              const float* part_lse, const int32_t* seq_lens,
                              const int32_t* counts, int group, int num_seqs, int num_heads,
                              int partition_tokens, int max_parts, cudaStream_t stream,
                              bool* supported);

// 4-bit cache: write and read-back of tokens by slot.  src / dst rows of one
// token are num_kv_heads * head_size elements of `dtype`, `stride` elements
// apart.
struct Fp4Pool {
  uint8_t* cache;
  int64_t num_slots;
  int num_kv_heads;
  int head_size;
  int log2_block_size;
};
cudaError_t launch_fp4_write(const Fp4Pool& pool, const void* key, const void* value, int dtype,
                             int64_t key_stride, int64_t value_stride,
                             const int64_t* slot_mapping, int num_tokens, float key_scale,
                             float value_scale, unsigned int* err, cudaStream_t stream);
cudaError_t launch_fp4_gather(const Fp4Pool& pool, void* key, void* value, int dtype,
                              const int64_t* slot_mapping, int num_tokens, float key_scale,
                              float value_scale, unsigned int* err, cudaStream_t stream);

// Decode attention over a 4-bit cache.
struct Fp4DecodeParams;
size_t decode_fp4_workspace_bytes(int head_size, int group, int num_sms);
cudaError_t launch_decode_fp4(const Fp4DecodeParams& params, void* workspace, int dtype,
                              int num_sms, cudaStream_t stream);

// 8-bit cache: write and read-back of tokens by slot, as for the 4-bit cache.
struct Int8Pool {
  uint8_t* cache;
  int64_t num_slots;
  int num_kv_heads;
  int head_size;
  int log2_block_size;
};
cudaError_t launch_int8_write(const Int8Pool& pool, const void* key, const void* value, int dtype,
                              int64_t key_stride, int64_t value_stride,
                              const int64_t* slot_mapping, int num_tokens, int num_sms,
                              unsigned int* err, cudaStream_t stream);
cudaError_t launch_int8_gather(const Int8Pool& pool, void* key, void* value, int dtype,
                               const int64_t* slot_mapping, int num_tokens, unsigned int* err,
                               cudaStream_t stream);

// Decode attention over an 8-bit cache; num_seqs and max_blocks of the calls that keep
// weights (0: none).
struct Int8DecodeParams;
size_t decode_int8_workspace_bytes(int head_size, int num_heads, int group, int block_size,
                                   int64_t num_seqs, int64_t max_blocks, int num_sms);
cudaError_t launch_decode_int8(const Int8DecodeParams& params, void* workspace, int dtype,
                               int num_sms, cudaStream_t stream);

// Eviction of the blocks with the least weight.
struct EvictParams;
cudaError_t launch_evict_blocks(const EvictParams& params, int num_sms, cudaStream_t stream);

// Norms of queries and keys, and rotation.
cudaError_t launch_norm_rope(const pa_norm_rope_args& args, int num_sms, unsigned int* err,
                             cudaStream_t stream);

// Limit of the tensor-core decodes' pipeline waits (pa_set_decode_wait_limit).
long long decode_wait_limit();

// Block tables, slot map and positions from request lengths.
struct TablesParams;
cudaError_t launch_extend_tables(const TablesParams& params, int num_sms, cudaStream_t stream);

}  // namespace pa
