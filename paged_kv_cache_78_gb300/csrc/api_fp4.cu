// C entry points of the 4-bit pool and of the device-side tables: argument
// checks and launches.  See include/pa.h for the contract.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "api_checks.h"
#include "decode_fp4.cuh"
#include "extend_tables.cuh"
#include "pa.h"
#include "pa_launch.h"

namespace {

using namespace pa;

constexpr int kFp4MaxGroup = 16;

// A power of two in [2^-32, 2^32].
bool tensor_scale_ok(float s) {
  int e = 0;
  return std::isfinite(s) && s > 0.f && std::frexp(s, &e) == 0.5f && e >= -31 && e <= 33;
}

pa_status check_call(const pa_cache_desc* desc, int32_t dtype, float key_scale, float value_scale) {
  const pa_status st = pa::check_fp4_desc(desc);
  if (st != PA_OK) return st;
  if (!dtype_ok(dtype) || !tensor_scale_ok(key_scale) || !tensor_scale_ok(value_scale))
    return PA_ERR_INVALID_ARG;
  return PA_OK;
}

// One grid holds the call: a CTA per eight tokens and two heads, or more.
bool grid_ok(const pa_cache_desc* d, int64_t num_tokens) {
  return (num_tokens + 7) / 8 * d->num_kv_heads < (1ll << 31);
}

int64_t pool_bytes(const pa_cache_desc* d) { return d->num_blocks * pa::fp4_block_bytes(d); }
pa::Fp4Pool pool_of(const void* cache, const pa_cache_desc* d) {
  pa::Fp4Pool p;
  p.cache = static_cast<uint8_t*>(const_cast<void*>(cache));
  p.num_slots = (int64_t)d->num_blocks * d->block_size;
  p.num_kv_heads = d->num_kv_heads;
  p.head_size = d->head_size;
  p.log2_block_size = ilog2(d->block_size);
  return p;
}

}  // namespace

namespace pa {

pa_status check_fp4_desc(const pa_cache_desc* d) {
  if (!d || d->dtype != PA_FP4) return PA_ERR_INVALID_ARG;
  if (d->num_blocks < 1 || d->num_kv_heads < 1 || d->head_size < 1) return PA_ERR_INVALID_ARG;
  if (!is_pow2(d->block_size) || d->block_size < 8 || d->block_size > 256)
    return PA_ERR_INVALID_ARG;
  if (d->head_size != 64 && d->head_size != 128 && d->head_size != 256) return PA_ERR_UNSUPPORTED;
  if (d->num_kv_heads > 65535 || fp4_block_bytes(d) > 0x7fffffff) return PA_ERR_UNSUPPORTED;
  return PA_OK;
}

int64_t fp4_block_bytes(const pa_cache_desc* d) {
  return (int64_t)d->num_kv_heads * (d->block_size / 8) * 9 * d->head_size;
}

}  // namespace pa

extern "C" {

pa_status pa_reshape_and_cache_fp4(void* cache, const pa_cache_desc* desc, const void* key,
                                   const void* value, int32_t dtype, int64_t key_stride,
                                   int64_t value_stride, const int64_t* slot_mapping,
                                   int32_t num_tokens, float key_scale, float value_scale,
                                   void* stream) {
  pa_status st = check_call(desc, dtype, key_scale, value_scale);
  if (st != PA_OK) return st;
  if (num_tokens < 0) return PA_ERR_INVALID_ARG;
  if (num_tokens == 0) return PA_OK;
  const int64_t row = (int64_t)desc->num_kv_heads * desc->head_size;
  if (!cache || !key || !value || !slot_mapping || !aligned(cache, 16) || !aligned(key, 16) ||
      !aligned(value, 16) || !aligned(slot_mapping, 8) || !stride_ok(key_stride, row, dtype) ||
      !stride_ok(value_stride, row, dtype) || !grid_ok(desc, num_tokens))
    return PA_ERR_INVALID_ARG;
  const Range buffers[] = {{cache, pool_bytes(desc), true},
                           {key, rows_bytes(num_tokens, key_stride, row, dtype), false},
                           {value, rows_bytes(num_tokens, value_stride, row, dtype), false},
                           {slot_mapping, num_tokens * 8ll, false}};
  if (conflict(buffers)) return PA_ERR_INVALID_ARG;
  unsigned int* err = nullptr;
  if ((st = pa::device_state(&err, nullptr)) != PA_OK) return st;
  return cuda_status(pa::launch_fp4_write(pool_of(cache, desc), key, value, dtype, key_stride,
                                          value_stride, slot_mapping, num_tokens, key_scale,
                                          value_scale, err, static_cast<cudaStream_t>(stream)));
}

pa_status pa_gather_cache_fp4(void* key, void* value, int32_t dtype, const void* cache,
                              const pa_cache_desc* desc, const int64_t* slot_mapping,
                              int32_t num_tokens, float key_scale, float value_scale,
                              void* stream) {
  pa_status st = check_call(desc, dtype, key_scale, value_scale);
  if (st != PA_OK) return st;
  if (num_tokens < 0) return PA_ERR_INVALID_ARG;
  if (num_tokens == 0) return PA_OK;
  const int64_t row = (int64_t)desc->num_kv_heads * desc->head_size;
  if (!cache || !key || !value || !slot_mapping || !aligned(cache, 16) || !aligned(key, 16) ||
      !aligned(value, 16) || !aligned(slot_mapping, 8) || !grid_ok(desc, num_tokens))
    return PA_ERR_INVALID_ARG;
  const Range buffers[] = {{key, num_tokens * row * elem_bytes(dtype), true},
                           {value, num_tokens * row * elem_bytes(dtype), true},
                           {cache, pool_bytes(desc), false},
                           {slot_mapping, num_tokens * 8ll, false}};
  if (conflict(buffers)) return PA_ERR_INVALID_ARG;
  unsigned int* err = nullptr;
  if ((st = pa::device_state(&err, nullptr)) != PA_OK) return st;
  return cuda_status(pa::launch_fp4_gather(pool_of(cache, desc), key, value, dtype, slot_mapping,
                                           num_tokens, key_scale, value_scale, err,
                                           static_cast<cudaStream_t>(stream)));
}

pa_status pa_decode_fp4_workspace_size(const pa_cache_desc* desc, int32_t num_heads,
                                       size_t* bytes) {
  pa_status st = pa::check_fp4_desc(desc);
  if (st != PA_OK) return st;
  if (!bytes || num_heads < 1 || num_heads % desc->num_kv_heads != 0) return PA_ERR_INVALID_ARG;
  if (num_heads / desc->num_kv_heads > kFp4MaxGroup) return PA_ERR_UNSUPPORTED;
  int sms = 0;
  if ((st = pa::device_state(nullptr, &sms)) != PA_OK) return st;
  if (sms > pa::kFp4MaxCtas) return PA_ERR_UNSUPPORTED;
  *bytes = pa::decode_fp4_workspace_bytes(desc->head_size, num_heads / desc->num_kv_heads, sms);
  return PA_OK;
}

pa_status pa_decode_fp4(void* out, const void* query, int32_t dtype, int64_t query_stride,
                        const void* cache, const pa_cache_desc* desc, float key_scale,
                        float value_scale, const int32_t* block_tables,
                        int32_t max_blocks_per_seq, const int32_t* seq_lens, int32_t num_seqs,
                        int32_t num_heads, float scale, void* workspace, size_t workspace_bytes,
                        void* stream) {
  pa_status st = check_call(desc, dtype, key_scale, value_scale);
  if (st != PA_OK) return st;
  if (num_seqs < 0 || num_seqs > 65535 || max_blocks_per_seq < 1 || !std::isfinite(scale))
    return PA_ERR_INVALID_ARG;
  if (num_heads < 1 || num_heads % desc->num_kv_heads != 0) return PA_ERR_INVALID_ARG;
  if (num_heads / desc->num_kv_heads > kFp4MaxGroup || (int64_t)num_seqs * num_heads >= (1ll << 31))
    return PA_ERR_UNSUPPORTED;
  if (num_seqs == 0) return PA_OK;
  if (!out || !query || !cache || !block_tables || !seq_lens || !workspace ||
      !aligned(workspace, 256) || !aligned(out, 16) ||
      !aligned(query, 16) || !aligned(cache, 16) || !aligned(block_tables, 4) ||
      !aligned(seq_lens, 4) ||
      !stride_ok(query_stride, (int64_t)num_heads * desc->head_size, dtype))
    return PA_ERR_INVALID_ARG;
  const int64_t row = (int64_t)num_heads * desc->head_size;
  // The workspace, whose size needs the device, is looked at below.
  Range buffers[] = {{out, num_seqs * row * elem_bytes(dtype), true},
                     {workspace, 0, true},
                     {query, rows_bytes(num_seqs, query_stride, row, dtype), false},
                     {cache, pool_bytes(desc), false},
                     {block_tables, (int64_t)num_seqs * max_blocks_per_seq * 4, false},
                     {seq_lens, num_seqs * 4ll, false}};
  if (conflict(buffers)) return PA_ERR_INVALID_ARG;
  pa::Fp4DecodeParams p = {};
  p.scale_log2 = (float)((double)scale * key_scale * 1.4426950408889634);
  if (!std::isfinite(p.scale_log2)) return PA_ERR_INVALID_ARG;
  int sms = 0;
  if ((st = pa::device_state(&p.err, &sms)) != PA_OK) return st;
  size_t need = 0;
  if ((st = pa_decode_fp4_workspace_size(desc, num_heads, &need)) != PA_OK) return st;
  buffers[1].bytes = (int64_t)need;
  if (workspace_bytes < need || conflict(buffers)) return PA_ERR_INVALID_ARG;
  p.out = out;
  p.query = query;
  p.cache = static_cast<const uint8_t*>(cache);
  p.block_tables = block_tables;
  p.seq_lens = seq_lens;
  p.query_stride = query_stride;
  p.value_scale = value_scale;
  p.num_blocks = desc->num_blocks;
  p.log2_block_size = ilog2(desc->block_size);
  p.num_kv_heads = desc->num_kv_heads;
  p.head_size = desc->head_size;
  p.num_heads = num_heads;
  p.num_seqs = num_seqs;
  p.group = num_heads / desc->num_kv_heads;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.wait_limit = pa::decode_wait_limit();
  return cuda_status(
      pa::launch_decode_fp4(p, workspace, dtype, sms, static_cast<cudaStream_t>(stream)));
}

pa_status pa_extend_tables(int32_t* block_tables, int32_t max_blocks_per_seq,
                           const int32_t* seq_lens, const int32_t* new_tokens, int32_t num_seqs,
                           int32_t block_size, int32_t num_blocks, const int32_t* free_blocks,
                           int32_t free_capacity, const int32_t* free_state,
                           int32_t* seq_lens_out, int32_t* free_state_out, int64_t* slot_mapping,
                           int32_t* positions, int32_t* token_starts, int32_t max_tokens,
                           void* stream) {
  if (num_seqs < 0 || num_seqs > PA_MAX_TABLE_REQUESTS || max_blocks_per_seq < 1 ||
      !is_pow2(block_size) || block_size > 256 || num_blocks < 1 || max_tokens < 0 ||
      max_tokens > PA_MAX_TABLE_TOKENS)
    return PA_ERR_INVALID_ARG;
  const bool ring = free_blocks || free_state || free_state_out || free_capacity != 0;
  if (ring && (!free_blocks || !free_state || !free_state_out || free_capacity < 1 ||
               free_capacity > (1 << 30) || !aligned(free_blocks, 4) || !aligned(free_state, 4) ||
               !aligned(free_state_out, 4)))
    return PA_ERR_INVALID_ARG;
  if (num_seqs > 0 && (!block_tables || !seq_lens || !new_tokens || !seq_lens_out ||
                       !aligned(block_tables, 4) || !aligned(seq_lens, 4) ||
                       !aligned(new_tokens, 4) || !aligned(seq_lens_out, 4)))
    return PA_ERR_INVALID_ARG;
  if ((max_tokens > 0 && !slot_mapping) || !aligned(slot_mapping, 8) || !aligned(positions, 4) ||
      !aligned(token_starts, 4))
    return PA_ERR_INVALID_ARG;
  // Lengths and the ring's state may be written in place; nothing else may overlap
  // what the step writes.
  const int64_t n = num_seqs;
  const Range buffers[] = {{block_tables, n * max_blocks_per_seq * 4, true},
                           {seq_lens_out, n * 4, true},
                           {free_state_out, 8, true},
                           {slot_mapping, max_tokens * 8ll, true},
                           {positions, max_tokens * 4ll, true},
                           {token_starts, (n + 1) * 4, true},
                           {seq_lens, n * 4, false},
                           {free_state, 8, false},
                           {new_tokens, n * 4, false},
                           {free_blocks, free_capacity * 4ll, false}};
  constexpr int kBuffers = sizeof buffers / sizeof buffers[0];
  for (int i = 0; i < kBuffers && buffers[i].written; ++i)
    for (int j = i + 1; j < kBuffers; ++j) {
      const bool in_place = ((i == 1 && j == 6) || (i == 2 && j == 7)) &&
                            buffers[i].p == buffers[j].p;
      if (!in_place && overlap(buffers[i], buffers[j])) return PA_ERR_INVALID_ARG;
    }
  pa::TablesParams p = {};
  int sms = 0;
  pa_status st = pa::device_state(&p.err, &sms);
  if (st != PA_OK) return st;
  p.in_place = seq_lens_out == seq_lens || (ring && free_state_out == free_state);
  p.block_tables = block_tables;
  p.seq_lens = seq_lens;
  p.new_tokens = new_tokens;
  p.free_blocks = free_blocks;
  p.free_state = free_state;
  p.seq_lens_out = seq_lens_out;
  p.free_state_out = free_state_out;
  p.slot_mapping = slot_mapping;
  p.positions = positions;
  p.token_starts = token_starts;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.num_seqs = num_seqs;
  p.log2_block_size = ilog2(block_size);
  p.num_blocks = num_blocks;
  p.free_capacity = free_capacity;
  p.max_tokens = max_tokens;
  return cuda_status(pa::launch_extend_tables(p, sms, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
