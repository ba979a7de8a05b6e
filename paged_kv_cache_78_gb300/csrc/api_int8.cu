// C entry points of the 8-bit pool, of the eviction and of the norms with rotation:
// argument checks and launches.  See include/pa.h for the contract.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "api_checks.h"
#include "decode_int8.cuh"
#include "evict_blocks.cuh"
#include "pa.h"
#include "pa_int8.cuh"
#include "pa_launch.h"

namespace {

using namespace pa;

constexpr int kInt8MaxGroup = 16;

pa_status check_call(const pa_cache_desc* desc, int32_t dtype) {
  const pa_status st = pa::check_int8_desc(desc);
  if (st != PA_OK) return st;
  return dtype_ok(dtype) ? PA_OK : PA_ERR_INVALID_ARG;
}

int64_t pool_bytes(const pa_cache_desc* d) { return d->num_blocks * pa::int8_block_bytes(d); }

pa::Int8Pool pool_of(const void* cache, const pa_cache_desc* d) {
  pa::Int8Pool p;
  p.cache = static_cast<uint8_t*>(const_cast<void*>(cache));
  p.num_slots = (int64_t)d->num_blocks * d->block_size;
  p.num_kv_heads = d->num_kv_heads;
  p.head_size = d->head_size;
  p.log2_block_size = ilog2(d->block_size);
  return p;
}

// One grid holds the call: a CTA per eight tokens and two heads, or more (read-back), or
// per eight heads and sides of 32 tokens (write).
bool grid_ok(const pa_cache_desc* d, int64_t num_tokens) {
  return (num_tokens + 7) / 8 * d->num_kv_heads < (1ll << 31);
}

// Tables whose blocks' weights are kept: 32 bits count their entries (and 64 the bytes of the
// workspace: 2^32 entries of up to 16 cells, 2^20 heads, 8 bytes).
bool tables_ok(int64_t num_seqs, int64_t max_blocks) { return num_seqs * max_blocks < (1ll << 32); }

}  // namespace

namespace pa {

pa_status check_int8_desc(const pa_cache_desc* d) {
  if (!d || d->dtype != PA_INT8) return PA_ERR_INVALID_ARG;
  if (d->num_blocks < 1 || d->num_kv_heads < 1 || d->head_size < 1) return PA_ERR_INVALID_ARG;
  if (!is_pow2(d->block_size) || d->block_size < 8 || d->block_size > 256)
    return PA_ERR_INVALID_ARG;
  if (d->head_size != 64 && d->head_size != 128 && d->head_size != 256) return PA_ERR_UNSUPPORTED;
  if (d->num_kv_heads > 65535 || int8_block_bytes(d) > 0x7fffffff) return PA_ERR_UNSUPPORTED;
  return PA_OK;
}

int64_t int8_block_bytes(const pa_cache_desc* d) {
  return (int64_t)d->num_kv_heads * (d->block_size / kInt8Tile) * int8_tile_bytes(d->head_size);
}

}  // namespace pa

extern "C" {

pa_status pa_reshape_and_cache_int8(void* cache, const pa_cache_desc* desc, const void* key,
                                    const void* value, int32_t dtype, int64_t key_stride,
                                    int64_t value_stride, const int64_t* slot_mapping,
                                    int32_t num_tokens, void* stream) {
  pa_status st = check_call(desc, dtype);
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
  int sms = 0;
  if ((st = pa::device_state(&err, &sms)) != PA_OK) return st;
  return cuda_status(pa::launch_int8_write(pool_of(cache, desc), key, value, dtype, key_stride,
                                           value_stride, slot_mapping, num_tokens, sms, err,
                                           static_cast<cudaStream_t>(stream)));
}

pa_status pa_gather_cache_int8(void* key, void* value, int32_t dtype, const void* cache,
                               const pa_cache_desc* desc, const int64_t* slot_mapping,
                               int32_t num_tokens, void* stream) {
  pa_status st = check_call(desc, dtype);
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
  return cuda_status(pa::launch_int8_gather(pool_of(cache, desc), key, value, dtype, slot_mapping,
                                            num_tokens, err, static_cast<cudaStream_t>(stream)));
}

pa_status pa_decode_int8_workspace_size(const pa_cache_desc* desc, int32_t num_heads,
                                        int32_t num_seqs, int32_t max_blocks_per_seq,
                                        size_t* bytes) {
  pa_status st = pa::check_int8_desc(desc);
  if (st != PA_OK) return st;
  if (!bytes || num_heads < 1 || num_heads % desc->num_kv_heads != 0 || num_seqs < 0 ||
      num_seqs > 65535 || max_blocks_per_seq < 0)
    return PA_ERR_INVALID_ARG;
  if (num_heads / desc->num_kv_heads > kInt8MaxGroup || !tables_ok(num_seqs, max_blocks_per_seq))
    return PA_ERR_UNSUPPORTED;
  int sms = 0;
  if ((st = pa::device_state(nullptr, &sms)) != PA_OK) return st;
  if (sms > pa::kInt8MaxCtas) return PA_ERR_UNSUPPORTED;
  *bytes = pa::decode_int8_workspace_bytes(desc->head_size, num_heads,
                                           num_heads / desc->num_kv_heads, desc->block_size,
                                           num_seqs, num_seqs ? max_blocks_per_seq : 0, sms);
  return PA_OK;
}

pa_status pa_decode_int8(void* out, const void* query, int32_t dtype, int64_t query_stride,
                         const void* cache, const pa_cache_desc* desc,
                         const int32_t* block_tables, int32_t max_blocks_per_seq,
                         const int32_t* seq_lens, int32_t num_seqs, int32_t num_heads,
                         float scale, const float* block_weights, float* block_weights_out,
                         float decay, void* workspace, size_t workspace_bytes, void* stream) {
  pa_status st = check_call(desc, dtype);
  if (st != PA_OK) return st;
  if (num_seqs < 0 || num_seqs > 65535 || max_blocks_per_seq < 1 || !std::isfinite(scale) ||
      !std::isfinite(decay) || (block_weights && !block_weights_out))
    return PA_ERR_INVALID_ARG;
  if (num_heads < 1 || num_heads % desc->num_kv_heads != 0) return PA_ERR_INVALID_ARG;
  if (num_heads / desc->num_kv_heads > kInt8MaxGroup || (int64_t)num_seqs * num_heads >= (1ll << 31) ||
      (block_weights_out && !tables_ok(num_seqs, max_blocks_per_seq)))
    return PA_ERR_UNSUPPORTED;
  if (num_seqs == 0) return PA_OK;
  const int64_t row = (int64_t)num_heads * desc->head_size;
  if (!out || !query || !cache || !block_tables || !seq_lens || !workspace ||
      !aligned(workspace, 256) || !aligned(out, 16) || !aligned(query, 16) || !aligned(cache, 16) ||
      !aligned(block_tables, 4) || !aligned(seq_lens, 4) || !aligned(block_weights, 4) ||
      !aligned(block_weights_out, 4) || !stride_ok(query_stride, row, dtype))
    return PA_ERR_INVALID_ARG;
  const int64_t entries = (int64_t)num_seqs * max_blocks_per_seq * 4;
  // The workspace, whose size needs the device, is looked at below.
  Range buffers[] = {{out, num_seqs * row * elem_bytes(dtype), true},
                     {workspace, 0, true},
                     {block_weights_out, entries, true},
                     {query, rows_bytes(num_seqs, query_stride, row, dtype), false},
                     {cache, pool_bytes(desc), false},
                     {block_tables, entries, false},
                     {seq_lens, num_seqs * 4ll, false},
                     {block_weights == block_weights_out ? nullptr : block_weights, entries, false}};
  if (conflict(buffers)) return PA_ERR_INVALID_ARG;
  pa::Int8DecodeParams p = {};
  p.scale_log2 = (float)((double)scale * 1.4426950408889634);
  if (!std::isfinite(p.scale_log2)) return PA_ERR_INVALID_ARG;
  int sms = 0;
  if ((st = pa::device_state(&p.err, &sms)) != PA_OK) return st;
  size_t need = 0;
  if ((st = pa_decode_int8_workspace_size(desc, num_heads, block_weights_out ? num_seqs : 0,
                                          max_blocks_per_seq, &need)) != PA_OK)
    return st;
  buffers[1].bytes = (int64_t)need;
  if (workspace_bytes < need || conflict(buffers)) return PA_ERR_INVALID_ARG;
  p.out = out;
  p.query = query;
  p.cache = static_cast<const uint8_t*>(cache);
  p.block_tables = block_tables;
  p.seq_lens = seq_lens;
  p.block_weights = block_weights;
  p.block_weights_out = block_weights_out;
  p.decay = decay;
  p.query_stride = query_stride;
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
      pa::launch_decode_int8(p, workspace, dtype, sms, static_cast<cudaStream_t>(stream)));
}

pa_status pa_evict_blocks(const int32_t* block_tables, const float* block_weights,
                          int32_t max_blocks_per_seq, const int32_t* seq_lens, int32_t num_seqs,
                          int32_t block_size, int32_t max_blocks, int32_t keep_first,
                          int32_t keep_last, int32_t* free_blocks, int32_t free_capacity,
                          const int32_t* free_state, const int32_t* evicted_tokens,
                          int32_t* block_tables_out, float* block_weights_out,
                          int32_t* seq_lens_out, int32_t* free_state_out,
                          int32_t* evicted_tokens_out, void* stream) {
  if (num_seqs < 0 || num_seqs > PA_MAX_TABLE_REQUESTS || max_blocks_per_seq < 1 ||
      max_blocks_per_seq > PA_MAX_EVICT_BLOCKS || !is_pow2(block_size) || block_size > 256 ||
      keep_first < 0 || keep_last < 1 || (int64_t)keep_first + keep_last > max_blocks)
    return PA_ERR_INVALID_ARG;
  const bool ring = free_blocks || free_state || free_state_out || free_capacity != 0;
  if (ring && (!free_blocks || !free_state || !free_state_out || free_capacity < 1 ||
               free_capacity > (1 << 30) || !aligned(free_blocks, 4) || !aligned(free_state, 4) ||
               !aligned(free_state_out, 4)))
    return PA_ERR_INVALID_ARG;
  if (!evicted_tokens != !evicted_tokens_out || !aligned(evicted_tokens, 4) ||
      !aligned(evicted_tokens_out, 4))
    return PA_ERR_INVALID_ARG;
  if (num_seqs == 0) {
    // The state after a call that does nothing is the state before it.
    if (free_state_out == free_state) return PA_OK;
  } else if (!block_tables || !block_weights || !seq_lens || !block_tables_out ||
             !block_weights_out || !seq_lens_out || !aligned(block_tables, 4) ||
             !aligned(block_weights, 4) || !aligned(seq_lens, 4) || !aligned(block_tables_out, 4) ||
             !aligned(block_weights_out, 4) || !aligned(seq_lens_out, 4)) {
    return PA_ERR_INVALID_ARG;
  }
  const int64_t n = num_seqs, entries = n * max_blocks_per_seq * 4;
  // Each output may be its input, six places behind it; nothing else may overlap what the
  // call writes.
  const Range buffers[] = {{block_tables_out, entries, true}, {block_weights_out, entries, true},
                           {seq_lens_out, n * 4, true},       {free_state_out, 8, true},
                           {evicted_tokens_out, n * 4, true}, {free_blocks, free_capacity * 4ll, true},
                           {block_tables, entries, false},    {block_weights, entries, false},
                           {seq_lens, n * 4, false},          {free_state, 8, false},
                           {evicted_tokens, n * 4, false}};
  constexpr int kBuffers = sizeof buffers / sizeof buffers[0];
  for (int i = 0; i < kBuffers && buffers[i].written; ++i)
    for (int j = i + 1; j < kBuffers; ++j) {
      const bool in_place = j == i + 6 && buffers[i].p == buffers[j].p;
      if (!in_place && overlap(buffers[i], buffers[j])) return PA_ERR_INVALID_ARG;
    }
  pa::EvictParams p = {};
  int sms = 0;
  const pa_status st = pa::device_state(&p.err, &sms);
  if (st != PA_OK) return st;
  p.block_tables = block_tables;
  p.block_weights = block_weights;
  p.seq_lens = seq_lens;
  p.free_state = free_state;
  p.evicted_tokens = evicted_tokens;
  p.free_blocks = free_blocks;
  p.block_tables_out = block_tables_out;
  p.block_weights_out = block_weights_out;
  p.seq_lens_out = seq_lens_out;
  p.free_state_out = free_state_out;
  p.evicted_tokens_out = evicted_tokens_out;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.num_seqs = num_seqs;
  p.log2_block_size = ilog2(block_size);
  p.free_capacity = free_capacity;
  p.max_blocks = max_blocks;
  p.keep_first = keep_first;
  p.keep_last = keep_last;
  return cuda_status(pa::launch_evict_blocks(p, sms, static_cast<cudaStream_t>(stream)));
}

pa_status pa_norm_rope(const pa_norm_rope_args* args, void* stream) {
  if (!args) return PA_ERR_INVALID_ARG;
  const pa_norm_rope_args& a = *args;
  if (!dtype_ok(a.dtype) || a.num_tokens < 0 || a.num_heads < 1 || a.num_kv_heads < 1 ||
      a.head_size < 1 || !std::isfinite(a.eps) || a.eps < 0.f ||
      (a.interleaved != 0 && a.interleaved != 1))
    return PA_ERR_INVALID_ARG;
  if (a.head_size != 64 && a.head_size != 128 && a.head_size != 256) return PA_ERR_UNSUPPORTED;
  if (a.rotary_dim < 0 || a.rotary_dim > a.head_size || a.rotary_dim % 16 != 0 ||
      (a.rotary_dim > 0 && (a.max_position < 1 || !a.cos_sin)))
    return PA_ERR_INVALID_ARG;
  const int64_t heads = (int64_t)a.num_heads + a.num_kv_heads;
  // A token's heads fit an int, all tokens' 32 bits.
  if (heads > (1 << 20) || a.num_tokens * heads >= (1ll << 32)) return PA_ERR_UNSUPPORTED;
  if (a.num_tokens == 0) return PA_OK;
  const int64_t n = a.num_tokens;
  const int64_t q_row = (int64_t)a.num_heads * a.head_size, k_row = (int64_t)a.num_kv_heads * a.head_size;
  if (!a.query_out || !a.key_out || !a.query || !a.key || !a.positions || !aligned(a.query_out, 16) ||
      !aligned(a.key_out, 16) || !aligned(a.query, 16) || !aligned(a.key, 16) ||
      !aligned(a.query_weight, 16) || !aligned(a.key_weight, 16) || !aligned(a.cos_sin, 16) ||
      !aligned(a.positions, 4) || !aligned(a.position_offsets, 4) ||
      !stride_ok(a.query_out_stride, q_row, a.dtype) || !stride_ok(a.query_stride, q_row, a.dtype) ||
      !stride_ok(a.key_out_stride, k_row, a.dtype) || !stride_ok(a.key_stride, k_row, a.dtype))
    return PA_ERR_INVALID_ARG;
  // Rows may lie between one another's (query and key of one projection); whether they
  // overlap is a question of their places in a common stride then.
  struct Rows {
    const void* p;
    int64_t stride, row;
    bool written;
  };
  const int64_t elem = elem_bytes(a.dtype);
  const Rows rows[] = {{a.query_out, a.query_out_stride * elem, q_row * elem, true},
                       {a.key_out, a.key_out_stride * elem, k_row * elem, true},
                       {a.query, a.query_stride * elem, q_row * elem, false},
                       {a.key, a.key_stride * elem, k_row * elem, false}};
  auto apart = [&](const Rows& x, const Rows& y) {
    if (!overlap({x.p, (n - 1) * x.stride + x.row, true}, {y.p, (n - 1) * y.stride + y.row, true}))
      return true;
    if (x.stride != y.stride || n == 1) return false;
    const int64_t d = reinterpret_cast<intptr_t>(y.p) - reinterpret_cast<intptr_t>(x.p);
    const int64_t m = ((d % x.stride) + x.stride) % x.stride;  // y's place in x's row
    return m >= x.row && m + y.row <= x.stride;
  };
  for (int i = 0; i < 4 && rows[i].written; ++i)
    for (int j = i + 1; j < 4; ++j) {
      const bool in_place = j == i + 2 && rows[i].p == rows[j].p && rows[i].stride == rows[j].stride;
      if (!in_place && !apart(rows[i], rows[j])) return PA_ERR_INVALID_ARG;
    }
  const Range read[] = {{a.query_weight, a.head_size * elem, false},
                        {a.key_weight, a.head_size * elem, false},
                        {a.cos_sin, (int64_t)a.max_position * a.rotary_dim * 4, false},
                        {a.positions, n * 4, false},
                        {a.position_offsets, n * 4, false}};
  for (int i = 0; i < 2; ++i)
    for (const Range& r : read)
      if (overlap({rows[i].p, (n - 1) * rows[i].stride + rows[i].row, true}, r)) return PA_ERR_INVALID_ARG;
  unsigned int* err = nullptr;
  int sms = 0;
  const pa_status st = pa::device_state(&err, &sms);
  if (st != PA_OK) return st;
  return cuda_status(pa::launch_norm_rope(a, sms, err, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
