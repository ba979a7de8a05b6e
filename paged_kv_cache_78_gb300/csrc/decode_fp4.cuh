// Arguments of the decode attention over a 4-bit pool (see pa_decode_fp4).
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace pa {

struct Fp4DecodeParams {
  void* out;
  const void* query;
  const uint8_t* cache;
  const int32_t* block_tables;
  const int32_t* seq_lens;
  unsigned int* err;
  int64_t query_stride;
  float scale_log2;   // scale * key_scale * log2(e)
  float value_scale;
  int num_blocks, log2_block_size, num_kv_heads, head_size, num_heads, num_seqs, group;
  int max_blocks_per_seq;
};

}  // namespace pa
