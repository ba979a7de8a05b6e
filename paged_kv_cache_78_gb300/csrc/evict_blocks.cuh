// Arguments of the eviction (see pa_evict_blocks).
#pragma once

#include <stdint.h>

namespace pa {

struct EvictParams {
  const int32_t* block_tables;
  const float* block_weights;
  const int32_t* seq_lens;
  const int32_t* free_state;      // NULL: no ring
  const int32_t* evicted_tokens;  // may be NULL
  int32_t* free_blocks;
  int32_t* block_tables_out;
  float* block_weights_out;
  int32_t* seq_lens_out;
  int32_t* free_state_out;
  int32_t* evicted_tokens_out;
  unsigned int* err;
  bool alone;  // the rows' launch writes lengths and ring state, as nothing that is read is written
  int max_blocks_per_seq, num_seqs, log2_block_size, free_capacity;
  int max_blocks, keep_first, keep_last;
};

}  // namespace pa
