// Arguments of the table extension (see pa_extend_tables).
#pragma once

#include <stdint.h>

namespace pa {

struct TablesParams {
  int32_t* block_tables;
  const int32_t* seq_lens;
  const int32_t* new_tokens;
  const int32_t* free_blocks;  // NULL: the tables hold every block already
  const int32_t* free_state;
  int32_t* seq_lens_out;
  int32_t* free_state_out;
  int64_t* slot_mapping;
  int32_t* positions;     // may be NULL
  int32_t* token_starts;  // may be NULL
  unsigned int* err;
  bool in_place;  // an output is its input: the CTAs are one cluster
  int max_blocks_per_seq, num_seqs, log2_block_size, num_blocks, free_capacity, max_tokens;
};

}  // namespace pa
