// Arguments of the decode attention over an 8-bit pool (see pa_decode_int8), and the sizes
// that its launch and its workspace share.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace pa {

constexpr int kInt8MostWarps = 16;      // of a CTA; one CTA per SM
constexpr int kInt8Gather = 16;         // parts that are merged at once
constexpr int kInt8MaxCtas = kInt8Gather * kInt8Gather;
constexpr int kInt8Rows = 16;           // heads of a unit at most, each merged by itself
// Counters; then, in the header's last words, what keeps the blocks' weights from being added up: the
// call was refused on the device (each call writes it), a wait of it gave up (set by the warp, cleared
// by the sums' launch), and how many CTAs of that launch have seen the latter.
constexpr int kInt8HeaderBytes = kInt8MaxCtas * 3 * kInt8Rows * 4 + 256;
constexpr int kInt8Refused = kInt8HeaderBytes / 4 - 1;
constexpr int kInt8GaveUp = kInt8HeaderBytes / 4 - 2;
constexpr int kInt8Seen = kInt8HeaderBytes / 4 - 3;

// Warps of a CTA: 16 where a thread's accumulators and query fragments leave room in 128
// registers, which hide each other's waits (with 8, 64 sequences of up to 2048 tokens with weights and
// heads of 64 take 10% longer, fp32 14%, 8 x 32768 tokens of 128 with weights 3%), else 8.
// But 8 for heads of 128 where no weights are kept: they copy 8 KB at a time, not 4, which the
// memory gives faster (with 16, 8 x 32768 tokens take 2% longer, 384 x 1500 4%), and for
// fp32 of 128 (8%), whose registers would spill.
__host__ __device__ constexpr int int8_warps(int head_size, int heads, bool fp32, bool weights) {
  return head_size == 64 ? (heads == 16 && fp32 ? 8 : 16)
                         : head_size == 128 && heads == 8 && !fp32 && weights ? 16 : 8;
}
// Tokens of a stage, the unit of copies, waits and of the work's division: 4 or 8 KB of codes.
__host__ __device__ constexpr int int8_stage(int head_size, int warps) {
  return (warps == 16 ? 2048 : 4096) / head_size;
}
// Tokens that a warp computes at a time.
__host__ __device__ constexpr int int8_step(int head_size, int warps) {
  return int8_stage(head_size, warps) < 32 ? 16 : 32;
}

// Query heads of a unit of work (columns of the matrix instructions): 8, or 16 where the
// registers hold them (16 heads of 128 take 13% longer than eight, not twice as long);
// groups past eight heads of 256 elements read the keys and values once per eight heads.
__host__ __device__ constexpr int int8_heads(int head_size, int group) {
  return group <= 8 || head_size == 256 ? 8 : 16;
}
// Rows (query heads) of a pair, and the floats of a partial result: weighted values, then
// each row's maximum, sum and value scale (rows are handed on one by one).
__host__ __device__ constexpr int int8_unit_rows(int heads, int group) {
  return group < heads ? group : heads;
}
__host__ __device__ constexpr int int8_partial_floats(int rows, int head_size) {
  return (rows * (head_size + 3) + 3) / 4 * 4;
}
// Floats of a warp's ended chains of sums: for each of a lane's columns (two per tile of
// eight) its maximum, sum and weighted values; and the value scale.
__host__ __device__ constexpr int int8_chain_floats(int head_size, int heads) {
  return 32 * (2 * (heads / 8) * (head_size / 8 + 2) + 1);
}

// Tokens of a cell, whose weight is handed on for the blocks' sums.
__host__ __device__ constexpr int int8_log2_cell(int log2_block_size) {
  return log2_block_size < 4 ? log2_block_size : 4;
}

struct Int8DecodeParams {
  void* out;
  const void* query;
  const uint8_t* cache;
  const int32_t* block_tables;
  const int32_t* seq_lens;
  const float* block_weights;  // may be NULL
  float* block_weights_out;    // NULL: no weights
  unsigned int* err;
  unsigned int* counters;  // [CTAs][3][kInt8Rows], zero between calls; the header's last words
  float* warp_partials;    // [CTAs][warps][partial]
  float* cta_partials;     // [CTAs][4][partial]: of CTAs, then of groups of CTAs
  float* chains;           // [CTAs][warps][int8_chain_floats]
  float2* rows;            // [num_seqs][num_heads]: maximum and sum
  float2* cells;           // [num_seqs][cells][num_heads]: sum of weights, and their maximum
  long long wait_limit;
  int64_t query_stride;
  float scale_log2;  // scale * log2(e)
  float decay;
  int num_blocks, log2_block_size, num_kv_heads, head_size, num_heads, num_seqs, group;
  int max_blocks_per_seq;
};

}  // namespace pa
