// Arguments of the decode attention over a 4-bit pool (see pa_decode_fp4),
// and the sizes that its launch and its workspace share.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace pa {

constexpr int kFp4Step = 32;           // tokens that a warp computes at a time

// Tokens of a stage, the unit of copies, waits and of the work's division: 64 where
// heads are small, whose steps are short beside what comes with each stage (8 x 32768
// tokens, 8 KV heads of 64, groups of four and eight: 41.7 and 44.5 us, 45.2 and 47.2
// with 32).  At 128 and 256, 64 would leave rings of one stage or none.
__host__ __device__ constexpr int fp4_stage(int head_size) { return head_size == 64 ? 64 : 32; }

constexpr int kFp4Gather = 16;         // parts that are merged at once
constexpr int kFp4MaxCtas = kFp4Gather * kFp4Gather;
constexpr int kFp4Units = 32;          // units of a pair that are merged by themselves
constexpr int kFp4HeaderBytes = kFp4MaxCtas * 3 * kFp4Units * 4;  // three counters per CTA and unit

// Query heads of a unit of work (columns of the matrix instructions): 4, 8, or
// 16 where the registers hold them; groups past eight heads of 256 elements read
// the keys and values once per eight heads.  Up to four heads use the eight columns
// twice (8 x 32768 tokens, heads of 128: 59 us, 63 us as eight heads; fp32 88 and 90;
// a decode step of 128 sequences 74 and 78).  Sixteen heads of 128 take 99 us where
// eight take 65, so twice eight would take 130 (fp32 142 and 185; of 64, 59 and 90).
__host__ __device__ constexpr int fp4_heads(int head_size, int group) {
  return group <= 4 ? 4 : group <= 8 || head_size == 256 ? 8 : 16;
}

// Warps of a CTA (one CTA per SM): 16 where a thread's accumulators, query fragments and
// weight fragments leave room in 128 registers, else 8.  Left of the bound 16 warps hide
// each other's waits (8 x 32768 tokens, four heads of 128: 59 us, 74 us with 8 warps;
// sixteen heads of 64: 58 and 67, although a few registers spill), right of it what
// spills is read again in every step (four heads of 128, fp32: 88 us, 83 to 137 with 16,
// by where the compiler spills; eight: 92 and 170; sixteen, bf16: 99 and 174; at 256 the
// rings would not fit).  With 8 warps sixteen heads of 128 and eight of 256 spill in fp32,
// 40 and 16 bytes a thread.
__host__ __device__ constexpr int fp4_warps(int head_size, int heads, bool fp32) {
  const int parts = fp32 ? 2 : 1;
  const int accumulators = heads == 4 ? head_size / 8 : head_size / 32 * heads;
  const int queries = head_size / 8 * (heads == 16 ? 2 : 1) * parts;
  const int weights = (heads == 4 ? 8 : heads / 2) * parts;
  return accumulators + queries + weights <= 56 ? 16 : 8;
}

// Rows (query heads) of a pair; the units of a head that are merged by
// themselves; and the floats of a partial result: weighted values, then each
// unit's maximum, then each unit's sum (units are handed on one by one, so each
// has its own).
__host__ __device__ constexpr int fp4_unit_rows(int heads, int group) {
  return group < heads ? group : heads;
}
__host__ __device__ constexpr int fp4_splits(int head_size, int rows, int warps) {
  return head_size > 64 && 2 * rows <= warps ? 2 : 1;
}
__host__ __device__ constexpr int fp4_partial_floats(int rows, int head_size, int splits) {
  return (rows * (head_size + 2 * splits) + 3) / 4 * 4;
}

// Floats of a warp's ended chains of sums: for each of a lane's columns (two per tile of
// eight, which four heads use twice) its maximum, its sum and its weighted values.
__host__ __device__ constexpr int fp4_chain_floats(int head_size, int heads) {
  return heads == 4 ? 32 * 2 * (head_size / 16 + 2) : 32 * 2 * (heads / 8) * (head_size / 8 + 2);
}

struct Fp4DecodeParams {
  void* out;
  const void* query;
  const uint8_t* cache;
  const int32_t* block_tables;
  const int32_t* seq_lens;
  unsigned int* err;
  unsigned int* counters;  // [CTAs][3][kFp4Units], zero between calls
  float* warp_partials;    // [CTAs][warps][partial]
  float* cta_partials;     // [CTAs][4][partial]: of CTAs, then of groups of CTAs
  float* chains;           // [CTAs][warps][fp4_chain_floats]
  long long wait_limit;
  int64_t query_stride;
  float scale_log2;   // scale * key_scale * log2(e)
  float value_scale;
  int num_blocks, log2_block_size, num_kv_heads, head_size, num_heads, num_seqs, group;
  int max_blocks_per_seq;
};

}  // namespace pa
