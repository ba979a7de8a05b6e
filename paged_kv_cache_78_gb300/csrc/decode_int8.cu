// Dispatch of the 8-bit decode over element types and head sizes, its workspace, and the
// sums of the blocks' weights.
#include "decode_int8.cuh"
#include "pa_device.cuh"
#include "pa_launch.h"

namespace pa {

cudaError_t launch_decode_int8_bf16_d64(const Int8DecodeParams&, int num_sms, cudaStream_t);
cudaError_t launch_decode_int8_bf16_d128(const Int8DecodeParams&, int num_sms, cudaStream_t);
cudaError_t launch_decode_int8_bf16_d256(const Int8DecodeParams&, int num_sms, cudaStream_t);
cudaError_t launch_decode_int8_f32_d64(const Int8DecodeParams&, int num_sms, cudaStream_t);
cudaError_t launch_decode_int8_f32_d128(const Int8DecodeParams&, int num_sms, cudaStream_t);
cudaError_t launch_decode_int8_f32_d256(const Int8DecodeParams&, int num_sms, cudaStream_t);

namespace {

// What follows the header, in floats, each part a multiple of 64 (256 bytes).
struct Layout {
  size_t warps, ctas, chains, rows, cells;
};
size_t up(size_t floats) { return (floats + 63) / 64 * 64; }
Layout layout(int head_size, int num_heads, int group, int log2_block_size, size_t num_seqs,
              size_t max_blocks, int num_sms) {
  const int heads = int8_heads(head_size, group);
  const size_t part = int8_partial_floats(int8_unit_rows(heads, group), head_size);
  Layout l;
  l.warps = up(num_sms * kInt8MostWarps * part);
  l.ctas = up(num_sms * 4 * part);
  l.chains = up((size_t)num_sms * kInt8MostWarps * int8_chain_floats(head_size, heads));
  const size_t cells = (max_blocks << log2_block_size) >> int8_log2_cell(log2_block_size);
  l.rows = max_blocks ? up(num_seqs * num_heads * 2) : 0;
  l.cells = up(num_seqs * cells * num_heads * 2);
  return l;
}

// A block's weight: the sum over heads and cells of weights / the row's sum, at the row's
// maximum.  A warp takes a block, lanes the heads, so that a cell's are read in one piece;
// 8 bytes per cell and head, written by the decode's kernel just before.  Which of the tables' entries
// are blocks is known from the lengths: a warp looks at 32 of its entries at once, a lane each, and
// goes on with those that are there, so that the width of a table costs a length per entry, 32 at a
// time, and no cell is read but the sequences' own.
__global__ void __launch_bounds__(256) block_weights_kernel(const Int8DecodeParams p) {
  const int lane = threadIdx.x & 31;
  const unsigned warps = gridDim.x * (blockDim.x / 32), width = (unsigned)p.max_blocks_per_seq;
  const int l2bs = p.log2_block_size, l2cell = int8_log2_cell(l2bs);
  const int per_block = 1 << (l2bs - l2cell);
  const int64_t cells = (int64_t)p.max_blocks_per_seq * per_block;
  const unsigned blocks = (unsigned)p.num_seqs * width;  // below 2^32
  grid_dependents_launch();
  grid_dependency_wait();
  const uint2 state = *reinterpret_cast<const uint2*>(p.counters + kInt8GaveUp);  // gave up, refused
  for (uint64_t at0 = blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32; at0 < blocks; at0 += 32ull * warps) {
    const uint64_t mine = at0 + (uint64_t)lane * warps;
    unsigned my_s = 0;
    int my_b = 0, my_len = 0;
    bool there = false;
    if (mine < blocks) {
      my_s = (unsigned)mine / width;
      my_b = (int)((unsigned)mine - my_s * width);
      my_len = p.seq_lens[my_s];
      there = !(state.x | state.y) && my_len > 0 && (my_len - 1) >> l2bs < p.max_blocks_per_seq &&
              my_b <= (my_len - 1) >> l2bs;
    }
    for (uint32_t left = __ballot_sync(0xffffffffu, there); left; left &= left - 1) {
      const int i = __ffs(left) - 1;
      const unsigned s = __shfl_sync(0xffffffffu, my_s, i), at = (unsigned)at0 + i * warps;
      const int b = __shfl_sync(0xffffffffu, my_b, i), len = __shfl_sync(0xffffffffu, my_len, i);
      const float old = p.block_weights ? p.block_weights[at] : 0.f;
      const float2* row = p.rows + (size_t)s * p.num_heads;
      const float2* cell = p.cells + (s * cells + (int64_t)b * per_block) * p.num_heads;
      const int n = min(per_block, ((len - 1) >> l2cell) + 1 - b * per_block);
      float sum = 0.f;
      for (int h = lane; h < p.num_heads; h += 32) {
        const float2 r = row[h], v = cell[h];
        float weight = v.x * fast_exp2(v.y - r.x);
        for (int c = 1; c < n; ++c) {
          const float2 u = cell[(size_t)c * p.num_heads + h];
          weight = fmaf(u.x, fast_exp2(u.y - r.x), weight);
        }
        sum += __fdiv_rn(weight, r.y);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (lane == 0) p.block_weights_out[at] = fmaf(p.decay, old, sum);
    }
  }
  if (state.x) {
    // The next call's weights are added up again: the last CTA that has seen the word clears it.
    __syncthreads();
    if (threadIdx.x == 0 && atomicAdd(p.counters + kInt8Seen, 1u) == gridDim.x - 1) {
      p.counters[kInt8Seen] = 0u;
      p.counters[kInt8GaveUp] = 0u;
    }
  }
}

}  // namespace

size_t decode_int8_workspace_bytes(int head_size, int num_heads, int group, int block_size,
                                   int64_t num_seqs, int64_t max_blocks, int num_sms) {
  int l2bs = 0;
  while ((1 << l2bs) < block_size) ++l2bs;
  const Layout l = layout(head_size, num_heads, group, l2bs, (size_t)num_seqs, (size_t)max_blocks,
                          num_sms);
  return kInt8HeaderBytes + 4 * (l.warps + l.ctas + l.chains + l.rows + l.cells);
}

cudaError_t launch_decode_int8(const Int8DecodeParams& params, void* workspace, int dtype,
                               int num_sms, cudaStream_t stream) {
  Int8DecodeParams p = params;
  const Layout l = layout(p.head_size, p.num_heads, p.group, p.log2_block_size, p.num_seqs,
                          p.block_weights_out ? p.max_blocks_per_seq : 0, num_sms);
  p.counters = static_cast<unsigned int*>(workspace);
  p.warp_partials = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kInt8HeaderBytes);
  p.cta_partials = p.warp_partials + l.warps;
  p.chains = p.cta_partials + l.ctas;
  p.rows = reinterpret_cast<float2*>(p.chains + l.chains);
  p.cells = reinterpret_cast<float2*>(p.chains + l.chains + l.rows);
  const bool half = dtype == PA_BF16;
  cudaError_t e;
  switch (p.head_size) {
    case 64:
      e = half ? launch_decode_int8_bf16_d64(p, num_sms, stream)
               : launch_decode_int8_f32_d64(p, num_sms, stream);
      break;
    case 128:
      e = half ? launch_decode_int8_bf16_d128(p, num_sms, stream)
               : launch_decode_int8_f32_d128(p, num_sms, stream);
      break;
    default:
      e = half ? launch_decode_int8_bf16_d256(p, num_sms, stream)
               : launch_decode_int8_f32_d256(p, num_sms, stream);
  }
  if (e != cudaSuccess || !p.block_weights_out) return e;
  const int64_t blocks = (int64_t)p.num_seqs * p.max_blocks_per_seq;
  const int64_t most = 8ll * num_sms, ctas = (blocks + 7) / 8;
  void* args[] = {&p};
  return launch_overlapped((const void*)block_weights_kernel,
                           dim3((unsigned)(ctas < most ? ctas : most)), dim3(256), 0, stream, args);
}

}  // namespace pa
