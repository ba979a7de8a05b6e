// Eviction of the blocks with the least accumulated attention (pa_evict_blocks), for
// sm_103a.
//
// How many blocks leave a sequence follows from its length alone, so every CTA finds by
// itself, from all lengths, whether the call goes ahead and where its sequences' blocks go
// in the ring; none waits for another.  Where lengths or ring state are written in place, that is
// a second launch's work, one CTA, after all have read them.
//
// A sequence's weights become keys in shared memory whose unsigned order is theirs.  The
// k-th smallest key is found by counting, three bits at a time, until a value parts k keys from the
// others or all bits are known; keys below it leave, and as many of those equal to it, from
// the lowest index on, as are left to go.  Then the row is
// gone through once, eight chunks of a thread per entry at a time, with one barrier: what stays moves
// down (so that a row may be its own output: nothing is written before it was read), and what leaves
// goes to the ring and is kept aside in shared memory for the row's end.
// Latency is all there is to it: 256 sequences of up to 130 blocks, of which one or two leave, take
// 4.8 us (launch, lengths, weights, about six counts, entries; with all eleven counts and two barriers
// a chunk 6.2), with lengths written in place 2 more; 16 sequences of 8192 blocks, of which three quarters
// leave, 18 us, half of it the counts of one CTA (21 before, bit by bit 28).
#include <atomic>
#include <climits>

#include "evict_blocks.cuh"
#include "pa_device.cuh"
#include "pa_launch.h"

namespace pa {

namespace {

constexpr int kEvictThreads = 1024;

struct EvictTotals {
  int before, all;  // blocks that leave sequences before `s`, and all sequences
  bool refused;
};

__device__ __forceinline__ int blocks_of(const EvictParams& p, int len) {
  return (int)(((unsigned)len + (1u << p.log2_block_size) - 1) >> p.log2_block_size);
}
__device__ __forceinline__ int leaving(const EvictParams& p, int len) {
  return max(blocks_of(p, len) - p.max_blocks, 0);
}

// Whole CTA.  Counts are below 2^29 (8192 sequences of 49152 blocks).
__device__ __forceinline__ EvictTotals evict_totals(const EvictParams& p, int s, bool record) {
  __shared__ int sums[3][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  int before = 0, all = 0;
  bool bad = false;
  for (int i = threadIdx.x; i < p.num_seqs; i += blockDim.x) {
    const int len = p.seq_lens[i];
    if (len < 0 || blocks_of(p, len) > p.max_blocks_per_seq) {
      bad = true;
    } else {
      const int k = leaving(p, len);
      all += k;
      if (i < s) before += k;
    }
  }
  before = __reduce_add_sync(0xffffffffu, before);
  all = __reduce_add_sync(0xffffffffu, all);
  bad = __any_sync(0xffffffffu, bad);
  __syncthreads();  // of an earlier use of sums
  if (lane == 0) {
    sums[0][warp] = before;
    sums[1][warp] = all;
    sums[2][warp] = bad;
  }
  __syncthreads();
  EvictTotals r;
  r.before = __reduce_add_sync(0xffffffffu, lane < warps ? sums[0][lane] : 0);
  r.all = __reduce_add_sync(0xffffffffu, lane < warps ? sums[1][lane] : 0);
  const bool lens_bad = __any_sync(0xffffffffu, lane < warps && sums[2][lane]);
  bool ring_bad = false;
  if (p.free_state) {
    const int front = p.free_state[0], count = p.free_state[1];
    ring_bad = front < 0 || front >= p.free_capacity || count < 0 || count > p.free_capacity ||
               r.all > p.free_capacity - count;
  }
  if (record && threadIdx.x == 0) {
    if (lens_bad) record_error(p.err, PA_DEVERR_SEQ_LEN);
    else if (ring_bad) record_error(p.err, PA_DEVERR_BLOCKS);
  }
  r.refused = lens_bad || ring_bad;
  return r;
}

// Unsigned order of the result is the order of numbers: -0 with 0, NaNs last.
__device__ __forceinline__ uint32_t weight_key(float w) {
  const uint32_t b = __float_as_uint(w + 0.f);
  if ((b & 0x7fffffffu) > 0x7f800000u) return 0xffffffffu;
  return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}

// Length and count of a sequence that k blocks leave.
__device__ __forceinline__ void write_state(const EvictParams& p, int s, int len, int k) {
  const int moved = k << p.log2_block_size;
  p.seq_lens_out[s] = len - moved;
  if (p.evicted_tokens) p.evicted_tokens_out[s] = p.evicted_tokens[s] + moved;
}

__global__ void __launch_bounds__(kEvictThreads) evict_rows_kernel(const EvictParams p) {
  extern __shared__ uint32_t keys[];
  constexpr int kBatch = 8;  // chunks whose entries are on their way at once
  __shared__ uint32_t counts[2][kBatch][32];
  __shared__ uint4 digits[2][32];
  const int tid = threadIdx.x, threads = blockDim.x;
  const int lane = tid & 31, warp = tid >> 5, warps = threads >> 5;
  const int per = (p.num_seqs + gridDim.x - 1) / gridDim.x;
  const int s0 = min((int)blockIdx.x * per, p.num_seqs), s1 = min(s0 + per, p.num_seqs);
  grid_dependents_launch();
  grid_dependency_wait();
  const EvictTotals totals = evict_totals(p, s0, blockIdx.x == 0);
  // Where the next block that leaves goes: below twice the capacity before it is brought back.
  int ring = 0;
  auto in_ring = [&](int i) { return i >= p.free_capacity ? i - p.free_capacity : i; };
  if (p.alone && p.free_state && blockIdx.x == 0 && tid == 0) {
    p.free_state_out[0] = p.free_state[0];
    p.free_state_out[1] = p.free_state[1] + (totals.refused ? 0 : totals.all);
  }
  if (p.free_state && !totals.refused)
    ring = in_ring(p.free_state[0] + p.free_state[1] + totals.before);
  for (int s = s0; s < s1; ++s) {
    const int len = p.seq_lens[s];
    const int n = len < 0 ? 0 : min(blocks_of(p, len), p.max_blocks_per_seq);
    const int k = totals.refused ? 0 : leaving(p, len);
    const size_t row = (size_t)s * p.max_blocks_per_seq;
    const int32_t* ids = p.block_tables + row;
    const float* weights = p.block_weights + row;
    int32_t* ids_out = p.block_tables_out + row;
    float* weights_out = p.block_weights_out + row;
    if (p.alone && tid == 0) write_state(p, s, len, k);
    if (k == 0) {
      if (ids != ids_out)
        for (int i = tid; i < n; i += threads) ids_out[i] = ids[i];
      if (weights != weights_out)
        for (int i = tid; i < n; i += threads) weights_out[i] = weights[i];
      continue;
    }
    const int first = p.keep_first, m = n - first - p.keep_last;  // candidates; k <= m
    // A thread's own keys, several on their way at once.
#pragma unroll 8
    for (int i = tid; i < m; i += threads) keys[i] = weight_key(weights[first + i]);
    // The k-th smallest key: the largest value that fewer than k keys are below, three bits at
    // a time from the top: seven values are tried at once, their counts two to a word (a
    // warp's are at most 1536, all warps' 49152).
    uint32_t kth = 0;
    int below = 0;
#pragma unroll 1
    for (int shift = 30, turn = 0; shift >= 0; shift -= 3, turn ^= 1) {
      // A thread's keys (48 at most) by their next three bits, eight counts of a byte.  Keys
      // below those with the bits so far count as 0, above them as 7: neither is ever below a value
      // that it should not be below.
      uint64_t by = 0;
#pragma unroll 4
      for (int i = tid; i < m; i += threads) {
        const uint32_t key = keys[i];
        by += 1ull << (8 * (key < kth ? 0u : min((key - kth) >> shift, 7u)));
      }
      // Values 2 w and 2 w + 1 (keys below 0: none): running sums of counts.
      uint32_t c[4], sum = 0;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        c[w] = sum;
        sum += (uint32_t)(by >> (16 * w)) & 0xff;
        c[w] |= sum << 16;
        sum += (uint32_t)(by >> (16 * w + 8)) & 0xff;
      }
#pragma unroll
      for (int w = 0; w < 4; ++w) c[w] = __reduce_add_sync(0xffffffffu, c[w]);
      if (lane == 0) digits[turn][warp] = make_uint4(c[0], c[1], c[2], c[3]);
      __syncthreads();
      const uint4 all = lane < warps ? digits[turn][lane] : make_uint4(0u, 0u, 0u, 0u);
      c[0] = __reduce_add_sync(0xffffffffu, all.x);
      c[1] = __reduce_add_sync(0xffffffffu, all.y);
      c[2] = __reduce_add_sync(0xffffffffu, all.z);
      c[3] = __reduce_add_sync(0xffffffffu, all.w);
      uint32_t digit = 0;
      bool all_leave = false;  // the keys of the digit
#pragma unroll
      for (int v = 1; v < 8; ++v) {
        const int n_below = (c[v / 2] >> (16 * (v & 1))) & 0xffff;
        if (n_below < k) {
          digit = v;
          below = n_below;
        }
        all_leave |= n_below == k;
      }
      kth += digit << shift;
      // Where exactly k keys are below one of the values, the least such value parts them as well as
      // the k-th key.  (At the top values past the third are 2^32 and more.)
      if (all_leave && shift < 30) {
        kth += 1u << shift;
        below = k;
        break;
      }
    }
    const int equal = k - below;  // of the keys equal to it, the first so many leave
    int less = 0, ties = 0;       // so far
    for (int b0 = 0, turn = 0; b0 < n; b0 += kBatch * threads, turn ^= 1) {
      int id[kBatch];
      float w[kBatch];
#pragma unroll
      for (int c = 0; c < kBatch; ++c) {
        const int i = b0 + c * threads + tid;
        id[c] = i < n ? ids[i] : 0;
        w[c] = i < n ? weights[i] : 0.f;
      }
      // Keys that are less and that are equal: a bit of the thread's, and the two counts of its
      // chunk's warps in a word (of at most 1024 a chunk).
      uint32_t is_less = 0, is_tie = 0;
#pragma unroll
      for (int c = 0; c < kBatch; ++c) {
        const int i = b0 + c * threads + tid;
        bool l = false, t = false;
        if (i >= first && i < first + m) {
          const uint32_t key = keys[i - first];
          l = key < kth;
          t = key == kth;
        }
        is_less |= (uint32_t)l << c;
        is_tie |= (uint32_t)t << c;
        const uint32_t sum = __popc(__ballot_sync(0xffffffffu, l)) | __popc(__ballot_sync(0xffffffffu, t)) << 16;
        if (lane == 0) counts[turn][c][warp] = sum;
      }
      // Everything of the batch is read.  One barrier a batch: the other turn's counts are
      // written when all have passed the barrier after they read them.
      __syncthreads();
#pragma unroll
      for (int c = 0; c < kBatch; ++c) {
        if (b0 + c * threads >= n) break;
        const int i = b0 + c * threads + tid;
        const bool l = is_less >> c & 1, t = is_tie >> c & 1;
        const uint32_t sum = lane < warps ? counts[turn][c][lane] : 0;
        const uint32_t of_warps = __reduce_add_sync(0xffffffffu, lane < warp ? sum : 0);
        const uint32_t of_all = __reduce_add_sync(0xffffffffu, sum);
        const uint32_t lower = (1u << lane) - 1;
        const int tied = ties + (int)(of_warps >> 16) + __popc(__ballot_sync(0xffffffffu, t) & lower);
        const int before = less + (int)(of_warps & 0xffff) +
                           __popc(__ballot_sync(0xffffffffu, l) & lower) + min(tied, equal);
        less += of_all & 0xffff;
        ties += of_all >> 16;
        if (l || (t && tied < equal)) {
          keys[before] = (uint32_t)id[c];  // before <= i - first: a key that was read
          if (p.free_state) p.free_blocks[in_ring(ring + before)] = id[c];
        } else if (i < n) {
          ids_out[i - before] = id[c];
          weights_out[i - before] = w[c];
        }
      }
    }
    __syncthreads();
    for (int i = tid; i < k; i += threads) {
      ids_out[n - k + i] = (int32_t)keys[i];
      weights_out[n - k + i] = 0.f;
    }
    if (p.free_state) ring = in_ring(ring + k);
    __syncthreads();  // keys and counts are free again
  }
}

__global__ void __launch_bounds__(kEvictThreads) evict_state_kernel(const EvictParams p) {
  grid_dependents_launch();
  grid_dependency_wait();
  const EvictTotals totals = evict_totals(p, 0, false);
  int front = 0, count = 0;
  if (p.free_state && threadIdx.x == 0) {
    front = p.free_state[0];
    count = p.free_state[1];
  }
  __syncthreads();  // every read of the lengths and the ring's state for the totals is done
  for (int i = threadIdx.x; i < p.num_seqs; i += blockDim.x) {
    const int len = p.seq_lens[i];
    write_state(p, i, len, totals.refused ? 0 : leaving(p, len));
  }
  if (p.free_state && threadIdx.x == 0) {
    p.free_state_out[0] = front;
    p.free_state_out[1] = count + (totals.refused ? 0 : totals.all);
  }
}

}  // namespace

cudaError_t launch_evict_blocks(const EvictParams& params, int num_sms, cudaStream_t stream) {
  // Raised on the first call of a device whatever its size: how much a launch may have unasked is
  // 48 KB less the kernel's own arrays.
  static std::atomic<bool> configured[64];
  const size_t smem = (size_t)params.max_blocks_per_seq * 4;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!configured[dev].load(std::memory_order_relaxed)) {
    e = cudaFuncSetAttribute(evict_rows_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             PA_MAX_EVICT_BLOCKS * 4);
    if (e != cudaSuccess) return e;
    configured[dev].store(true, std::memory_order_relaxed);
  }
  const int threads = params.max_blocks_per_seq <= 1024 ? 256 : kEvictThreads;
  int ctas = params.num_seqs < 2 * num_sms ? params.num_seqs : 2 * num_sms;
  if (ctas < 1) ctas = 1;
  EvictParams p = params;
  p.alone = p.seq_lens_out != p.seq_lens && (!p.free_state || p.free_state_out != p.free_state);
  void* args[] = {&p};
  e = launch_overlapped((const void*)evict_rows_kernel, dim3((unsigned)ctas), dim3(threads), smem,
                        stream, args);
  if (e != cudaSuccess || p.alone) return e;
  return launch_overlapped((const void*)evict_state_kernel, dim3(1),
                           dim3(p.num_seqs <= 256 ? 256 : kEvictThreads), 0, stream, args);
}

}  // namespace pa
