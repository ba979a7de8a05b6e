// Eviction of the blocks with the least accumulated attention (pa_evict_blocks), for
// sm_103a.
//
// How many blocks leave a sequence follows from its length alone, so every CTA finds by
// itself, from all lengths, whether the call goes ahead and where its sequences' blocks go
// in the ring; none waits for another.  The first launch only reads lengths and ring state,
// the second, one CTA, writes them: they may be written in place.
//
// A sequence's weights become keys in shared memory whose unsigned order is theirs.  The
// k-th smallest key is found bit by bit from the top, by counting; keys below it leave, and as many
// of those equal to it, from the lowest index on, as are left to go.  Then the row is
// gone through once, a chunk of a thread per entry at a time: what stays moves down (so that a
// row may be its own output: nothing is written before it was read), and what leaves
// goes to the ring and is kept aside in shared memory for the row's end.
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

__global__ void __launch_bounds__(kEvictThreads) evict_rows_kernel(const EvictParams p) {
  extern __shared__ uint32_t keys[];
  __shared__ int counts[2][32];
  const int tid = threadIdx.x, threads = blockDim.x;
  const int lane = tid & 31, warp = tid >> 5, warps = threads >> 5;
  const int per = (p.num_seqs + gridDim.x - 1) / gridDim.x;
  const int s0 = min((int)blockIdx.x * per, p.num_seqs), s1 = min(s0 + per, p.num_seqs);
  grid_dependents_launch();
  grid_dependency_wait();
  const EvictTotals totals = evict_totals(p, s0, blockIdx.x == 0);
  int64_t ring = 0;  // where the next block that leaves goes
  if (p.free_state && !totals.refused)
    ring = ((int64_t)p.free_state[0] + p.free_state[1] + totals.before) % p.free_capacity;
  // Exclusive count of a flag over the CTA's threads, and all of them.  One barrier a use:
  // `which` alternates between uses, so that a use's writers have passed the barrier that the
  // readers of the use before the last came to after they had read.
  auto count = [&](bool flag, int which, int* all) -> int {
    const uint32_t b = __ballot_sync(0xffffffffu, flag);
    if (lane == 0) counts[which][warp] = __popc(b);
    __syncthreads();
    const int c = lane < warps ? counts[which][lane] : 0;
    *all = __reduce_add_sync(0xffffffffu, c);
    return __reduce_add_sync(0xffffffffu, lane < warp ? c : 0) + __popc(b & ((1u << lane) - 1));
  };
  for (int s = s0; s < s1; ++s) {
    const int len = p.seq_lens[s];
    const int n = len < 0 ? 0 : min(blocks_of(p, len), p.max_blocks_per_seq);
    const int k = totals.refused ? 0 : leaving(p, len);
    const size_t row = (size_t)s * p.max_blocks_per_seq;
    const int32_t* ids = p.block_tables + row;
    const float* weights = p.block_weights + row;
    int32_t* ids_out = p.block_tables_out + row;
    float* weights_out = p.block_weights_out + row;
    if (k == 0) {
      if (ids != ids_out)
        for (int i = tid; i < n; i += threads) ids_out[i] = ids[i];
      if (weights != weights_out)
        for (int i = tid; i < n; i += threads) weights_out[i] = weights[i];
      continue;
    }
    const int first = p.keep_first, m = n - first - p.keep_last;  // candidates; k <= m
    for (int i = tid; i < m; i += threads) keys[i] = weight_key(weights[first + i]);
    // The k-th smallest key: the largest value that fewer than k keys are below.
    uint32_t kth = 0;
    int below = 0;
#pragma unroll 1
    for (int bit = 31; bit >= 0; --bit) {
      const uint32_t trial = kth | (1u << bit);
      int c = 0;
      for (int i = tid; i < m; i += threads) c += keys[i] < trial;  // a thread's own keys
      c = __reduce_add_sync(0xffffffffu, c);
      if (lane == 0) counts[bit & 1][warp] = c;
      __syncthreads();
      c = __reduce_add_sync(0xffffffffu, lane < warps ? counts[bit & 1][lane] : 0);
      if (c < k) {
        kth = trial;
        below = c;
      }
    }
    const int equal = k - below;  // of the keys equal to it, the first so many leave
    int gone = 0, ties = 0;       // so far
    for (int i0 = 0; i0 < n; i0 += threads) {
      const int i = i0 + tid;
      int id = 0;
      float w = 0.f;
      bool less = false, tie = false;
      if (i < n) {
        id = ids[i];
        w = weights[i];
        if (i >= first && i < first + m) {
          const uint32_t key = keys[i - first];
          less = key < kth;
          tie = key == kth;
        }
      }
      int all;
      const int tied = ties + count(tie, 1, &all);
      ties += all;
      const bool leaves = less || (tie && tied < equal);
      const int before = gone + count(leaves, 0, &all);  // everything of the chunk is read
      gone += all;
      if (leaves) {
        keys[before] = (uint32_t)id;  // before <= i - first: a key that was read
        if (p.free_state) p.free_blocks[(ring + before) % p.free_capacity] = id;
      } else if (i < n) {
        ids_out[i - before] = id;
        weights_out[i - before] = w;
      }
    }
    __syncthreads();
    for (int i = tid; i < k; i += threads) {
      ids_out[n - k + i] = (int32_t)keys[i];
      weights_out[n - k + i] = 0.f;
    }
    if (p.free_state) ring = (ring + k) % p.free_capacity;
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
    const int moved = totals.refused ? 0 : leaving(p, len) << p.log2_block_size;
    const int past = p.evicted_tokens ? p.evicted_tokens[i] : 0;
    p.seq_lens_out[i] = len - moved;
    if (p.evicted_tokens) p.evicted_tokens_out[i] = past + moved;
  }
  if (p.free_state && threadIdx.x == 0) {
    p.free_state_out[0] = front;
    p.free_state_out[1] = count + (totals.refused ? 0 : totals.all);
  }
}

}  // namespace

cudaError_t launch_evict_blocks(const EvictParams& params, int num_sms, cudaStream_t stream) {
  static std::atomic<bool> configured[64];
  const size_t smem = (size_t)params.max_blocks_per_seq * 4;
  if (smem > 47 * 1024) {
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
  }
  const int threads = params.max_blocks_per_seq <= 1024 ? 256 : kEvictThreads;
  int ctas = params.num_seqs < 2 * num_sms ? params.num_seqs : 2 * num_sms;
  if (ctas < 1) ctas = 1;
  void* args[] = {const_cast<EvictParams*>(&params)};
  cudaError_t e = launch_overlapped((const void*)evict_rows_kernel, dim3((unsigned)ctas),
                                    dim3(threads), smem, stream, args);
  if (e != cudaSuccess) return e;
  return launch_overlapped((const void*)evict_state_kernel, dim3(1),
                           dim3(params.num_seqs <= 256 ? 256 : kEvictThreads), 0, stream, args);
}

}  // namespace pa
