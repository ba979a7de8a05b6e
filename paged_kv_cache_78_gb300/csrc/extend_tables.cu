// Block tables, slot map and positions from request lengths (pa_extend_tables).
//
// Latency is all there is to it for a decode step: one CTA, dependent reads
// (lengths, then a block id) and stores; 256 requests with a token each take 7.0 us
// in a row of graph replays, most of it the launch and four dependent trips to
// memory.  Steps with many tokens are shared out (500 requests with 125000 tokens,
// 1.5 MB written: 4.7 us, 8.5 us with new blocks from the ring).
// Every CTA scans all requests' token and block counts into its own shared
// memory (at most 8192 requests, 64 KB read from L2), so none waits for another;
// a thread then takes four consecutive tokens, with one binary search of the
// starts.  Where an output is its input, a barrier has to stand between the last
// read of the lengths and the ring's state and their first write: the CTAs are
// then one cluster of eight at most.
#include <atomic>
#include <climits>

#include "extend_tables.cuh"
#include "pa_device.cuh"
#include "pa_launch.h"

namespace pa {

namespace {

constexpr int kTablesThreads = 1024;
constexpr int kTablesCluster = 8;
constexpr int kTablesRun = 4;  // tokens of a thread
// Sums stop here: past every max_tokens, and 32 of them are below 2^32.
constexpr int kTablesCap = PA_MAX_TABLE_TOKENS + 1;

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

// Exclusive scan of v (0 .. kTablesCap) over the CTA; its total, kTablesCap or
// more where the sums went past that, in *all.
__device__ __forceinline__ int block_scan(int v, int* warp_sums, unsigned* all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  int sum = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum = min(sum + u, kTablesCap);
  }
  if (lane == 31) warp_sums[warp] = sum;
  __syncthreads();
  const unsigned other = lane < warps ? (unsigned)warp_sums[lane] : 0u;
  *all = __reduce_add_sync(0xffffffffu, other);
  return (int)__reduce_add_sync(0xffffffffu, lane < warp ? other : 0u) + sum - v;
}

__global__ void __launch_bounds__(kTablesThreads) extend_tables_kernel(const TablesParams p) {
  extern __shared__ int32_t scans[];  // first token, then first new block, of every request
  __shared__ int sums[2][32];
  int32_t* first_token = scans;
  int32_t* first_block = scans + p.num_seqs + 1;
  const int tid = threadIdx.x, threads = blockDim.x;
  const int n = p.num_seqs;
  const int l2bs = p.log2_block_size, BS = 1 << l2bs;
  const int per = (n + threads - 1) / threads;
  const int r0 = min(n, tid * per), r1 = min(n, r0 + per);
  grid_dependents_launch();
  grid_dependency_wait();
  const int head = p.free_blocks ? p.free_state[0] : 0;
  const int available = p.free_blocks ? p.free_state[1] : 0;
  int tokens = 0, blocks = 0;
  bool bad = false;
  for (int r = r0; r < r1; ++r) {
    const int len = p.seq_lens[r], add = p.new_tokens[r];
    const long long after = (long long)len + add;
    bad |= len < 0 || add < 0 || after > INT_MAX - 256 ||
           ((after + BS - 1) >> l2bs) > p.max_blocks_per_seq;
    if (!bad) {
      tokens = (int)min((long long)tokens + add, (long long)kTablesCap);
      blocks = min(blocks + (((int)after + BS - 1) >> l2bs) - ((len + BS - 1) >> l2bs), kTablesCap);
    }
  }
  unsigned all_tokens, all_blocks;
  tokens = block_scan(tokens, sums[0], &all_tokens);
  blocks = block_scan(blocks, sums[1], &all_blocks);
  bool refused = __syncthreads_or(bad) || all_tokens > (unsigned)p.max_tokens;
  // A ring state outside the ring is as good as an empty ring.
  const bool short_of =
      p.free_blocks && (head < 0 || head >= p.free_capacity || available < 0 ||
                        available > p.free_capacity || all_blocks > (unsigned)available);
  if ((refused || short_of) && blockIdx.x == 0 && tid == 0)
    record_error(p.err, refused ? PA_DEVERR_SEQ_LEN : PA_DEVERR_BLOCKS);
  refused = refused || short_of;
  const int total = refused ? 0 : (int)all_tokens;
  if (!refused) {
    for (int r = r0; r < r1; ++r) {
      first_token[r] = tokens;
      first_block[r] = blocks;
      const int len = p.seq_lens[r], add = p.new_tokens[r];
      tokens += add;
      blocks += ((len + add + BS - 1) >> l2bs) - ((len + BS - 1) >> l2bs);
    }
    if (tid == 0) first_token[n] = total;
  }
  __syncthreads();

  bool bad_id = false;
  const bool wide = ((reinterpret_cast<uintptr_t>(p.slot_mapping) |
                      reinterpret_cast<uintptr_t>(p.positions)) & 15) == 0;
  for (int t0 = (blockIdx.x * threads + tid) * kTablesRun; t0 < p.max_tokens;
       t0 += gridDim.x * threads * kTablesRun) {
    // The last request that starts at or before t0 (the ones that get no token
    // start where the next one does).
    int lo = 0, hi = n - 1;
    if (t0 < total)
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (first_token[mid] <= t0) lo = mid;
        else hi = mid - 1;
      }
    int64_t slot[kTablesRun];
    int pos[kTablesRun];
    int block = -1, id = -1, len = 0;  // the block of the token before
#pragma unroll
    for (int i = 0; i < kTablesRun; ++i) {
      const int t = t0 + i;
      slot[i] = -1;
      pos[i] = -1;
      if (t >= total) continue;
      if (i == 0 || t >= first_token[lo + 1]) {
        while (t >= first_token[lo + 1]) ++lo;
        len = p.seq_lens[lo];
        block = -1;
      }
      pos[i] = len + (t - first_token[lo]);
      const int b = pos[i] >> l2bs;
      if (b != block) {
        block = b;
        int32_t* entry = p.block_tables + (size_t)lo * p.max_blocks_per_seq + b;
        const int have = (len + BS - 1) >> l2bs;
        if (p.free_blocks && b >= have) {
          int at = head + first_block[lo] + (b - have);
          if (at >= p.free_capacity) at -= p.free_capacity;
          id = p.free_blocks[at];
          if ((pos[i] & (BS - 1)) == 0) *entry = id;
        } else {
          id = *entry;
        }
      }
      if (id >= 0 && id < p.num_blocks) slot[i] = ((int64_t)id << l2bs) + (pos[i] & (BS - 1));
      else bad_id = true;
    }
    if (wide && t0 + kTablesRun <= p.max_tokens) {
      longlong2* s2 = reinterpret_cast<longlong2*>(p.slot_mapping + t0);
      s2[0] = make_longlong2(slot[0], slot[1]);
      s2[1] = make_longlong2(slot[2], slot[3]);
      if (p.positions)
        *reinterpret_cast<int4*>(p.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
    } else {
#pragma unroll
      for (int i = 0; i < kTablesRun; ++i)
        if (t0 + i < p.max_tokens) {
          p.slot_mapping[t0 + i] = slot[i];
          if (p.positions) p.positions[t0 + i] = pos[i];
        }
    }
  }
  if (bad_id) record_error(p.err, PA_DEVERR_BLOCK_ID);
  if (p.token_starts)
    for (int r = blockIdx.x * threads + tid; r <= n; r += gridDim.x * threads)
      p.token_starts[r] = refused ? 0 : first_token[r];
  // Every CTA has read the lengths and the ring's state.
  if (p.in_place && gridDim.x > 1) cluster_sync();
  else __syncthreads();
  for (int r = blockIdx.x * threads + tid; r < n; r += gridDim.x * threads)
    p.seq_lens_out[r] = p.seq_lens[r] + (refused ? 0 : p.new_tokens[r]);
  if (p.free_blocks && blockIdx.x == 0 && tid == 0) {
    const int used = refused ? 0 : (int)all_blocks;
    int front = head + used;
    if (!refused && front >= p.free_capacity) front -= p.free_capacity;
    p.free_state_out[0] = front;
    p.free_state_out[1] = available - used;
  }
}

}  // namespace

cudaError_t launch_extend_tables(const TablesParams& params, int num_sms, cudaStream_t stream) {
  static std::atomic<bool> configured[64];
  const size_t smem = (size_t)(2 * params.num_seqs + 1) * 4;
  if (smem > 47 * 1024) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!configured[dev].load(std::memory_order_relaxed)) {
      e = cudaFuncSetAttribute(extend_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               (2 * PA_MAX_TABLE_REQUESTS + 1) * 4);
      if (e != cudaSuccess) return e;
      configured[dev].store(true, std::memory_order_relaxed);
    }
  }
  // A CTA takes 4096 tokens in one pass.  In place, where a cluster's barrier is
  // needed, eight CTAs are the most that every GPU allows; otherwise all SMs (500
  // requests with 250 tokens each: 10.1 us in place, 4.7 us into other memory).
  int ctas = (params.max_tokens + kTablesRun * kTablesThreads - 1) / (kTablesRun * kTablesThreads);
  if (ctas > num_sms) ctas = num_sms;
  if (ctas < 1) ctas = 1;
  if (params.in_place && ctas > 1) ctas = kTablesCluster;
  const int most = params.num_seqs > params.max_tokens ? params.num_seqs : params.max_tokens;
  // Few requests and tokens: scans over eight warps, not 32 (8.9 -> 7.0 us for 256
  // requests, with the 32-bit scans that came with it).
  const int threads = most <= 256 ? 256 : kTablesThreads;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = params.in_place && ctas > 1 ? 2 : 1;
  void* args[] = {const_cast<TablesParams*>(&params)};
  return cudaLaunchKernelExC(&cfg, (const void*)extend_tables_kernel, args);
}

}  // namespace pa
