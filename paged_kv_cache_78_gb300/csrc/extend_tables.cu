// Block tables, slot map and positions from request lengths (pa_extend_tables).
//
// One cluster of up to eight CTAs.  Every CTA scans all requests' token and
// block counts into its own shared memory (at most 8192 requests, 64 KB read
// from L2), so none has to wait for another; the tokens are then shared out
// over the cluster, each finding its request by a binary search of the starts.
// The inputs may be updated in place: a cluster barrier stands between the
// last read of the lengths and the ring's state and their first write.
#include <atomic>
#include <climits>

#include "extend_tables.cuh"
#include "pa_device.cuh"
#include "pa_launch.h"

namespace pa {

namespace {

constexpr int kTablesThreads = 1024;
constexpr int kTablesCluster = 8;

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

// Exclusive scan of a and b over the CTA; totals in ta and tb.
__device__ __forceinline__ void block_scan2(long long& a, long long& b, long long& ta,
                                            long long& tb) {
  __shared__ long long wa[32], wb[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  long long ia = a, ib = b;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long ua = __shfl_up_sync(0xffffffffu, ia, o);
    const long long ub = __shfl_up_sync(0xffffffffu, ib, o);
    if (lane >= o) {
      ia += ua;
      ib += ub;
    }
  }
  if (lane == 31) {
    wa[warp] = ia;
    wb[warp] = ib;
  }
  __syncthreads();
  ta = 0;
  tb = 0;
  long long ba = 0, bb = 0;
  for (int w = 0; w < warps; ++w) {
    if (w == warp) {
      ba = ta;
      bb = tb;
    }
    ta += wa[w];
    tb += wb[w];
  }
  a = ba + ia - a;
  b = bb + ib - b;
}

__global__ void __launch_bounds__(kTablesThreads) extend_tables_kernel(const TablesParams p) {
  extern __shared__ int32_t scans[];  // first token, then first new block, of every request
  int32_t* first_token = scans;
  int32_t* first_block = scans + p.num_seqs + 1;
  grid_dependents_launch();
  grid_dependency_wait();
  const int tid = threadIdx.x, threads = blockDim.x;
  const int n = p.num_seqs;
  const int BS = 1 << p.log2_block_size;
  const int per = (n + threads - 1) / threads;
  const int r0 = min(n, tid * per), r1 = min(n, r0 + per);
  long long tokens = 0, blocks = 0;
  bool bad = false;
  for (int r = r0; r < r1; ++r) {
    const long long len = p.seq_lens[r], add = p.new_tokens[r];
    const long long have = (len + BS - 1) >> p.log2_block_size;
    const long long after = (len + add + BS - 1) >> p.log2_block_size;
    bad |= len < 0 || add < 0 || after > p.max_blocks_per_seq || len + add > INT_MAX - 256;
    tokens += add;
    blocks += after - have;
  }
  long long all_tokens, all_blocks;
  block_scan2(tokens, blocks, all_tokens, all_blocks);
  const int head = p.free_blocks ? p.free_state[0] : 0;
  const int available = p.free_blocks ? p.free_state[1] : 0;
  bool refused = __syncthreads_or(bad) || all_tokens > p.max_tokens;
  // A ring state outside the ring is as good as an empty ring.
  const bool short_of = p.free_blocks && (head < 0 || head >= p.free_capacity ||
                                          available > p.free_capacity || all_blocks > available);
  if ((refused || short_of) && blockIdx.x == 0 && tid == 0)
    record_error(p.err, refused ? PA_DEVERR_SEQ_LEN : PA_DEVERR_BLOCKS);
  refused = refused || short_of;
  const int total = refused ? 0 : (int)all_tokens;
  if (!refused) {
    for (int r = r0; r < r1; ++r) {
      first_token[r] = (int)tokens;
      first_block[r] = (int)blocks;
      const int len = p.seq_lens[r], add = p.new_tokens[r];
      tokens += add;
      blocks += ((len + add + BS - 1) >> p.log2_block_size) - ((len + BS - 1) >> p.log2_block_size);
    }
    if (tid == 0) first_token[n] = total;
  }
  __syncthreads();

  bool bad_id = false;
  for (int t = blockIdx.x * threads + tid; t < p.max_tokens; t += gridDim.x * threads) {
    int64_t slot = -1;
    int pos = -1;
    if (t < total) {
      // The last request that starts at or before t (the ones that get no
      // token start where the next one does).
      int lo = 0, hi = n - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (first_token[mid] <= t) lo = mid;
        else hi = mid - 1;
      }
      const int len = p.seq_lens[lo];
      pos = len + (t - first_token[lo]);
      const int b = pos >> p.log2_block_size;
      const int have = (len + BS - 1) >> p.log2_block_size;
      int32_t* entry = p.block_tables + (size_t)lo * p.max_blocks_per_seq + b;
      int id;
      if (p.free_blocks && b >= have) {
        int at = head + first_block[lo] + (b - have);
        if (at >= p.free_capacity) at -= p.free_capacity;
        id = p.free_blocks[at];
        if ((pos & (BS - 1)) == 0) *entry = id;
      } else {
        id = *entry;
      }
      if (id >= 0 && id < p.num_blocks)
        slot = ((int64_t)id << p.log2_block_size) + (pos & (BS - 1));
      else
        bad_id = true;
    }
    p.slot_mapping[t] = slot;
    if (p.positions) p.positions[t] = pos;
  }
  if (bad_id) record_error(p.err, PA_DEVERR_BLOCK_ID);
  if (p.token_starts)
    for (int r = blockIdx.x * threads + tid; r <= n; r += gridDim.x * threads)
      p.token_starts[r] = refused ? 0 : first_token[r];
  // Every CTA has read the lengths and the ring's state.
  cluster_sync();
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

cudaError_t launch_extend_tables(const TablesParams& params, cudaStream_t stream) {
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
  const int ctas = params.max_tokens > 4 * kTablesThreads ? kTablesCluster : 1;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kTablesThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  void* args[] = {const_cast<TablesParams*>(&params)};
  return cudaLaunchKernelExC(&cfg, (const void*)extend_tables_kernel, args);
}

}  // namespace pa
