// Decode attention over the 4-bit pool for sm_103a.
//
// For one sequence and KV head, with the query heads of its group as columns,
//   S [tokens x heads]  = K [tokens x D] . Q^T [D x heads]
//   O^T [D x heads]    += V^T [D x tokens] . P^T [tokens x heads],
// P = 2^(S - m) with a running maximum m.  Reading the pool bounds it: an SM
// gets about 23 bytes of codes and scales per clock, 41 elements, each of which
// has to become fp16 before a product.  Two conversions (one instruction per
// pair of codes, one multiplication per pair by the scales, exact) and the
// matrix instructions take about 60% of the SM's issue slots at that rate, so
// the codes go from shared memory to registers once, are converted there, and
// are used there: the operands of mma.sync are the converting thread's own
// registers.  Tensor-memory or shared-memory operands would put a second trip
// of 2 bytes per element on a path that has no room for it (82 bytes written
// and 82 read per clock of 128).  The pool's layout is made for this: a tile's
// key rows and value groups are the matrix instructions' fragments.
//
// Every warp works for itself.  The stages of 32 tokens of all (sequence, KV
// head) pairs, laid end to end, are cut into equal ranges, one per CTA, and
// those into equal parts, one per warp; a warp streams its part through a ring
// of its own (bulk copies that its lanes issue, one per block; no barrier with
// other warps) and keeps S, P, m and O in registers.  A pair that a warp saw
// whole is written out; parts of a pair are merged over the CTA's warps at the
// end, and over CTAs by whichever finishes last, always in the same order.
#pragma once

#include <cuda_bf16.h>
#include <math.h>

#include "decode_fp4.cuh"
#include "pa_fp4.cuh"

namespace pa {

constexpr float kFp4Lift = 7.f;   // weights are 2^(S - m + 7): fp16 keeps small ones
constexpr float kFp4Slack = 8.f;  // scores may pass the running maximum by this before it moves
constexpr int kFp4RingBytes = 216 * 1024;

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

__device__ __forceinline__ uint32_t lds_u8(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=h"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds_u16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds_u32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds_u64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}

// c += a . b: a 16 x 16, b 16 x 8, fp16 with fp32 sums.
__device__ __forceinline__ void mma_f16(float* c, const uint32_t* a, const uint32_t* b) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

// The 8 x 8 matrix of 16-bit elements that the warp holds, transposed.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

template <int S>
__device__ __forceinline__ float group_max(float v) {  // over lanes that differ in bits >= S
#pragma unroll
  for (int o = S; o < 32; o <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// A warp's place in the work: stage k of the n stages of pair (s, hp).
struct Fp4Place {
  int s, hp, k, n, len;
};

// What a warp needs to know of a stage that is in its ring.
struct __align__(16) Fp4Record {
  int s, hp;
  int k;
  int info;  // tokens (1..32), then flags
};
constexpr int kRecBegin = 1 << 8;   // first stage of the pair
constexpr int kRecFinish = 1 << 9;  // last stage of the pair
constexpr int kRecLast = 1 << 10;   // last stage of the warp's part
constexpr int kFp4Records = 8;      // ring of records, at least the stages in flight + 1

// The parts of pairs that a warp leaves behind for the merge: a (ended inside
// its part, begun before it) in global memory, b (reaches the part's end) in
// its ring.  Pair numbers, or -1.
struct Fp4Left {
  int a, b;
};

template <typename T, int D, int NT>
struct Fp4Config {
  static constexpr bool kF32 = sizeof(T) == 4;
  static constexpr int kWarps = fp4_warps(D, NT, kF32);
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kTileBytes = fp4_tile_bytes(D);
  static constexpr int kStageBytes = kFp4Stage / kFp4Tile * kTileBytes;
  static constexpr int kFit = kFp4RingBytes / kWarps / kStageBytes;
  static constexpr int kStages = kFit < 6 ? kFit : 6;
  static constexpr int kWarpRing = kStages * kStageBytes;
  static constexpr int kBars = kWarps * kWarpRing;
  static constexpr int kRecs = kBars + 8 * kWarps * kStages;
  static constexpr int kPre = (kRecs + kWarps * kFp4Records * 16 + 15) / 16 * 16;
  static constexpr int kLeft = kPre + 8 * (kThreads + 34);
  static constexpr int kMisc = kLeft + 8 * kWarps;
  static constexpr int kRuns = kMisc + 64;
  static constexpr int kSmem = kRuns + 4 * (2 * kWarps + 2);
  static_assert(kStages >= 2 && kStages < kFp4Records, "ring");
  static_assert(kSmem <= 227 * 1024, "shared memory");
  static_assert(fp4_partial_floats(8 * NT, D) * 4 <= kWarpRing, "a part fits its warp's ring");
};

template <typename T, int D, int NT>
__global__ void __launch_bounds__(Fp4Config<T, D, NT>::kThreads, 1)
    decode_fp4_kernel(const Fp4DecodeParams p) {
  using C = Fp4Config<T, D, NT>;
  constexpr bool kF32 = C::kF32;
  constexpr int W = C::kWarps;
  constexpr int NS = C::kStages;
  constexpr int kSteps = D / 16;      // of QK; and 16-row tiles of O^T
  constexpr int kQParts = kF32 ? 2 : 1;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  const int G = p.group;
  const int head_tiles = (G + 8 * NT - 1) / (8 * NT);
  const int rows = fp4_unit_rows(NT, G);
  const int per_seq = p.num_kv_heads * head_tiles;  // pairs of a sequence
  const int l2bs = p.log2_block_size;
  const int part_floats = fp4_partial_floats(rows, D);

  extern __shared__ __align__(128) uint8_t smem[];
  const uint32_t ring = smem_u32(smem) + (uint32_t)warp * C::kWarpRing;
  const uint32_t bars = smem_u32(smem) + C::kBars + (uint32_t)warp * NS * 8;
  Fp4Record* recs = reinterpret_cast<Fp4Record*>(smem + C::kRecs) + warp * kFp4Records;
  long long* pre = reinterpret_cast<long long*>(smem + C::kPre);
  Fp4Left* left = reinterpret_cast<Fp4Left*>(smem + C::kLeft);
  volatile int* misc = reinterpret_cast<volatile int*>(smem + C::kMisc);
  int* runs = reinterpret_cast<int*>(smem + C::kRuns);

  if (lane == 0) {
    for (int i = 0; i < NS; ++i) mbar_init(bars + 8u * i, 1);
    fence_mbar_init();
  }
  grid_dependency_wait();
  grid_dependents_launch();

  // ---- the work: stages of every sequence, scanned ----
  auto stages_of = [&](int s, int* len_out) -> int {
    const int len = p.seq_lens[s];
    *len_out = len;
    if (len <= 0) return 0;
    if ((((long long)len + (1 << l2bs) - 1) >> l2bs) > p.max_blocks_per_seq) return 0;
    return (len + kFp4Stage - 1) / kFp4Stage;
  };
  const int chunk = (p.num_seqs + C::kThreads - 1) / C::kThreads;
  {
    long long mine = 0;
    for (int i = 0; i < chunk; ++i) {
      const int s = tid * chunk + i;
      if (s >= p.num_seqs) break;
      int len;
      const int n = stages_of(s, &len);
      if (n == 0 && len > 0 && blockIdx.x == 0) record_error(p.err, PA_DEVERR_SEQ_LEN);
      mine += n;
    }
    mine *= per_seq;
    long long sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += v;
    }
    long long* warp_sums = pre + C::kThreads + 1;
    if (lane == 31) warp_sums[warp] = sum;
    __syncthreads();
    long long base = 0;
    for (int w = 0; w < warp; ++w) base += warp_sums[w];
    pre[tid] = base + sum - mine;
    if (tid == C::kThreads - 1) pre[C::kThreads] = base + sum;
    __syncthreads();
  }
  const long long total = pre[C::kThreads];
  // Stages of a CTA: an equal share, at least half a stage per warp (fewer
  // parts to merge where there is little work).
  long long share = (total + gridDim.x - 1) / gridDim.x;
  if (share < W / 2) share = W / 2;
  const long long cta0 = share * blockIdx.x;
  const long long cta1 = cta0 + share < total ? cta0 + share : total;

  auto locate = [&](long long at) -> Fp4Place {
    int lo = 0, hi = C::kThreads - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (pre[mid] <= at) lo = mid;
      else hi = mid - 1;
    }
    long long acc = pre[lo];
    Fp4Place pl;
    pl.s = lo * chunk;
    while (true) {
      pl.n = stages_of(pl.s, &pl.len);
      const long long next = acc + (long long)pl.n * per_seq;
      if (next > at) break;
      acc = next;
      ++pl.s;
    }
    const long long rem = at - acc;
    pl.hp = (int)(rem / pl.n);
    pl.k = (int)(rem - (long long)pl.hp * pl.n);
    return pl;
  };

  bool ok = true;
  if (lane == 0) left[warp] = Fp4Left{-1, -1};
  const long long share_w = (share + W - 1) / W;
  const long long my0 = cta0 + share_w * warp;
  const long long my1 = my0 + share_w < cta1 ? my0 + share_w : cta1;
  if (my0 < my1) {
    const int count = (int)(my1 - my0);  // a launch has far fewer than 2^31 stages per warp
    Fp4Place pp = locate(my0);           // the next stage to prepare
    int prepared = 0, issued = 0;
    int ids[NS];  // table entries of prepared stages, one block per lane

    // Record the next stage and fetch its table entries.
    auto prepare = [&]() -> int {
      const int tok0 = pp.k * kFp4Stage;
      const int tokens = min(kFp4Stage, pp.len - tok0);
      if (lane == 0) {
        Fp4Record r;
        r.s = pp.s;
        r.hp = pp.hp;
        r.k = pp.k;
        r.info = tokens | (pp.k == 0 ? kRecBegin : 0) | (pp.k + 1 == pp.n ? kRecFinish : 0) |
                 (prepared + 1 == count ? kRecLast : 0);
        recs[prepared % kFp4Records] = r;
      }
      const int first = tok0 >> l2bs;
      const int blocks = ((tok0 + tokens - 1) >> l2bs) - first + 1;
      int id = 0;
      if (lane < blocks) id = __ldg(p.block_tables + (size_t)pp.s * p.max_blocks_per_seq + first + lane);
      if (++prepared < count && ++pp.k == pp.n) {
        pp.k = 0;
        if (++pp.hp == per_seq) {
          pp.hp = 0;
          do {
            ++pp.s;
            pp.n = stages_of(pp.s, &pp.len);
          } while (pp.n == 0);
        }
      }
      return id;
    };
    // Copy the next stage's tiles into its slot: one range per block.
    auto issue = [&](int id) {
      __syncwarp();
      const Fp4Record r = recs[issued % kFp4Records];
      const int slot = issued % NS;
      const int tokens = r.info & 255;
      const int tiles = (tokens + kFp4Tile - 1) / kFp4Tile;
      const int tok0 = r.k * kFp4Stage;
      const int in_block = (tok0 & ((1 << l2bs) - 1)) >> 3;  // first tile (blocks of 64 and more)
      const int per_block = l2bs >= 5 ? kFp4Stage / kFp4Tile : 1 << (l2bs - 3);
      const int mine = min(per_block, tiles - lane * per_block);
      const bool live = mine > 0;
      const bool good = live && id >= 0 && id < p.num_blocks;
      const uint32_t bar = bars + 8u * slot;
      const uint32_t dst = ring + slot * C::kStageBytes + lane * per_block * C::kTileBytes;
      const uint32_t bytes = good ? (uint32_t)mine * C::kTileBytes : 0u;
      const uint32_t sum = __reduce_add_sync(0xffffffffu, bytes);
      if (lane == 0) mbar_arrive_expect_tx(bar, sum);
      __syncwarp();
      if (good) {
        const int h = r.hp / head_tiles;
        const size_t tile = (((size_t)id * p.num_kv_heads + h) << (l2bs - 3)) + in_block;
        bulk_load(dst, p.cache + tile * C::kTileBytes, bytes, bar);
      } else if (live) {
        // A block outside the pool: zero keys and values.
        record_error(p.err, PA_DEVERR_BLOCK_ID);
        for (int i = 0; i < mine * C::kTileBytes; i += 16)
          asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(dst + i), "r"(0u) : "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      }
      ++issued;
    };

    // Prologue: fill the ring, every table entry on its way before the first
    // is needed.
#pragma unroll
    for (int i = 0; i < NS; ++i) ids[i] = i < count ? prepare() : 0;
#pragma unroll
    for (int i = 0; i < NS; ++i)
      if (i < count) issue(ids[i]);
    int next_id = NS < count ? prepare() : 0;

    uint32_t q[kQParts][NT][kSteps][2];  // Q^T: head g of tile nt, this thread's elements
    float o[NT][kSteps][4];              // O^T: rows 2j, 2j + 1 of chunk g; heads 2t, 2t + 1
    float cs[NT][2], m[NT][2], l[NT][2];

    for (int i = 0; i < count; ++i) {
      const int slot = i % NS;
      __syncwarp();
      const Fp4Record r = recs[i % kFp4Records];
      const int tokens = r.info & 255;
      const int h = r.hp / head_tiles, ht = r.hp - h * head_tiles;
      const int head0 = h * G + ht * 8 * NT;  // first query head of the unit
      const int heads = min(8 * NT, G - ht * 8 * NT);
      if (i == 0 || (r.info & kRecBegin)) {
        // ---- the pair's queries ----
        // fp16 holds a row scaled by a power of two to a maximum in [2^13, 2^14)
        // (bf16 exactly, unless an element is 2^-30 of the largest).
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const int head = nt * 8 + g;
          float x[D / 4];
          if (head < heads) {
            const T* src = static_cast<const T*>(p.query) + r.s * p.query_stride +
                           (size_t)(head0 + head) * D + t * (D / 4);
            constexpr int kPer = ElemTraits<T>::kPerChunk;
#pragma unroll
            for (int c = 0; c < D / 4 / kPer; ++c)
              ElemTraits<T>::unpack(ldg_nc_v4(src + c * kPer), x + c * kPer);
          } else {
#pragma unroll
            for (int e = 0; e < D / 4; ++e) x[e] = 0.f;
          }
          uint32_t top = 0;
#pragma unroll
          for (int e = 0; e < D / 4; ++e) top = max(top, __float_as_uint(x[e]) & 0x7fffffffu);
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
          const uint32_t ex = max(top >> 23, 14u);
          const float up = __uint_as_float((267u - ex) << 23);
          const float down = __uint_as_float((ex - 13u) << 23);
          cs[nt][0] = __shfl_sync(0xffffffffu, down, 8 * t) * p.scale_log2;
          cs[nt][1] = __shfl_sync(0xffffffffu, down, 8 * t + 4) * p.scale_log2;
#pragma unroll
          for (int j = 0; j < kSteps; ++j)
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              const float x0 = x[4 * j + 2 * b] * up, x1 = x[4 * j + 2 * b + 1] * up;
              const uint32_t hi = pack_half2(x0, x1);
              q[0][nt][j][b] = hi;
              if constexpr (kF32) q[1][nt][j][b] = pack_half2(x0 - half_lo(hi), x1 - half_hi(hi));
            }
          m[nt][0] = m[nt][1] = -INFINITY;
          l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
          for (int j = 0; j < kSteps; ++j)
#pragma unroll
            for (int c = 0; c < 4; ++c) o[nt][j][c] = 0.f;
        }
      }
      {
        const bool w = mbar_wait_bounded(bars + 8u * slot, (i / NS) & 1, p.err, p.wait_limit);
        ok = __all_sync(0xffffffffu, w);
        if (!ok) break;
      }
      const uint32_t stage = ring + slot * C::kStageBytes;

      // ---- scores of 32 tokens: rows g (tile 2u) and g + 8 (tile 2u + 1) ----
      float sc[2][NT][4];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 4; ++c) sc[u][nt][c] = 0.f;
        constexpr int kWords = D / 32;  // of a thread's quarter row
        uint32_t kw[2][kWords], ks[2][D / 64];  // codes; scales of 16 elements as pairs
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t tile = stage + (2 * u + e) * C::kTileBytes;
          const uint32_t row = tile + g * (D / 2) + t * (D / 8);
          const uint32_t sca = tile + fp4_key_scales(D) + g * (D / 16) + t * (D / 64);
          if constexpr (D == 64) {
            const uint2 v = lds_u64(row);
            kw[e][0] = v.x;
            kw[e][1] = v.y;
            const uint32_t two = e4m3x2_to_half2(lds_u8(sca));
            ks[e][0] = __byte_perm(two, 0, 0x1010);
          } else {
#pragma unroll
            for (int c = 0; c < kWords / 4; ++c) {
              const uint4 v = lds128(row + 16 * c);
              kw[e][4 * c] = v.x;
              kw[e][4 * c + 1] = v.y;
              kw[e][4 * c + 2] = v.z;
              kw[e][4 * c + 3] = v.w;
              const uint32_t two = e4m3x2_to_half2(lds_u16(sca + 2 * c));
              ks[e][2 * c] = __byte_perm(two, 0, 0x1010);
              ks[e][2 * c + 1] = __byte_perm(two, 0, 0x3232);
            }
          }
        }
#pragma unroll
        for (int w = 0; w < kWords; ++w) {
          uint32_t lo[4], hi[4];
          e2m1x8_to_half2(kw[0][w], lo);
          e2m1x8_to_half2(kw[1][w], hi);
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            lo[b] = half2_mul(lo[b], ks[0][w / 2]);
            hi[b] = half2_mul(hi[b], ks[1][w / 2]);
          }
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            const uint32_t a[4] = {lo[2 * b], hi[2 * b], lo[2 * b + 1], hi[2 * b + 1]};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int part = 0; part < kQParts; ++part)
                mma_f16(sc[u][nt], a, q[part][nt][2 * w + b]);
          }
        }
      }

      // ---- softmax: the maximum moves only when a score passes it by 2^8 ----
      const bool whole = tokens == kFp4Stage;
      float over = -INFINITY;
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            sc[u][nt][c] *= cs[nt][c & 1];
            if (!whole && u * 16 + (c >> 1) * 8 + g >= tokens) sc[u][nt][c] = -INFINITY;
            over = fmaxf(over, sc[u][nt][c] - m[nt][c & 1]);
          }
      if (__any_sync(0xffffffffu, over > kFp4Lift + kFp4Slack)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const float top = group_max<4>(fmaxf(fmaxf(sc[0][nt][c], sc[0][nt][c + 2]),
                                                 fmaxf(sc[1][nt][c], sc[1][nt][c + 2])));
            const float m_new = fmaxf(m[nt][c], top - kFp4Lift);
            const float alpha = m_new == -INFINITY ? 1.f : fast_exp2(m[nt][c] - m_new);
            m[nt][c] = m_new;
            l[nt][c] *= alpha;
#pragma unroll
            for (int j = 0; j < kSteps; ++j) {
              o[nt][j][c] *= alpha;
              o[nt][j][c + 2] *= alpha;
            }
          }
      }
      uint32_t pt[kQParts][2][NT][2];  // P^T: head g; tokens 2t, 2t + 1 of tile 2u (+ 1)
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float w0 = fast_exp2(sc[u][nt][2 * e] - m[nt][0]);
            const float w1 = fast_exp2(sc[u][nt][2 * e + 1] - m[nt][1]);
            l[nt][0] += w0;
            l[nt][1] += w1;
            const uint32_t two = pack_half2(w0, w1);
            pt[0][u][nt][e] = transpose8x8(two);
            if constexpr (kF32)
              pt[1][u][nt][e] = transpose8x8(pack_half2(w0 - half_lo(two), w1 - half_hi(two)));
          }

      // ---- values ----
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        constexpr int kParts = D == 256 ? 2 : 1;  // groups of a thread's chunk of D / 8 elements
        constexpr int kWords = D == 64 ? 1 : 2;   // words of a part, per token
#pragma unroll
        for (int part = 0; part < kParts; ++part) {
          uint32_t x[2][kWords], y[2][kWords], vs[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t tile = stage + (2 * u + e) * C::kTileBytes;
            const int group = D == 64 ? g >> 1 : g * kParts + part;
            uint32_t wa[kWords], wb[kWords];
            if constexpr (D == 64) {
              const uint32_t at = tile + fp4_value_codes(D) + group * 64 + t * 16 + (g & 1) * 4;
              wa[0] = lds_u32(at);
              wb[0] = lds_u32(at + 8);
            } else {
              const uint4 v = lds128(tile + fp4_value_codes(D) + group * 64 + t * 16);
              wa[0] = v.x;
              wa[1] = v.y;
              wb[0] = v.z;
              wb[1] = v.w;
            }
            uint32_t two = lds_u16(tile + fp4_value_scales(D) + group * 8 + 2 * t);
            if (!whole) {
              // Rows past the sequence's end hold anything: a zero scale.
              const int tok = u * 16 + e * 8 + 2 * t;
              if (tok >= tokens) two = 0;
              else if (tok + 1 >= tokens) two &= 0xffu;
            }
            vs[e] = e4m3x2_to_half2(two);
            // Bytes of the two tokens' codes of one element.
#pragma unroll
            for (int w = 0; w < kWords; ++w) {
              x[e][w] = (wa[w] & 0x0f0f0f0fu) | ((wb[w] << 4) & 0xf0f0f0f0u);
              y[e][w] = ((wa[w] >> 4) & 0x0f0f0f0fu) | (wb[w] & 0xf0f0f0f0u);
            }
          }
#pragma unroll
          for (int w = 0; w < kWords; ++w) {
            uint32_t x0[4], y0[4], x1[4], y1[4];
            e2m1x8_to_half2(x[0][w], x0);
            e2m1x8_to_half2(y[0][w], y0);
            e2m1x8_to_half2(x[1][w], x1);
            e2m1x8_to_half2(y[1][w], y1);
#pragma unroll
            for (int b = 0; b < 4; ++b) {
              const uint32_t a[4] = {half2_mul(x0[b], vs[0]), half2_mul(y0[b], vs[0]),
                                     half2_mul(x1[b], vs[1]), half2_mul(y1[b], vs[1])};
              const int j = part * 8 + w * 4 + b;
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int qp = 0; qp < kQParts; ++qp) mma_f16(o[nt][j], a, pt[qp][u][nt]);
            }
          }
        }
      }

      // ---- the slot is free: the next stage ----
      if (issued < count) {
        issue(next_id);
        if (prepared < count) next_id = prepare();
      }

      // ---- the end of the pair, or of the warp's part ----
      if (r.info & (kRecFinish | kRecLast)) {
        const bool begun = (r.info & kRecFinish) ? i - r.k >= 0 : false;
        // Sums over the tokens' lanes.
        float ls[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float v = l[nt][c];
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
            ls[nt][c] = v;
          }
        if (begun) {
          // The whole pair: final rows.
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const int head = nt * 8 + 2 * t + c;
              if (head >= heads) continue;
              const float inv = p.value_scale / ls[nt][c];
              T* dst = static_cast<T*>(p.out) +
                       ((size_t)r.s * p.num_heads + head0 + head) * D + g * (D / 8);
              if constexpr (kF32) {
#pragma unroll
                for (int j = 0; j < kSteps; j += 2)
                  *reinterpret_cast<float4*>(dst + 2 * j) =
                      make_float4(o[nt][j][c] * inv, o[nt][j][c + 2] * inv, o[nt][j + 1][c] * inv,
                                  o[nt][j + 1][c + 2] * inv);
              } else {
#pragma unroll
                for (int j = 0; j < kSteps; j += 4) {
                  uint32_t w[4];
#pragma unroll
                  for (int b = 0; b < 4; ++b)
                    w[b] = pack_bf16x2(o[nt][j + b][c] * inv, o[nt][j + b][c + 2] * inv);
                  stg_v4(dst + 2 * j, make_uint4(w[0], w[1], w[2], w[3]));
                }
              }
            }
        } else {
          // A part: to the ring at the end of the warp's part (every copy has
          // landed and been read), to global memory before.
          const bool last = (r.info & kRecLast) != 0;
          float* dst = last ? reinterpret_cast<float*>(smem + warp * C::kWarpRing)
                            : p.warp_partials + ((size_t)blockIdx.x * W + warp) * part_floats;
          __syncwarp();
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const int head = nt * 8 + 2 * t + c;
              if (head >= heads) continue;
              float* od = dst + head * D + g * (D / 8);
#pragma unroll
              for (int j = 0; j < kSteps; j += 2)
                *reinterpret_cast<float4*>(od + 2 * j) =
                    make_float4(o[nt][j][c], o[nt][j][c + 2], o[nt][j + 1][c], o[nt][j + 1][c + 2]);
              if (g == 0) {
                dst[rows * D + head] = m[nt][c];
                dst[rows * D + rows + head] = ls[nt][c];
              }
            }
          if (lane == 0) {
            const int pair = r.s * per_seq + r.hp;
            if (last) left[warp].b = pair;
            else left[warp].a = pair;
          }
        }
      }
    }
    if (!ok) {
      // A wait gave up: this warp's copies in flight end before it leaves.
      for (int i = max(0, issued - NS); i < issued; ++i)
        mbar_wait_bounded(bars + 8u * (i % NS), (i / NS) & 1, p.err);
    }
  }

  // ---- zero rows of empty sequences ----
  for (int s = blockIdx.x * W + warp; s < p.num_seqs; s += gridDim.x * W)
    if (p.seq_lens[s] <= 0) {
      uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(p.out) + (size_t)s * p.num_heads * D);
      for (int i = lane; i < p.num_heads * D * (int)sizeof(T) / 16; i += 32)
        stg_v4(dst + i, make_uint4(0u, 0u, 0u, 0u));
    }

  // ---- merge over the CTA's warps ----
  if (cta0 >= cta1) return;  // the same for the whole CTA
  __syncthreads();
  // The pairs that reach over the CTA's ends (the same for every thread).
  const Fp4Place first = locate(cta0), final_ = locate(cta1 - 1);
  const int head_pair = first.k > 0 ? first.s * per_seq + first.hp : -1;
  const int tail_pair = final_.k + 1 < final_.n ? final_.s * per_seq + final_.hp : -1;
  // Runs of parts of one pair: part 2w is warp w's a, part 2w + 1 its b; runs[]
  // holds the first part of each run, and the end.
  if (tid == 0) {
    int count = 0, last_pair = -1, end = 0;
    for (int i = 0; i < 2 * W; ++i) {
      const int pair = (i & 1) ? left[i >> 1].b : left[i >> 1].a;
      if (pair < 0) continue;
      if (pair != last_pair) runs[count++] = i;
      last_pair = pair;
      end = i + 1;
    }
    runs[count] = end;
    misc[0] = count;
  }
  __syncthreads();
  const int num_runs = misc[0];
  auto part_at = [&](int i) -> const float* {
    return (i & 1) ? reinterpret_cast<const float*>(smem + (i >> 1) * C::kWarpRing)
                   : p.warp_partials + ((size_t)blockIdx.x * W + (i >> 1)) * part_floats;
  };
  auto part_pair = [&](int i) { return (i & 1) ? left[i >> 1].b : left[i >> 1].a; };
  constexpr int kLaneCols = D / 32;
  auto write_row = [&](int pair, int head, const float* acc, float sum) {
    const int s = pair / per_seq, hp = pair - s * per_seq;
    const int h = hp / head_tiles, ht = hp - h * head_tiles;
    const float inv = p.value_scale / sum;
    T* dst = static_cast<T*>(p.out) +
             ((size_t)s * p.num_heads + h * G + ht * 8 * NT + head) * D + lane * kLaneCols;
#pragma unroll
    for (int e = 0; e < kLaneCols; ++e) dst[e] = ElemTraits<T>::from_float(acc[e] * inv);
  };
  auto heads_of = [&](int pair) {
    const int ht = pair % head_tiles;  // per_seq is a multiple of head_tiles
    return min(8 * NT, G - ht * 8 * NT);
  };
  for (int unit = warp; unit < num_runs * rows; unit += W) {
    const int run = unit / rows, head = unit - run * rows;
    const int i0 = runs[run], i1 = runs[run + 1];
    const int pair = part_pair(i0);
    if (head >= heads_of(pair)) continue;
    float top = -INFINITY;
    for (int i = i0; i < i1; ++i)
      if (part_pair(i) == pair) top = fmaxf(top, part_at(i)[rows * D + head]);
    float acc[kLaneCols], sum = 0.f;
#pragma unroll
    for (int e = 0; e < kLaneCols; ++e) acc[e] = 0.f;
    for (int i = i0; i < i1; ++i) {
      if (part_pair(i) != pair) continue;
      const float* src = part_at(i);
      const float mi = src[rows * D + head];
      const float w = mi == top ? 1.f : fast_exp2(mi - top);
      sum = fmaf(src[rows * D + rows + head], w, sum);
#pragma unroll
      for (int e = 0; e < kLaneCols; ++e)
        acc[e] = fmaf(src[head * D + lane * kLaneCols + e], w, acc[e]);
    }
    if (pair != head_pair && pair != tail_pair) {
      write_row(pair, head, acc, sum);
    } else {
      float* dst = p.cta_partials +
                   ((size_t)blockIdx.x * 2 + (pair == head_pair ? 0 : 1)) * part_floats;
#pragma unroll
      for (int e = 0; e < kLaneCols; ++e) dst[head * D + lane * kLaneCols + e] = acc[e];
      if (lane == 0) {
        dst[rows * D + head] = top;
        dst[rows * D + rows + head] = sum;
      }
    }
  }
  if (head_pair < 0 && tail_pair < 0) return;

  // ---- merge over CTAs, by the last of a pair's CTAs to arrive ----
  __threadfence();
  __syncthreads();
  // CTAs of a pair: from the one with its first stage to the one with its last.
  const long long head_at = cta0 - first.k, tail_at = cta1 - 1 - final_.k;
  for (int which = 0; which < 2; ++which) {
    const int pair = which == 0 ? head_pair : tail_pair;
    if (pair < 0 || (which == 1 && tail_pair == head_pair)) continue;
    const long long at = which == 0 ? head_at : tail_at;
    const int n = which == 0 ? first.n : final_.n;
    const int c0 = (int)(at / share), c1 = (int)((at + n - 1) / share);
    if (tid == 0) {
      const unsigned int before = atomicAdd(p.counters + c0, 1u);
      const bool last = before == (unsigned)(c1 - c0);
      if (last) p.counters[c0] = 0u;
      misc[1] = last;
    }
    __syncthreads();
    const bool last = misc[1] != 0;
    __syncthreads();
    if (!last) continue;
    __threadfence();
    for (int head = warp; head < heads_of(pair); head += W) {
      auto src_of = [&](int c) {
        return p.cta_partials + ((size_t)c * 2 + (c == c0 ? 1 : 0)) * part_floats;
      };
      float top = -INFINITY;
      for (int c = c0 + lane; c <= c1; c += 32) top = fmaxf(top, __ldcg(src_of(c) + rows * D + head));
      top = group_max<1>(top);
      float acc[kLaneCols], sum = 0.f;
#pragma unroll
      for (int e = 0; e < kLaneCols; ++e) acc[e] = 0.f;
#pragma unroll 4
      for (int c = c0; c <= c1; ++c) {
        const float* src = src_of(c);
        const float mi = __ldcg(src + rows * D + head);
        const float w = mi == top ? 1.f : fast_exp2(mi - top);
        sum = fmaf(__ldcg(src + rows * D + rows + head), w, sum);
#pragma unroll
        for (int e = 0; e < kLaneCols; ++e)
          acc[e] = fmaf(__ldcg(src + head * D + lane * kLaneCols + e), w, acc[e]);
      }
      write_row(pair, head, acc, sum);
    }
  }
}

}  // namespace pa
