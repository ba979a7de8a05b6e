// Decode attention over the 8-bit pool for sm_103a.
//
// For one sequence and KV head, with the query heads of its group as columns,
//   S [tokens x heads]  = K [tokens x D] . Q^T [D x heads] * key scale of the token's block
//   O^T [D x heads]    += V^T [D x tokens] . (P * value scale)^T [tokens x heads],
// P = 2^(S - m) with a running maximum m.  Reading the pool bounds it.  A code becomes fp16
// (exactly) by a byte permutation and a subtraction per pair in the registers of the thread
// that uses it as an operand of mma.sync; with the matrix instructions a step of 32 tokens
// of 128 elements takes a warp about 640 instructions, and an SM, which gets the step's 8 KB in
// 370 clocks at HBM's rate, could issue 1480.  (tcgen05 would take its operands from shared or
// tensor memory: the fp16 codes would have to be written there and read again, 4 bytes a code beside
// the one that comes.  e4m3 codes, which it takes as they are, would round queries and weights to
// four bits.)  The pool's layout is made for this: ldmatrix gives a tile's keys, and with .trans
// its values, as the matrix instructions' fragments.
//
// Every warp works for itself.  The stages of 16 to 64 tokens of all (sequence, KV head)
// pairs, laid end to end, are cut into equal ranges, one per CTA, and those into equal
// parts, one per warp; a warp streams its part through a ring of its own (bulk copies that
// its lanes issue, one per block; no barrier with other warps) and keeps S, P, m and O in
// registers.  A pair that a warp saw whole is written out; parts of a pair are merged over
// the CTA's warps at the end, and over CTAs by whichever finishes last, always in the
// same order.
//
// Two stages a warp, 132 KB on their way per SM: with three (198 KB) the memory gives less (8 x
// 32768 tokens take 8% longer, 384 x 1500 10%), and so it does without the hint that L2 may drop
// the lines first (1%; 128 sequences of up to 2100 tokens 6%).
//
// Weights times value scales enter their product as one fp16 number in bf16 calls, half a step 2^-11 of
// it, and as two in fp32 calls.  Of the bf16 outputs one in eleven is thereby the other neighbour of the exact
// result than the one that exact weights give (1% more error against 64 bits than the output's own rounding
// makes).  Two for bf16 as well take 0.5% longer for 8 x 32768 tokens, 1 to 5% for smaller
// batches, 6% where the blocks' weights are kept, 16% for 16 heads a group: not taken.
//
// Value scales: O is kept in units of the pair's largest value scale so far (rounded up
// to a power of two, so that nothing but the ratios' own rounding is lost), which moves with the
// maximum.
//
// kWeights: every cell (16 tokens, or a block of 8) hands on, for each head, the sum of its
// weights and the maximum that they are relative to; a second launch adds them up when
// the rows' maxima and sums are known.
//
// Measured (graph replays in a row, data larger than L2, 6776 GB/s = 100%):
//   8 x 32768 tokens, 32 heads on 8 of 128, bf16     84 us    538 MB  94%  (with weights 91 us)
//   the same with blocks of 256                      82 us            97%
//   the same with 64 heads, with 128 heads on 8      86, 97 us        92%, 82%
//   the same in fp32                                 85 us            93%
//   16 x 32768 tokens, 32 heads on 8 of 64           86 us    539 MB  93%
//   8 x 32768 tokens, 32 heads on 4 of 256           88 us    538 MB  90%
//   384 x 1500 tokens, 32 heads on 8 of 128         185 us   1.19 GB  95%
//   128 sequences of 0 .. 2100 tokens                50 us    273 MB  80%  (56 us)
//   32 sequences of 1 .. 2048 tokens, 40 heads       53 us    311 MB  86%
//   64 sequences of 0 .. 2048 tokens, 14 on 2 of 64  13.0 us               (16.8 us)
//   four sequences of up to 100 tokens                6.1 us
// One box differs from another by 1%.
// What is left of the short ones is the launch (2.5 us), lengths, tables and first copies one
// after another (4 us), steps of a lone warp (1.5 us each) and merges over CTAs (3 to 4 us);
// 16 heads of 128 are bound by instructions (8 warps, two column tiles).
#pragma once

#include <cuda_bf16.h>
#include <float.h>
#include <math.h>

#include "decode_int8.cuh"
#include "pa_int8.cuh"
#include "warp_decode.cuh"

namespace pa {

// Weights are 2^(S - m + lift), and scores may pass the running maximum by the slack before
// it moves: lift + slack = 15, the most that fp16 holds.  fp16 has steps of 2^-24, so a
// weight is off by up to 2^-25 where the largest is 2^lift or more.
__host__ __device__ constexpr float int8_lift(bool fp32) { return fp32 ? 11.f : 7.f; }
constexpr float kInt8Top = 15.f;
// Units of a launch are at most about this many, so that two sums of them fit an int.
constexpr int kInt8MaxWork = (1 << 30) - 1;
// Tokens of a chain of sums: rounded additions drop whatever is below half a step of a sum, so
// a chain's sums are added to the piece's in global memory.
constexpr int kInt8Chain = 4096;
// A pair's queries and its end count as this many stages (at one, 128 sequences of up to 2100 tokens
// take 3% longer, 32 of 40 pairs each 0.5%).
constexpr int kInt8PairCost = 2;
constexpr int kInt8Whole = 512;  // tokens of a pair that may stay whole with a warp (256, 1024: the same)

// Four 8 x 8 matrices of 16-bit elements (rows of 16 bytes at the lanes' addresses), as they
// lie or transposed.
__device__ __forceinline__ void ldmatrix4(uint32_t* r, uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at));
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t* r, uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at));
}

// A power of two at or above a scale, and never so small that its reciprocal is not a number.
__device__ __forceinline__ float int8_unit(float scale) {
  const uint32_t b = (__float_as_uint(fmaxf(scale, 0x1p-120f)) + 0x7fffffu) & 0x7f800000u;
  return __uint_as_float(min(b, 0x7e800000u));  // 2^126
}

// A warp's place: stage k, at unit `at`, of the n stages of pair (s, hp).
struct Int8Place {
  int s, hp, k, n, len;
  int at;
};

// A piece: consecutive stages of one pair in a warp's part.
struct Int8Piece {
  int s, hp;       // the pair
  int k0, stages;  // its first stage, and how many
  int n, len;      // stages and tokens of the sequence
  int at;          // the unit of its first stage
};

// The parts of one pair in a CTA: warps `first` .. w, w the last of them,
// whose run it is.  A part that reaches its warp's end lies in the warp's ring,
// one that ends before it in global memory.  The pair has parts in `ctas` CTAs
// from cta0 on; s < 0: no run.
struct Int8Run {
  int s, head0, heads;  // the pair's sequence and query heads
  int first, cta0, ctas;
};

template <typename T, int D, int H, bool kWeights>
struct Int8Config {
  static constexpr bool kF32 = sizeof(T) == 4;
  static constexpr int kWarps = int8_warps(D, H, kF32, kWeights);
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kTileBytes = int8_tile_bytes(D);
  static constexpr int kStep = int8_step(D, kWarps);
  static constexpr int kStage = int8_stage(D, kWarps);
  static constexpr int kStageBytes = kStage / kInt8Tile * kTileBytes;
  static constexpr int kWholeStages = kWarps * kStep / kStage;  // a step per warp
  static constexpr int kStages = 2;
  static constexpr int kWarpRing = kStages * kStageBytes;
  // Ring of a warp's pieces: when a piece ends, the stages in flight, the one that waits
  // for a slot and the one after it may all have entered pieces of their own.
  static constexpr int kPieceRing = kStages + 3 <= 8 ? 8 : 16;
  static constexpr int kBars = kWarps * kWarpRing;
  static constexpr int kPieces = kBars + 8 * kWarps * kStages;
  static constexpr int kPre = (kPieces + kWarps * kPieceRing * (int)sizeof(Int8Piece) + 15) / 16 * 16;
  static constexpr int kRuns = (kPre + 4 * (kThreads + 2 * kWarps) + 15) / 16 * 16;
  static constexpr int kSmem = kRuns + (int)sizeof(Int8Run) * 2 * kWarps;
  static_assert(kStages >= 2 && kStages + 3 <= kPieceRing, "rings");
  static_assert(kBars % 16 == 0, "barriers are aligned");
  static_assert(kSmem <= 227 * 1024, "shared memory");
  static_assert(int8_partial_floats(H, D) * 4 <= kWarpRing, "a part fits its warp's ring");
  static_assert(H <= kInt8Rows, "counters");
};

template <typename T, int D, int H, bool kWeights>
__global__ void __launch_bounds__(Int8Config<T, D, H, kWeights>::kThreads, 1)
    decode_int8_kernel(const Int8DecodeParams p) {
  using C = Int8Config<T, D, H, kWeights>;
  constexpr bool kF32 = C::kF32;
  constexpr int W = C::kWarps;
  constexpr int NS = C::kStages;
  constexpr int U = C::kStep / 16;          // row tiles of a step
  constexpr int NT = H / 8;                 // tiles of eight columns
  constexpr int kChunks = D / 16;           // of 16 elements
  constexpr int kQParts = kF32 ? 2 : 1;
  constexpr float kLift = int8_lift(kF32);
  constexpr int TB = C::kTileBytes;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  const int G = p.group;
  const int head_tiles = D == 256 ? (G + 7) / 8 : 1;  // units of a KV head
  const int rows = int8_unit_rows(H, G);
  const int per_seq = p.num_kv_heads * head_tiles;  // pairs of a sequence
  const int l2bs = p.log2_block_size;
  constexpr int kVec = D / 32;  // columns of a lane in a merge
  const int part_floats = int8_partial_floats(rows, D);

  extern __shared__ __align__(128) uint8_t smem[];
  const uint32_t ring = smem_u32(smem) + (uint32_t)warp * C::kWarpRing;
  const uint32_t bars = smem_u32(smem) + C::kBars + (uint32_t)warp * NS * 8;
  Int8Piece* pieces = reinterpret_cast<Int8Piece*>(smem + C::kPieces) + warp * C::kPieceRing;
  // First query head and heads of a pair.
  auto heads_of = [&](int hp, int* heads) -> int {
    const int h = hp / head_tiles, ht = hp - h * head_tiles;
    *heads = min(H, G - ht * H);
    return h * G + ht * H;
  };
  // Units before each thread's sequences; the warps' sums and their sequences.
  int* warp_sums = reinterpret_cast<int*>(smem + C::kPre);
  int* warp_seqs = warp_sums + W;
  int* pre = warp_seqs + W;
  Int8Run* runs = reinterpret_cast<Int8Run*>(smem + C::kRuns);  // [warp][ended before, at its end]
  if (lane == 0) {
    for (int i = 0; i < NS; ++i) mbar_init(bars + 8u * i, 1);
    runs[2 * warp].s = runs[2 * warp + 1].s = -1;
  }
  if (lane == 0) fence_mbar_init();
  grid_dependency_wait();
  grid_dependents_launch();

  // ---- the work: units of every sequence, scanned ----
  auto stages_of = [&](int s, int* len_out) -> int {
    const int len = p.seq_lens[s];
    *len_out = len;
    if (len <= 0) return 0;
    if (((len - 1) >> l2bs) >= p.max_blocks_per_seq) return 0;
    return (int)((unsigned)(len - 1) / C::kStage) + 1;
  };
  // Sums stop at kInt8MaxWork: an error then, and nothing is computed.
  const int chunk = (p.num_seqs + C::kThreads - 1) / C::kThreads;
  int total, pairs;
  {
    int mine = 0, seqs = 0;
    for (int s = tid * chunk; s < min((tid + 1) * chunk, p.num_seqs); ++s) {
      int len;
      const int n = stages_of(s, &len);
      if (n == 0 && len > 0 && blockIdx.x == 0) record_error(p.err, PA_DEVERR_SEQ_LEN);
      seqs += n > 0;
      if (n > 0)
        mine = (int)min(mine + (long long)(n + kInt8PairCost) * per_seq, (long long)kInt8MaxWork);
    }
    int sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum = min(sum + v, kInt8MaxWork);
    }
    seqs = __reduce_add_sync(0xffffffffu, seqs);
    if (lane == 31) {
      warp_sums[warp] = sum;
      warp_seqs[warp] = seqs;
    }
    __syncthreads();
    const unsigned other = lane < W ? (unsigned)warp_sums[lane] : 0u;
    const unsigned base = __reduce_add_sync(0xffffffffu, lane < warp ? other : 0u);
    // The warps' sum may pass 32 bits, that of their upper halves does not.
    const unsigned all = __reduce_add_sync(0xffffffffu, other);
    const bool most = __reduce_add_sync(0xffffffffu, other >> 16) >= (kInt8MaxWork >> 16);
    pre[tid] = (int)base + sum - mine;
    if (tid == 0 && blockIdx.x == 0) {
      if (most) record_error(p.err, PA_DEVERR_SEQ_LEN);
      if (kWeights) p.counters[kInt8Refused] = most;  // no weights to add up
    }
    total = most ? 0 : (int)all;
    pairs = __reduce_add_sync(0xffffffffu, lane < W ? warp_seqs[lane] : 0) * per_seq;
    __syncthreads();
  }
  // Units of a CTA: an equal share, at least a step per two warps (fewer parts to
  // merge where there is little work).
  const int share = max((total + (int)gridDim.x - 1) / (int)gridDim.x, C::kWholeStages / 2);
  int cta0 = (int)min((long long)share * blockIdx.x, (long long)total);
  int cta1 = min(cta0 + share, total);

  // The first stage whose unit is `unit` or a later one of the same pair.  All
  // lanes look: the last thread whose sequences begin at or before the unit, then
  // the sequence.
  auto locate = [&](int unit) -> Int8Place {
    constexpr int kSpan = C::kThreads / 32;
    const int seg = __popc(__ballot_sync(0xffffffffu, pre[lane * kSpan] <= unit)) - 1;
    const int own = lane < kSpan ? pre[seg * kSpan + lane] : 0x7fffffff;
    const int off = __popc(__ballot_sync(0xffffffffu, own <= unit)) - 1;
    int acc = __shfl_sync(0xffffffffu, own, off);
    Int8Place pl;
    pl.s = (seg * kSpan + off) * chunk;
    while (true) {
      pl.n = stages_of(pl.s, &pl.len);
      const int next = pl.n > 0 ? acc + (pl.n + kInt8PairCost) * per_seq : acc;
      if (next > unit) break;
      acc = next;
      ++pl.s;
    }
    const int size = pl.n + kInt8PairCost;
    pl.hp = (unit - acc) / size;
    const int at = acc + pl.hp * size + kInt8PairCost;
    pl.k = max(unit - at, 0);
    pl.at = at + pl.k;
    return pl;
  };

  // Ends of CTAs' and warps' parts that would cut a short pair move behind it: the
  // pair stays whole with the warp (or, of several warps, the CTA) of its first unit,
  // and nothing is left to merge.  Short is a pair of no more stages than a warp's part
  // has, and of kInt8Whole tokens at most (whole pairs leave the warps less even); for a
  // CTA whose share is at most a step per warp, one of up to that.  Both only where the
  // average pair is short.
  // The CTA's two ends, then the warp's: a loop, as one-time code is paid by its length.
  bool ok = true;
  const int per_warp = (share + W - 1) / W;
  auto short_of = [&](int stages) {  // the average pair has at most about so many
    return total <= (long long)pairs * (stages + kInt8PairCost);
  };
  const bool few = share <= C::kWholeStages && short_of(C::kWholeStages);
  const int most_w = min(per_warp, kInt8Whole / C::kStage);
  const int whole_w = !few && short_of(most_w) ? most_w : 0;
  const int whole_cta = few ? C::kWholeStages : whole_w;
  int share_w = 0, my0 = 0, my1 = 0;
  Int8Place pp = {};  // the next stage to copy
#pragma unroll 1
  for (int i = whole_cta ? 0 : 3; i < 4; ++i) {
    if (i == 2 || (i == 3 && !whole_w)) {
      share_w = (cta1 - cta0 + W - 1) / W;
      my1 = min(cta0 + share_w * (warp + 1), cta1);
      if (!whole_w) i = 3;
    }
    int unit = i == 0 ? cta0 : i == 1 ? cta1 : i == 2 ? my1 : cta0 + share_w * warp;
    if (i == 3) my0 = unit;
    if (i == 3 ? unit >= my1 : unit <= 0 || unit >= total) continue;
    pp = locate(unit);
    const int first = pp.at - pp.k - kInt8PairCost;  // the pair's first unit
    if (unit > first && pp.n <= (i < 2 ? whole_cta : whole_w)) {
      unit = first + kInt8PairCost + pp.n;
      pp.k = 0;
      pp.at = unit + kInt8PairCost;
      if (i == 3 && unit < my1 && ++pp.hp == per_seq) {
        pp.hp = 0;
        do {
          ++pp.s;
          pp.n = stages_of(pp.s, &pp.len);
        } while (pp.n == 0);
      }
    }
    if (i == 0) cta0 = unit;
    else if (i == 1) cta1 = unit;
    else if (i == 2) my1 = unit;
    else my0 = unit;
  }
  if (my0 < my1 && pp.at < my1) {
    const int per_block = min(C::kStage / kInt8Tile, 1 << (l2bs - 3));  // tiles of a copy
    const uint32_t lane_dst = (uint32_t)(lane * per_block) * TB;
    const uint32_t block_bytes = ((uint32_t)p.num_kv_heads << (l2bs - 3)) * TB;

    // ---- producer: the next stage to copy, its table entry already fetched ----
    int entered = 0, issued = 0;
    bool more = true;                // there is a stage after the ones fetched
    const int32_t* table = nullptr;  // the sequence's row, from this lane's block
    const uint8_t* head_base = nullptr;
    auto enter = [&]() {  // a piece begins
      table = p.block_tables + (size_t)pp.s * p.max_blocks_per_seq + lane;
      const int h = pp.hp / head_tiles;
      head_base = p.cache + ((size_t)h << (l2bs - 3)) * TB;
      if (lane == 0)
        pieces[entered % C::kPieceRing] =
            Int8Piece{pp.s, pp.hp, pp.k, min(pp.n - pp.k, my1 - pp.at), pp.n, pp.len, pp.at};
      ++entered;
    };
    enter();
    struct Next {
      int id, tiles;
      const uint8_t* base;
    };
    auto fetch = [&]() -> Next {
      const int tok0 = pp.k * C::kStage;
      Next nx;
      nx.tiles = min(C::kStage / kInt8Tile, (pp.len - tok0 + kInt8Tile - 1) >> 3);
      nx.base = head_base + ((tok0 & ((1 << l2bs) - 1)) >> 3) * TB;
      nx.id = lane * per_block < nx.tiles ? __ldg(table + (tok0 >> l2bs)) : 0;
      // On to the next stage, if it is this warp's.
      ++pp.at;
      if (++pp.k == pp.n) {
        pp.at += kInt8PairCost;
        pp.k = 0;
        more = pp.at < my1;
        if (more) {
          if (++pp.hp == per_seq) {
            pp.hp = 0;
            do {
              ++pp.s;
              pp.n = stages_of(pp.s, &pp.len);
            } while (pp.n == 0);
          }
          enter();
        }
      } else {
        more = pp.at < my1;
      }
      return nx;
    };
    // One copy per block into slot `slot`.
    auto issue = [&](const Next& nx, int slot) {
      const uint32_t bar = bars + 8u * slot;
      const uint32_t dst = ring + slot * C::kStageBytes + lane_dst;
      const int mine = min(per_block, nx.tiles - lane * per_block);
      const bool bad = (unsigned)nx.id >= (unsigned)p.num_blocks;  // false in lanes without a block
      __syncwarp();
      if (!__any_sync(0xffffffffu, bad)) {
        if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)nx.tiles * TB);
        if (mine > 0)
          bulk_load_once(dst, nx.base + (uint64_t)(uint32_t)nx.id * block_bytes, (uint32_t)mine * TB, bar);
      } else {
        // A block outside the pool: scales of zero.
        const uint32_t bytes = mine > 0 && !bad ? (uint32_t)mine * TB : 0u;
        const uint32_t sum = __reduce_add_sync(0xffffffffu, bytes);
        if (lane == 0) mbar_arrive_expect_tx(bar, sum);
        if (bytes) bulk_load_once(dst, nx.base + (uint64_t)(uint32_t)nx.id * block_bytes, bytes, bar);
        if (bad) {
          record_error(p.err, PA_DEVERR_BLOCK_ID);
          for (int i = 0; i < mine; ++i)
            asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(dst + i * TB), "r"(0u)
                         : "memory");
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
        __syncwarp();  // other lanes read the zeros, which no barrier announces
      }
      ++issued;
    };

    Next next;
    bool have = false;  // `next` waits for a slot
    {
      // Fill the ring, every table entry on its way before the first is needed.
      Next first[NS];
      int n = 0;
#pragma unroll
      for (int i = 0; i < NS; ++i)
        if (more) {
          first[i] = fetch();
          ++n;
        }
      if ((have = more)) next = fetch();
#pragma unroll
      for (int i = 0; i < NS; ++i)
        if (i < n) issue(first[i], i);
    }

    uint32_t q[kQParts][NT][kChunks][2];  // Q^T: head g of tile nt, elements 4t .. 4t + 3 of a chunk
    float o[NT][kChunks][4];  // O^T: rows 2g, 2g + 1 of a chunk; columns 2t, 2t + 1
    float cs[NT][2], m[NT][2], l[NT][2];
    float unit = 0.f, inv_unit = 0.f;  // of the values: a power of two
    int slot = 0;
    uint32_t parity = 0;
    bool fresh = true;  // the piece has no maximum yet
    int rows_here = 0;  // the pair's heads
    // Where the lane's row of a step's ldmatrix lies: matrix i is tile i of the step (U == 2),
    // or tile i mod 2 of chunk i / 2 (U == 1); for keys always the latter, of a row tile.
    const uint32_t key_lane = kInt8Header + ((lane >> 3) & 1) * TB + (lane >> 4) * 128 + (lane & 7) * 16;
    const uint32_t value_lane =
        (uint32_t)int8_value_codes(D) + (U == 2 ? (lane >> 3) * TB + (lane & 7) * 16
                                                : ((lane >> 3) & 1) * TB + (lane >> 4) * 128 + (lane & 7) * 16);

    // One step in `stage`, its first `tokens` tokens valid.  One body for whole
    // and for ragged steps: the branches below are small and the same for the
    // warp, where a second body would be fetched anew at every sequence's end.
    // `cell`: the first of the step's cells of this pair's heads, if weights are handed on.
    auto attend = [&](const uint32_t stage, const int tokens, float2* cell) {
      const bool ragged = tokens < C::kStep;
      float ks[2 * U], vs[2 * U];  // scales of the step's tiles; no value where no token is
      float vmax = 0.f;
#pragma unroll
      for (int e = 0; e < 2 * U; ++e) {
        const uint2 v = lds_u64(stage + e * TB);
        ks[e] = __uint_as_float(v.x);
        vs[e] = 8 * e < tokens ? __uint_as_float(v.y) : 0.f;
        vmax = fmaxf(vmax, vs[e]);
      }
      // ---- scores: rows g (tile 2u) and g + 8 (tile 2u + 1) ----
      float sc[U][NT][4];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        // The matrix unit cuts its sums off towards zero.  For fp32 they are kept short, 64
        // elements, and added up with rounding.
        constexpr int kSum = kF32 ? 4 : kChunks;  // chunks of one chain
        float own[NT][4];
#pragma unroll
        for (int j = 0; j < kChunks; j += 2) {
          uint32_t w[4];
          ldmatrix4(w, stage + 2 * u * TB + j * 128 + key_lane);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const uint32_t a[4] = {int8x2_to_half2<0, 1>(w[2 * c]), int8x2_to_half2<0, 1>(w[2 * c + 1]),
                                   int8x2_to_half2<2, 3>(w[2 * c]), int8x2_to_half2<2, 3>(w[2 * c + 1])};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int part = kQParts - 1; part >= 0; --part) {  // small parts first
                if ((j + c) % kSum == 0 && part == kQParts - 1)
                  mma_f16_first(own[nt], a, q[part][nt][j + c]);
                else
                  mma_f16(own[nt], a, q[part][nt][j + c]);
              }
          }
          if ((j + 2) % kSum == 0)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int c = 0; c < 4; ++c)
                sc[u][nt][c] = j + 2 == kSum ? own[nt][c] : sc[u][nt][c] + own[nt][c];
        }
      }
      // Rounded here, so that the largest less the maximum is exact.
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 4; ++c)
            sc[u][nt][c] = __fmul_rn(sc[u][nt][c], __fmul_rn(cs[nt][c & 1], ks[2 * u + (c >> 1)]));

      // ---- softmax: the maximum moves only when a score passes it by the slack ----
      float y[U][NT][4];
      auto weigh = [&]() {  // exponents; their maximum of this thread
        float over = -INFINITY;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 4; ++c)
              y[u][nt][c] = __fsub_rn(sc[u][nt][c], m[nt][c & 1]);
        if (ragged) {
#pragma unroll
          for (int u = 0; u < U; ++u)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int c = 0; c < 4; ++c)
                if (u * 16 + (c >> 1) * 8 + g >= tokens) y[u][nt][c] = -INFINITY;
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 4; ++c) over = fmaxf(over, y[u][nt][c]);
        return over;
      };
      if (fresh || __any_sync(0xffffffffu, weigh() > kInt8Top || vmax > unit)) {
        const float unit_new = int8_unit(fmaxf(unit, vmax));
        const float shrink = unit * (1.f / unit_new);  // exact: powers of two
        unit = unit_new;
        inv_unit = 1.f / unit;
        fresh = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float top = -INFINITY;
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
              for (int e = c; e < 4; e += 2)
                if (u * 16 + (e >> 1) * 8 + g < tokens) top = fmaxf(top, sc[u][nt][e]);
            top = group_max<4>(top);
            // Rounded up, so that no weight passes 2^lift where the steps are wide.  Never
            // minus infinity: scores below the least number weigh nothing then.
            const float m_new = fmaxf(fmaxf(m[nt][c], __fsub_ru(top, kLift)), -FLT_MAX);
            const float alpha = fast_exp2(m[nt][c] - m_new);
            m[nt][c] = m_new;
            l[nt][c] *= alpha;
            const float both = alpha * shrink;
#pragma unroll
            for (int j = 0; j < kChunks; ++j) {
              o[nt][j][c] *= both;
              o[nt][j][c + 2] *= both;
            }
          }
        weigh();
      }
      uint32_t pt[kQParts][U][NT][2];  // P^T: head g; tokens 2t, 2t + 1 of tile 2u (+ 1)
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float w[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            w[c] = fast_exp2(y[u][nt][c]);
            l[nt][c & 1] += w[c];
          }
          if constexpr (kWeights) {
            // Sums over the tokens of a cell: both halves of the rows, or each.
            const int l2cell = int8_log2_cell(l2bs);
            float a[4] = {w[0], w[1], w[2], w[3]};
            if (l2cell == 4) a[0] += a[2], a[1] += a[3];
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) {
              a[0] += __shfl_xor_sync(0xffffffffu, a[0], off);
              a[1] += __shfl_xor_sync(0xffffffffu, a[1], off);
            }
            if (l2cell == 3)
#pragma unroll
              for (int off = 4; off < 32; off <<= 1) {
                a[2] += __shfl_xor_sync(0xffffffffu, a[2], off);
                a[3] += __shfl_xor_sync(0xffffffffu, a[3], off);
              }
            if (g == 0)
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                const int half = c >> 1, head = nt * 8 + 2 * t + (c & 1);
                if ((half == 0 || l2cell == 3) && 16 * u + 8 * half < tokens && head < rows_here)
                  cell[((16 * u + 8 * half) >> l2cell) * (size_t)p.num_heads + head] =
                      make_float2(a[c], m[nt][c & 1]);
              }
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float r = vs[2 * u + e] * inv_unit;
            const float w0 = w[2 * e] * r, w1 = w[2 * e + 1] * r;
            const uint32_t two = pack_half2(w0, w1);
            pt[0][u][nt][e] = transpose8x8(two);
            if constexpr (kF32)
              pt[1][u][nt][e] = transpose8x8(pack_half2(w0 - half_lo(two), w1 - half_hi(two)));
          }
        }

      // ---- values: the matrix unit's chains end with the step, and are added with rounding ----
      auto add = [&](int j, const uint32_t (*w)[2]) {  // w[u]: tiles 2u, 2u + 1
        float own[NT][4];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const uint32_t a[4] = {int8x2_to_half2<0, 2>(w[u][0]), int8x2_to_half2<1, 3>(w[u][0]),
                                 int8x2_to_half2<0, 2>(w[u][1]), int8x2_to_half2<1, 3>(w[u][1])};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int part = kQParts - 1; part >= 0; --part) {  // small parts first
              if (u == 0 && part == kQParts - 1) mma_f16_first(own[nt], a, pt[part][u][nt]);
              else mma_f16(own[nt], a, pt[part][u][nt]);
            }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 4; ++c) o[nt][j][c] += own[nt][c];
      };
      if constexpr (U == 2) {
#pragma unroll
        for (int j = 0; j < kChunks; ++j) {
          uint32_t w[4];
          ldmatrix4_trans(w, stage + j * 128 + value_lane);
          const uint32_t both[2][2] = {{w[0], w[1]}, {w[2], w[3]}};
          add(j, both);
        }
      } else {
#pragma unroll
        for (int j = 0; j < kChunks; j += 2) {
          uint32_t w[4];
          ldmatrix4_trans(w, stage + j * 128 + value_lane);
          const uint32_t one[1][2] = {{w[0], w[1]}}, two[1][2] = {{w[2], w[3]}};
          add(j, one);
          add(j + 1, two);
        }
      }
    };

    bool last = false;
    for (int piece = 0; !last; ++piece) {
      __syncwarp();
      // What is needed of the record at the piece's end is read then, as registers are
      // short between.
      const Int8Piece& rec = pieces[piece % C::kPieceRing];
      const int len = rec.len;
      float2* cells = nullptr;  // of the pair's first head
      // ---- the pair's queries ----
      {
        int heads;
        const int head0 = heads_of(rec.hp, &heads);
        if constexpr (kWeights) {
          rows_here = heads;
          cells = p.cells + (size_t)rec.s * ((size_t)p.max_blocks_per_seq << (l2bs - int8_log2_cell(l2bs))) *
                                p.num_heads + head0;
        }
        // fp16 holds a row scaled by a power of two to a maximum in [2^13, 2^14)
        // (bf16 exactly, unless an element is 2^-30 of the largest).
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const int head = nt * 8 + g;
          float x[D / 4];
          if (head < heads) {
            const T* src = static_cast<const T*>(p.query) + rec.s * p.query_stride +
                           (size_t)(head0 + head) * D + 4 * t;
#pragma unroll
            for (int j = 0; j < kChunks; ++j) {
              if constexpr (kF32) {
                ElemTraits<T>::unpack(ldg_nc_v4(src + 16 * j), x + 4 * j);
              } else {
                const uint2 v = __ldg(reinterpret_cast<const uint2*>(src + 16 * j));
                x[4 * j] = bf16_lo(v.x);
                x[4 * j + 1] = bf16_hi(v.x);
                x[4 * j + 2] = bf16_lo(v.y);
                x[4 * j + 3] = bf16_hi(v.y);
              }
            }
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
          for (int j = 0; j < kChunks; ++j)
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
          for (int j = 0; j < kChunks; ++j)
#pragma unroll
            for (int c = 0; c < 4; ++c) o[nt][j][c] = 0.f;
        }
      }
      fresh = true;
      unit = 0.f;
      constexpr int kChainStages = kInt8Chain / C::kStage;
      for (int k = rec.k0; k < rec.k0 + rec.stages;) {
        const int chain_end = min(k + kChainStages, rec.k0 + rec.stages);
        for (; k < chain_end; ++k) {
          if (ok) {
            const bool w = wait_phase(bars + 8u * slot, parity, p.err, p.wait_limit);
            ok = __all_sync(0xffffffffu, w);
          }
          if (ok)
#pragma unroll 1
            for (int t0 = 0; t0 < C::kStage && k * C::kStage + t0 < len; t0 += C::kStep)
              attend(ring + slot * C::kStageBytes + t0 / kInt8Tile * TB,
                     min(len - k * C::kStage - t0, C::kStep),
                     kWeights ? cells + (size_t)((k * C::kStage + t0) >> int8_log2_cell(l2bs)) * p.num_heads
                              : nullptr);
          // The slot is free: the next stage.  After a wait that gave up nothing is
          // copied or computed any more, but the parts are still handed on, so that
          // the counters come out even.
          if (have) {
            if (ok) issue(next, slot);
            if ((have = more)) next = fetch();
          }
          if (++slot == NS) {
            slot = 0;
            parity ^= 1;
          }
        }
        if (__builtin_expect(rec.stages > kChainStages, 0)) {
          // The sums of the piece's chains that ended before are added to this one's, at
          // its maximum and unit; then they are put away for the next.
          const bool first = k - rec.k0 == kChainStages, final = k == rec.k0 + rec.stages;
          float* past =
              p.chains + ((size_t)blockIdx.x * W + warp) * int8_chain_floats(D, H) + lane;
          const float shrink = first ? 0.f : past[0] * inv_unit;
          past[0] = unit;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              float* at = past + (1 + (nt * 2 + c) * (2 * kChunks + 2)) * 32;
              const float w = first ? 0.f : fast_exp2(at[0] - m[nt][c]);
              auto join = [&](int i, float by, float& sum) {
                if (!first) sum = fmaf(at[32 * i], by, sum);
                if (!final) {
                  at[32 * i] = sum;
                  sum = 0.f;
                }
              };
              join(1, w, l[nt][c]);
#pragma unroll
              for (int j = 0; j < kChunks; ++j) {
                join(2 * j + 2, w * shrink, o[nt][j][c]);
                join(2 * j + 3, w * shrink, o[nt][j][c + 2]);
              }
              at[0] = m[nt][c];
            }
        }
      }
      const Int8Piece pc = rec;
      int heads;
      const int head0 = heads_of(pc.hp, &heads);
      const bool ends = pc.k0 + pc.stages == pc.n;
      last = pc.at + pc.stages + (ends ? kInt8PairCost : 0) >= my1;

      // ---- the piece is done ----
      const bool whole = pc.k0 == 0 && pc.stages == pc.n;
      // A part goes to the ring at the end of the warp's part (every copy has
      // landed and been read), to global memory before.
      float* to = last ? reinterpret_cast<float*>(smem + warp * C::kWarpRing)
                       : p.warp_partials + ((size_t)blockIdx.x * W + warp) * part_floats;
      __syncwarp();
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float sum = l[nt][c];  // over the tokens' lanes
#pragma unroll
          for (int off = 4; off < 32; off <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
          const int head = nt * 8 + 2 * t + c;
          if (head >= heads) continue;
          if (whole) {
            const float inv = 1.f / sum;
            const size_t row = (size_t)pc.s * p.num_heads + head0 + head;
            T* dst = static_cast<T*>(p.out) + row * D + 2 * g;
#pragma unroll
            for (int j = 0; j < kChunks; ++j) {
              const float v0 = o[nt][j][c] * inv * unit, v1 = o[nt][j][c + 2] * inv * unit;
              if constexpr (kF32) *reinterpret_cast<float2*>(dst + 16 * j) = make_float2(v0, v1);
              else *reinterpret_cast<uint32_t*>(dst + 16 * j) = pack_bf16x2(v0, v1);
            }
            if (kWeights && g == 0) p.rows[row] = make_float2(m[nt][c], sum);
          } else {
            float* dst = to + head * D + 2 * g;
#pragma unroll
            for (int j = 0; j < kChunks; ++j)
              *reinterpret_cast<float2*>(dst + 16 * j) = make_float2(o[nt][j][c], o[nt][j][c + 2]);
            if (g == 0) {
              to[rows * D + head] = m[nt][c];
              to[rows * D + rows + head] = sum;
              to[rows * D + 2 * rows + head] = unit;
            }
          }
        }
      if (!whole) {
        // The warp with the pair's last part in this CTA says where the parts are.
        if (lane == 0 && (ends || pc.at + pc.stages == cta1)) {
          const int at = pc.at - pc.k0;  // the pair's first stage
          const bool here = at >= cta0 && at + pc.n <= cta1;
          const int c0 = here ? (int)blockIdx.x : at / share;
          runs[2 * warp + last] = Int8Run{pc.s, head0, heads, at <= cta0 ? 0 : (at - cta0) / share_w,
                                          c0, here ? 1 : (at + pc.n - 1) / share - c0 + 1};
        }
      }
    }
    if (!ok) {
      // A wait gave up: cells and rows of this call are missing, and the weights stay.
      if (kWeights && lane == 0) p.counters[kInt8GaveUp] = 1u;
      // This warp's copies in flight end before it leaves.
      // Slot i's last copy is its (issued - 1 - i) / NS + 1-th.
      for (int i = 0; i < NS && i < issued; ++i)
        mbar_wait_bounded(bars + 8u * i, ((issued - 1 - i) / NS) & 1, p.err);
    }
  }

  // ---- zero rows of empty sequences ----
  for (int s = blockIdx.x * W + warp; s < p.num_seqs; s += gridDim.x * W)
    if (p.seq_lens[s] <= 0) {
      uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(p.out) + (size_t)s * p.num_heads * D);
      for (int i = lane; i < p.num_heads * D * (int)sizeof(T) / 16; i += 32)
        stg_v4(dst + i, make_uint4(0u, 0u, 0u, 0u));
    }

  // ---- merges ----
  // A warp takes one head of a pair, first over the CTA's warps; then, for a pair with
  // parts in other CTAs, the last warp to arrive with its head merges those, up to
  // kInt8Gather at a time: the groups of the pair's CTAs, then their results.  Of a CTA's
  // counters for each head the first is for the group of the pair that it continues, the second for
  // the first group of the pair that it begins, the third for the results of that pair's
  // groups; its four slots hold its part of the pair that it continues, of the one that it
  // begins, and the groups' results likewise.  One short loop for all levels: code that runs
  // once is paid by its length.
  if (cta0 >= cta1) return;  // the same for the whole CTA
  __syncthreads();
  static_assert(W <= kInt8Gather, "merges");
  uint32_t live = __ballot_sync(0xffffffffu, lane < 2 * W && runs[lane % (2 * W)].s >= 0);
  for (int u0 = 0; live; live &= live - 1, u0 += rows) {
    // Head u of all runs' is warp u mod W's.
    int head = (warp - u0) & (W - 1);
    if (head >= rows) continue;
    const int which = __ffs(live) - 1;
    const Int8Run run = runs[which];
    for (; head < run.heads; head += W) {
      const int col = head * D + lane * kVec;
      // Parts i < n lie `step` bytes apart from `base` on, but for part `odd`.
      const uint8_t* base = smem + run.first * C::kWarpRing;
      uint32_t step = C::kWarpRing;
      int n = (which >> 1) - run.first + 1;
      int odd = (which & 1) ? -1 : n - 1;
      const float* odd_part =
          p.warp_partials + ((size_t)blockIdx.x * W + (which >> 1)) * part_floats;
      for (int level = 0;; ++level) {
        auto part = [&](int i) {
          return i == odd ? odd_part : reinterpret_cast<const float*>(base + i * step);
        };
        float mi = -INFINITY, li = 0.f, ui = 0.f, acc[kVec];
        if (lane < n) {
          const float* src = part(lane) + rows * D + head;
          mi = src[0];
          li = src[rows];
          ui = src[2 * rows];
        }
        // Four parts at a time (past the last, that one again, with no weight); the
        // first ones are on their way with the maxima and sums.
        constexpr int kBatch = 4;
        float top = 0.f, w = 0.f, sum = 0.f, unit = 0.f;
#pragma unroll
        for (int e = 0; e < kVec; ++e) acc[e] = 0.f;
#pragma unroll 1
        for (int i0 = 0; i0 < n; i0 += kBatch) {
          alignas(16) float v[kBatch][kVec];
#pragma unroll
          for (int i = 0; i < kBatch; ++i) {
            const float* src = part(min(i0 + i, n - 1)) + col;
            if constexpr (kVec == 2) {
              *reinterpret_cast<float2*>(v[i]) = *reinterpret_cast<const float2*>(src);
            } else {
#pragma unroll
              for (int e = 0; e < kVec; e += 4)
                *reinterpret_cast<float4*>(v[i] + e) = *reinterpret_cast<const float4*>(src + e);
            }
          }
          if (i0 == 0) {
            top = warp_max_redux(mi);
            unit = warp_max_redux(ui);
            w = lane >= n ? 0.f : mi == top ? 1.f : fast_exp2(mi - top);
            sum = lane < n ? li * w : 0.f;
            w *= ui * (1.f / unit);  // exact: powers of two
#pragma unroll
            for (int o = 1; o < kInt8Gather; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            sum = __shfl_sync(0xffffffffu, sum, 0);
          }
#pragma unroll
          for (int i = 0; i < kBatch; ++i) {
            const float wi = __shfl_sync(0xffffffffu, w, i0 + i);
#pragma unroll
            for (int e = 0; e < kVec; ++e) acc[e] = fmaf(v[i][e], wi, acc[e]);
          }
        }
        const int group = ((int)blockIdx.x - run.cta0) / kInt8Gather;
        const int groups = (run.ctas + kInt8Gather - 1) / kInt8Gather;
        if (level == (run.ctas == 1 ? 0 : groups == 1 ? 1 : 2)) {
          const float inv = 1.f / sum;
          const size_t row = (size_t)run.s * p.num_heads + run.head0;
          T* dst = static_cast<T*>(p.out) + row * D + col;
#pragma unroll
          for (int e = 0; e < kVec; e += 2) {
            const float v0 = acc[e] * inv * unit, v1 = acc[e + 1] * inv * unit;
            if constexpr (kF32) *reinterpret_cast<float2*>(dst + e) = make_float2(v0, v1);
            else *reinterpret_cast<uint32_t*>(dst + e) = pack_bf16x2(v0, v1);
          }
          if (kWeights && lane == 0) p.rows[row + head] = make_float2(top, sum);
          break;
        }
        // Hand the part on; whoever is last takes the next level.  Lane 0's atomic
        // releases what the warp's lanes wrote before and acquires, for all of
        // them, what the others' released.
        const int at = level == 0 ? (int)blockIdx.x : run.cta0 + group * kInt8Gather;
        float* to =
            p.cta_partials + ((size_t)at * 4 + 2 * level + (at == run.cta0)) * part_floats;
#pragma unroll
        for (int e = 0; e < kVec; e += 2)
          *reinterpret_cast<float2*>(to + col + e) = make_float2(acc[e], acc[e + 1]);
        if (lane == 0) {
          to[rows * D + head] = top;
          to[rows * D + rows + head] = sum;
          to[rows * D + 2 * rows + head] = unit;
        }
        __syncwarp();
        const int first = level == 0 ? run.cta0 + group * kInt8Gather : run.cta0;
        const int parts = level == 0 ? min(kInt8Gather, run.ctas - group * kInt8Gather) : groups;
        int go = 0;
        if (lane == 0) {
          unsigned int* counter =
              p.counters + (first * 3 + (level == 1 ? 2 : first == run.cta0)) * kInt8Rows + head;
          unsigned int before;
          asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;"
                       : "=r"(before)
                       : "l"(counter)
                       : "memory");
          go = before == (unsigned)parts - 1;
          if (go) *counter = 0u;
        }
        if (!__shfl_sync(0xffffffffu, go, 0)) break;
        __syncwarp();
        n = parts;
        const float* slot0 = p.cta_partials + ((size_t)first * 4 + 2 * level) * part_floats;
        base = reinterpret_cast<const uint8_t*>(slot0);
        step = (level == 0 ? 1u : (uint32_t)kInt8Gather) * 16u * part_floats;
        odd = first == run.cta0 ? 0 : -1;
        odd_part = slot0 + part_floats;
      }
    }
  }
}

}  // namespace pa
