// Decode attention over the 4-bit pool for sm_103a.
//
// For one sequence and KV head, with the query heads of its group as columns,
//   S [tokens x heads]  = K [tokens x D] . Q^T [D x heads]
//   O^T [D x heads]    += V^T [D x tokens] . P^T [tokens x heads],
// P = 2^(S - m) with a running maximum m.  Reading the pool bounds it: at the rate
// of HBM an SM gets about 23 bytes of codes and scales per clock, 41 elements,
// each of which has to become fp16 before a product.  A conversion takes one
// instruction per pair of codes and one multiplication per pair by the scales
// (exact), on pipes that pass 16 lanes per clock and scheduler; with the matrix
// instructions a step of 32 tokens of 128 elements takes a warp about 400
// instructions and an SM 140 to 150 clocks (measured: 1.34 per instruction on such
// a pipe and 4.6 per matrix instruction, per scheduler), 30 to 32 bytes per clock:
// 1.3 times what the memory gives, so nothing more fits.  So the codes go
// from shared memory to registers once, are converted there, and are used there: the
// operands of mma.sync are the converting thread's own registers.  Tensor-memory or
// shared-memory operands would put a second trip of 2 bytes per element on the
// path (82 bytes written and 82 read per clock of 128).  The pool's layout is made
// for this: a tile's key rows and value groups are the matrix instructions'
// fragments.
//
// Every warp works for itself.  The stages of 32 or 64 tokens of all (sequence, KV
// head) pairs, laid end to end, are cut into equal ranges, one per CTA, and
// those into equal parts, one per warp; a warp streams its part through a ring
// of its own (bulk copies that its lanes issue, one per block; no barrier with
// other warps) and keeps S, P, m and O in registers.  A pair that a warp saw
// whole is written out; parts of a pair are merged over the CTA's warps at the
// end, and over CTAs by whichever finishes last, always in the same order.
//
// Measured (graph replays in a row, data larger than L2, 6766 GB/s = 100%):
//   8 x 32768 tokens, 32 heads on 8 of 128, bf16   59 us  302 MB  5.1 TB/s  75%
//   the same with 64 heads on 8                    65 us                    69%
//   the same with 64 heads on 8 of 64              45 us  151 MB            50%
//   8 x 32768 tokens, 64 heads on 8 of 128, fp32   92 us  302 MB            48%
//   32 sequences of 1 .. 2048 tokens, 40 heads     44 us  181 MB            61%
//   384 sequences of 1500 tokens, 32 heads on 8   125 us  670 MB            79%
//   64 sequences of 0 .. 2048 tokens, 14 on 2 of 64  14.5 us
//   four sequences of up to 100 tokens               10 us
// Of the long batch reading alone takes 57 us and the arithmetic alone 55; the
// launch, the lengths and the first copies take 5 to 6 us, and merges over CTAs 4,
// and these are what is left of the short ones.  Heads of 64 pay a step's fixed
// part (exponents, softmax) for half the elements; fp32 doubles the matrix
// instructions.
#pragma once

#include <cuda_bf16.h>
#include <float.h>
#include <math.h>

#include <type_traits>

#include "decode_fp4.cuh"
#include "pa_fp4.cuh"

namespace pa {

// Weights are 2^(S - m + lift), and scores may pass the running maximum by the slack before
// it moves: lift + slack = 15, the most that fp16 holds.  fp16 has steps of 2^-24, so a
// weight is off by up to 2^-25 where the largest is 2^lift or more: 2^-32 of it for bf16,
// whose half step that stays below for millions of them, and 2^-36 for fp32 (8 x 32768
// tokens as with 2^-32 to 0.4%; 2^-39 would cost 1%, as the maximum moves more often).
__host__ __device__ constexpr float fp4_lift(bool fp32) { return fp32 ? 11.f : 7.f; }
constexpr float kFp4Top = 15.f;
constexpr int kFp4RingBytes = 216 * 1024;
// Units of a launch are at most about this many (5 TB of reads at 128 elements, half a
// second and more; sequences may share blocks), so that two sums of them fit an int.
constexpr int kFp4MaxWork = (1 << 30) - 1;
// Tokens of a chain of sums.  Sums over more lose what is small beside them: the matrix
// unit cuts off, and rounded additions drop whatever is below half a step (a warp
// that sees a million tokens of a pair: bf16 1e-2 of the result, fp32 2.8e-4).  So a
// chain's sums are added, with rounding, to the piece's in global memory: fp32 outputs are
// then off by 1e-6 to 1.5e-6 up to 131072 tokens of a warp and 6e-6 at a million, bf16 ones
// by 4e-5 before their rounding.  At one in 128 stages it costs nothing; its code costs
// every call 0 to 0.7 us (four short sequences 9.7 -> 10.3).
constexpr int kFp4Chain = 4096;
// A pair's queries and its end count as this many stages (32 sequences of 40 pairs
// each: 52 us at 0, 43 at 1, 44 at 2).
constexpr int kFp4PairCost = 1;
constexpr int kFp4Whole = 512;  // tokens of a pair that may stay whole with a warp (see there)

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

// Wait for a phase of `bar`, at most `limit` cycles from the first look on; a
// wait that runs out records PA_DEVERR_TIMEOUT and returns false.
__device__ __forceinline__ bool wait_phase(uint32_t bar, uint32_t parity, unsigned int* err,
                                           long long limit) {
  if (mbar_test(bar, parity)) return true;
  const long long t0 = clock64();
  while (clock64() - t0 < limit)
    if (mbar_try_wait(bar, parity)) return true;
  record_error(err, PA_DEVERR_TIMEOUT);
  return false;
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
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

// c = a . b.
__device__ __forceinline__ void mma_f16_first(float* c, const uint32_t* a, const uint32_t* b) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%10, %10, %10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]), "f"(0.f));
}

// Products added to c: by the matrix unit, or (kShort) in a chain of their own that
// done() adds with rounding.  The unit cuts its sums off towards zero, which makes a
// sum over n products about 1e-8 n too small: over kFp4Chain tokens 4e-5.  That is less
// than bf16's half step of 2^-8 by far (short chains would cost 1% of the time at four
// heads of 128, 9% at eight), but not fp32's, where the unit's chains end with their step
// of 32 tokens.  The small parts of queries and weights go first, where they cut nothing off
// the large ones' sum (errors a fifth smaller).
template <bool kShort>
struct Fp4Sum {
  float* c;
  float own[4];
  __device__ __forceinline__ Fp4Sum(float* to) : c(to) {}
  __device__ __forceinline__ void operator()(const uint32_t* a, const uint32_t* b, bool first) {
    if (!kShort) mma_f16(c, a, b);
    else if (first) mma_f16_first(own, a, b);
    else mma_f16(own, a, b);
  }
  __device__ __forceinline__ void done() {
    if (kShort)
#pragma unroll
      for (int i = 0; i < 4; ++i) c[i] += own[i];
  }
};

// The 8 x 8 matrix of 16-bit elements that the warp holds, transposed.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// a times the low (kHigh: the high) half of s, which the multiplication takes
// as an operand's half without an instruction of its own.
template <bool kHigh>
__device__ __forceinline__ uint32_t half2_mul_by(uint32_t a, uint32_t s) {
  uint32_t r;
  if constexpr (kHigh)
    asm("{\n\t.reg .b16 l, h;\n\t.reg .b32 t;\n\tmov.b32 {l, h}, %2;\n\tmov.b32 t, {h, h};\n\t"
        "mul.rn.f16x2 %0, %1, t;\n\t}"
        : "=r"(r)
        : "r"(a), "r"(s));
  else
    asm("{\n\t.reg .b16 l, h;\n\t.reg .b32 t;\n\tmov.b32 {l, h}, %2;\n\tmov.b32 t, {l, l};\n\t"
        "mul.rn.f16x2 %0, %1, t;\n\t}"
        : "=r"(r)
        : "r"(a), "r"(s));
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

// The work in units: every pair is kFp4PairCost units (its queries, its end),
// then one per stage.  A stage belongs to the warp whose part its unit is in.
// A warp's place: stage k, at unit `at`, of the n stages of pair (s, hp).
struct Fp4Place {
  int s, hp, k, n, len;
  int at;
};

// A piece: consecutive stages of one pair in a warp's part.
struct Fp4Piece {
  int s, hp;       // the pair
  int k0, stages;  // its first stage, and how many
  int n, len;      // stages and tokens of the sequence
  int at;          // the unit of its first stage
};

// The parts of one pair in a CTA: warps `first` .. w, w the last of them,
// whose run it is.  A part that reaches its warp's end lies in the warp's ring,
// one that ends before it in global memory.  The pair has parts in `ctas` CTAs
// from cta0 on; s < 0: no run.
struct Fp4Run {
  int s, head0, heads;  // the pair's sequence and query heads
  int first, cta0, ctas;
};

template <typename T, int D, int H>
struct Fp4Config {
  static constexpr bool kF32 = sizeof(T) == 4;
  static constexpr int kWarps = fp4_warps(D, H, kF32);
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kTileBytes = fp4_tile_bytes(D);
  static constexpr int kStage = fp4_stage(D);
  static constexpr int kStageBytes = kStage / kFp4Tile * kTileBytes;
  static constexpr int kWholeStages = kWarps * kFp4Step / kStage;  // a step per warp
  static constexpr int kFit = kFp4RingBytes / kWarps / kStageBytes;
  static constexpr int kStages = kFit < 6 ? kFit : 6;
  static constexpr int kWarpRing = kStages * kStageBytes;
  // Ring of a warp's pieces: when a piece ends, the stages in flight, the one that waits
  // for a slot and the one after it may all have entered pieces of their own.
  static constexpr int kPieceRing = kStages + 3 <= 8 ? 8 : 16;
  static constexpr int kBars = kWarps * kWarpRing;
  static constexpr int kPieces = kBars + 8 * kWarps * kStages;
  static constexpr int kPre = (kPieces + kWarps * kPieceRing * (int)sizeof(Fp4Piece) + 15) / 16 * 16;
  static constexpr int kRuns = (kPre + 4 * (kThreads + 2 * kWarps) + 15) / 16 * 16;
  static constexpr int kSmem = kRuns + (int)sizeof(Fp4Run) * 2 * kWarps;
  static_assert(kStages >= 2 && kStages + 3 <= kPieceRing, "rings");
  static_assert(kSmem <= 227 * 1024, "shared memory");
  static_assert(fp4_partial_floats(H, D, 2) * 4 <= kWarpRing, "a part fits its warp's ring");
};

// H: query heads of a unit, 4, 8 or 16.  With four, the matrix instructions'
// eight columns are the heads twice, for a value's even and odd elements: a
// byte's two codes are then used as they come, as the two elements of one token
// (P zero in the other element's place), where otherwise the codes of two tokens
// have to be brought together first (measured at fp4_heads).
template <typename T, int D, int H>
__global__ void __launch_bounds__(Fp4Config<T, D, H>::kThreads, 1)
    decode_fp4_kernel(const Fp4DecodeParams p) {
  using C = Fp4Config<T, D, H>;
  constexpr bool kF32 = C::kF32;
  constexpr int W = C::kWarps;
  constexpr int NS = C::kStages;
  constexpr bool kNarrow = H == 4;
  constexpr int NT = H == 16 ? 2 : 1;               // tiles of eight columns
  constexpr int kSteps = D / 16;                    // of QK
  constexpr int kTiles = kNarrow ? D / 32 : D / 16;  // of O^T
  constexpr int kQParts = kF32 ? 2 : 1;
  constexpr float kLift = fp4_lift(kF32);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  const int G = p.group;
  const int head_tiles = D == 256 ? (G + 7) / 8 : 1;  // units of a KV head (see fp4_heads)
  const int rows = fp4_unit_rows(H, G);
  const int per_seq = p.num_kv_heads * head_tiles;  // pairs of a sequence
  const int l2bs = p.log2_block_size;
  // A merge's unit: a head, or half of one where there are two warps per head.
  constexpr int kSplit = fp4_splits(D, H, W);  // units of a head
  constexpr int kVec = D / 32 / kSplit;             // columns of a lane
  const int per_run = rows * kSplit;                // units of a pair
  const int part_floats = fp4_partial_floats(rows, D, kSplit);

  extern __shared__ __align__(128) uint8_t smem[];
  const uint32_t ring = smem_u32(smem) + (uint32_t)warp * C::kWarpRing;
  const uint32_t bars = smem_u32(smem) + C::kBars + (uint32_t)warp * NS * 8;
  Fp4Piece* pieces = reinterpret_cast<Fp4Piece*>(smem + C::kPieces) + warp * C::kPieceRing;
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
  Fp4Run* runs = reinterpret_cast<Fp4Run*>(smem + C::kRuns);   // [warp][ended before, at its end]
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
  // Sums stop at kFp4MaxWork: an error then, and nothing is computed.
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
        mine = (int)min(mine + (long long)(n + kFp4PairCost) * per_seq, (long long)kFp4MaxWork);
    }
    int sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum = min(sum + v, kFp4MaxWork);
    }
    seqs = __reduce_add_sync(0xffffffffu, seqs);
    if (lane == 31) {
      warp_sums[warp] = sum;
      warp_seqs[warp] = seqs;
    }
    __syncthreads();
    const unsigned other = lane < W ? (unsigned)warp_sums[lane] : 0u;
    const unsigned base = __reduce_add_sync(0xffffffffu, lane < warp ? other : 0u);
    const unsigned all = __reduce_add_sync(0xffffffffu, other);
    // The warps' sum may pass 32 bits, that of their upper halves does not.
    const bool most = __reduce_add_sync(0xffffffffu, other >> 16) >= (kFp4MaxWork >> 16);
    pre[tid] = (int)base + sum - mine;
    if (most && tid == 0 && blockIdx.x == 0) record_error(p.err, PA_DEVERR_SEQ_LEN);
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
  auto locate = [&](int unit) -> Fp4Place {
    constexpr int kSpan = C::kThreads / 32;
    const int seg = __popc(__ballot_sync(0xffffffffu, pre[lane * kSpan] <= unit)) - 1;
    const int own = lane < kSpan ? pre[seg * kSpan + lane] : 0x7fffffff;
    const int off = __popc(__ballot_sync(0xffffffffu, own <= unit)) - 1;
    int acc = __shfl_sync(0xffffffffu, own, off);
    Fp4Place pl;
    pl.s = (seg * kSpan + off) * chunk;
    while (true) {
      pl.n = stages_of(pl.s, &pl.len);
      const int next = pl.n > 0 ? acc + (pl.n + kFp4PairCost) * per_seq : acc;
      if (next > unit) break;
      acc = next;
      ++pl.s;
    }
    const int size = pl.n + kFp4PairCost;
    pl.hp = (unit - acc) / size;
    const int at = acc + pl.hp * size + kFp4PairCost;
    pl.k = max(unit - at, 0);
    pl.at = at + pl.k;
    return pl;
  };

  // Ends of CTAs' and warps' parts that would cut a short pair move behind it: the
  // pair stays whole with the warp (or, of several warps, the CTA) of its first unit,
  // and nothing is left to merge, which takes a CTA 6 us where every warp cuts one.
  // Short is a pair of no more stages than a warp's part has, and of kFp4Whole tokens at
  // most: whole pairs leave the warps less even, by up to a pair, which is little beside a
  // merge only while pairs are short (32 heads on 8 of 128: 256 sequences of 128 tokens
  // 29.4 -> 20.6 us, 512 of 300, 64 heads, 60.3 -> 52.3, 1024 of up to 300 60.3 -> 57.5; but
  // 512 of up to 500 49.3 -> 53.4, of up to 1000 73.8 and 92.7 without the bound, 384 of
  // 1500 125 and 169).
  // For a CTA whose share is at most a step per warp it is a pair of up to that: latency
  // is what counts there, and a merge over CTAs costs more than the stages that it
  // spares (64 sequences of up to 500 tokens 12.4 -> 10.4 us, four of up to 100 9.7 ->
  // 8.3; with up to four steps per warp, 64 sequences of up to 2048 tokens took 16.5, not
  // 14.5 us).  Both only where the average pair is short (one sequence of 1024 tokens
  // looked in vain for 1.9 us).
  // The CTA's two ends, then the warp's: a loop, as one-time code is paid by its length.
  bool ok = true;
  const int per_warp = (share + W - 1) / W;
  auto short_of = [&](int stages) {  // the average pair has at most about so many
    return total <= (long long)pairs * (stages + kFp4PairCost);
  };
  const bool few = share <= C::kWholeStages && short_of(C::kWholeStages);
  const int most_w = min(per_warp, kFp4Whole / C::kStage);
  const int whole_w = !few && short_of(most_w) ? most_w : 0;
  const int whole_cta = few ? C::kWholeStages : whole_w;
  int share_w = 0, my0 = 0, my1 = 0;
  Fp4Place pp = {};  // the next stage to copy
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
    const int first = pp.at - pp.k - kFp4PairCost;  // the pair's first unit
    if (unit > first && pp.n <= (i < 2 ? whole_cta : whole_w)) {
      unit = first + kFp4PairCost + pp.n;
      pp.k = 0;
      pp.at = unit + kFp4PairCost;
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
    const int per_block = min(C::kStage / kFp4Tile, 1 << (l2bs - 3));  // tiles of a copy
    const uint32_t lane_dst = (uint32_t)(lane * per_block) * C::kTileBytes;
    const uint32_t block_bytes = ((uint32_t)p.num_kv_heads << (l2bs - 3)) * C::kTileBytes;

    // ---- producer: the next stage to copy, its table entry already fetched ----
    int entered = 0, issued = 0;
    bool more = true;                // there is a stage after the ones fetched
    const int32_t* table = nullptr;  // the sequence's row, from this lane's block
    const uint8_t* head_base = nullptr;
    auto enter = [&]() {  // a piece begins
      table = p.block_tables + (size_t)pp.s * p.max_blocks_per_seq + lane;
      const int h = pp.hp / head_tiles;
      head_base = p.cache + ((size_t)h << (l2bs - 3)) * C::kTileBytes;
      if (lane == 0)
        pieces[entered % C::kPieceRing] =
            Fp4Piece{pp.s, pp.hp, pp.k, min(pp.n - pp.k, my1 - pp.at), pp.n, pp.len, pp.at};
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
      nx.tiles = min(C::kStage / kFp4Tile, (pp.len - tok0 + kFp4Tile - 1) >> 3);
      nx.base = head_base + ((tok0 & ((1 << l2bs) - 1)) >> 3) * C::kTileBytes;
      nx.id = lane * per_block < nx.tiles ? __ldg(table + (tok0 >> l2bs)) : 0;
      // On to the next stage, if it is this warp's.
      ++pp.at;
      if (++pp.k == pp.n) {
        pp.at += kFp4PairCost;
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
        if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)nx.tiles * C::kTileBytes);
        if (mine > 0)
          bulk_load(dst, nx.base + (uint64_t)(uint32_t)nx.id * block_bytes, (uint32_t)mine * C::kTileBytes, bar);
      } else {
        // A block outside the pool: zero keys and values.
        const uint32_t bytes = mine > 0 && !bad ? (uint32_t)mine * C::kTileBytes : 0u;
        const uint32_t sum = __reduce_add_sync(0xffffffffu, bytes);
        if (lane == 0) mbar_arrive_expect_tx(bar, sum);
        if (bytes) bulk_load(dst, nx.base + (uint64_t)(uint32_t)nx.id * block_bytes, bytes, bar);
        if (bad) {
          record_error(p.err, PA_DEVERR_BLOCK_ID);
          for (int i = 0; i < mine * C::kTileBytes; i += 16)
            asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(dst + i), "r"(0u)
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

    uint32_t q[kQParts][NT][kSteps][2];  // Q^T: head g of tile nt, this thread's elements
    float o[NT][kTiles][4];              // O^T: rows 2j, 2j + 1 of chunk g; columns 2t, 2t + 1
    float cs[NT][2], m[NT][2], l[NT][2];
    int slot = 0;
    uint32_t parity = 0;
    bool fresh = true;  // the piece has no maximum yet

    // One stage in `stage`, its first `tokens` tokens valid.  One body for whole
    // and for ragged stages: the branches below are small and the same for the
    // warp, where a second body would be fetched anew at every sequence's end.
    auto attend = [&](const uint32_t stage, const int tokens) {
      const bool ragged = tokens < kFp4Step;
      // ---- scores of 32 tokens: rows g (tile 2u) and g + 8 (tile 2u + 1) ----
      float sc[2][NT][4];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        constexpr int kWords = D / 32;  // of a thread's quarter row
        constexpr int kSum = !kF32 ? kWords : D == 64 ? 1 : 2;  // words of one chain
        float own[NT][4];
        uint32_t kw[2][kWords], ks[2][(D + 127) / 128];  // codes; scales, two to a word
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
            ks[e][0] = two;
          } else {
#pragma unroll
            for (int c = 0; c < kWords / 4; ++c) {
              const uint4 v = lds128(row + 16 * c);
              kw[e][4 * c] = v.x;
              kw[e][4 * c + 1] = v.y;
              kw[e][4 * c + 2] = v.z;
              kw[e][4 * c + 3] = v.w;
              const uint32_t two = e4m3x2_to_half2(lds_u16(sca + 2 * c));
              ks[e][c] = two;
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
            // Words 0, 1 of four have the first scale of a pair.
            lo[b] = w / 2 % 2 ? half2_mul_by<true>(lo[b], ks[0][w / 4])
                              : half2_mul_by<false>(lo[b], ks[0][w / 4]);
            hi[b] = w / 2 % 2 ? half2_mul_by<true>(hi[b], ks[1][w / 4])
                              : half2_mul_by<false>(hi[b], ks[1][w / 4]);
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            // The matrix unit cuts its sums off towards zero.  For fp32 they are kept
            // short, a quarter or half of a row, and added up with rounding: chains
            // over the whole row made outputs up to 2.8e-6 wrong (D = 256, 30000
            // tokens; now 9e-7, an unfused fp32 form 8e-7 to 3e-6).
            float* sum = kF32 ? own[nt] : sc[u][nt];
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              const uint32_t a[4] = {lo[2 * b], hi[2 * b], lo[2 * b + 1], hi[2 * b + 1]};
#pragma unroll
              for (int part = kQParts - 1; part >= 0; --part) {  // small parts first
                if (b == 0 && part == kQParts - 1 && w % kSum == 0)
                  mma_f16_first(sum, a, q[part][nt][2 * w + b]);
                else
                  mma_f16(sum, a, q[part][nt][2 * w + b]);
              }
            }
            if (kF32 && w % kSum == kSum - 1)
#pragma unroll
              for (int c = 0; c < 4; ++c)
                sc[u][nt][c] = w == kSum - 1 ? own[nt][c] : sc[u][nt][c] + own[nt][c];
          }
        }
      }

      // Rounded here, so that the largest less the maximum is exact: were the product
      // part of that difference, it would be off by half a step of the maximum, and
      // weights infinite or all zero where that is 8 or more (scores of 2^27 on).  (As one
      // instruction it took the same time.)
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 4; ++c) sc[u][nt][c] = __fmul_rn(sc[u][nt][c], cs[nt][c & 1]);

      // ---- softmax: the maximum moves only when a score passes it by the slack ----
      float y[2][NT][4];
      auto weigh = [&]() {  // exponents; their maximum of this thread
        float over = -INFINITY;
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 4; ++c)
              y[u][nt][c] = __fsub_rn(sc[u][nt][c], m[nt][c & 1]);
        if (ragged) {
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int c = 0; c < 4; ++c)
                if (u * 16 + (c >> 1) * 8 + g >= tokens) y[u][nt][c] = -INFINITY;
        }
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 4; ++c) over = fmaxf(over, y[u][nt][c]);
        return over;
      };
      if (fresh || __any_sync(0xffffffffu, weigh() > kFp4Top)) {
        fresh = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float top = -INFINITY;
#pragma unroll
            for (int u = 0; u < 2; ++u)
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
#pragma unroll
            for (int j = 0; j < kTiles; ++j) {
              o[nt][j][c] *= alpha;
              o[nt][j][c + 2] *= alpha;
            }
          }
        weigh();
      }
      uint32_t pt[kQParts][2][NT][2];  // P^T: head g; tokens 2t, 2t + 1 of tile 2u (+ 1)
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float w0 = fast_exp2(y[u][nt][2 * e]);
            const float w1 = fast_exp2(y[u][nt][2 * e + 1]);
            l[nt][0] += w0;
            l[nt][1] += w1;
            const uint32_t two = pack_half2(w0, w1);
            pt[0][u][nt][e] = transpose8x8(two);
            if constexpr (kF32)
              pt[1][u][nt][e] = transpose8x8(pack_half2(w0 - half_lo(two), w1 - half_hi(two)));
          }

      // ---- values ----
      constexpr int kParts = D == 256 ? 2 : 1;  // groups of a thread's chunk of D / 8 elements
      constexpr int kWords = D == 64 ? 1 : 2;   // words of a part, per token
#pragma unroll
      for (int part = 0; part < kParts; ++part) {
        // Codes and scales of tokens 2t (wa) and 2t + 1 (wb) of the stage's tiles.
        uint32_t wa[4][kWords], wb[4][kWords], vs[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t tile = stage + e * C::kTileBytes;
          const int group = D == 64 ? g >> 1 : g * kParts + part;
          if constexpr (D == 64) {
            const uint32_t at = tile + fp4_value_codes(D) + group * 64 + t * 16 + (g & 1) * 4;
            wa[e][0] = lds_u32(at);
            wb[e][0] = lds_u32(at + 8);
          } else {
            const uint4 v = lds128(tile + fp4_value_codes(D) + group * 64 + t * 16);
            wa[e][0] = v.x;
            wa[e][1] = v.y;
            wb[e][0] = v.z;
            wb[e][1] = v.w;
          }
          uint32_t two = lds_u16(tile + fp4_value_scales(D) + group * 8 + 2 * t);
          if (ragged) {
            // Rows past the sequence's end hold anything: a zero scale.
            const int tok = e * 8 + 2 * t;
            if (tok >= tokens) two = 0;
            else if (tok + 1 >= tokens) two &= 0xffu;
          }
          vs[e] = e4m3x2_to_half2(two);
        }
        if constexpr (kNarrow) {
          // Columns of even elements (g < 4) or of odd ones: the weight in that
          // half, of token 2t, then of token 2t + 1.
          const uint32_t first = g < 4 ? 0x4410u : 0x1044u;
          const uint32_t second = g < 4 ? 0x4432u : 0x3244u;
          uint32_t b2[4][kQParts][2];
#pragma unroll
          for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int qp = 0; qp < kQParts; ++qp) {
              b2[e][qp][0] = __byte_perm(pt[qp][e / 2][0][e % 2], 0, first);
              b2[e][qp][1] = __byte_perm(pt[qp][e / 2][0][e % 2], 0, second);
            }
#pragma unroll
          for (int w = 0; w < kWords; ++w) {
            Fp4Sum<kF32> add[2] = {o[0][part * 4 + w * 2], o[0][part * 4 + w * 2 + 1]};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t ha[4], hb[4];
              e2m1x8_to_half2(wa[e][w], ha);
              e2m1x8_to_half2(wb[e][w], hb);
#pragma unroll
              for (int b = 0; b < 2; ++b) {
                const uint32_t a[4] = {half2_mul_by<false>(ha[2 * b], vs[e]),
                                       half2_mul_by<false>(ha[2 * b + 1], vs[e]),
                                       half2_mul_by<true>(hb[2 * b], vs[e]),
                                       half2_mul_by<true>(hb[2 * b + 1], vs[e])};
#pragma unroll
                for (int qp = kQParts - 1; qp >= 0; --qp)  // small parts first
                  add[b](a, b2[e][qp], e == 0 && qp == kQParts - 1);
              }
            }
            add[0].done();
            add[1].done();
          }
        } else {
#pragma unroll
          for (int w = 0; w < kWords; ++w) {
            float own[NT][4][4];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              // Bytes of the two tokens' codes of one element: even, then odd ones.
              uint32_t even[2][4], odd[2][4];
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const uint32_t a2 = wa[2 * u + e][w], b2 = wb[2 * u + e][w];
                e2m1x8_to_half2((a2 & 0x0f0f0f0fu) | ((b2 << 4) & 0xf0f0f0f0u), even[e]);
                e2m1x8_to_half2(((a2 >> 4) & 0x0f0f0f0fu) | (b2 & 0xf0f0f0f0u), odd[e]);
              }
#pragma unroll
              for (int b = 0; b < 4; ++b) {
                const uint32_t a[4] = {
                    half2_mul(even[0][b], vs[2 * u]), half2_mul(odd[0][b], vs[2 * u]),
                    half2_mul(even[1][b], vs[2 * u + 1]), half2_mul(odd[1][b], vs[2 * u + 1])};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                  for (int qp = kQParts - 1; qp >= 0; --qp) {
                    if (!kF32) mma_f16(o[nt][part * 8 + w * 4 + b], a, pt[qp][u][nt]);
                    else if (u == 0 && qp == kQParts - 1) mma_f16_first(own[nt][b], a, pt[qp][u][nt]);
                    else mma_f16(own[nt][b], a, pt[qp][u][nt]);
                  }
              }
            }
            if constexpr (kF32)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int b = 0; b < 4; ++b)
#pragma unroll
                  for (int c = 0; c < 4; ++c) o[nt][part * 8 + w * 4 + b][c] += own[nt][b][c];
          }
        }
      }
    };

    bool last = false;
    for (int piece = 0; !last; ++piece) {
      __syncwarp();
      // What is needed of the record at the piece's end is read then, as registers are
      // short between.
      const Fp4Piece& rec = pieces[piece % C::kPieceRing];
      const int len = rec.len;
      // ---- the pair's queries ----
      {
        int heads;
        const int head0 = heads_of(rec.hp, &heads);
        // fp16 holds a row scaled by a power of two to a maximum in [2^13, 2^14)
        // (bf16 exactly, unless an element is 2^-30 of the largest).
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const int head = nt * 8 + (kNarrow ? g & 3 : g);
          float x[D / 4];
          if (head < heads) {
            const T* src = static_cast<const T*>(p.query) + rec.s * p.query_stride +
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
          for (int j = 0; j < kTiles; ++j)
#pragma unroll
            for (int c = 0; c < 4; ++c) o[nt][j][c] = 0.f;
        }
      }
      fresh = true;
      constexpr int kChainStages = kFp4Chain / C::kStage;
      for (int k = rec.k0; k < rec.k0 + rec.stages;) {
        const int chain_end = min(k + kChainStages, rec.k0 + rec.stages);
        for (; k < chain_end; ++k) {
          if (ok) {
            const bool w = wait_phase(bars + 8u * slot, parity, p.err, p.wait_limit);
            ok = __all_sync(0xffffffffu, w);
          }
          if (ok)
#pragma unroll 1
            for (int t0 = 0; t0 < C::kStage && k * C::kStage + t0 < len; t0 += kFp4Step)
              attend(ring + slot * C::kStageBytes + t0 / kFp4Tile * C::kTileBytes,
                     min(len - k * C::kStage - t0, kFp4Step));
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
          // its maximum; then they are put away for the next.
          const bool first = k - rec.k0 == kChainStages, final = k == rec.k0 + rec.stages;
          float* past =
              p.chains + ((size_t)blockIdx.x * W + warp) * fp4_chain_floats(D, H) + lane;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              float* at = past + (nt * 2 + c) * (2 * kTiles + 2) * 32;
              const float w = first ? 0.f : fast_exp2(at[0] - m[nt][c]);
              auto join = [&](int i, float& sum) {
                if (!first) sum = fmaf(at[32 * i], w, sum);
                if (!final) {
                  at[32 * i] = sum;
                  sum = 0.f;
                }
              };
              join(1, l[nt][c]);
#pragma unroll
              for (int j = 0; j < kTiles; ++j) {
                join(2 * j + 2, o[nt][j][c]);
                join(2 * j + 3, o[nt][j][c + 2]);
              }
              at[0] = m[nt][c];
            }
        }
      }
      const Fp4Piece pc = rec;
      int heads;
      const int head0 = heads_of(pc.hp, &heads);
      const bool ends = pc.k0 + pc.stages == pc.n;
      last = pc.at + pc.stages + (ends ? kFp4PairCost : 0) >= my1;

      // ---- the piece is done ----
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
      const bool whole = pc.k0 == 0 && pc.stages == pc.n;
      // A part goes to the ring at the end of the warp's part (every copy has
      // landed and been read), to global memory before.
      float* to = last ? reinterpret_cast<float*>(smem + warp * C::kWarpRing)
                       : p.warp_partials + ((size_t)blockIdx.x * W + warp) * part_floats;
      __syncwarp();
      // Chunk g of one head: a final row, or a part's.
      auto put = [&](int head, const float* v, float max_, float sum) {
        if (head >= heads) return;
        if (whole) {
          const float inv = __fdividef(p.value_scale, sum);
          T* dst = static_cast<T*>(p.out) +
                   ((size_t)pc.s * p.num_heads + head0 + head) * D + g * (D / 8);
          if constexpr (kF32) {
#pragma unroll
            for (int e = 0; e < D / 8; e += 4)
              *reinterpret_cast<float4*>(dst + e) =
                  make_float4(v[e] * inv, v[e + 1] * inv, v[e + 2] * inv, v[e + 3] * inv);
          } else {
#pragma unroll
            for (int e = 0; e < D / 8; e += 8)
              stg_v4(dst + e, make_uint4(pack_bf16x2(v[e] * inv, v[e + 1] * inv),
                                         pack_bf16x2(v[e + 2] * inv, v[e + 3] * inv),
                                         pack_bf16x2(v[e + 4] * inv, v[e + 5] * inv),
                                         pack_bf16x2(v[e + 6] * inv, v[e + 7] * inv)));
          }
        } else {
          float* dst = to + head * D + g * (D / 8);
#pragma unroll
          for (int e = 0; e < D / 8; e += 4)
            *reinterpret_cast<float4*>(dst + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
          if (g == 0)
#pragma unroll
            for (int sp = 0; sp < kSplit; ++sp) {
              to[rows * D + head * kSplit + sp] = max_;
              to[rows * D + per_run + head * kSplit + sp] = sum;
            }
        }
      };
      float v[D / 8];
      if constexpr (kNarrow) {
        // Lanes t and t ^ 2 have the even and the odd elements of two heads: one
        // head whole to each.
        const bool low = t < 2;
#pragma unroll
        for (int j = 0; j < kTiles; ++j)
#pragma unroll
          for (int c = 0; c < 4; c += 2) {
            const float keep = low ? o[0][j][c] : o[0][j][c + 1];
            const float got =
                __shfl_xor_sync(0xffffffffu, low ? o[0][j][c + 1] : o[0][j][c], 2);
            v[4 * j + c] = low ? keep : got;
            v[4 * j + c + 1] = low ? got : keep;
          }
        put((t & 1) * 2 + (t >> 1), v, low ? m[0][0] : m[0][1], low ? ls[0][0] : ls[0][1]);
      } else {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
#pragma unroll
            for (int j = 0; j < kTiles; ++j) {
              v[2 * j] = o[nt][j][c];
              v[2 * j + 1] = o[nt][j][c + 2];
            }
            put(nt * 8 + 2 * t + c, v, m[nt][c], ls[nt][c]);
          }
      }
      if (!whole) {
        // The warp with the pair's last part in this CTA says where the parts are.
        if (lane == 0 && (ends || pc.at + pc.stages == cta1)) {
          const int at = pc.at - pc.k0;  // the pair's first stage
          const bool here = at >= cta0 && at + pc.n <= cta1;
          const int c0 = here ? (int)blockIdx.x : at / share;
          runs[2 * warp + last] = Fp4Run{pc.s, head0, heads, at <= cta0 ? 0 : (at - cta0) / share_w,
                                         c0, here ? 1 : (at + pc.n - 1) / share - c0 + 1};
        }
      }
    }
    if (!ok) {
      // A wait gave up: this warp's copies in flight end before it leaves.
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
  // A warp takes some columns of one head of a pair, first over the CTA's warps;
  // then, for a pair with parts in other CTAs, the last warp to arrive with its
  // columns merges those, up to kFp4Gather at a time (one SM would take 8 us for
  // a part of 8 heads of 256 elements from every SM; a level costs 1.3 us to hand
  // on and 2 to 3 us to read): the groups of the pair's
  // CTAs, then their results.  Of a CTA's counters for each unit the first is
  // for the group of the pair that it continues, the second for the first group
  // of the pair that it begins, the third for the results of that pair's groups;
  // its four slots hold its part of the pair that it continues, of the one that
  // it begins, and the groups' results likewise.  One short loop for all levels:
  // code that runs once is paid by its length (unrolled over 16 parts it took
  // 2 us longer).
  if (cta0 >= cta1) return;  // the same for the whole CTA
  __syncthreads();
  static_assert(W <= kFp4Gather && H * kSplit <= kFp4Units, "merges");
  uint32_t live = __ballot_sync(0xffffffffu, lane < 2 * W && runs[lane % (2 * W)].s >= 0);
  for (int u0 = 0; live; live &= live - 1, u0 += per_run) {
    // Unit u of all runs' is warp u mod W's.
    int unit = (warp - u0) & (W - 1);
    if (unit >= per_run) continue;
    const int which = __ffs(live) - 1;
    const Fp4Run run = runs[which];
    for (; unit < run.heads * kSplit; unit += W) {
      const int col = unit * 32 * kVec + lane * kVec;
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
        float mi = -INFINITY, li = 0.f, acc[kVec];
        if (lane < n) {
          const float* src = part(lane) + rows * D + unit;
          mi = src[0];
          li = src[per_run];
        }
        // Four parts at a time (past the last, that one again, with no weight); the
        // first ones are on their way with the maxima and sums.
        constexpr int kBatch = 4;
        float top = 0.f, w = 0.f, sum = 0.f;
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
            w = lane >= n ? 0.f : mi == top ? 1.f : fast_exp2(mi - top);
            sum = lane < n ? li * w : 0.f;
#pragma unroll
            for (int o = 1; o < kFp4Gather; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            sum = __shfl_sync(0xffffffffu, sum, 0);
          }
#pragma unroll
          for (int i = 0; i < kBatch; ++i) {
            const float wi = __shfl_sync(0xffffffffu, w, i0 + i);
#pragma unroll
            for (int e = 0; e < kVec; ++e) acc[e] = fmaf(v[i][e], wi, acc[e]);
          }
        }
        const int group = ((int)blockIdx.x - run.cta0) / kFp4Gather;
        const int groups = (run.ctas + kFp4Gather - 1) / kFp4Gather;
        if (level == (run.ctas == 1 ? 0 : groups == 1 ? 1 : 2)) {
          const float inv = __fdividef(p.value_scale, sum);
          T* dst = static_cast<T*>(p.out) + ((size_t)run.s * p.num_heads + run.head0) * D + col;
#pragma unroll
          for (int e = 0; e < kVec; e += 2) {
            if constexpr (kF32)
              *reinterpret_cast<float2*>(dst + e) = make_float2(acc[e] * inv, acc[e + 1] * inv);
            else
              *reinterpret_cast<uint32_t*>(dst + e) = pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
          }
          break;
        }
        // Hand the part on; whoever is last takes the next level.  Lane 0's atomic
        // releases what the warp's lanes wrote before and acquires, for all of
        // them, what the others' released.
        const int at = level == 0 ? (int)blockIdx.x : run.cta0 + group * kFp4Gather;
        float* to =
            p.cta_partials + ((size_t)at * 4 + 2 * level + (at == run.cta0)) * part_floats;
#pragma unroll
        for (int e = 0; e < kVec; e += 2)
          *reinterpret_cast<float2*>(to + col + e) = make_float2(acc[e], acc[e + 1]);
        if (lane == 0) {
          to[rows * D + unit] = top;
          to[rows * D + per_run + unit] = sum;
        }
        __syncwarp();
        const int first = level == 0 ? run.cta0 + group * kFp4Gather : run.cta0;
        const int parts = level == 0 ? min(kFp4Gather, run.ctas - group * kFp4Gather) : groups;
        int go = 0;
        if (lane == 0) {
          unsigned int* counter =
              p.counters + (first * 3 + (level == 1 ? 2 : first == run.cta0)) * kFp4Units + unit;
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
        step = (level == 0 ? 1u : (uint32_t)kFp4Gather) * 16u * part_floats;
        odd = first == run.cta0 ? 0 : -1;
        odd_part = slot0 + part_floats;
      }
    }
  }
}

}  // namespace pa
