// Quantising write into the 8-bit pool, and reading tokens back, for sm_103a.
//
// The scale of a block, head and side (keys or values) is that of all its tokens, so what a
// call puts into one block, a run, is found and written together: a block's tokens are
// neighbours in the call.  A lane has 16 elements of a row, which are one 16-byte piece of the
// pool.  A decode batch's runs are single tokens, whose latency counts: a row is a group of D / 16
// lanes, a warp has several heads and sides.  A prompt's are blocks: a warp, or several for
// large blocks and small prompts, holds a run's rows in registers from the one reading on, so
// that each byte moves once.  One launch has CTAs for either kind.  A block that goes on has
// its scale read beside the rows, and its codes read and rounded again only where it grows.
//
// Measured (graph replays in a row, data larger than L2), 8 heads of 128, bf16, blocks of 16: 16384
// tokens of a prompt 23.3 us (4.3 TB/s, 64% of the copy rate: three dependent trips a run -
// slots, rows, codes - and about 450 instructions for 1024 elements, most of which a warp needs
// once for a run and side, however many rows: maxima, barrier, quotients, headers; 32 warps per SM
// hide each other's waits to 2.4 a clock; fp32 31.7 us, 5.3 TB/s; heads of 64 21.5, blocks of 8
// 21.7, of 256 31), 128 tokens of as many sequences 2.7 us, 1024 5.3 us, 8000 29 to 33 us (with one at a
// time on its way to a warp a sixth longer).
// Each kind by itself, the other kind's kernel taking it: single tokens by whole warps 17 us
// (1024), prompts by groups 26 us (500 tokens; 2000 in blocks of 256 330 us).
//
// These are writes whose scales stay, as those of a pass that is repeated do.  A decode batch's do not: of like
// rows token i of a block raises each of its scales with probability 1 / (i + 1), and the codes that
// the block holds are rounded again, a warp's growing scales one after another and each piece stored before
// the next is asked for.  Steps as they come, 8 heads of 128 (in brackets: repeated; where
// every scale grows): 64 sequences 11 us (3.3; 15), 256 13 us (3.8; 19), 1024 17 us (4.4; 25), 64 of 2 heads of
// 64 6.1 us (2.6; 8.8); in blocks of 256, 64 sequences 94 us (3.4; 168), 256 132 us (5.8; 267).
//
// Reading back takes 16 elements of a token's key and of its value per thread: 65536 tokens
// 61.7 us, 96% of the copy rate.
#include <type_traits>

#include "pa_int8.cuh"
#include "pa_launch.h"

namespace pa {

namespace {

constexpr int kInt8Threads = 256;   // of a CTA that reads back
constexpr int kWriteThreads = 128;

// ---- write --------------------------------------------------------------------

// What a run does to its block's scale.
struct Scale {
  float s, inv;
  float lean;  // int8_lean's, for bf16 rows with a maximum of their own; or 0
  bool grows;  // and the codes are rounded again
};
template <typename T>
__device__ __forceinline__ Scale scale_of(uint32_t top, float old, bool begins) {
  Scale r;
  r.s = int8_scale(top);
  // Grown, or NaN now; a block whose scale is NaN keeps it.
  r.grows = !begins && !(r.s <= old) && old == old;
  const bool own = begins || r.grows;
  if (!own) r.s = old;
  r.inv = r.s >= kInt8Small ? 1.f / r.s : 0.f;
  r.lean = sizeof(T) == 2 && own && r.s >= kInt8Small ? int8_lean(__uint_as_float(top), r.s, r.inv) : 0.f;
  return r;
}

// 16 elements of a row.
template <typename T>
struct Piece {
  uint4 w[sizeof(T)];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T); ++i) w[i] = make_uint4(0u, 0u, 0u, 0u);
  }
  __device__ __forceinline__ void load(const T* p, bool wide) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T); i += 2)
      load32(reinterpret_cast<const uint4*>(p) + i, &w[i], wide);
  }
  // The largest |x|, as bits (which order NaN above infinity above numbers).
  __device__ __forceinline__ uint32_t largest() const {
    if constexpr (sizeof(T) == 2) {
      uint32_t top = 0;  // a pair, whose signs mean nothing
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t v[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          asm("max.NaN.xorsign.abs.bf16x2 %0, %0, %1;" : "+r"(top) : "r"(v[e]));
      }
      return max((top << 16) & 0x7fff0000u, top & 0x7fff0000u);
    } else {
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        top = max(max(top, max(w[i].x & 0x7fffffffu, w[i].y & 0x7fffffffu)),
                  max(w[i].z & 0x7fffffffu, w[i].w & 0x7fffffffu));
      return top;
    }
  }
  // kOwn: the scale is these rows' own.
  template <bool kOwn>
  __device__ __forceinline__ uint4 codes(const Scale& sc) const {
    constexpr int kPer = ElemTraits<T>::kPerChunk;
    const float s = sc.s;
    float x[16];
#pragma unroll
    for (int i = 0; i < (int)sizeof(T); ++i) ElemTraits<T>::unpack(w[i], x + i * kPer);
    uint32_t c[16];
    bool sure = s >= kInt8Small;
    if constexpr (sizeof(T) == 2) {
      if (kOwn || sc.lean != 0.f) {
#pragma unroll
        for (int e = 0; e < 16; e += 2) int8_plain(x[e], x[e + 1], sc.lean, c + e);
      } else {
#pragma unroll
        for (int e = 0; e < 16; ++e) c[e] = int8_near_bf16(x[e], sc.inv, s);
        sure = sure && !int8_few_bits(s);
      }
    } else {
      float off = 0.f;
#pragma unroll
      for (int e = 0; e < 16; ++e) c[e] = int8_near(x[e], sc.inv, &off);
      sure = sure && off < kInt8Sure;
    }
    if (!sure) {
      // A tie or beside one (fp32: one piece in 1000); or a scale that is small, zero or NaN
      // (zeros then).
      const float lift = int8_lift_of(s), sl = s * lift, by = 1.f / sl;
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const float y = x[e] * lift;
        c[e] = s > 0.f ? int8_exact(y * by, y, 0.f, sl) : kInt8Bias;
      }
    }
    return make_uint4(low_bytes(c[0], c[1], c[2], c[3]), low_bytes(c[4], c[5], c[6], c[7]),
                      low_bytes(c[8], c[9], c[10], c[11]), low_bytes(c[12], c[13], c[14], c[15]));
  }
};

// A piece of codes whose scale grows from old to s.
__device__ __forceinline__ uint4 again(const uint4& v, float old, float s) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t r[4];
  const float lift = int8_lift_of(s), was = old * lift, sl = s * lift, ratio = was / sl;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint32_t c[4];
    float off = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) c[e] = int8_near((float)int8_code(w[k], e), ratio, &off);
    if (!(off < kInt8Sure) || !(s > 0.f))
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float x = (float)int8_code(w[k], e), hi = x * was;
        c[e] = s > 0.f ? int8_exact(x * ratio, hi, fmaf(x, was, -hi), sl) : kInt8Bias;
      }
    r[k] = low_bytes(c[0], c[1], c[2], c[3]);
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

// Codes of one side of a block, 16-byte piece i of D / 2 to a tile, in any order of lanes.
template <int D>
__device__ __forceinline__ void grow(uint8_t* base, int codes, int l2bs, float old, float s,
                                     int first, int step) {
  for (int i = first; i < (D / 2) << (l2bs - 3); i += step) {
    uint4* at = reinterpret_cast<uint4*>(base + i / (D / 2) * int8_tile_bytes(D) + codes + i % (D / 2) * 16);
    *at = again(*at, old, s);
  }
}

// Where the first 16 codes of the token at `off` in a block are, after the block's first; its others
// follow every 128 bytes.
template <int D>
__device__ __forceinline__ int place_of(int off) {
  return (off >> 3) * int8_tile_bytes(D) + (off & 7) * 16;
}

struct WriteParams {
  Int8Pool pool;
  const void* key;
  const void* value;
  int64_t key_stride, value_stride;
  const int64_t* slots;
  unsigned int* err;
  int num_tokens;
  bool wide;         // rows are on 32-byte boundaries
  int single_ctas;   // the first CTAs of the grid, which take runs of one token
  int single_window; // tokens of a warp of theirs
  int window;        // tokens that a run of the others begins in
  int row_warps, l2_row_warps;  // warps of a team: they share a run's rows
  unsigned teams, per, more;  // per pairs of a window and a side each; the first `more` teams one more
  __device__ __forceinline__ int block_of(int64_t slot) const {  // -1: padding, or no slot
    return (uint64_t)slot < (uint64_t)pool.num_slots ? (int)(slot >> pool.log2_block_size) : -1;
  }
  __device__ __forceinline__ int block_at(int64_t t) const {
    return t >= 0 && t < num_tokens ? block_of(__ldg(slots + t)) : -1;
  }
};

template <typename T>
__device__ __forceinline__ const T* row_of(const WriteParams& p, int side, int64_t t, int at) {
  return (side & 1 ? static_cast<const T*>(p.value) + t * p.value_stride
                   : static_cast<const T*>(p.key) + t * p.key_stride) + at;
}

// Steps of rows that a warp holds, and CTAs of an SM: bf16's 16 registers of rows leave room for
// eight (16384 tokens of a prompt take 3% and 12% longer with seven and six, 45% with half the rows), while
// fp32 rather has its loads on their way at once (half the rows and seven CTAs 5% longer, five CTAs 22%).
template <typename T>
__host__ __device__ constexpr int write_steps() {
  return sizeof(T) == 2 ? 2 : 4;
}

template <typename T>
__host__ __device__ constexpr int write_ctas() {
  return sizeof(T) == 2 ? 8 : 4;
}

// Runs of one token, as a decode batch has them: a warp takes some tokens and as many heads
// and sides as it has groups of a row's D / 16 lanes.
template <typename T, int D>
__device__ __forceinline__ void write_singles(const WriteParams& p) {
  constexpr int kLanes = D / 16, kGroups = 32 / kLanes;
  const int lane = threadIdx.x & 31, j = lane % kLanes;
  const int sides = 2 * p.pool.num_kv_heads;
  const unsigned parts = (unsigned)((sides + kGroups - 1) / kGroups);
  const unsigned unit = blockIdx.x * (kWriteThreads / 32) + threadIdx.x / 32;
  const int side = (int)(unit % parts) * kGroups + lane / kLanes, h = side >> 1, kv = side & 1;
  const bool on = side < sides;
  const int64_t t0 = (int64_t)(unit / parts) * p.single_window;
  if (t0 >= p.num_tokens) return;
  const int l2bs = p.pool.log2_block_size, last = (1 << l2bs) - 1;
  const int codes = kv ? int8_value_codes(D) : int8_key_codes();
  // One token: its row is on its way before its slot is known.
  Piece<T> x;
  const bool early = p.single_window == 1;
  if (early && on) x.load(row_of<T>(p, side, t0, h * D + j * 16), p.wide);
  const int64_t t = t0 + lane;
  const bool mine = lane < p.single_window && t < p.num_tokens;
  const int64_t slot = mine ? __ldg(p.slots + t) : -1;
  const int block = p.block_of(slot);
  // Bad slots are recorded here, by the first heads and sides.
  if (slot >= p.pool.num_slots && unit % parts == 0) record_error(p.err, PA_DEVERR_SLOT);
  const bool alone = block >= 0 && p.block_at(t - 1) != block && p.block_at(t + 1) != block;
  uint32_t singles = __ballot_sync(0xffffffffu, alone);
  // The next token's row and scale are on their way while a token is written.
  uint8_t* base = p.pool.cache;
  float held = 0.f;
  auto fetch = [&](int i, bool row) {
    const int b = __shfl_sync(0xffffffffu, block, i);
    if (!on) return;
    base = p.pool.cache + int8_block_offset(b, h, p.pool.num_kv_heads, l2bs, D);
    held = reinterpret_cast<const float*>(base)[kv];
    if (row) x.load(row_of<T>(p, side, t0 + i, h * D + j * 16), p.wide);
  };
  if (singles) fetch(__ffs(singles) - 1, !early);
  for (; singles; singles &= singles - 1) {
    const int off = __shfl_sync(0xffffffffu, (int)slot, __ffs(singles) - 1) & last;
    const bool begins = off == 0;
    const Piece<T> now = x;
    uint8_t* const to = base;
    const float old = held;
    if (singles & (singles - 1)) fetch(__ffs(singles & (singles - 1)) - 1, true);
    uint32_t top = on ? now.largest() : 0;
#pragma unroll
    for (int o = 1; o < kLanes; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    const Scale sc = scale_of<T>(top, old, begins || !on);
    // Blocks whose scale grows, each by the whole warp.
    uint32_t growing = __ballot_sync(0xffffffffu, j == 0 && sc.grows);
    for (; growing; growing &= growing - 1) {
      const int g = __ffs(growing) - 1;
      uint8_t* at = reinterpret_cast<uint8_t*>(__shfl_sync(0xffffffffu, (unsigned long long)to, g));
      grow<D>(at, __shfl_sync(0xffffffffu, codes, g), l2bs, __shfl_sync(0xffffffffu, old, g),
              __shfl_sync(0xffffffffu, sc.s, g), lane, 32);
    }
    __syncwarp();
    if (on) {
      if (begins || sc.grows)
        for (int k = j; k < 1 << (l2bs - 3); k += kLanes)
          (reinterpret_cast<float*>(to) + kv)[k * (int8_tile_bytes(D) / 4)] = sc.s;
      stg_v4(to + codes + place_of<D>(off) + j * 128, now.template codes<false>(sc));
    }
  }
}

// Longer runs, a prompt's blocks: teams of warps take (window of tokens, some heads and sides).
// The runs that begin in the window are the team's work, one after another; a run's rows go
// over the team's lanes, which hold them from the one reading on.
template <typename T, int D>
__device__ __forceinline__ void write_runs(const WriteParams& p, unsigned cta) {
  constexpr int kLanes = D / 16, kRows = 32 / kLanes;  // lanes of a row, rows of a step
  constexpr int kSteps = write_steps<T>(), kWarps = kWriteThreads / 32;
  __shared__ uint32_t tops[2][kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  const int team = warp >> p.l2_row_warps, rank = warp & (p.row_warps - 1);
  const int j = lane % kLanes;
  const int row0 = rank * kRows + lane / kLanes, step = p.row_warps * kRows;  // the lane's rows
  const int batch = kSteps * step;  // rows that the team holds
  const unsigned sides = 2u * p.pool.num_kv_heads;
  const int l2bs = p.pool.log2_block_size, last = (1 << l2bs) - 1;
  // With a number that the compiler knows: one from a register takes all 16 barriers of a CTA,
  // and four CTAs those of the SM.
  auto sync = [&]() {
    if (p.row_warps == 1) __syncwarp();
    else if (team == 0) asm volatile("bar.sync 1, %0;" ::"r"(32 * p.row_warps) : "memory");
    else asm volatile("bar.sync 2, %0;" ::"r"(32 * p.row_warps) : "memory");
  };
  // The team's part of all (window, side) pairs, which are as many for each team or one more.
  const unsigned me = cta * (kWarps >> p.l2_row_warps) + team;
  if (me >= p.teams) return;  // the whole team
  const unsigned first = me * p.per + min(me, p.more);
  int left = (int)(p.per + (me < p.more ? 1 : 0));
  unsigned window = first / sides;
  int side0 = (int)(first - window * sides);
  int turn = 0;
  for (; left > 0; ++window) {
    const int side1 = min(side0 + left, (int)sides);
    left -= side1 - side0;
    unsigned at = window * p.window;
    const unsigned num_tokens = p.num_tokens, end = min(at + p.window, num_tokens);
    // The window's rows of the first side are on their way to L2 while its slots are read.
    constexpr int kLines = D * sizeof(T) / 128;
    for (unsigned t = at + (rank * 32 + lane) / kLines; t < end; t += 32 / kLines * p.row_warps)
      prefetch_l2(row_of<T>(p, side0, t, (side0 >> 1) * D + lane % kLines * (D / kLines)));
    while (at < end) {
      // The slots from here on; the next run of two tokens or more that begins.
      const int64_t slot = at + lane < num_tokens ? __ldg(p.slots + at + lane) : -1;
      const int mine = p.block_of(slot);
      int before = __shfl_up_sync(0xffffffffu, mine, 1), after = __shfl_down_sync(0xffffffffu, mine, 1);
      if (lane == 0) before = p.block_at((int64_t)at - 1);
      if (lane == 31) after = p.block_at((int64_t)at + 32);
      const uint32_t starts = __ballot_sync(
          0xffffffffu, mine >= 0 && mine != before && mine == after && at + lane < end);
      if (!starts) {
        at += 32;
        continue;
      }
      const int skip = __ffs(starts) - 1;
      const int block = __shfl_sync(0xffffffffu, mine, skip);
      const uint32_t other = ~__ballot_sync(0xffffffffu, mine == block) & (0xffffffffu << skip);
      at += skip;
      const int seen = 32 - skip;  // slots of the run that lanes may hold
      int n = other ? __ffs(other) - 1 - skip : seen;
      bool begins = __any_sync(0xffffffffu, lane >= skip && lane < skip + n && ((int)slot & last) == 0);
      if (!other)
        for (uint32_t same = 0xffffffffu; same == 0xffffffffu;) {
          const unsigned i = at + n + lane;
          const int64_t s = i < num_tokens ? __ldg(p.slots + i) : -1;
          same = __ballot_sync(0xffffffffu, p.block_of(s) == block);
          const int more = same == 0xffffffffu ? 32 : __ffs(~same) - 1;
          begins |= __any_sync(0xffffffffu, lane < more && ((int)s & last) == 0);
          n += more;
        }
      int places[kSteps];  // of the lane's tokens in the block
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const int r = row0 + i * step;
        int off = (int)__shfl_sync(0xffffffffu, (int)slot, skip + r) & last;
        if (r >= seen && r < n) off = (int)__ldg(p.slots + (at + r)) & last;
        places[i] = place_of<D>(off);
      }
      const T* rows[2];  // the lane's first, of the first head
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) rows[kv] = row_of<T>(p, kv, (int64_t)at + row0, j * 16);
      uint8_t* const tiles = p.pool.cache + int8_block_offset(block, 0, p.pool.num_kv_heads, l2bs, D);
      auto write = [&](auto plain) {
        constexpr bool kPlain = decltype(plain)::value;
#pragma unroll 1
        for (int side = side0; side < side1; ++side, turn ^= 1) {
          const int kv = side & 1;
          uint8_t* base = tiles + (size_t)(side >> 1) * (int8_tile_bytes(D) << (l2bs - 3));
          float* head = reinterpret_cast<float*>(base) + kv;
          const float held = kPlain ? 0.f : *head;
          const int64_t stride = (kv ? p.value_stride : p.key_stride);
          const T* src = (kv ? rows[1] : rows[0]) + (side >> 1) * D;
          Piece<T> x[kSteps];
          auto load = [&](int r0) {
#pragma unroll
            for (int i = 0; i < kSteps; ++i) {
              const int r = r0 + i * step;
              if (kPlain) x[i].load(src + r * stride, true);
              else if (row0 + r < n) x[i].load(src + r * stride, p.wide);
              else x[i].clear();
            }
          };
          // Batch after batch for the maximum; the last one stays, and those before it are read
          // again, from its end on.
          uint32_t top = 0;
          int r0 = 0;
#pragma unroll 1
          for (;; r0 += batch) {
            load(r0);
#pragma unroll
            for (int i = 0; i < kSteps; ++i) top = max(top, x[i].largest());
            if (r0 + batch >= n) break;
          }
          top = __reduce_max_sync(0xffffffffu, top);
          if (p.row_warps > 1) {
            if (lane == 0) tops[turn][warp] = top;
            sync();
            for (int i = 0; i < p.row_warps; ++i) top = max(top, tops[turn][warp - rank + i]);
          }
          const Scale sc = scale_of<T>(top, held, kPlain || begins);
          uint8_t* to = base + (kv ? int8_value_codes(D) : int8_key_codes());
          if (!kPlain && sc.grows) {
            // All codes of the block, those that are written below among them.
            grow<D>(base, (int)(to - base), l2bs, held, sc.s, rank * 32 + lane, p.row_warps * 32);
            sync();  // before other lanes' codes of the new tokens
          }
          if (kPlain || begins || sc.grows)
            for (int i = rank * 32 + lane; i < 1 << (l2bs - 3); i += p.row_warps * 32)
              head[i * (int8_tile_bytes(D) / 4)] = sc.s;
          to += j * 128;
          const bool many = r0 > 0;
#pragma unroll 1
          for (;;) {
#pragma unroll
            for (int i = 0; i < kSteps; ++i) {
              const int r = r0 + row0 + i * step;
              if (kPlain || r < n)
                stg_v4(to + (many ? place_of<D>((int)__ldg(p.slots + (at + r)) & last) : places[i]),
                       x[i].template codes<kPlain>(sc));
            }
            if (r0 == 0) break;
            r0 -= batch;
            load(r0);
          }
        }
      };
      // Whole batches that begin their block, as nearly all of a prompt do, have nothing to ask.
      if (begins && p.wide && n % batch == 0) write(std::true_type{});
      else write(std::false_type{});
      at += n;
    }
    side0 = 0;
  }
}

// One launch for both: CTAs that find no run of their kind are done at once.
template <typename T, int D>
__global__ void __launch_bounds__(kWriteThreads, write_ctas<T>())
    int8_write_kernel(const WriteParams p) {
  grid_dependents_launch();
  grid_dependency_wait();
  if (blockIdx.x < p.single_ctas) write_singles<T, D>(p);
  else write_runs<T, D>(p, blockIdx.x - p.single_ctas);
}

// ---- read-back ----------------------------------------------------------------

template <typename T, int D>
__global__ void __launch_bounds__(kInt8Threads)
    int8_gather_kernel(Int8Pool pool, T* __restrict__ key, T* __restrict__ value,
                       const int64_t* __restrict__ slot_mapping, int num_tokens, bool wide,
                       unsigned int* err) {
  // Consecutive (eight tokens, head) units; lanes are a group's tokens, then the next group.
  constexpr int kUnits = kInt8Tile * D / kInt8Group;  // of one head of eight tokens
  constexpr int kHeads = kInt8Threads / kUnits;
  const unsigned head = blockIdx.x * kHeads + threadIdx.x / kUnits;  // of all tokens' heads
  const unsigned eight = head / (unsigned)pool.num_kv_heads;
  const int h = (int)(head - eight * pool.num_kv_heads);
  const int i = threadIdx.x % kUnits, j = i / kInt8Tile;
  const int64_t t = (int64_t)eight * kInt8Tile + i % kInt8Tile;
  grid_dependents_launch();
  grid_dependency_wait();
  if (t >= num_tokens) return;
  const int64_t slot = __ldg(slot_mapping + t);
  if (slot < 0) return;
  if (slot >= pool.num_slots) {
    if (h == 0 && j == 0) record_error(err, PA_DEVERR_SLOT);
    return;
  }
  const int l2bs = pool.log2_block_size;
  const int off = (int)(slot & ((1 << l2bs) - 1));
  const uint8_t* tile = pool.cache +
                        int8_block_offset(slot >> l2bs, h, pool.num_kv_heads, l2bs, D) +
                        (off >> 3) * int8_tile_bytes(D);
  const float2 scale = *reinterpret_cast<const float2*>(tile);
  const uint8_t* codes = tile + int8_key_codes() + j * 128 + (off & 7) * 16;
  const uint4 w[2] = {*reinterpret_cast<const uint4*>(codes),
                      *reinterpret_cast<const uint4*>(codes + 8 * D)};
  const int64_t to = (t * pool.num_kv_heads + h) * D + j * kInt8Group;
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    const float s = kv ? scale.y : scale.x;
    const uint32_t v[4] = {w[kv].x, w[kv].y, w[kv].z, w[kv].w};
    float x[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) x[e] = (float)int8_code(v[e / 4], e % 4) * s;
    T* dst = (kv ? value : key) + to;
    if constexpr (sizeof(T) == 2) {
      uint32_t p[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) p[e] = pack_bf16x2(x[2 * e], x[2 * e + 1]);
      store32(dst, p, wide);
    } else {
      store32(dst, reinterpret_cast<const uint32_t*>(x), wide);
      store32(dst + 8, reinterpret_cast<const uint32_t*>(x) + 8, wide);
    }
  }
}

template <typename T, int D>
cudaError_t launch_write(WriteParams p, int num_sms, cudaStream_t stream) {
  constexpr int kWarps = kWriteThreads / 32, kRows = 512 / D;
  const int64_t n = p.num_tokens, sides = 2ll * p.pool.num_kv_heads;
  // Warps of either kind that are worth having at once (32 an SM: 64 prompts of 37 tokens take 17%
  // longer).
  const int64_t resident = 24ll * num_sms;
  const int64_t parts = (sides + kRows - 1) / kRows;
  p.single_window = 1;
  if (n * parts > 2 * resident)
    while (p.single_window < 32 && (n + p.single_window - 1) / p.single_window * parts > resident)
      p.single_window *= 2;
  p.single_ctas = (int)(((n + p.single_window - 1) / p.single_window * parts + kWarps - 1) / kWarps);
  const int block = 1 << p.pool.log2_block_size;
  p.window = block;
  const int64_t windows = (n + block - 1) / block, pairs = windows * sides;
  // Rows of a warp: as many as it holds, fewer where there are few runs.
  p.row_warps = 1, p.l2_row_warps = 0;
  while (p.row_warps < kWarps && (p.row_warps * write_steps<T>() * kRows < block ||
                                  (p.row_warps * kRows < block && pairs * p.row_warps * 2 <= resident)))
    p.row_warps *= 2, ++p.l2_row_warps;
  // Teams share the pairs evenly, twice as many as are there at once: with as many a team that is
  // slow ends alone (a fifth longer), with four times as many they look for runs more often.
  const int team_ctas = kWarps / p.row_warps;  // teams of a CTA
  const int64_t most = (int64_t)num_sms * write_ctas<T>() * team_ctas;
  p.teams = (unsigned)(pairs < 2 * most ? pairs : 2 * most);
  p.per = (unsigned)(pairs / p.teams);
  p.more = (unsigned)(pairs % p.teams);
  const int64_t grid = p.single_ctas + (p.teams + team_ctas - 1) / team_ctas;
  void* args[] = {&p};
  return launch_overlapped((const void*)int8_write_kernel<T, D>, dim3((unsigned)grid),
                           dim3(kWriteThreads), 0, stream, args);
}

template <typename T, int D>
cudaError_t launch_gather(const Int8Pool& pool, void* key, void* value,
                          const int64_t* slot_mapping, int num_tokens, unsigned int* err,
                          cudaStream_t stream) {
  constexpr int kHeads = kInt8Threads / (kInt8Tile * D / kInt8Group);
  const int64_t all = ((int64_t)num_tokens + kInt8Tile - 1) / kInt8Tile * pool.num_kv_heads;
  bool wide = ((reinterpret_cast<uintptr_t>(key) | reinterpret_cast<uintptr_t>(value)) & 31) == 0;
  void* args[] = {const_cast<Int8Pool*>(&pool), &key, &value, &slot_mapping, &num_tokens, &wide,
                  &err};
  return launch_overlapped((const void*)int8_gather_kernel<T, D>,
                           dim3((unsigned)((all + kHeads - 1) / kHeads)), dim3(kInt8Threads), 0,
                           stream, args);
}

}  // namespace

cudaError_t launch_int8_write(const Int8Pool& pool, const void* key, const void* value, int dtype,
                              int64_t key_stride, int64_t value_stride,
                              const int64_t* slot_mapping, int num_tokens, int num_sms,
                              unsigned int* err, cudaStream_t stream) {
  const bool half = dtype == PA_BF16;
  WriteParams p = {};
  p.pool = pool;
  p.key = key;
  p.value = value;
  p.key_stride = key_stride;
  p.value_stride = value_stride;
  p.slots = slot_mapping;
  p.err = err;
  p.num_tokens = num_tokens;
  p.wide = ((reinterpret_cast<uintptr_t>(key) | reinterpret_cast<uintptr_t>(value)) & 31) == 0 &&
           (key_stride | value_stride) * (half ? 2 : 4) % 32 == 0;
  switch (pool.head_size) {
    case 64:
      return half ? launch_write<__nv_bfloat16, 64>(p, num_sms, stream)
                  : launch_write<float, 64>(p, num_sms, stream);
    case 128:
      return half ? launch_write<__nv_bfloat16, 128>(p, num_sms, stream)
                  : launch_write<float, 128>(p, num_sms, stream);
    default:
      return half ? launch_write<__nv_bfloat16, 256>(p, num_sms, stream)
                  : launch_write<float, 256>(p, num_sms, stream);
  }
}

cudaError_t launch_int8_gather(const Int8Pool& pool, void* key, void* value, int dtype,
                               const int64_t* slot_mapping, int num_tokens, unsigned int* err,
                               cudaStream_t stream) {
  auto run = [&](auto* launch) {
    return launch(pool, key, value, slot_mapping, num_tokens, err, stream);
  };
  const bool half = dtype == PA_BF16;
  switch (pool.head_size) {
    case 64: return half ? run(launch_gather<__nv_bfloat16, 64>) : run(launch_gather<float, 64>);
    case 128:
      return half ? run(launch_gather<__nv_bfloat16, 128>) : run(launch_gather<float, 128>);
    default: return half ? run(launch_gather<__nv_bfloat16, 256>) : run(launch_gather<float, 256>);
  }
}

}  // namespace pa
