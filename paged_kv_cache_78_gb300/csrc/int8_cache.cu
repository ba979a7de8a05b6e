// Quantising write into the 8-bit pool, and reading tokens back, for sm_103a.
//
// The scale of a block, head and side (keys or values) is that of all its tokens, so a
// warp takes what a call puts into one block for one head and side: the block's tokens are
// neighbours in the call, the first of them finds the others.  Their rows are read once
// where they fit in registers (up to 4 KB: 16 tokens of a bf16 head of 128), the maximum goes
// over the warp, and every 16 elements of a token are one 16-byte piece of the pool.  A
// block that goes on has its scale read beside the rows, and its codes read and rounded
// again only where the scale grows.
// Reading back takes 16 elements of a token's key and of its value per thread.
#include "pa_int8.cuh"
#include "pa_launch.h"

namespace pa {

namespace {

constexpr int kInt8Threads = 256;

// ---- write --------------------------------------------------------------------

// The maximum of |x| over 16 bytes, as bits.
__device__ __forceinline__ uint32_t largest_bits(const uint4& w, const __nv_bfloat16*) {
  uint32_t top = 0;
  const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) top = __vmaxu2(top, v[e] & 0x7fff7fffu);
  return max(top & 0xffff0000u, top << 16);
}
__device__ __forceinline__ uint32_t largest_bits(const uint4& w, const float*) {
  return max(max(w.x & 0x7fffffffu, w.y & 0x7fffffffu), max(w.z & 0x7fffffffu, w.w & 0x7fffffffu));
}

// Codes of kPer numbers in a 16-byte chunk, packed from byte 0 on.
template <typename T>
__device__ __forceinline__ uint2 quantise_chunk(const uint4& w, float s, float inv) {
  constexpr int kPer = ElemTraits<T>::kPerChunk;
  float x[kPer];
  ElemTraits<T>::unpack(w, x);
  uint32_t c[kPer];
  bool sure = true;
#pragma unroll
  for (int e = 0; e < kPer; ++e) c[e] = int8_near(x[e] * inv, &sure);
  if (s >= 0x1p-100f) {
    if (!sure)
#pragma unroll
      for (int e = 0; e < kPer; ++e) c[e] = int8_exact(x[e] * inv, x[e], 0.f, s);
  } else {
    // A scale of zero or NaN holds zeros; other small ones leave fp32's normal numbers.
    const bool zeros = !(s > 0.f);
#pragma unroll 1
    for (int e = 0; e < kPer; ++e) {
      const uint32_t v = zeros ? kInt8Bias : int8_exact_small((double)x[e], s);
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (i == e) c[i] = v;
    }
  }
  uint2 r = make_uint2(0u, 0u);
  r.x = __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
  if constexpr (kPer == 8)
    r.y = __byte_perm(__byte_perm(c[4], c[5], 0x0040), __byte_perm(c[6], c[7], 0x0040), 0x5410);
  return r;
}

// What a call puts into one block, for one head and side: tokens t0 .. t0 + n - 1, whose
// slots lie in `block`.
template <typename T, int D>
__device__ __forceinline__ void write_run(const Int8Pool& pool, const T* __restrict__ src,
                                          int64_t stride, const int64_t* __restrict__ slots,
                                          int n, int64_t block, bool begins, int h, int kv) {
  constexpr int kPer = ElemTraits<T>::kPerChunk;
  constexpr int kChunks = D / kPer;                             // of a row
  constexpr int kLanes = kChunks < 32 ? kChunks : 32;           // of a row at a time
  constexpr int kRows = 32 / kLanes;                            // rows at a time
  constexpr int kCols = kChunks / kLanes;                       // chunks of a lane in a row
  constexpr int kHeld = 8;                                      // chunks of a lane in registers
  constexpr int kSteps = kHeld / kCols;                         // steps of kRows rows
  const int lane = threadIdx.x & 31;
  const int row = lane / kLanes, col = lane % kLanes;
  const int l2bs = pool.log2_block_size;
  uint8_t* base = pool.cache + int8_block_offset(block, h, pool.num_kv_heads, l2bs, D);
  float* head = reinterpret_cast<float*>(base) + kv;
  const float old = begins ? 0.f : *head;
  const T* from = src + row * stride + col * kPer;
  // The rows, or the first of them.
  uint4 w[kSteps][kCols];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const bool live = i * kRows + row < n;
#pragma unroll
    for (int c = 0; c < kCols; ++c) {
      w[i][c] = live ? ldg_nc_v4(from + (int64_t)i * kRows * stride + c * kLanes * kPer)
                     : make_uint4(0u, 0u, 0u, 0u);
      top = max(top, largest_bits(w[i][c], static_cast<const T*>(nullptr)));
    }
  }
#pragma unroll 1
  for (int i = kSteps * kRows + row; i < n; i += kRows)
#pragma unroll
    for (int c = 0; c < kCols; ++c)
      top = max(top, largest_bits(ldg_nc_v4(src + i * stride + (c * kLanes + col) * kPer),
                                  static_cast<const T*>(nullptr)));
  top = __reduce_max_sync(0xffffffffu, top);
  float s = int8_scale(top);
  // Grown, or NaN now; a block whose scale is NaN keeps it.
  const bool grows = !begins && !(s <= old) && !isnan(old);
  if (!begins && !grows) s = old;
  const int codes = kv ? int8_value_codes(D) : int8_key_codes();
  if (grows) {
    // All codes of the block, those that are written below among them.
    const float ratio = old / s;
    for (int i = lane; i < (D / 2) << (l2bs - 3); i += 32) {  // 16-byte pieces, D / 2 to a tile
      uint8_t* at = base + i / (D / 2) * int8_tile_bytes(D) + codes + i % (D / 2) * 16;
      uint4 v = *reinterpret_cast<const uint4*>(at);
      uint32_t* words = &v.x;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t c[4];
        bool sure = true;
#pragma unroll
        for (int e = 0; e < 4; ++e) c[e] = int8_near((float)int8_code(words[k], e) * ratio, &sure);
        if (s >= 0x1p-100f) {
          if (!sure)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float x = (float)int8_code(words[k], e), hi = x * old;
              c[e] = int8_exact(x * ratio, hi, fmaf(x, old, -hi), s);
            }
        } else {
          const bool zeros = !(s > 0.f);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            c[e] = zeros ? kInt8Bias
                         : int8_exact_small((double)int8_code(words[k], e) * (double)old, s);
        }
        words[k] = __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040),
                               0x5410);
      }
      stg_v4(at, v);
    }
    __syncwarp();  // before other lanes' codes of the new tokens
  }
  if (begins || grows)
    for (int i = lane; i < 1 << (l2bs - 3); i += 32)
      head[i * (int8_tile_bytes(D) / 4)] = s;
  const float inv = s > 0.f ? 1.f / s : 0.f;
  auto put = [&](int i, int c, const uint4& v) {  // row i, chunk c * kLanes + col
    const int off = (int)(slots[i] & ((1 << l2bs) - 1));
    const int chunk = c * kLanes + col;
    uint8_t* at = base + (off >> 3) * int8_tile_bytes(D) + codes +
                  chunk * kPer / kInt8Group * 128 + (off & 7) * 16 + chunk * kPer % kInt8Group;
    const uint2 q = quantise_chunk<T>(v, s, inv);
    if constexpr (kPer == 8) *reinterpret_cast<uint2*>(at) = q;
    else *reinterpret_cast<uint32_t*>(at) = q.x;
  };
#pragma unroll
  for (int i = 0; i < kSteps; ++i)
    if (i * kRows + row < n)
#pragma unroll
      for (int c = 0; c < kCols; ++c) put(i * kRows + row, c, w[i][c]);
#pragma unroll 1
  for (int i = kSteps * kRows + row; i < n; i += kRows)
#pragma unroll
    for (int c = 0; c < kCols; ++c)
      put(i, c, ldg_nc_v4(src + i * stride + (c * kLanes + col) * kPer));
}

// Warps take (window of tokens, head, side); the window's tokens that are the first of
// their block's in the call are the warp's work, one after another.
template <typename T, int D>
__global__ void __launch_bounds__(kInt8Threads)
    int8_write_kernel(Int8Pool pool, const T* __restrict__ key, const T* __restrict__ value,
                      int64_t key_stride, int64_t value_stride,
                      const int64_t* __restrict__ slot_mapping, int num_tokens, int window,
                      unsigned int* err) {
  const int lane = threadIdx.x & 31;
  const int64_t unit = (int64_t)blockIdx.x * (kInt8Threads / 32) + threadIdx.x / 32;
  const int sides = 2 * pool.num_kv_heads;
  const int64_t w0 = unit / sides * window;
  const int side = (int)(unit % sides), h = side >> 1, kv = side & 1;
  const int l2bs = pool.log2_block_size;
  grid_dependents_launch();
  grid_dependency_wait();
  if (w0 >= num_tokens) return;
  const int64_t t = w0 + lane;
  const bool mine = lane < window && t < num_tokens;
  const int64_t slot = mine ? __ldg(slot_mapping + t) : -1;
  const int64_t before = mine && t > 0 ? __ldg(slot_mapping + t - 1) : -1;
  if (slot >= pool.num_slots && side == 0) record_error(err, PA_DEVERR_SLOT);
  auto valid = [&](int64_t s) { return s >= 0 && s < pool.num_slots; };
  const bool first = valid(slot) && !(valid(before) && (before >> l2bs) == (slot >> l2bs));
  uint32_t firsts = __ballot_sync(0xffffffffu, first);
  for (; firsts; firsts &= firsts - 1) {
    const int at = __ffs(firsts) - 1;
    const int64_t block = __shfl_sync(0xffffffffu, slot, at) >> l2bs;
    const int64_t t0 = w0 + at;
    // The run's length, and whether one of its tokens begins the block.
    int n = 0;
    bool begins = false;
    for (uint32_t same = 0xffffffffu; same == 0xffffffffu;) {
      const int64_t i = t0 + n + lane;
      const int64_t s = i < num_tokens ? __ldg(slot_mapping + i) : -1;
      const bool in = valid(s) && (s >> l2bs) == block;
      same = __ballot_sync(0xffffffffu, in);
      const int more = __ffs(~same) - 1;  // -1: all
      const bool counted = more < 0 || lane < more;
      begins |= __any_sync(0xffffffffu, counted && (s & ((1 << l2bs) - 1)) == 0);
      n += more < 0 ? 32 : more;
    }
    const T* src = (kv ? value + t0 * value_stride : key + t0 * key_stride) + h * D;
    write_run<T, D>(pool, src, kv ? value_stride : key_stride, slot_mapping + t0, n, block, begins,
                    h, kv);
  }
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
cudaError_t launch_write(const Int8Pool& pool, const void* key, const void* value,
                         int64_t key_stride, int64_t value_stride, const int64_t* slot_mapping,
                         int num_tokens, int num_sms, unsigned int* err, cudaStream_t stream) {
  // A token a warp while all warps are resident at once or nearly (64 warps an SM), so that
  // a batch's tokens, each with a block of its own, do not wait for one another; else
  // windows, so that a prompt's tokens do not each cost a warp.
  const int64_t sides = 2ll * pool.num_kv_heads;
  int window = 1;
  while (window < 32 && (num_tokens + window - 1) / window * sides > 64ll * num_sms) window *= 2;
  const int64_t warps = (num_tokens + window - 1) / window * sides;
  constexpr int kPerCta = kInt8Threads / 32;
  void* args[] = {const_cast<Int8Pool*>(&pool), &key, &value, &key_stride, &value_stride,
                  &slot_mapping, &num_tokens, &window, &err};
  return launch_overlapped((const void*)int8_write_kernel<T, D>,
                           dim3((unsigned)((warps + kPerCta - 1) / kPerCta)), dim3(kInt8Threads),
                           0, stream, args);
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
  auto run = [&](auto* launch) {
    return launch(pool, key, value, key_stride, value_stride, slot_mapping, num_tokens, num_sms,
                  err, stream);
  };
  const bool half = dtype == PA_BF16;
  switch (pool.head_size) {
    case 64: return half ? run(launch_write<__nv_bfloat16, 64>) : run(launch_write<float, 64>);
    case 128: return half ? run(launch_write<__nv_bfloat16, 128>) : run(launch_write<float, 128>);
    default: return half ? run(launch_write<__nv_bfloat16, 256>) : run(launch_write<float, 256>);
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
