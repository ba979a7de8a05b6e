// Quantising write into the 4-bit pool, and reading tokens back, for sm_103a.
//
// Both move a group of 16 elements of a token's key and the same of its value
// per thread: 32 bytes (bf16) or 64 bytes (fp32) each on one side, eight bytes of
// codes and one scale byte on the other, and are bound by memory; a thread takes
// key and value so that addresses are worked out once for both (one of them per
// thread spent 62% of the issue slots, most of it on addresses).  A CTA takes
// consecutive (eight tokens, head) units, the heads of a token next to each other,
// lanes a group's tokens, then the next group.  Tokens that follow one another
// usually lie in one tile, so that a warp's codes and scales are whole sectors of 32
// bytes, and the wide side is anyway.  (Units of one token block only would leave
// threads idle where heads are few: one head of 64, 150 MB, 59 us instead of 24.)
//
// Measured on 8 heads of 128, bf16, in a row of graph replays: the write of 65536
// tokens 51.7 us (344 MB, 6.7 TB/s, 98% of the copy rate, part of it L2's), the
// read-back 55.0 us (6.3 TB/s, 92%; fp32 75 to 89%, the lower where a token's row is
// a power of two); of 16381 tokens 15.1 and 16.3 us (5.7 and 5.3
// TB/s), where the L1 cache is at 72% (write) and 84% (read-back, its stores) of its
// rate.  777 tokens of 4 heads of 64 take 5.2 us and 64 tokens of 2 heads 3.1 us a
// call, which is the launch and two dependent reads.
#include "pa_fp4.cuh"
#include "pa_launch.h"

namespace pa {

namespace {

constexpr int kFp4Threads = 256;

// The thread's token, head and group; false where there is none.
template <int D>
__device__ __forceinline__ bool fp4_unit(int num_tokens, int num_kv_heads, int* t, int* h, int* j) {
  constexpr int kUnits = kFp4Tile * D / kFp4Group;  // of one head of eight tokens
  constexpr int kHeads = kFp4Threads / kUnits;
  const unsigned head = blockIdx.x * kHeads + threadIdx.x / kUnits;  // of all tokens' heads
  const unsigned block = head / (unsigned)num_kv_heads;
  const int i = threadIdx.x % kUnits;
  *h = (int)(head - block * num_kv_heads);
  *t = (int)min((unsigned long long)block * kFp4Tile + i % kFp4Tile, 0x7fffffffull);
  *j = i / kFp4Tile;
  return *t < num_tokens;
}

// Where group j of a tile's row has its codes and its scale.
template <int D>
__device__ __forceinline__ void fp4_places(int row, int j, int kv, int* codes, int* scale) {
  *codes = kv ? fp4_value_codes(D) + j * 64 + row * 8 : row * (D / 2) + j * 8;
  *scale = kv ? fp4_value_scales(D) + j * 8 + row : fp4_key_scales(D) + row * (D / kFp4Group) + j;
}

// The group's largest magnitude; a NaN if there is one.
__device__ __forceinline__ float largest(const uint4* w, const __nv_bfloat16*) {
  __nv_bfloat162 top = __float2bfloat162_rn(0.f);
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const uint32_t v[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
#pragma unroll
    for (int e = 0; e < 4; ++e)
      top = __hmax2_nan(top, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&v[e])));
  }
  return __bfloat162float(__hmax_nan(top.x, top.y));
}
__device__ __forceinline__ float largest(const uint4* w, const float*) {
  uint32_t top = 0;  // bits order NaNs above everything
#pragma unroll
  for (int c = 0; c < 4; ++c)
    top = max(max(top, max(w[c].x & 0x7fffffffu, w[c].y & 0x7fffffffu)),
              max(w[c].z & 0x7fffffffu, w[c].w & 0x7fffffffu));
  return __uint_as_float(top);
}

// A group to its codes; returns the scale's code.
template <typename T>
__device__ __forceinline__ uint32_t quantise16(const uint4* w, float tensor_scale, uint2* codes) {
  constexpr int kPer = ElemTraits<T>::kPerChunk;
  float x[16], q[16];
#pragma unroll
  for (int c = 0; c < 16 / kPer; ++c) ElemTraits<T>::unpack(w[c], x + c * kPer);
  const float inv_tensor = fast_rcp(tensor_scale);  // exact: a power of two
  const uint32_t code = fp4_scale_code(largest(w, static_cast<const T*>(nullptr)) * inv_tensor);
  const float s = e4m3_to_float(code);
  const float r = s > 0.f ? fast_rcp(s) * inv_tensor : 0.f;
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int e = 0; e < 16; ++e) q[e] = fp4_quotient_bf16(x[e], r);
  } else {
    bool sure = true;
#pragma unroll
    for (int e = 0; e < 16; ++e) q[e] = fp4_quotient_f32(x[e], r, &sure);
    if (!sure)
#pragma unroll
      for (int e = 0; e < 16; ++e) q[e] = fp4_exact_quotient_f32(x[e], s * tensor_scale, r);
  }
  *codes = make_uint2(e2m1_pack8(q), e2m1_pack8(q + 8));
  return code;
}

// 32 bytes as one sector (`wide`: the address is a multiple of 32) or as halves.  A
// warp's lanes ask for whole lines once then, not for halves of them twice, which
// takes the L1 cache to 89% of its rate (65536 tokens 51.7 and 65.0 us).
__device__ __forceinline__ void load32(const void* p, uint4* w, bool wide) {
  if (wide) {
    asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(w[0].x), "=r"(w[0].y), "=r"(w[0].z), "=r"(w[0].w), "=r"(w[1].x),
                   "=r"(w[1].y), "=r"(w[1].z), "=r"(w[1].w)
                 : "l"(p));
  } else {
    w[0] = ldg_nc_v4(p);
    w[1] = ldg_nc_v4(static_cast<const uint8_t*>(p) + 16);
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kFp4Threads)
    fp4_write_kernel(Fp4Pool pool, const T* __restrict__ key, const T* __restrict__ value,
                     int64_t key_stride, int64_t value_stride,
                     const int64_t* __restrict__ slot_mapping, int num_tokens, float key_scale,
                     float value_scale, bool wide, unsigned int* err) {
  constexpr int kChunks = sizeof(T);  // 16-byte parts of a group
  int t, h, j;
  const bool live = fp4_unit<D>(num_tokens, pool.num_kv_heads, &t, &h, &j);
  grid_dependents_launch();
  grid_dependency_wait();
  if (!live) return;
  const int64_t slot = __ldg(slot_mapping + t);
  // The rows are read whatever the slot says: the loads need not wait for it.
  uint4 w[2][kChunks];
  const T* src[2] = {key + t * key_stride + h * D + j * 16,
                     value + t * value_stride + h * D + j * 16};
#pragma unroll
  for (int kv = 0; kv < 2; ++kv)
#pragma unroll
    for (int c = 0; c < kChunks; c += 2)
      load32(reinterpret_cast<const uint4*>(src[kv]) + c, &w[kv][c], wide);
  if (slot < 0) return;
  if (slot >= pool.num_slots) {
    if (h == 0 && j == 0) record_error(err, PA_DEVERR_SLOT);
    return;
  }
  uint8_t* tile =
      pool.cache + fp4_tile_offset(slot, h, pool.num_kv_heads, pool.log2_block_size, D);
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    uint2 codes;
    const uint32_t scale = quantise16<T>(w[kv], kv ? value_scale : key_scale, &codes);
    int at_codes, at_scale;
    fp4_places<D>((int)(slot & 7), j, kv, &at_codes, &at_scale);
    *reinterpret_cast<uint2*>(tile + at_codes) = codes;
    tile[at_scale] = (uint8_t)scale;
  }
}

// 32 bytes as one sector (`wide`: the address is a multiple of 32) or as halves (the
// read-back of 65536 tokens 55.0 and 80.4 us).
__device__ __forceinline__ void store32(void* p, const uint32_t* w, bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]),
                 "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    stg_v4(p, make_uint4(w[0], w[1], w[2], w[3]));
    stg_v4(static_cast<uint8_t*>(p) + 16, make_uint4(w[4], w[5], w[6], w[7]));
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kFp4Threads)
    fp4_gather_kernel(Fp4Pool pool, T* __restrict__ key, T* __restrict__ value,
                      const int64_t* __restrict__ slot_mapping, int num_tokens, float key_scale,
                      float value_scale, bool wide, unsigned int* err) {
  int t, h, j;
  const bool live = fp4_unit<D>(num_tokens, pool.num_kv_heads, &t, &h, &j);
  grid_dependents_launch();
  grid_dependency_wait();
  if (!live) return;
  const int64_t slot = __ldg(slot_mapping + t);
  if (slot < 0) return;
  if (slot >= pool.num_slots) {
    if (h == 0 && j == 0) record_error(err, PA_DEVERR_SLOT);
    return;
  }
  const uint8_t* tile =
      pool.cache + fp4_tile_offset(slot, h, pool.num_kv_heads, pool.log2_block_size, D);
  uint2 codes[2];
  uint32_t scales[2];
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    int at_codes, at_scale;
    fp4_places<D>((int)(slot & 7), j, kv, &at_codes, &at_scale);
    codes[kv] = *reinterpret_cast<const uint2*>(tile + at_codes);
    scales[kv] = tile[at_scale];
  }
  const int64_t to = ((int64_t)t * pool.num_kv_heads + h) * D + j * 16;
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    const float s = e4m3_to_float(scales[kv]) * (kv ? value_scale : key_scale);
    uint32_t c[8];
    e2m1x8_to_half2(codes[kv].x, c);
    e2m1x8_to_half2(codes[kv].y, c + 4);
    float x[16];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      x[2 * e] = half_lo(c[e]) * s;
      x[2 * e + 1] = half_hi(c[e]) * s;
    }
    T* dst = (kv ? value : key) + to;
    if constexpr (sizeof(T) == 2) {
      uint32_t w[8];  // six significant bits: exact in bf16
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = pack_bf16x2(x[2 * e], x[2 * e + 1]);
      store32(dst, w, wide);
    } else {
      store32(dst, reinterpret_cast<const uint32_t*>(x), wide);
      store32(dst + 8, reinterpret_cast<const uint32_t*>(x) + 8, wide);
    }
  }
}

unsigned fp4_grid(const Fp4Pool& pool, int num_tokens) {
  const unsigned heads = kFp4Threads / (kFp4Tile * pool.head_size / kFp4Group);
  const unsigned all = ((unsigned)num_tokens + kFp4Tile - 1) / kFp4Tile * pool.num_kv_heads;
  return (all + heads - 1) / heads;
}

template <typename T, int D>
cudaError_t launch_write(const Fp4Pool& pool, const void* key, const void* value,
                         int64_t key_stride, int64_t value_stride, const int64_t* slot_mapping,
                         int num_tokens, float key_scale, float value_scale,
                         unsigned int* err, cudaStream_t stream) {
  bool wide = ((reinterpret_cast<uintptr_t>(key) | reinterpret_cast<uintptr_t>(value)) & 31) == 0 &&
              (key_stride | value_stride) * (int)sizeof(T) % 32 == 0;
  void* args[] = {const_cast<Fp4Pool*>(&pool), &key, &value, &key_stride, &value_stride,
                  &slot_mapping, &num_tokens, &key_scale, &value_scale, &wide, &err};
  return launch_overlapped((const void*)fp4_write_kernel<T, D>, dim3(fp4_grid(pool, num_tokens)),
                           dim3(kFp4Threads), 0, stream, args);
}

template <typename T, int D>
cudaError_t launch_gather(const Fp4Pool& pool, void* key, void* value,
                          const int64_t* slot_mapping, int num_tokens, float key_scale,
                          float value_scale, unsigned int* err, cudaStream_t stream) {
  bool wide = ((reinterpret_cast<uintptr_t>(key) | reinterpret_cast<uintptr_t>(value)) & 31) == 0;
  void* args[] = {const_cast<Fp4Pool*>(&pool), &key, &value, &slot_mapping, &num_tokens,
                  &key_scale, &value_scale, &wide, &err};
  return launch_overlapped((const void*)fp4_gather_kernel<T, D>, dim3(fp4_grid(pool, num_tokens)),
                           dim3(kFp4Threads), 0, stream, args);
}

}  // namespace

cudaError_t launch_fp4_write(const Fp4Pool& pool, const void* key, const void* value, int dtype,
                             int64_t key_stride, int64_t value_stride,
                             const int64_t* slot_mapping, int num_tokens, float key_scale,
                             float value_scale, unsigned int* err, cudaStream_t stream) {
  auto run = [&](auto* launch) {
    return launch(pool, key, value, key_stride, value_stride, slot_mapping, num_tokens, key_scale,
                  value_scale, err, stream);
  };
  const bool half = dtype == PA_BF16;
  switch (pool.head_size) {
    case 64: return half ? run(launch_write<__nv_bfloat16, 64>) : run(launch_write<float, 64>);
    case 128: return half ? run(launch_write<__nv_bfloat16, 128>) : run(launch_write<float, 128>);
    default: return half ? run(launch_write<__nv_bfloat16, 256>) : run(launch_write<float, 256>);
  }
}

cudaError_t launch_fp4_gather(const Fp4Pool& pool, void* key, void* value, int dtype,
                              const int64_t* slot_mapping, int num_tokens, float key_scale,
                              float value_scale, unsigned int* err, cudaStream_t stream) {
  auto run = [&](auto* launch) {
    return launch(pool, key, value, slot_mapping, num_tokens, key_scale, value_scale, err, stream);
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
