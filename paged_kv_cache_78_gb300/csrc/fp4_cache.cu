// Quantising write into the 4-bit pool, and reading tokens back, for sm_103a.
//
// Both move a group of 16 elements per thread: 32 bytes (bf16) or 64 bytes
// (fp32) on one side, eight bytes of codes and one scale byte on the other.
// Consecutive threads take a token's groups, then its heads, so the wide side
// is read or written in whole lines.
#include "pa_fp4.cuh"
#include "pa_launch.h"

namespace pa {

namespace {

// The thread's group: token t, keys or values, head h, group j.
struct Fp4Unit {
  int64_t t;
  int kv, h, j;
};

__device__ __forceinline__ Fp4Unit fp4_unit(int64_t i, int groups, int num_kv_heads) {
  const int row_units = num_kv_heads * groups;
  Fp4Unit u;
  u.t = i / (2 * row_units);
  int r = (int)(i - u.t * 2 * row_units);
  u.kv = r >= row_units;
  r -= u.kv ? row_units : 0;
  u.h = r / groups;
  u.j = r - u.h * groups;
  return u;
}

// Where the group's codes and scale lie in its tile.
template <int D>
__device__ __forceinline__ void fp4_places(const Fp4Unit& u, int row, int* codes, int* scale) {
  constexpr int kGroups = D / kFp4Group;
  *codes = u.kv ? fp4_value_codes(D) + u.j * 64 + row * 8 : row * (D / 2) + u.j * 8;
  *scale = u.kv ? fp4_value_scales(D) + u.j * 8 + row : fp4_key_scales(D) + row * kGroups + u.j;
}

template <typename T>
__device__ __forceinline__ void load16(const T* src, float* x) {
  constexpr int kPer = ElemTraits<T>::kPerChunk;
#pragma unroll
  for (int c = 0; c < 16 / kPer; ++c) ElemTraits<T>::unpack(ldg_nc_v4(src + c * kPer), x + c * kPer);
}

template <typename T, int D>
__global__ void __launch_bounds__(256)
    fp4_write_kernel(Fp4Pool pool, const T* __restrict__ key, const T* __restrict__ value,
                     int64_t key_stride, int64_t value_stride,
                     const int64_t* __restrict__ slot_mapping, int64_t num_tokens, float key_scale,
                     float value_scale, unsigned int* err) {
  grid_dependents_launch();
  grid_dependency_wait();
  constexpr int kGroups = D / kFp4Group;
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= num_tokens * 2 * pool.num_kv_heads * kGroups) return;
  const Fp4Unit u = fp4_unit(i, kGroups, pool.num_kv_heads);
  const int64_t slot = __ldg(slot_mapping + u.t);
  if (slot < 0) return;
  if (slot >= pool.num_slots) {
    if (u.kv == 0 && u.h == 0 && u.j == 0) record_error(err, PA_DEVERR_SLOT);
    return;
  }
  const T* src = (u.kv ? value + u.t * value_stride : key + u.t * key_stride) + u.h * D + u.j * 16;
  float x[16];
  load16(src, x);
  const float tensor_scale = u.kv ? value_scale : key_scale;
  // The largest magnitude by its bits, which order NaNs above everything.
  uint32_t top = 0;
#pragma unroll
  for (int e = 0; e < 16; ++e) top = max(top, __float_as_uint(x[e]) & 0x7fffffffu);
  const float inv_tensor = __frcp_rn(tensor_scale);
  const uint32_t code = fp4_scale_code(__uint_as_float(top) * inv_tensor);
  const float s = e4m3_to_float(code);
  const float r = s > 0.f ? __frcp_rn(s) * inv_tensor : 0.f;
  float q[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    if constexpr (sizeof(T) == 2) q[e] = fp4_quotient_bf16(x[e], r);
    else q[e] = fp4_quotient_f32(x[e], s * tensor_scale, r);
  }
  int at_codes, at_scale;
  fp4_places<D>(u, (int)(slot & 7), &at_codes, &at_scale);
  uint8_t* tile = pool.cache +
                  fp4_tile_offset(slot, u.h, pool.num_kv_heads, pool.log2_block_size, D);
  *reinterpret_cast<uint2*>(tile + at_codes) = make_uint2(e2m1_pack8(q), e2m1_pack8(q + 8));
  tile[at_scale] = (uint8_t)code;
}

template <typename T, int D>
__global__ void __launch_bounds__(256)
    fp4_gather_kernel(Fp4Pool pool, T* __restrict__ key, T* __restrict__ value,
                      const int64_t* __restrict__ slot_mapping, int64_t num_tokens,
                      float key_scale, float value_scale, unsigned int* err) {
  grid_dependents_launch();
  grid_dependency_wait();
  constexpr int kGroups = D / kFp4Group;
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= num_tokens * 2 * pool.num_kv_heads * kGroups) return;
  const Fp4Unit u = fp4_unit(i, kGroups, pool.num_kv_heads);
  const int64_t slot = __ldg(slot_mapping + u.t);
  if (slot < 0) return;
  if (slot >= pool.num_slots) {
    if (u.kv == 0 && u.h == 0 && u.j == 0) record_error(err, PA_DEVERR_SLOT);
    return;
  }
  int at_codes, at_scale;
  fp4_places<D>(u, (int)(slot & 7), &at_codes, &at_scale);
  const uint8_t* tile = pool.cache +
                        fp4_tile_offset(slot, u.h, pool.num_kv_heads, pool.log2_block_size, D);
  const uint2 w = *reinterpret_cast<const uint2*>(tile + at_codes);
  const float s = e4m3_to_float(tile[at_scale]) * (u.kv ? value_scale : key_scale);
  uint32_t h[8];
  e2m1x8_to_half2(w.x, h);
  e2m1x8_to_half2(w.y, h + 4);
  float x[16];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    x[2 * e] = half_lo(h[e]) * s;
    x[2 * e + 1] = half_hi(h[e]) * s;
  }
  T* dst = (u.kv ? value : key) + (u.t * pool.num_kv_heads + u.h) * D + u.j * 16;
  uint4* d4 = reinterpret_cast<uint4*>(dst);
  if constexpr (sizeof(T) == 2) {
    // Six significant bits: exact in bf16.
#pragma unroll
    for (int c = 0; c < 2; ++c)
      stg_v4(d4 + c, make_uint4(pack_bf16x2(x[8 * c], x[8 * c + 1]),
                                pack_bf16x2(x[8 * c + 2], x[8 * c + 3]),
                                pack_bf16x2(x[8 * c + 4], x[8 * c + 5]),
                                pack_bf16x2(x[8 * c + 6], x[8 * c + 7])));
  } else {
#pragma unroll
    for (int c = 0; c < 4; ++c)
      stg_v4(d4 + c, make_uint4(__float_as_uint(x[4 * c]), __float_as_uint(x[4 * c + 1]),
                                __float_as_uint(x[4 * c + 2]), __float_as_uint(x[4 * c + 3])));
  }
}

constexpr int kFp4Threads = 256;

unsigned fp4_grid(const Fp4Pool& pool, int64_t num_tokens) {
  const int64_t units = num_tokens * 2 * pool.num_kv_heads * (pool.head_size / kFp4Group);
  return (unsigned)((units + kFp4Threads - 1) / kFp4Threads);
}

template <typename T, int D>
cudaError_t launch_write(const Fp4Pool& pool, const void* key, const void* value,
                         int64_t key_stride, int64_t value_stride, const int64_t* slot_mapping,
                         int64_t num_tokens, float key_scale, float value_scale,
                         unsigned int* err, cudaStream_t stream) {
  void* args[] = {const_cast<Fp4Pool*>(&pool), &key, &value, &key_stride, &value_stride,
                  &slot_mapping, &num_tokens, &key_scale, &value_scale, &err};
  return launch_overlapped((const void*)fp4_write_kernel<T, D>, dim3(fp4_grid(pool, num_tokens)),
                           dim3(kFp4Threads), 0, stream, args);
}

template <typename T, int D>
cudaError_t launch_gather(const Fp4Pool& pool, void* key, void* value,
                          const int64_t* slot_mapping, int64_t num_tokens, float key_scale,
                          float value_scale, unsigned int* err, cudaStream_t stream) {
  void* args[] = {const_cast<Fp4Pool*>(&pool), &key, &value, &slot_mapping, &num_tokens,
                  &key_scale, &value_scale, &err};
  return launch_overlapped((const void*)fp4_gather_kernel<T, D>, dim3(fp4_grid(pool, num_tokens)),
                           dim3(kFp4Threads), 0, stream, args);
}

}  // namespace

cudaError_t launch_fp4_write(const Fp4Pool& pool, const void* key, const void* value, int dtype,
                             int64_t key_stride, int64_t value_stride,
                             const int64_t* slot_mapping, int64_t num_tokens, float key_scale,
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
                              const int64_t* slot_mapping, int64_t num_tokens, float key_scale,
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
