// The 8-bit pool: where a block's codes and scales lie, and the conversions between
// numbers and codes (see include/pa.h).
#pragma once

#include <stdint.h>

#include "pa_device.cuh"
#include "warp_decode.cuh"

namespace pa {

constexpr int kInt8Tile = 8;       // tokens of a tile
constexpr int kInt8Header = 16;    // bytes: key scale, value scale, zeros
constexpr int kInt8Group = 16;     // elements that lie together
constexpr int kInt8Bias = 128;     // codes are stored plus this

// Bytes of a tile of head size D, and of its value codes' offset.
__host__ __device__ constexpr int int8_tile_bytes(int D) { return 16 * (D + 1); }
__host__ __device__ constexpr int int8_key_codes() { return kInt8Header; }
__host__ __device__ constexpr int int8_value_codes(int D) { return kInt8Header + 8 * D; }

// First byte of the tiles of block `block` and KV head h.
__device__ __forceinline__ size_t int8_block_offset(int64_t block, int h, int num_kv_heads,
                                                    int log2_block_size, int D) {
  return (((size_t)block * num_kv_heads + h) << (log2_block_size - 3)) * int8_tile_bytes(D);
}

// Two stored codes of w, bytes kFirst and kSecond, as an fp16 pair (exact): the bytes
// under fp16's 1024 are 1024 + 128 + code, and 1152 less is the code.
template <int kFirst, int kSecond>
__device__ __forceinline__ uint32_t int8x2_to_half2(uint32_t w) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;"
      : "=r"(r)
      : "r"(__byte_perm(w, 0x64646464u, 0x4040 | kFirst | (kSecond << 8))), "r"(0x64806480u));
  return r;
}

// A stored code as a whole number.
__device__ __forceinline__ int int8_code(uint32_t w, int byte) {
  return (int)((w >> (8 * byte)) & 0xffu) - kInt8Bias;
}

// max |x| / 127 rounded to fp32, from the bits of max |x| (which order NaN above infinity
// above numbers); NaN where that is no number.
__device__ __forceinline__ float int8_scale(uint32_t most) {
  return most >= 0x7f800000u ? __uint_as_float(0x7fffffffu)
                             : __fdiv_rn(__uint_as_float(most), 127.f);
}

// x / s to the nearest whole number, ties to even, decided on the exact quotient, plus 128;
// x = hi + lo (lo at most half a step of hi), |x| <= 127.5 s, s >= 2^-100, from the
// approximate quotient t, off by 2^-16 at the most.  hi - c s has no more bits than fp32
// holds: for c = 0 it is hi, for c = 1 hi and s are within a factor of two, and from there on hi is a
// multiple of s's last place and the difference below 2^24 of those.  Neither is |hi - c s| -
// s / 2 rounded where it is near zero, and a sum's sign is not rounded ever.  (In fp64,
// of which the GPU has little: the write of 16385 tokens 190 us, as one chunk in 60 has
// a quotient beside a tie.)
__device__ __forceinline__ uint32_t int8_exact(float t, float hi, float lo, float s) {
  float c = rintf(t);
  const float e = fmaf(-c, s, hi);
  const float past = (fabsf(e) - 0.5f * s) + (e < 0.f ? -lo : lo);
  const bool odd = (int)c & 1;
  if (past > 0.f || (past == 0.f && odd)) c += e < 0.f ? -1.f : 1.f;
  return (uint32_t)((int)c + kInt8Bias);
}

// The same in fp64 for scales below that.  A quotient of numbers of 32 bits and 24 that is no
// tie is 2^-33 (relative) away from one at the least, and fp64 keeps 2^-53.
static __device__ __noinline__ uint32_t int8_exact_small(double x, float s) {
  const double q = rint(x / (double)s);
  return (uint32_t)((int)fmin(fmax(q, -127.0), 127.0) + kInt8Bias);
}

// The same from the approximate quotient t = x * (1 / s), off by 2^-16 at the most up to
// 128 (half a step of 2^-24 for 1 / s and for the product): beside a tie, *sure turns
// false.  1.5 * 2^23 as a summand leaves the nearest whole number in the sum's low bits.
__device__ __forceinline__ uint32_t int8_near(float t, bool* sure) {
  constexpr float kGrid = 12582912.f;
  const float r = t + kGrid;
  const float off = fabsf(t - (r - kGrid));
  *sure = *sure && off < 0.5f - 0x1p-15f;
  return __float_as_uint(r) + kInt8Bias;  // the low byte
}

}  // namespace pa
