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
// of which the GPU has little: the write of 16385 tokens 190 us, for one piece in 60.)
// Scales below 2^-100 are lifted first, and what they divide with them.
constexpr float kInt8Small = 0x1p-100f;
__device__ __forceinline__ float int8_lift_of(float s) { return s < kInt8Small ? 0x1p100f : 1.f; }
__device__ __forceinline__ uint32_t int8_exact(float t, float hi, float lo, float s) {
  float c = rintf(t);
  const float e = fmaf(-c, s, hi);
  const float past = (fabsf(e) - 0.5f * s) + (e < 0.f ? -lo : lo);
  const bool odd = (int)c & 1;
  if (past > 0.f || (past == 0.f && odd)) c += e < 0.f ? -1.f : 1.f;
  return (uint32_t)((int)c + kInt8Bias);
}

// The nearest whole number to x * inv, plus 128, in the low byte; *off: how far x * inv is
// from it at the most so far.  1.5 * 2^23 as a summand leaves whole numbers in a sum's
// low bits, and neither product is rounded before it is added.  inv = 1 / s is off by
// half a step: x * inv is by 2^-17 up to 128, so that no quotient is on the other
// side of a tie while *off stays below a half less 2^-15.
constexpr float kInt8Sure = 0.5f - 0x1p-15f;
__device__ __forceinline__ uint32_t int8_near(float x, float inv, float* off) {
  constexpr float kGrid = 12582912.f;
  const float r = fmaf(x, inv, kGrid + kInt8Bias);
  *off = fmaxf(*off, fabsf(fmaf(x, inv, (kGrid + kInt8Bias) - r)));
  return __float_as_uint(r);
}

// bf16 x, whose scale s is the rounded m / 127 of a bf16 maximum m: 127 x / m is a tie or 2^-16
// (relative) away from one, as both have eight bits.  One in a hundred is a tie, and x / s
// then lies beside it, on the side that the rounding of s gives, the same for all.  So the
// reciprocal is taken off by 2^-21 that way (int8_lean): ties fall on their side, and nothing else
// moves past one.  Where s is m / 127 exactly, m is 127 times a power of two, which s and its reciprocal
// are then, and ties are ties.
__device__ __forceinline__ float int8_lean(float m, float s, float inv) {
  const float e = fmaf(s, 127.f, -m);  // exact: the rounding of s, times 127
  return e == 0.f ? inv : inv + (e > 0.f ? -inv : inv) * 0x1p-21f;
}

// Any bf16 x: the nearest whole number c, then the one nearest to c + e / s with the
// exact remainder e = x - c s, again as a sum whose rounding is ties to even.  x is a multiple of
// s's last place where it counts (|x| > s / 4), so 2 |e| is s or differs from it by a last
// place of s, more than 2^-24 of s, and inv is off by less: e * inv is on e / s's side of a
// half.  That 2 |e| is s takes a scale of no more bits than x has (int8_few_bits).
__device__ __forceinline__ bool int8_few_bits(float s) { return (__float_as_uint(s) & 0xffffu) == 0; }
__device__ __forceinline__ uint32_t int8_near_bf16(float x, float inv, float s) {
  constexpr float kGrid = 12582912.f + kInt8Bias;
  const float r = fmaf(x, inv, kGrid);
  return __float_as_uint(fmaf(fmaf(kGrid - r, s, x), inv, r));
}
// Two at a time.
__device__ __forceinline__ void int8_plain(float x, float y, float inv, uint32_t* c) {
  constexpr float kGrid = 12582912.f + kInt8Bias;
  const float2 r = parts(fma2(two(x, y), two(inv, inv), two(kGrid, kGrid)));
  c[0] = __float_as_uint(r.x), c[1] = __float_as_uint(r.y);
}

// The low bytes of four words.
__device__ __forceinline__ uint32_t low_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

}  // namespace pa
