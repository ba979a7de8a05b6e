// The 4-bit pool: where a token's codes and scales lie, and the conversions
// between numbers and codes (e2m1 codes, one e4m3 scale per 16 elements, see
// include/pa.h).
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "pa_device.cuh"

namespace pa {

constexpr int kFp4Tile = 8;    // tokens of a tile
constexpr int kFp4Group = 16;  // elements that share a scale

// Byte offsets inside a tile of head size D.
__host__ __device__ constexpr int fp4_tile_bytes(int D) { return 9 * D; }
__host__ __device__ constexpr int fp4_value_codes(int D) { return 4 * D; }
__host__ __device__ constexpr int fp4_key_scales(int D) { return 8 * D; }
__host__ __device__ constexpr int fp4_value_scales(int D) { return 8 * D + D / 2; }

// First byte of the tile that holds `slot` for KV head h.
__device__ __forceinline__ size_t fp4_tile_offset(int64_t slot, int h, int num_kv_heads,
                                                  int log2_block_size, int D) {
  const size_t block = (size_t)(slot >> log2_block_size);
  const size_t tile = (size_t)((slot & ((1 << log2_block_size) - 1)) >> 3);
  return (((block * num_kv_heads + h) << (log2_block_size - 3)) + tile) * fp4_tile_bytes(D);
}

// ---- codes to numbers ---------------------------------------------------------

// The two codes of each byte of w as fp16 pairs (exact), low nibble first.
__device__ __forceinline__ void e2m1x8_to_half2(uint32_t w, uint32_t* h) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

// Two e4m3 scales as an fp16 pair (exact; the code 0x7f is NaN).
__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
  return h;
}

// Code times scale: at most six significant bits between 2^-10 and 2688, so
// exact in fp16.
__device__ __forceinline__ uint32_t half2_mul(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__device__ __forceinline__ float half_lo(uint32_t h) {
  float f;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.f32.f16 %0, a;\n\t}" : "=f"(f) : "r"(h));
  return f;
}
__device__ __forceinline__ float half_hi(uint32_t h) {
  float f;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.f32.f16 %0, b;\n\t}" : "=f"(f) : "r"(h));
  return f;
}

// ---- numbers to codes ---------------------------------------------------------

// 1 / x, off by at most one last place; exact for powers of two.
__device__ __forceinline__ float fast_rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// e4m3 of max / 6 (nearest, ties to even, at most 448; NaN stays NaN).  A max past
// 6 * 448, infinity among them (a number may become one in the division by a tensor
// scale below 1), is as good as that.  The quotient is first rounded to fp32 (by one step of
// Newton's iteration on the rounded product, which is enough for a correctly
// rounded 1 / 6), which never moves it onto or past a border of e4m3: a border
// times six has at most seven significant bits, so a max other than that is
// off by one of its own last places, more than the rounding.
__device__ __forceinline__ uint32_t fp4_scale_code(float max_abs) {
  constexpr float kSixth = 1.f / 6.f, kMost = 6.f * 448.f;
  if (max_abs > kMost) max_abs = kMost;  // false for NaN
  const float p = max_abs * kSixth;
  const float q = fmaf(fmaf(-6.f, p, max_abs), kSixth, p);
  uint32_t r;
  asm("{\n\t.reg .b16 c;\n\tcvt.rn.satfinite.e4m3x2.f32 c, %2, %1;\n\tcvt.u32.u16 %0, c;\n\t}"
      : "=r"(r)
      : "f"(q), "f"(0.f));
  return r & 0xffu;
}

__device__ __forceinline__ float e4m3_to_float(uint32_t code) {
  return half_lo(e4m3x2_to_half2(code));
}

// Eight quotients to codes, the first in the lowest nibble (nearest, ties to
// even, at most 6).
__device__ __forceinline__ uint32_t e2m1_pack8(const float* q) {
  uint32_t w;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(w)
      : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]), "f"(q[4]), "f"(q[5]), "f"(q[6]), "f"(q[7]));
  return w;
}

// x / s for the conversion to e2m1, s an e4m3 number, r = 1 / s within 2^-22.  The
// borders of e2m1 are 0.25 .. 5; a quotient has to reach the conversion on its
// own side of each, or exactly on it.
//
// bf16 x: x and border * s are multiples of a common last place of eight
// significant bits, so a quotient that is not a border is 2^-8 (relative)
// away from it.  x * r is off by 2^-22; added to 1.5 * 2^12 it rounds to a
// multiple of 2^-11, which puts a border's own quotient on the border (they
// are multiples) and moves no other onto or past one (0.25 * 2^-8 > 2^-12).
// A NaN or infinite sum is as good: the group's scale decides, or 6 does.
__device__ __forceinline__ float fp4_quotient_bf16(float x, float r) {
  constexpr float kGrid = 6144.f;
  return fmaf(x, r, kGrid) - kGrid;
}

// fp32 x: x * r, off by 2^-22 (relative), is rounded to a multiple of 2^-16 in the
// sum with 1.5 * 2^7; that is off by less than 2^-16 up to 8, so it lies on x / s's
// side of every border that it is not on.  *sure turns false where it may be on one:
// on a multiple of 1/4, which the sum's low bits show.
__device__ __forceinline__ float fp4_quotient_f32(float x, float r, bool* sure) {
  constexpr float kGrid = 192.f;
  const float t = fmaf(x, r, kGrid);
  *sure = *sure && (__float_as_uint(t) & 0x3fffu) != 0;
  return t - kGrid;
}

// Then: the rounded quotient, and where it fell on a number with few bits (as
// borders are) one last place towards the side that the remainder's sign gives.
// (About one group of random numbers in 1000, and those with zeros.  For every element
// it made the write of fp32 rows bound by instructions: 8 heads of 128, 150 MB, 30.8 us
// at 72% of the copy rate.)
__device__ __forceinline__ float fp4_exact_quotient_f32(float x, float s, float r) {
  float q = x * r;
  if (!(fabsf(q) > 0.2f && fabsf(q) < 8.f)) return q;  // zero, or 6
  q = fmaf(fmaf(-q, s, x), r, q);
  const float rest = fmaf(-q, s, x);
  if ((__float_as_uint(q) & 0xfffffu) == 0 && rest != 0.f)
    q = __uint_as_float(__float_as_uint(q) + ((rest > 0.f) == (q > 0.f) ? 1u : 0xffffffffu));
  return q;
}

}  // namespace pa
