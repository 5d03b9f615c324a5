// The 8-bit paged cache: e4m3 codes, one power-of-two scale for each block of 16 tokens
// and KV head, and where their bytes sit inside a block.
//
// A value is code * 2^(e - 127), `e` the block's scale byte of that KV head, read as
// clamp(e, 10, 246).  A code has four significant bits and lies between 2^-9 and 448, so
// with those e every value is a normal bfloat16: attention over this cache is attention
// over a bfloat16 cache of the same values.  (A float32 scale would fill the codes' range
// up to 448 exactly; e4m3 is a floating-point type, so that changes the number of binades
// below the largest value by less than one and no rounding above them, and it would cost
// bfloat16's exactness, and that of bringing rows to a larger scale.)
//
// A block of one cache holds its KV heads one after the other, each in a chunk of 16 D
// code bytes, the scale byte and 15 zero bytes.  The order of the codes is the one the
// warp MMA's A fragments want, so that a lane of the decode kernel loads its part of 16
// tokens as D / 32 whole vectors, lane after lane, and nothing is shuffled:
//   K (a row is a token): vector j of lane 4 g + c is dims 64 (j % (D / 64)) + 16 c .. + 15
//     of token g + 8 (j / (D / 64));
//   V (a row is a dimension): vector j of lane 4 g + c is dims (D / 8) g + 4 j .. + 3, each
//     with tokens 2c, 2c + 1, 2c + 8, 2c + 9.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace pkv {

constexpr int kF8Block = 16;                 // tokens per cache block
constexpr int kF8MinScale = 10;              // 2^-9 2^(10 - 127) is bfloat16's smallest normal number
constexpr int kF8MaxScale = 246;             // 448 2^(246 - 127) = 1.75 2^127 is finite
constexpr int kF8Loud = 207;                 // up to here 2^31 values (below 2^89) times 2^8 add up to less than 2^128

__host__ __device__ constexpr int f8_code_bytes(int d) { return kF8Block * d; }
__host__ __device__ constexpr int f8_chunk_bytes(int d) { return kF8Block * d + 16; }

// A scale byte as it counts.
__device__ __forceinline__ int f8_scale(uint32_t byte) {
  return min(max(static_cast<int>(byte), kF8MinScale), kF8MaxScale);
}

// The scale of rows whose largest finite magnitude has these float32 bits: the smallest e
// with |x| <= 448 2^(e - 127), 448 = 1.75 2^8.
__device__ __forceinline__ int f8_scale_of(uint32_t bits) {
  const int e = static_cast<int>(bits >> 23) - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  return min(max(e, kF8MinScale), kF8MaxScale);
}

// 2^k, k in [-126, 127].
__device__ __forceinline__ float f8_pow2(int k) {
  return __uint_as_float(static_cast<uint32_t>(k + 127) << 23);
}

// The four codes of a word as two f16 pairs (exact; byte 0 in the low half of lo).
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

// As four floats.
__device__ __forceinline__ void e4m3x4_to_f32(uint32_t w, float (&x)[4]) {
  uint32_t lo, hi;
  e4m3x4_to_f16(w, lo, hi);
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  x[0] = a.x;
  x[1] = a.y;
  x[2] = b.x;
  x[3] = b.y;
}

// Four floats to codes, to nearest even, saturating at 448; NaN stays NaN.
__device__ __forceinline__ uint32_t f32x4_to_e4m3(float x0, float x1, float x2, float x3) {
  uint32_t r;
  asm("{\n\t.reg .b16 a, b;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 b, %4, %3;\n\t"
      "mov.b32 %0, {a, b};\n\t}"
      : "=r"(r)
      : "f"(x0), "f"(x1), "f"(x2), "f"(x3));
  return r;
}

// The codes of a word at a scale `down` = 2^-n times as fine, rounded again.
__device__ __forceinline__ uint32_t e4m3x4_rescale(uint32_t w, float down) {
  float x[4];
  e4m3x4_to_f32(w, x);
  return f32x4_to_e4m3(x[0] * down, x[1] * down, x[2] * down, x[3] * down);
}

// Byte offsets of token t's key and value codes of dimension d in a chunk.
template <int D>
__device__ __forceinline__ int f8_key_at(int t, int d) {
  return ((t >> 3) * (D / 64) + d / 64) * 512 + (t & 7) * 64 + d % 64;
}
template <int D>
__device__ __forceinline__ int f8_value_at(int t, int d) {
  constexpr int P = D / 8;
  return d % P / 4 * 512 + (d / P * 4 + (t & 7) / 2) * 16 + d % 4 * 4 + (t >> 3) * 2 + (t & 1);
}

}  // namespace pkv
