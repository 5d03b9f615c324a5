// The 4-bit paged cache: microscaled e2m1 rows (32 dimensions share one
// power-of-two scale) and where their bytes sit inside a 16-token block.
//
// A value is code * 2^(e - 127): `code` an e2m1 number (0, 0.5, 1, 1.5, 2, 3, 4,
// 6 and their negatives), `e` the scale byte of its 32 dimensions; e = 255
// makes the whole group NaN.  A block of one cache holds its KV heads one
// after the other, each in chunk_bytes = 17 D / 2 bytes: 16 rows of D / 2 code
// bytes, then 16 D / 32 scale bytes.
//
// The order inside a row is the one the tensor-core fragments want, so that
// the attention kernels load whole vectors and never shuffle codes between
// lanes.  With b = d / 32:
//   K: lane c of a quad (c = 0..3) takes dims 32 b + 8 c .. + 7 of every b, so
//      those 4 bytes of all b sit together: byte c D/8 + 4 b + (d % 8) / 2
//   V: lane group g (0..7) takes dims 32 b + 4 g .. + 3 of every b: byte
//      g D/16 + 2 b + (d % 4) / 2
// (even position of a pair in the low nibble).  K scales are in row order,
// t D/32 + b.  V scales of a token pair are interleaved two dimension groups
// at a time, (t / 2) D/16 + (b / 2) 4 + (t % 2) 2 + b % 2: one 32-bit word then
// holds both tokens of two groups, a half-word pair after a shift and a mask.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace pkv {

constexpr int kMxBlock = 16;    // tokens per cache block
constexpr int kMxGroup = 32;    // dimensions per scale

// Bytes of one KV head in one block, and the parts of it.
__host__ __device__ constexpr int mx_row_bytes(int d) { return d / 2; }
__host__ __device__ constexpr int mx_scale_off(int d) { return kMxBlock * d / 2; }
__host__ __device__ constexpr int mx_chunk_bytes(int d) { return kMxBlock * (d / 2 + d / kMxGroup); }

// 2^(e - 127) of a scale byte; NaN for 255, subnormal for 0.
__device__ __forceinline__ float mx_scale(uint32_t e) {
  const uint32_t bits = e == 0u ? 0x00400000u : e == 255u ? 0x7fffffffu : e << 23;
  return __uint_as_float(bits);
}

// Byte offset, inside a chunk, of the V scale of token t and group b.
template <int D>
__device__ __forceinline__ int mx_vscale_off(int t, int b) {
  return mx_scale_off(D) + (t >> 1) * (D / 16) + (b >> 1) * 4 + (t & 1) * 2 + (b & 1);
}

// Two scale bytes as bfloat16 powers of two, NaN for 255.
__device__ __forceinline__ uint32_t e8m0x2_to_bf16x2(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "mov.b32 {lo, hi}, %1;\n\t"
      "cvt.rn.bf16x2.ue8m0x2 %0, lo;\n\t}"
      : "=r"(r)
      : "r"(w));
  return r;
}

// The two codes of one byte as f16 values (even position in the low half).
__device__ __forceinline__ uint32_t e2m1x2_to_f16x2(uint32_t byte) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t}"
      : "=r"(r)
      : "r"(byte));
  return r;
}

// The eight codes of a word as four f16 pairs.
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&r)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(w));
}

// Eight floats to eight codes, round to nearest even, saturating at 6.
__device__ __forceinline__ uint32_t f32x8_to_e2m1(const float (&x)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return r;
}

}  // namespace pkv
