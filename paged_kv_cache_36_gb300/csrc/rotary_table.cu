// The table of rotary angles that the RoPE entry points read: row p holds the cosines,
// then the sines, of (start + p) f_i for the rotary_dim / 2 frequencies f_i, times a factor.
//
// Of an angle only the remainder modulo a turn counts, and in float32 the remainder of a far
// position has no correct digits.  So frequencies are turns per position in fixed point, 64
// bits behind the point: the product with a position modulo 2^64 is the remainder, exact but
// for the frequency's own rounding (2^-65 turns, times the position, beside the 2^-55 that a
// frequency in 64-bit floating point may be off by itself), in integer arithmetic; 64-bit
// floating point, of which this GPU has little, takes 145 us for 131072 rows of 128.
//
// The nearest quarter turn is taken off.  What is left, r within an eighth of a turn, rounds to
// float32 and goes through the Taylor polynomials of factor sin(2 pi r) and factor cos(2 pi r),
// in r, so that nothing multiplies what has been rounded: the factor (in [1, 2), a power of two
// comes last) and the powers of 2 pi are in the coefficients, of which the cosine's first two and
// the sine's first take two floats.  In units of 2^-24 of the factor, at r = 1/8, the worst: the cosine is off by 0.71 for
// its last rounding, 0.28 for r's, 0.29 for r^2's and 0.34 for those of the sums before; the
// sine by 0.71, 0.28 and 0.47.  So 2 is a bound; the most of 20 million angles with nine factors
// was 1.33.  (A polynomial in radians, times the factor, was off by up to 2.67.)
//
// A thread keeps its four frequencies and goes down the rows by adding a step to each
// remainder.  131072 rows of 128 (67 MB) take 13.0 us, 5.2 TB/s.
#include <cuda_runtime.h>

#include <cstdint>

#include "kernels.h"
#include "pkv_device.cuh"

namespace pkv {

namespace {

constexpr int kThreads = 256;

// f times cosine and sine of `turn` 2^-64 turns, times `unit`.
__device__ __forceinline__ void cos_sin(uint64_t turn, const RotarySeries& f, float& c, float& s) {
  // an eighth of a turn further the quarter's two bits lead, and the 32 behind them count from
  // the quarter's middle
  const uint32_t hi = static_cast<uint32_t>(turn >> 32) + (1u << 29);
  const uint32_t rest = __funnelshift_l(static_cast<uint32_t>(turn), hi, 2) ^ (1u << 31);
  const float r = static_cast<float>(static_cast<int32_t>(rest)) * 0x1p-34f;
  const float r2 = r * r;
  const float q = fmaf(r2, fmaf(r2, fmaf(r2, fmaf(r2, f.s[4], f.s[3]), f.s[2]), f.s[1]), f.s_low);
  const float w = fmaf(r2, fmaf(r2, fmaf(r2, fmaf(r2, f.c[5], f.c[4]), f.c[3]), f.c[2]), f.c1_low);
  const float sn = fmaf(r, f.s[0], r * q);
  const float cs = f.c[0] + fmaf(r2, f.c[1], fmaf(r2, w, f.c_low));
  const bool odd = hi & (1u << 30);
  const uint32_t a = __float_as_uint(odd ? sn : cs), b = __float_as_uint(odd ? cs : sn);
  c = __uint_as_float(a ^ ((hi ^ hi << 1) & (1u << 31))) * f.unit;  // negative in quarters 1 and 2
  s = __uint_as_float(b ^ (hi & (1u << 31))) * f.unit;              // in 2 and 3
}

// kVec frequencies a thread, half / kVec threads a row.
template <int kVec>
__global__ void __launch_bounds__(kThreads, 4) rotary_table_kernel(const RotaryFrequencies f, float* __restrict__ out,
                                                                int64_t rows, int64_t start, int32_t half,
                                                                const RotarySeries series) {
  // (reads nothing that another kernel writes, but `out` may still be read by one)
  grid_dependency_wait();
  if (threadIdx.x == 0) grid_launch_dependents();
  const int cols = half / kVec;
  const uint32_t me = blockIdx.x * kThreads + threadIdx.x;
  const uint32_t step = gridDim.x * kThreads / cols;  // rows at once
  const uint32_t first = me / cols;
  if (first >= step) return;
  const int k = (me - first * cols) * kVec;
  uint64_t turn[kVec], more[kVec];
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const uint64_t w = f.turns[k + i];
    turn[i] = w * static_cast<uint64_t>(start + first);
    more[i] = w * step;
  }
  float* row = out + static_cast<int64_t>(first) * (2 * half) + k;
  for (int64_t p = first; p < rows; p += step, row += static_cast<int64_t>(step) * (2 * half)) {
    float c[kVec], s[kVec];
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      cos_sin(turn[i], series, c[i], s[i]);
      turn[i] += more[i];
    }
    if constexpr (kVec == 4) {
      *reinterpret_cast<float4*>(row) = make_float4(c[0], c[1], c[2], c[3]);
      *reinterpret_cast<float4*>(row + half) = make_float4(s[0], s[1], s[2], s[3]);
    } else {
      row[0] = c[0];
      row[half] = s[0];
    }
  }
}

}  // namespace

cudaError_t launch_rotary_table(const RotaryFrequencies& f, float* out, int64_t rows, int64_t start,
                                int32_t rotary_dim, const RotarySeries& series, cudaStream_t stream) {
  if (rows == 0) return cudaSuccess;
  const int half = rotary_dim / 2;
  const bool vec = half % 4 == 0;
  const int64_t items = rows * (half / (vec ? 4 : 1));
  const int64_t blocks = (items + kThreads - 1) / kThreads;
  const int64_t cap = 4 * static_cast<int64_t>(current_sm_count());  // one wave
  const dim3 grid(static_cast<unsigned>(blocks < cap ? blocks : cap));
  return launch_programmatic(vec ? rotary_table_kernel<4> : rotary_table_kernel<1>, grid, dim3(kThreads), 0, stream,
                             f, out, rows, start, half, series);
}

}  // namespace pkv
