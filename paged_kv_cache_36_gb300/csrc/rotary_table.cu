// The table of rotary angles that the RoPE entry points read: row p holds the cosines,
// then the sines, of (start + p) f_i for the rotary_dim / 2 frequencies f_i, times a factor.
//
// Of an angle only the remainder modulo a turn counts, and in float32 the remainder of a far
// position has no correct digits.  So frequencies are turns per position in fixed point, 64
// bits behind the point: the product with a position modulo 2^64 is the remainder, exact but
// for the frequency's own rounding (2^-65 turns, times the position), in integer arithmetic;
// 64-bit floating point, of which this GPU has little, takes 145 us for 131072 rows of 128.
// The nearest quarter turn is taken off, and what is left, within pi / 4, rounds once to
// float32 (2^-25 of a radian at most) and goes through the sine's and cosine's Taylor
// polynomials (the first terms left out are below 2^-29).
//
// A thread keeps its four frequencies and goes down the rows by adding a step to each
// remainder.  131072 rows of 128 (67 MB) take 13.7 us, 4.9 TB/s: 40 instructions an angle, 72 %
// of the issue slots (counters of the same call).
#include <cuda_runtime.h>

#include <cstdint>

#include "kernels.h"
#include "pkv_device.cuh"

namespace pkv {

namespace {

constexpr int kThreads = 256;

// factor times cosine and sine of `turn` 2^-64 turns.
__device__ __forceinline__ void cos_sin(uint64_t turn, float factor, float& c, float& s) {
  // the nearest quarter, and the rest: a signed fraction of a turn within an eighth
  const uint64_t shifted = turn + (uint64_t{1} << 61);
  const uint32_t quarter = static_cast<uint32_t>(shifted >> 62);
  const int64_t rest = static_cast<int64_t>(turn - (static_cast<uint64_t>(quarter) << 62));
  // 2 pi 2^-32 and 2^-64
  const float x = fmaf(static_cast<float>(static_cast<int32_t>(rest >> 32)), 1.46291807927e-9f,
                       static_cast<float>(static_cast<uint32_t>(rest)) * 3.40612158009e-19f);
  const float x2 = x * x;
  const float sn = fmaf(x * x2, fmaf(x2, fmaf(x2, fmaf(x2, 1.f / 362880, -1.f / 5040), 1.f / 120), -1.f / 6), x);
  const float cs = fmaf(x2, fmaf(x2, fmaf(x2, fmaf(x2, fmaf(x2, -1.f / 3628800, 1.f / 40320), -1.f / 720), 1.f / 24), -0.5f), 1.f);
  const float a = (quarter & 1u) ? sn : cs, b = (quarter & 1u) ? cs : sn;
  c = (quarter == 1u || quarter == 2u ? -factor : factor) * a;
  s = (quarter >= 2u ? -factor : factor) * b;
}

// kVec frequencies a thread, half / kVec threads a row.
template <int kVec>
__global__ void __launch_bounds__(kThreads, 4) rotary_table_kernel(const RotaryFrequencies f, float* __restrict__ out,
                                                                int64_t rows, int64_t start, int32_t half,
                                                                float factor) {
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
      cos_sin(turn[i], factor, c[i], s[i]);
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
                                int32_t rotary_dim, float factor, cudaStream_t stream) {
  if (rows == 0) return cudaSuccess;
  const int half = rotary_dim / 2;
  const bool vec = half % 4 == 0;
  const int64_t items = rows * (half / (vec ? 4 : 1));
  const int64_t blocks = (items + kThreads - 1) / kThreads;
  const int64_t cap = 4 * static_cast<int64_t>(current_sm_count());  // one wave
  const dim3 grid(static_cast<unsigned>(blocks < cap ? blocks : cap));
  return launch_programmatic(vec ? rotary_table_kernel<4> : rotary_table_kernel<1>, grid, dim3(kThreads), 0, stream,
                             f, out, rows, start, half, factor);
}

}  // namespace pkv
