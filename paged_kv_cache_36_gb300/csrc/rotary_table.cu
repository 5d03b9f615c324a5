// The table of rotary angles that the RoPE entry points read: row p holds the cosines,
// then the sines, of (start + p) f_i for the rotary_dim / 2 frequencies f_i, times a factor.
//
// The frequencies come from the host, in 64 bits.  An angle is a product of some 2^20 by a
// frequency, of which only the remainder modulo 2 pi counts: in float32 the remainder of a
// far position has no correct digits, so the product, the number of whole turns and the
// remainder are 64-bit, and only what is left, within a half turn, goes to float32's sine
// and cosine, with its rounding error put back to first order:
//   sin(r + d) = sin r + d cos r,  cos(r + d) = cos r - d sin r,  |d| <= 2^-24 |r|.
//
// What bounds it: writing the table.  131072 rows of 128 are 67 MB.
#include <cuda_runtime.h>

#include <cstdint>

#include "kernels.h"
#include "pkv_device.cuh"

namespace pkv {

namespace {

constexpr int kThreads = 256;

__global__ void __launch_bounds__(kThreads) rotary_table_kernel(const RotaryFrequencies f, float* __restrict__ out,
                                                                int64_t rows, int64_t start, int32_t half,
                                                                float factor) {
  // (reads nothing that another kernel writes, but `out` may still be read by one)
  grid_dependency_wait();
  if (threadIdx.x == 0) grid_launch_dependents();
  const int64_t total = rows * half;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * kThreads) {
    const int64_t p = i / half;
    const int k = static_cast<int>(i - p * half);
    const double turns = static_cast<double>(start + p) * f.turns[k];
    const double r = (turns - rint(turns)) * 6.283185307179586476925;
    const float hi = static_cast<float>(r);
    const float lo = static_cast<float>(r - static_cast<double>(hi));
    float s, c;
    sincosf(hi, &s, &c);
    float* row = out + p * (2 * half);
    row[k] = factor * fmaf(-lo, s, c);
    row[half + k] = factor * fmaf(lo, c, s);
  }
}

}  // namespace

cudaError_t launch_rotary_table(const RotaryFrequencies& f, float* out, int64_t rows, int64_t start,
                                int32_t rotary_dim, float factor, cudaStream_t stream) {
  if (rows == 0) return cudaSuccess;
  const int64_t blocks = (rows * (rotary_dim / 2) + kThreads - 1) / kThreads;
  const int64_t cap = 32 * static_cast<int64_t>(current_sm_count());
  return launch_programmatic(rotary_table_kernel, dim3(static_cast<unsigned>(blocks < cap ? blocks : cap)),
                             dim3(kThreads), 0, stream, f, out, rows, start, rotary_dim / 2, factor);
}

}  // namespace pkv
