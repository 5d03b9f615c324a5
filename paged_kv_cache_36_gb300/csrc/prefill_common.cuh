// Pieces shared by the tensor-core prefill kernels: the order in which CTAs take
// query tiles, a register transpose for the epilogue, warp-wide bounded waits.
#pragma once

#include <cstdint>

#include "pkv_device.cuh"
#include "tcgen05.cuh"

namespace pkv {

// The it-th tile of CTA cid, or -1 when there is none.  Within a request
// later query tiles see more keys, so tiles are taken from the highest index
// down, ncta at a time, in alternating direction: each CTA starts with one of
// the heaviest tiles and heavy and light ones pair up.
__device__ __forceinline__ int cta_tile(int it, int cid, int ncta, int total) {
  const int lin = it * ncta + ((it & 1) ? ncta - 1 - cid : cid);
  return lin < total ? total - 1 - lin : -1;
}

// Transposes NV x NV blocks of 16-byte values across groups of NV lanes
// (NV a power of two <= 32): afterwards lane NV g + j holds in v[k] what lane
// NV g + k held in v[j].  Butterfly exchanges, log2(NV) rounds of shuffles.
template <int NV>
__device__ __forceinline__ void transpose_lane_groups(uint4 (&v)[NV], int lane) {
#pragma unroll
  for (int s = 1; s < NV; s <<= 1) {
    const bool hi = (lane & s) != 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (i & s) continue;
      // pair (i, i + s): the low lane sends v[i + s], the high lane v[i]
      const uint4 x = hi ? v[i] : v[i + s];
      uint4 y;
      y.x = __shfl_xor_sync(0xffffffffu, x.x, s);
      y.y = __shfl_xor_sync(0xffffffffu, x.y, s);
      y.z = __shfl_xor_sync(0xffffffffu, x.z, s);
      y.w = __shfl_xor_sync(0xffffffffu, x.w, s);
      if (hi) v[i] = y; else v[i + s] = y;
    }
  }
}

// max(a, b, c) in one instruction (the three-input form of max.f32).
__device__ __forceinline__ float fmax3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// All lanes of the calling warp wait; the result is made warp-uniform.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, uint32_t* err,
                                          volatile int* abort) {
  return __all_sync(0xffffffffu, mbar_wait_or_abort(bar, parity, err, abort));
}

}  // namespace pkv
