// Pieces shared by the tensor-core prefill kernels: the order in which CTAs take
// query tiles, a register transpose for the epilogue, bounded waits, and short loops over
// scores and sums in tensor memory.
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

// Like mbar_wait_or_abort, but the hardware may hold the warp for a while before
// it answers "not yet", so that waiting warps leave the issue slots to the
// others (they wake when the phase completes).
__device__ __forceinline__ bool held_wait(uint64_t* bar, uint32_t parity, uint32_t* err,
                                          volatile int* abort) {
  const uint32_t addr = smem_u32(bar);
  auto ready = [&]() {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(addr), "r"(parity), "r"(20000u)  // nanoseconds, at most
        : "memory");
    return done != 0;
  };
  if (ready()) return true;
  const long long t0 = clock64();
  while (!ready()) {
    if (*abort) return false;
    if (clock64() - t0 > kWaitLimitCycles) {
      atomicOr(err, PKV_ERR_TIMEOUT);
      *abort = 1;
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ bool held_warp_wait(uint64_t* bar, uint32_t parity, uint32_t* err,
                                               volatile int* abort) {
  return __all_sync(0xffffffffu, held_wait(bar, parity, err, abort));
}

template <int kRegs, bool kMore>
__device__ __forceinline__ void set_registers() {
  if constexpr (kMore)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
  else
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// -inf into this row's columns from `visible` on, of 64; `first` is the smallest such
// column of the warp's rows.
__device__ __forceinline__ void mask_scores(uint32_t cols, int first, int visible) {
#pragma unroll 1
  for (int c = max(first, 0) & ~7; c < 64; c += 8) {
    uint32_t r[8];
    tmem_ld8(cols + c, r);
    tmem_wait_ld();
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (c + e >= visible) r[e] = 0xff800000u;
    tmem_st8(cols + c, r);
  }
  tmem_wait_st();
}

// Rescales N columns of O from `cols` on.
template <int N>
__device__ __forceinline__ void rescale(uint32_t cols, float alpha) {
#pragma unroll 1
  for (int c = 0; c < N; c += 32) {
    uint32_t r32[32];
    tmem_ld32(cols + c, r32);
    tmem_wait_ld();
#pragma unroll
    for (int e = 0; e < 32; ++e) r32[e] = __float_as_uint(__uint_as_float(r32[e]) * alpha);
    tmem_st32(cols + c, r32);
  }
  tmem_wait_st();
}

}  // namespace pkv
