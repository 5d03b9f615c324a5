// Attention over the 4-bit paged cache on CUDA cores, one warp per (query row,
// query head): query row t of request r at position p attends keys j <= p of
// its KV head with an online softmax,
//   out = sum_j softmax_j(scale <q, K_j>) V_j.
// Lane i owns dims [i D/32, (i + 1) D/32).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "kernels.h"
#include "mxfp4.cuh"
#include "pkv_device.cuh"

namespace pkv {

namespace {

// The E consecutive values from dim d0 (E divides 8; d0 a multiple of E).
template <int D, bool kIsKey>
__device__ __forceinline__ void read_dims(const uint8_t* chunk, int t, int d0,
                                          float (&x)[D / 32]) {
  constexpr int E = D / 32;
  const int b = d0 >> 5;
  const uint8_t* row = chunk + t * (D / 2);
  const int byte = kIsKey ? ((d0 & 31) >> 3) * (D / 8) + 4 * b + ((d0 & 7) >> 1)
                          : ((d0 & 31) >> 2) * (D / 16) + 2 * b + ((d0 & 3) >> 1);
  const uint32_t e =
      kIsKey ? chunk[mx_scale_off(D) + t * (D / 32) + b] : chunk[mx_vscale_off<D>(t, b)];
  const float s = mx_scale(e);
#pragma unroll
  for (int i = 0; i < E / 2; ++i) {
    const uint32_t p = e2m1x2_to_f16x2(row[byte + i]);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&p));
    x[2 * i] = f.x * s;
    x[2 * i + 1] = f.y * s;
  }
}

template <int D>
__global__ void __launch_bounds__(256) attn_rows_mxfp4_kernel(const AttnArgs a, float scale_log2) {
  grid_dependency_wait();
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t wid = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const int64_t t = wid / a.num_heads;
  const int h = static_cast<int>(wid - t * a.num_heads);
  if (t >= a.num_tokens) return;
  int lo = 0, hi = a.num_reqs;  // the largest r with qsl[r] <= t
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(a.qsl + mid) <= t) lo = mid; else hi = mid;
  }
  const int r = lo;
  const int q0 = __ldg(a.qsl + r);
  const int qlen = __ldg(a.qsl + r + 1) - q0;
  const int nc = __ldg(a.num_computed + r);
  const int seq = __ldg(a.seq_lens + r);
  if (t - q0 >= qlen || qlen <= 1) return;  // rows behind the last request, decode rows
  if (nc < 0 || seq != nc + qlen || (seq - 1) / kMxBlock >= a.bt_width) {
    if (lane == 0) atomicOr(a.err, PKV_ERR_METADATA);
    return;
  }
  const int pos = nc + static_cast<int>(t - q0);
  const int g = h / (a.num_heads / a.num_kv_heads);
  const __nv_bfloat16* qrow =
      static_cast<const __nv_bfloat16*>(a.q) + t * a.q_stride + static_cast<int64_t>(h) * D;
  float qv[E];
#pragma unroll
  for (int i = 0; i < E; ++i) qv[i] = __bfloat162float(qrow[lane * E + i]);
  const uint8_t* kc = static_cast<const uint8_t*>(a.key_cache);
  const uint8_t* vc = static_cast<const uint8_t*>(a.value_cache);
  const int32_t* row = a.block_table + static_cast<int64_t>(r) * a.bt_stride;
  const int64_t block_bytes = static_cast<int64_t>(a.num_kv_heads) * mx_chunk_bytes(D);
  float m = -INFINITY, l = 0.f, acc[E] = {};
  for (int j = 0; j <= pos; ++j) {
    const int32_t blk = __ldg(row + j / kMxBlock);
    float kv[E] = {}, vv[E] = {};
    if (blk < 0 || blk >= a.num_blocks) {
      if (lane == 0) atomicOr(a.err, PKV_ERR_BLOCK_ID);  // such a block reads as zeros
    } else {
      const int64_t off = blk * block_bytes + g * mx_chunk_bytes(D);
      read_dims<D, true>(kc + off, j % kMxBlock, lane * E, kv);
      read_dims<D, false>(vc + off, j % kMxBlock, lane * E, vv);
    }
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) dot += qv[i] * kv[i];
#pragma unroll
    for (int sh = 16; sh; sh >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, sh);
    const float s = dot * scale_log2;
    const float mn = fmaxf(m, s);
    const float alpha = exp2f(m - mn);
    const float pj = exp2f(s - mn);
    l = l * alpha + pj;
#pragma unroll
    for (int i = 0; i < E; ++i) acc[i] = acc[i] * alpha + pj * vv[i];
    m = mn;
  }
  __nv_bfloat16* orow =
      static_cast<__nv_bfloat16*>(a.out) + t * a.out_stride + static_cast<int64_t>(h) * D;
  const float inv = 1.f / l;
#pragma unroll
  for (int i = 0; i < E; ++i) orow[lane * E + i] = __float2bfloat16_rn(acc[i] * inv);
}

}  // namespace

cudaError_t launch_attn_rows_mxfp4(const AttnArgs& a, cudaStream_t stream) {
  const int64_t warps = a.num_tokens * a.num_heads;
  if (warps == 0) return cudaSuccess;
  const int64_t blocks = (warps + 7) / 8;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  const float scale_log2 = static_cast<float>(static_cast<double>(a.scale) * 1.4426950408889634);
  const dim3 grid(static_cast<unsigned>(blocks));
  if (a.head_dim == 128)
    return launch_programmatic(attn_rows_mxfp4_kernel<128>, grid, dim3(256), 0, stream, a, scale_log2);
  if (a.head_dim == 64)
    return launch_programmatic(attn_rows_mxfp4_kernel<64>, grid, dim3(256), 0, stream, a, scale_log2);
  return cudaErrorNotSupported;
}

}  // namespace pkv
