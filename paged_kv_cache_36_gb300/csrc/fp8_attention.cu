// Attention over the 8-bit paged cache of the rows of requests with several query tokens, one
// warp per (token, query head): each lane takes
// a key for the scores and D / 32 dimensions of the values, with a running maximum and sum.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "fp8.cuh"
#include "kernels.h"
#include "pkv_device.cuh"

namespace pkv {

namespace {

struct Params {
  const __nv_bfloat16* q;
  int64_t q_stride;
  const uint8_t* key_cache;
  const uint8_t* value_cache;
  const int32_t* block_table;
  int32_t bt_stride, bt_width;
  const int32_t *qsl, *seq_lens, *num_computed;
  __nv_bfloat16* out;
  int64_t out_stride, num_tokens;
  int32_t num_reqs, num_blocks, hkv, group;
  float scale_log2;
  uint32_t* err;
};

template <int D>
__global__ void __launch_bounds__(256) attention_fp8_kernel(const Params p) {
  grid_dependency_wait();
  if (threadIdx.x == 0) grid_launch_dependents();
  __shared__ float qs[8][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int heads = p.hkv * p.group;
  const int64_t items = p.num_tokens * heads;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 8 + warp; i < items; i += static_cast<int64_t>(gridDim.x) * 8) {
    const int64_t t = i / heads;
    const int head = static_cast<int>(i - t * heads), h = head / p.group;
    int r = 0;
    while (r < p.num_reqs && !(__ldg(p.qsl + r) <= t && t < __ldg(p.qsl + r + 1))) ++r;
    if (r == p.num_reqs) continue;
    const int q0 = __ldg(p.qsl + r);
    const int qlen = static_cast<int>(static_cast<uint32_t>(__ldg(p.qsl + r + 1)) - static_cast<uint32_t>(q0));
    const int seq = __ldg(p.seq_lens + r), nc = __ldg(p.num_computed + r);
    if (qlen == 1) continue;
    if (q0 < 0 || qlen <= 0 || nc < 0 || nc > 0x7fffff00 - qlen || seq != nc + qlen || (seq - 1) / kF8Block >= p.bt_width ||
        q0 + qlen > p.num_tokens) {
      if (lane == 0) atomicOr(p.err, PKV_ERR_METADATA);
      continue;
    }
    __syncwarp();
    for (int d = lane; d < D; d += 32)
      qs[warp][d] = __bfloat162float(p.q[t * p.q_stride + static_cast<int64_t>(head) * D + d]);
    __syncwarp();
    const int keys = nc + static_cast<int>(t - q0) + 1;
    float m = -INFINITY, l = 0.f, o[D / 32] = {};
    for (int j0 = 0; j0 < keys; j0 += 32) {
      const int j = j0 + lane;
      float s = -INFINITY;
      int64_t chunk = -1;
      if (j < keys) {
        const int id = __ldg(p.block_table + static_cast<int64_t>(r) * p.bt_stride + j / kF8Block);
        if (static_cast<uint32_t>(id) < static_cast<uint32_t>(p.num_blocks))
          chunk = (static_cast<int64_t>(id) * p.hkv + h) * f8_chunk_bytes(D);
        else
          atomicOr(p.err, PKV_ERR_BLOCK_ID);
        float sum = 0.f;
        if (chunk >= 0) {
          const float scale = f8_pow2(f8_scale(p.key_cache[chunk + f8_code_bytes(D)]) - 127);
          for (int d = 0; d < D; d += 4) {
            float k[4];
            e4m3x4_to_f32(*reinterpret_cast<const uint32_t*>(p.key_cache + chunk + f8_key_at<D>(j % kF8Block, d)), k);
            for (int c = 0; c < 4; ++c) sum = fmaf(qs[warp][d + c], k[c] * scale, sum);
          }
        }
        s = sum * p.scale_log2;
      }
      float mx = s;
      for (int x = 1; x < 32; x <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
      const float mn = fmaxf(m, mx);
      const float alpha = exp2_approx(m - mn);
      m = mn;
      const float w = j < keys ? exp2_approx(s - m) : 0.f;
      l = l * alpha + w;
      for (int d = 0; d < D / 32; ++d) o[d] *= alpha;
      for (int k = 0; k < 32 && j0 + k < keys; ++k) {
        const float wk = __shfl_sync(0xffffffffu, w, k);
        const int64_t c = __shfl_sync(0xffffffffu, chunk, k);
        if (c < 0) continue;
        const float scale = f8_pow2(f8_scale(p.value_cache[c + f8_code_bytes(D)]) - 127);
        for (int d = 0; d < D / 32; ++d) {
          float v[4];
          e4m3x4_to_f32(p.value_cache[c + f8_value_at<D>((j0 + k) % kF8Block, d * 32 + lane)], v);
          o[d] = fmaf(wk, v[0] * scale, o[d]);
        }
      }
    }
    for (int x = 1; x < 32; x <<= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
    for (int d = 0; d < D / 32; ++d)
      p.out[t * p.out_stride + static_cast<int64_t>(head) * D + d * 32 + lane] = __float2bfloat16(o[d] / l);
  }
}

}  // namespace

cudaError_t launch_attention_fp8(const AttnArgs& a, int sms, cudaStream_t stream) {
  Params p;
  p.q = static_cast<const __nv_bfloat16*>(a.q);
  p.q_stride = a.q_stride;
  p.key_cache = static_cast<const uint8_t*>(a.key_cache);
  p.value_cache = static_cast<const uint8_t*>(a.value_cache);
  p.block_table = a.block_table;
  p.bt_stride = a.bt_stride;
  p.bt_width = a.bt_width;
  p.qsl = a.qsl;
  p.seq_lens = a.seq_lens;
  p.num_computed = a.num_computed;
  p.out = static_cast<__nv_bfloat16*>(a.out);
  p.out_stride = a.out_stride;
  p.num_tokens = a.num_tokens;
  p.num_reqs = a.num_reqs;
  p.num_blocks = static_cast<int32_t>(a.num_blocks);
  p.hkv = a.num_kv_heads;
  p.group = a.num_heads / a.num_kv_heads;
  p.scale_log2 = static_cast<float>(static_cast<double>(a.scale) * 1.4426950408889634);
  p.err = a.err;
  const int64_t want = (a.num_tokens * a.num_heads + 7) / 8, cap = 8 * static_cast<int64_t>(sms);
  const dim3 grid(static_cast<unsigned>(want < cap ? want : cap));
  return a.head_dim == 128 ? launch_programmatic(attention_fp8_kernel<128>, grid, dim3(256), 0, stream, p)
                           : launch_programmatic(attention_fp8_kernel<64>, grid, dim3(256), 0, stream, p);
}

}  // namespace pkv
