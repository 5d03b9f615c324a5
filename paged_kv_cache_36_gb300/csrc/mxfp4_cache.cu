// reshape_and_cache into the 4-bit paged cache, and its inverse.
//
// Quantisation of one group of 32 dimensions ("microscaling", OCP MX formats
// v1.0): with amax = max |x|,
//   e = clamp(floor(log2 amax) - 2 + 127, 1, 254),  code = RNE_e2m1(x 2^(127 - e))
// saturating at 6 (2 = the exponent of the largest e2m1 binade, so amax lands
// in [4, 8)).  The scaling is by a power of two and exact in float32; the one
// rounding is the code's.  An all-zero group has e = 127; a group with a NaN or
// an infinity has e = 255 and zero codes, which reads as NaN.
//
// One warp per token: lane i of a pass takes 8 consecutive dimensions of the K
// row or the V row (one 32-bit word of codes), so 4 lanes share a scale and
// find amax with two shuffles.
//
// Both directions are bound by memory, four fifths of it the rows' side.  8 KV
// heads of 128 in bfloat16, nothing in L2: 8192 tokens (33.6 MB read, 8.9 MB
// written, and back) take 21.0 us for the write and the gather together, 4.0
// TB/s; a gather of 16384 tokens 19.1 us, 4.4 TB/s, and 14.9 us, 5.7 TB/s, where
// L2 still holds what it reads and writes.
#include <cuda_runtime.h>

#include <cstdint>

#include "kernels.h"
#include "mxfp4.cuh"
#include "pkv_device.cuh"

namespace pkv {

namespace {

// Passes whose loads a lane has in flight at once.  With one, a warp waits for
// memory n / 32 times a token.  8 KV heads of 128, caches and rows not in L2: a
// write of 8192 tokens and its gather take 22.5 us with one, 21.0 with two, 22.2
// with four (whose registers cost warps).
constexpr int kAhead = 2;

template <typename T>
struct Eight;  // eight consecutive elements of a row

template <>
struct Eight<__nv_bfloat16> {
  uint4 v;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    v = __ldg(reinterpret_cast<const uint4*>(p));
  }
  __device__ __forceinline__ void unpack(float (&x)[8]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  __device__ __forceinline__ static void store(__nv_bfloat16* p, const float (&x)[8]) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]),
                                              pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
  }
};

template <>
struct Eight<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __ldg(reinterpret_cast<const float4*>(p));
    b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void unpack(float (&x)[8]) const {
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
  __device__ __forceinline__ static void store(float* p, const float (&x)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
  }
};

// Codes and scale byte of this lane's 8 dimensions; the group's 32 are held by
// the 4 lanes of a quad (all lanes of the warp call this).
__device__ __forceinline__ uint32_t quantise8(float (&x)[8], uint32_t& e) {
  // |x| as bits: order of the bit patterns is the order of the magnitudes,
  // with infinity and NaN above everything finite
  uint32_t m = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(x[i]) & 0x7fffffffu);
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
  if (m >= 0x7f800000u) {
    e = 255u;
    return 0u;
  }
  const uint32_t field = m >> 23;  // floor(log2 amax) + 127, 0 below 2^-126
  e = m == 0u ? 127u : field > 3u ? field - 2u : 1u;
  const float inv = __uint_as_float((254u - e) << 23);  // 2^(127 - e), e <= 252
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] *= inv;
  return f32x8_to_e2m1(x);
}

template <typename T, int D>
__global__ void __launch_bounds__(256) reshape_and_cache_mxfp4_kernel(
    const T* __restrict__ key, const T* __restrict__ value, int64_t key_stride,
    int64_t value_stride, uint8_t* __restrict__ key_cache, uint8_t* __restrict__ value_cache,
    const int64_t* __restrict__ slot_mapping, int64_t num_tokens, int64_t num_slots, int32_t hkv,
    uint32_t* __restrict__ err) {
  // a programmatic dependent of the kernel before it, which may still read
  // the cache or write the new rows
  grid_dependency_wait();
  if (threadIdx.x == 0) grid_launch_dependents();
  constexpr int kWords = D / 8;  // words of codes in one head's row
  const int lane = threadIdx.x & 31;
  const int64_t wpb = blockDim.x >> 5;
  const int n = hkv * kWords;
  const int64_t block_bytes = static_cast<int64_t>(hkv) * mx_chunk_bytes(D);
  for (int64_t t = blockIdx.x * wpb + (threadIdx.x >> 5); t < num_tokens; t += gridDim.x * wpb) {
    const int64_t slot = __ldg(slot_mapping + t);
    if (slot >= num_slots && lane == 0 && err) atomicOr(err, PKV_ERR_SLOT);
    if (slot < 0 || slot >= num_slots) continue;  // the whole warp has one token
    const int off = static_cast<int>(slot & (kMxBlock - 1));
    uint8_t* kblk = key_cache + slot / kMxBlock * block_bytes;
    uint8_t* vblk = value_cache + slot / kMxBlock * block_bytes;
    for (int base = 0; base < n; base += 32 * kAhead) {
      // quads are wholly inside or outside the row
      Eight<T> kr[kAhead], vr[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int i = base + 32 * u + lane;
        if (i < n) {
          kr[u].load(key + t * key_stride + 8 * i);
          vr[u].load(value + t * value_stride + 8 * i);
        }
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        if (base + 32 * u >= n) break;
        const int i = base + 32 * u + lane;
        const int h = i / kWords, wi = i % kWords, b = wi >> 2, c = wi & 3;
        float kx[8] = {}, vx[8] = {};
        if (i < n) {
          kr[u].unpack(kx);
          vr[u].unpack(vx);
        }
        uint32_t ke, ve;
        const uint32_t kw = quantise8(kx, ke);
        const uint32_t vw = quantise8(vx, ve);
        if (i < n) {
          uint8_t* kc = kblk + h * mx_chunk_bytes(D);
          uint8_t* vc = vblk + h * mx_chunk_bytes(D);
          *reinterpret_cast<uint32_t*>(kc + off * (D / 2) + c * (D / 8) + 4 * b) = kw;
          uint8_t* vrow = vc + off * (D / 2) + 2 * b;
          *reinterpret_cast<uint16_t*>(vrow + (2 * c) * (D / 16)) = static_cast<uint16_t>(vw);
          *reinterpret_cast<uint16_t*>(vrow + (2 * c + 1) * (D / 16)) = static_cast<uint16_t>(vw >> 16);
          if (c == 0) {
            kc[mx_scale_off(D) + off * (D / 32) + b] = static_cast<uint8_t>(ke);
            vc[mx_vscale_off<D>(off, b)] = static_cast<uint8_t>(ve);
          }
        }
      }
    }
  }
}

__device__ __forceinline__ void dequantise8(uint32_t w, uint32_t e, float (&x)[8]) {
  uint32_t p[4];
  e2m1x8_to_f16(w, p);
  const float s = mx_scale(e);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&p[i]));
    x[2 * i] = f.x * s;
    x[2 * i + 1] = f.y * s;
  }
}

// One warp per token, 8 dimensions per lane; every value is exact in either
// output type.
template <typename T, int D>
__global__ void __launch_bounds__(256) gather_cache_mxfp4_kernel(
    const uint8_t* __restrict__ key_cache, const uint8_t* __restrict__ value_cache,
    const int64_t* __restrict__ slot_mapping, T* __restrict__ key_out, T* __restrict__ value_out,
    int64_t key_stride, int64_t value_stride, int64_t num_tokens, int64_t num_slots, int32_t hkv,
    uint32_t* __restrict__ err) {
  grid_dependency_wait();  // the kernel before it may write the cache
  if (threadIdx.x == 0) grid_launch_dependents();
  constexpr int kWords = D / 8;
  const int lane = threadIdx.x & 31;
  const int64_t wpb = blockDim.x >> 5;
  const int n = hkv * kWords;
  const int64_t block_bytes = static_cast<int64_t>(hkv) * mx_chunk_bytes(D);
  for (int64_t t = blockIdx.x * wpb + (threadIdx.x >> 5); t < num_tokens; t += gridDim.x * wpb) {
    const int64_t slot = __ldg(slot_mapping + t);
    if (slot < 0) continue;
    const bool in = slot < num_slots;
    if (!in && lane == 0 && err) atomicOr(err, PKV_ERR_SLOT);
    const int off = static_cast<int>(slot & (kMxBlock - 1));
    const int64_t blk = in ? slot / kMxBlock : 0;
    const uint8_t* kblk = key_cache + blk * block_bytes;
    const uint8_t* vblk = value_cache + blk * block_bytes;
    for (int base = 0; base < n; base += 32 * kAhead) {
      uint32_t kw[kAhead], vw[kAhead], ke[kAhead], ve[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int i = base + 32 * u + lane;
        const int h = i / kWords, wi = i % kWords, b = wi >> 2, c = wi & 3;
        kw[u] = vw[u] = ke[u] = ve[u] = 0u;
        if (in && i < n) {
          const uint8_t* kc = kblk + h * mx_chunk_bytes(D);
          const uint8_t* vc = vblk + h * mx_chunk_bytes(D);
          kw[u] = *reinterpret_cast<const uint32_t*>(kc + off * (D / 2) + c * (D / 8) + 4 * b);
          const uint8_t* vrow = vc + off * (D / 2) + 2 * b;
          vw[u] = *reinterpret_cast<const uint16_t*>(vrow + (2 * c) * (D / 16)) |
                  static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(vrow + (2 * c + 1) * (D / 16)))
                      << 16;
          ke[u] = kc[mx_scale_off(D) + off * (D / 32) + b];
          ve[u] = vc[mx_vscale_off<D>(off, b)];
        }
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int i = base + 32 * u + lane;
        if (i < n) {
          float kx[8], vx[8];
          dequantise8(kw[u], ke[u], kx);  // zero codes where the slot is refused
          dequantise8(vw[u], ve[u], vx);
          Eight<T>::store(key_out + t * key_stride + 8 * i, kx);
          Eight<T>::store(value_out + t * value_stride + 8 * i, vx);
        }
      }
    }
  }
}

unsigned token_grid(int64_t num_tokens) {
  const int64_t blocks = (num_tokens + 7) / 8;  // 8 warps, one token each
  // one token a warp up to eight waves: with one wave of warps that walk several
  // tokens, the gather of 16384 takes 20.2 us instead of 19.1
  const int64_t cap = static_cast<int64_t>(current_sm_count()) * 64;
  return static_cast<unsigned>(blocks < cap ? blocks : cap);
}

template <typename T, int D>
cudaError_t write_t(const MxCacheArgs& a, cudaStream_t stream) {
  return launch_programmatic(reshape_and_cache_mxfp4_kernel<T, D>, dim3(token_grid(a.num_tokens)),
                             dim3(256), 0, stream, static_cast<const T*>(a.key),
                             static_cast<const T*>(a.value), a.key_stride, a.value_stride,
                             a.key_cache, a.value_cache, a.slot_mapping, a.num_tokens, a.num_slots,
                             a.num_kv_heads, a.err);
}

template <typename T, int D>
cudaError_t gather_t(const MxCacheArgs& a, cudaStream_t stream) {
  return launch_programmatic(
      gather_cache_mxfp4_kernel<T, D>, dim3(token_grid(a.num_tokens)), dim3(256), 0, stream,
      static_cast<const uint8_t*>(a.key_cache), static_cast<const uint8_t*>(a.value_cache),
      a.slot_mapping, static_cast<T*>(const_cast<void*>(a.key)),
      static_cast<T*>(const_cast<void*>(a.value)), a.key_stride, a.value_stride, a.num_tokens,
      a.num_slots, a.num_kv_heads, a.err);
}

}  // namespace

cudaError_t launch_reshape_and_cache_mxfp4(const MxCacheArgs& a, cudaStream_t stream) {
  if (a.num_tokens == 0) return cudaSuccess;
  if (a.head_dim == 128)
    return a.bf16 ? write_t<__nv_bfloat16, 128>(a, stream) : write_t<float, 128>(a, stream);
  if (a.head_dim == 64)
    return a.bf16 ? write_t<__nv_bfloat16, 64>(a, stream) : write_t<float, 64>(a, stream);
  return cudaErrorNotSupported;
}

cudaError_t launch_gather_cache_mxfp4(const MxCacheArgs& a, cudaStream_t stream) {
  if (a.num_tokens == 0) return cudaSuccess;
  if (a.head_dim == 128)
    return a.bf16 ? gather_t<__nv_bfloat16, 128>(a, stream) : gather_t<float, 128>(a, stream);
  if (a.head_dim == 64)
    return a.bf16 ? gather_t<__nv_bfloat16, 64>(a, stream) : gather_t<float, 64>(a, stream);
  return cudaErrorNotSupported;
}

}  // namespace pkv
