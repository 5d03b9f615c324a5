// reshape_and_cache into the 8-bit paged cache, alone or with RoPE, and its inverse.
//
// The rows that a call writes to one block and KV head share a scale (fp8.cuh), and with
// those that the block holds already:
//   e = max(e_old, smallest e' with max |x| <= 448 2^(e' - 127)),  code = RNE_e4m3(x 2^(127 - e)).
// A call that writes row 0 of a block begins it anew: there is no e_old, and rows that it
// does not write become zero.  Where e grows, the rows that stay are rounded again,
// RNE(code 2^(e_old - e)); being powers of two, scales move only what falls below e4m3's
// normal numbers.  A NaN or an infinity has the code for NaN, which reads as NaN, and does
// not count for the scale.
//
// Who writes what.  A block is written by one warp per (KV head, K or V), whichever tokens
// of the call go to it: a CTA takes a window of tokens, finds those whose block the token
// before them does not share, and searches the call's slots for the blocks' other tokens.
// The block is its own if none of them comes earlier.  So there are no atomics and no
// second pass, the result depends on no order, and of a slot given twice the last token
// counts.  A batch in the order of its requests has one search per 16 tokens, T^2 / 2 bytes of
// slots; in the worst order there is one per two, 4 T^2 (8 KV heads of 128, bfloat16, in order and
// in none: 8192 tokens 17 and 60 us, 32768 80 and 283, 131072 503 and 2922, 2^20 24 and 183 ms).
//
// What bounds it.  8192 tokens that begin inside blocks, 8 KV heads of 128, bfloat16, nothing in
// L2: 17.4 us for 50 MB.  By its clocks (whole blocks, CTAs of 256 threads) a CTA has its leaders
// 2 us after its start, the other tokens 1.4 later, and a warp takes 2 to 2.7 us for each of its
// two items: latency of rows that follow from slots, of their maximum and of the stores.  With
// RoPE of 32 query heads 35.4 us for 184 MB, 5.2 TB/s.  64 tokens 5.5 us with RoPE or without.
#include <cuda_runtime.h>

#include <cstdint>

#include "fp8.cuh"
#include "kernels.h"
#include "pkv_device.cuh"

namespace pkv {

namespace {

constexpr int kThreads = 256;  // of a gather's CTA
constexpr int kWindow = 16;  // tokens of a gather's window, at most
// Of a write's.  8192 tokens in order, 8 heads of 128 (and CTAs of 256 threads): 19.9 us with 8,
// 20.7 with 4, 23.0 with 16 (half of the windows of 8 have no block to begin, and end at once; those of 16 leave
// some CTAs with twice the others' work).
constexpr int kWriteWindow = 8;

enum Rope { kNone, kHalf, kInterleaved };
// Threads of a write's CTA.  A window in which one block ends and another begins has twice the
// work.  8192 tokens, 8 heads of 128, that begin inside blocks: 17.4 us, with 256 threads
// 18.4; of whole blocks 16.5 and 15.6; with RoPE 39.0 and 35.4.
template <Rope kRope>
constexpr int write_threads() { return kRope == kNone ? 512 : 256; }

// N consecutive elements of a row.
template <typename T, int N>
struct Piece {
  static constexpr int kVecs = N * sizeof(T) / 16;
  static constexpr int kPer = 16 / sizeof(T);  // elements of a vector
  uint4 v[kVecs];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) v[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) v[i] = make_uint4(0u, 0u, 0u, 0u);
  }
  template <typename F>
  __device__ __forceinline__ void each(F&& f) {  // of the words
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      f(v[i].x);
      f(v[i].y);
      f(v[i].z);
      f(v[i].w);
    }
  }
  __device__ __forceinline__ float at(int i) const {  // i known when compiled
    const uint4& u = v[i / kPer];
    const int k = i % kPer;
    if constexpr (sizeof(T) == 4) {
      return __uint_as_float(k == 0 ? u.x : k == 1 ? u.y : k == 2 ? u.z : u.w);
    } else {
      const uint32_t w = k < 2 ? u.x : k < 4 ? u.y : k < 6 ? u.z : u.w;
      return __uint_as_float((k & 1) ? w & 0xffff0000u : w << 16);
    }
  }
};

constexpr uint32_t kInf = 0x7f800000u;

// |x| as bits: their order is that of the magnitudes, infinity and NaN above everything.
__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7fffffffu; }
// With NaN for an infinity, its finite magnitude to `most`.
__device__ __forceinline__ float without_infinity(float x, uint32_t& most) {
  const uint32_t m = magnitude(x);
  if (m >= kInf) return __uint_as_float(0x7fffffffu);
  most = max(most, m);
  return x;
}

// What a row's vectors need on their way to codes: elements of T in the words of a vector.
template <typename T>
struct Words;
template <>
struct Words<float> {
  __device__ __forceinline__ static void most(uint32_t w, uint32_t& m) { m = max(m, w & 0x7fffffffu); }
  __device__ __forceinline__ static uint32_t bits(uint32_t m) { return m; }  // of a float32
  __device__ __forceinline__ static uint32_t finite(uint32_t w, uint32_t& m) {
    return __float_as_uint(without_infinity(__uint_as_float(w), m));
  }
  __device__ __forceinline__ static uint32_t times(uint32_t w, float f) { return __float_as_uint(__uint_as_float(w) * f); }
};
template <>
struct Words<__nv_bfloat16> {  // two elements a word
  // (a NaN does not count, and needs nothing done about it)
  __device__ __forceinline__ static void most(uint32_t w, uint32_t& m) {
    const __nv_bfloat162 x = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&m),
                                     __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w)));
    m = *reinterpret_cast<const uint32_t*>(&x);
  }
  __device__ __forceinline__ static uint32_t bits(uint32_t m) { return max(m << 16, m & 0xffff0000u); }
  __device__ __forceinline__ static uint32_t finite(uint32_t w, uint32_t& m) {
    uint32_t lo = 0u, hi = 0u;
    if ((w & 0x7f80u) == 0x7f80u) w |= 0x40u; else lo = w & 0x7fffu;
    if ((w & 0x7f800000u) == 0x7f800000u) w |= 0x400000u; else hi = w & 0x7fff0000u;
    m = __vmaxu2(m, lo | hi);
    return w;
  }
  // (by a power of two: exact, but for what is far below any code)
  __device__ __forceinline__ static uint32_t times(uint32_t w, float f) {
    const __nv_bfloat162 h = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&w), __float2bfloat162_rn(f));
    return *reinterpret_cast<const uint32_t*>(&h);
  }
};

struct WriteParams {
  const void* key;
  const void* value;
  int64_t key_stride;    // elements
  int64_t value_stride;
  uint8_t* key_cache;
  uint8_t* value_cache;
  const int64_t* slot_mapping;
  int64_t num_slots;
  int32_t num_tokens;
  int32_t hkv;
  int32_t window;        // tokens of a window
  int32_t splits;        // CTAs of a window
  int32_t cache_ctas;    // the CTAs after them rotate the queries
  uint32_t* err;
  // RoPE
  const int64_t* positions;
  const float* table;    // [max_position][rotary_dim]: cosines, sines
  int64_t max_position;
  int32_t rotary_dim;
  int32_t heads;
  const void* query;
  void* query_out;
  int64_t query_stride;
  int64_t query_out_stride;
};

// M floats of the table (M even).
template <int M>
__device__ __forceinline__ void load_table(const float* p, float (&x)[M]) {
  if constexpr (M % 4 == 0) {
#pragma unroll
    for (int i = 0; i < M; i += 4) *reinterpret_cast<float4*>(x + i) = __ldg(reinterpret_cast<const float4*>(p + i));
  } else {
#pragma unroll
    for (int i = 0; i < M; i += 2) *reinterpret_cast<float2*>(x + i) = __ldg(reinterpret_cast<const float2*>(p + i));
  }
}

// The vector of elements d .. of a row, rotated by the angles of its table row `cs`.
template <typename T, Rope kRope>
__device__ __forceinline__ void rotated(const T* row, int d, const float* cs, int rd,
                                        float (&y)[16 / sizeof(T)]) {
  constexpr int N = 16 / sizeof(T);
  Piece<T, N> a;
  a.load(row + d);
  if (d >= rd) {
#pragma unroll
    for (int i = 0; i < N; ++i) y[i] = a.at(i);
    return;
  }
  const int half = rd >> 1;
  if constexpr (kRope == kHalf) {
    const bool upper = d >= half;
    const int at = upper ? d - half : d;
    Piece<T, N> b;
    b.load(row + (upper ? at : d + half));
    float c[N], s[N];
    load_table<N>(cs + at, c);
    load_table<N>(cs + half + at, s);
#pragma unroll
    for (int i = 0; i < N; ++i)
      y[i] = upper ? a.at(i) * c[i] + b.at(i) * s[i] : a.at(i) * c[i] - b.at(i) * s[i];
  } else {
    float c[N / 2], s[N / 2];
    load_table<N / 2>(cs + d / 2, c);
    load_table<N / 2>(cs + half + d / 2, s);
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      y[i] = a.at(i) * c[i / 2] - a.at(i + 1) * s[i / 2];
      y[i + 1] = a.at(i + 1) * c[i / 2] + a.at(i) * s[i / 2];
    }
  }
}

__device__ __forceinline__ uint32_t warp_max(uint32_t x) { return __reduce_max_sync(0xffffffffu, x); }

// The scale of a chunk with scale `e_old` (0 if it begins anew) that gets rows of magnitude
// `amax`; *grown: by how much the rows that stay have to come down.
__device__ __forceinline__ int new_scale(int e_old, uint32_t amax, int* grown) {
  const int e_new = f8_scale_of(amax);
  *grown = e_old == 0 ? 0 : max(e_new - e_old, 0);
  return max(e_new, e_old);
}

// The largest finite magnitude of the warp's pieces; where some are not finite, infinities
// become NaN.
template <typename T, typename Pc, int n>
__device__ __forceinline__ uint32_t most_of(Pc (&raw)[n]) {
  uint32_t m = 0u;
#pragma unroll
  for (int j = 0; j < n; ++j) raw[j].each([&](uint32_t& w) { Words<T>::most(w, m); });
  m = warp_max(Words<T>::bits(m));
  if (m >= kInf) {
    m = 0u;
#pragma unroll
    for (int j = 0; j < n; ++j) raw[j].each([&](uint32_t& w) { w = Words<T>::finite(w, m); });
    m = warp_max(Words<T>::bits(m));
  }
  return m;
}

// One block's keys of KV head h: rows[t] is the token whose key row t becomes, or -1.
template <typename T, int D, Rope kRope>
__device__ __forceinline__ void write_keys(const WriteParams& p, int64_t blk, int h, const int* rows, int lane) {
  constexpr int NV = D / 32;  // pieces of 16 codes a lane
  constexpr int N = 16 / sizeof(T);
  uint8_t* chunk = p.key_cache + (blk * p.hkv + h) * f8_chunk_bytes(D);
  const T* key = static_cast<const T*>(p.key) + static_cast<int64_t>(h) * D;
  const int tok[2] = {rows[lane >> 2], rows[(lane >> 2) + 8]};
  const bool anew = rows[0] >= 0;
  const int e_old = anew ? 0 : f8_scale(chunk[f8_code_bytes(D)]);
  uint32_t amax = 0u;
  // without RoPE the rows stay in registers; with it they are rotated twice, for the scale
  // and for the codes (64 more registers would halve the warps of an SM)
  Piece<T, 16> raw[kRope == kNone ? NV : 1];
  bool odd = false;  // infinities among the rotated ones
  const float* cs[2] = {nullptr, nullptr};
  auto rotate = [&](int j, int i, float (&y)[N]) {
    const int t = tok[j / (D / 64)], d = 64 * (j % (D / 64)) + (lane & 3) * 16 + i;
    rotated<T, kRope>(key + t * p.key_stride, d, cs[j / (D / 64)], p.rotary_dim, y);
  };
  if constexpr (kRope == kNone) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int t = tok[j / (D / 64)];
      if (t >= 0) raw[j].load(key + t * p.key_stride + 64 * (j % (D / 64)) + (lane & 3) * 16);
      else raw[j].zero();
    }
    amax = most_of<T>(raw);
  } else {
#pragma unroll
    for (int u = 0; u < 2; ++u)
      if (tok[u] >= 0) cs[u] = p.table + __ldg(p.positions + tok[u]) * p.rotary_dim;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (tok[j / (D / 64)] < 0) continue;
#pragma unroll
      for (int i = 0; i < 16; i += N) {
        float y[N];
        rotate(j, i, y);
#pragma unroll
        for (int k = 0; k < N; ++k) amax = max(amax, magnitude(y[k]));
      }
    }
    amax = warp_max(amax);
    if (amax >= kInf) {  // once more, for the finite ones
      odd = true;
      amax = 0u;
#pragma unroll 1
      for (int j = 0; j < NV; ++j)
#pragma unroll 1
        for (int i = 0; i < 16 && tok[j / (D / 64)] >= 0; i += N) {
          float y[N];
          rotate(j, i, y);
#pragma unroll
          for (int k = 0; k < N; ++k) without_infinity(y[k], amax);
        }
      amax = warp_max(amax);
    }
  }
  int grown;
  const int e = new_scale(e_old, amax, &grown);
  const float inv = f8_pow2(127 - e);
  const float down = f8_pow2(max(-grown, -126));
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    uint4* at = reinterpret_cast<uint4*>(chunk + j * 512 + lane * 16);
    if (tok[j / (D / 64)] >= 0) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 16; i += N) {
        float y[N];
        if constexpr (kRope == kNone) {
          if (i == 0) raw[j].each([&](uint32_t& word) { word = Words<T>::times(word, inv); });
#pragma unroll
          for (int k = 0; k < N; ++k) y[k] = raw[j].at(i + k);
        } else {
          rotate(j, i, y);
          if (odd) {
#pragma unroll
            for (int k = 0; k < N; ++k) y[k] = without_infinity(y[k], amax);
          }
#pragma unroll
          for (int k = 0; k < N; ++k) y[k] *= inv;
        }
#pragma unroll
        for (int k = 0; k < N; k += 4) w[(i + k) / 4] = f32x4_to_e4m3(y[k], y[k + 1], y[k + 2], y[k + 3]);
      }
      *at = make_uint4(w[0], w[1], w[2], w[3]);
    } else if (anew) {
      *at = make_uint4(0u, 0u, 0u, 0u);
    } else if (grown) {
      const uint4 o = *at;
      *at = make_uint4(e4m3x4_rescale(o.x, down), e4m3x4_rescale(o.y, down), e4m3x4_rescale(o.z, down),
                       e4m3x4_rescale(o.w, down));
    }
  }
  __syncwarp();
  if (lane == 0)
    *reinterpret_cast<uint4*>(chunk + f8_code_bytes(D)) = make_uint4(static_cast<uint32_t>(e), 0u, 0u, 0u);
}

// One block's values of KV head h.
template <typename T, int D>
__device__ __forceinline__ void write_values(const WriteParams& p, int64_t blk, int h, const int* rows, int lane) {
  constexpr int P = D / 8;  // dimensions a lane has of each of its four tokens
  uint8_t* chunk = p.value_cache + (blk * p.hkv + h) * f8_chunk_bytes(D);
  const T* value = static_cast<const T*>(p.value) + static_cast<int64_t>(h) * D + (lane >> 2) * P;
  const bool anew = rows[0] >= 0;
  const int e_old = anew ? 0 : f8_scale(chunk[f8_code_bytes(D)]);
  Piece<T, P> raw[4];
  uint32_t keep = 0u;  // bytes of a word that stay
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = rows[2 * (lane & 3) + (i >> 1) * 8 + (i & 1)];
    if (t >= 0) {
      raw[i].load(value + t * p.value_stride);
    } else {
      raw[i].zero();
      keep |= 0xffu << (8 * i);
    }
  }
  const uint32_t amax = most_of<T>(raw);
  int grown;
  const int e = new_scale(e_old, amax, &grown);
  const float inv = f8_pow2(127 - e);
  const float down = f8_pow2(max(-grown, -126));
  if (anew || grown || keep != 0xffffffffu) {
#pragma unroll
    for (int i = 0; i < 4; ++i) raw[i].each([&](uint32_t& w) { w = Words<T>::times(w, inv); });
#pragma unroll
    for (int j = 0; j < P / 4; ++j) {
      uint4* at = reinterpret_cast<uint4*>(chunk + j * 512 + lane * 16);
      uint4 o = make_uint4(0u, 0u, 0u, 0u);
      if (!anew && keep != 0u) o = *at;
      uint32_t w[4] = {o.x, o.y, o.z, o.w};
      if (grown) {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = e4m3x4_rescale(w[i], down);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t n = f32x4_to_e4m3(raw[0].at(4 * j + i), raw[1].at(4 * j + i), raw[2].at(4 * j + i),
                                         raw[3].at(4 * j + i));
        w[i] = (w[i] & keep) | (n & ~keep);
      }
      *at = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  __syncwarp();
  if (lane == 0)
    *reinterpret_cast<uint4*>(chunk + f8_code_bytes(D)) = make_uint4(static_cast<uint32_t>(e), 0u, 0u, 0u);
}

// Rotates the query heads of every token whose position is in the table, a warp a token: a
// lane takes the same vector (or two that hold the pairs) of every head, so it reads its
// cosines and sines once.  Behind the vectors that rotate come those that are copied.
template <typename T, int D, Rope kRope>
__device__ __forceinline__ void rotate_queries(const WriteParams& p, int64_t first, int64_t step, int lane) {
  constexpr int N = 16 / sizeof(T);
  constexpr int M = kRope == kHalf ? N : N / 2;  // table entries of a vector, each of cosines and sines
  constexpr int kAhead = 4;
  const int rot = p.rotary_dim / N / (kRope == kHalf ? 2 : 1);
  const int items = rot + (p.query == p.query_out ? 0 : (D - p.rotary_dim) / N);  // 32 at most
  const int per = 32 / items;  // heads at once
  const int j = lane % items, h0 = lane / items;
  if (h0 >= per) return;
  const int at = j < rot ? j : p.rotary_dim / N + j - rot;
  for (int64_t t = first; t < p.num_tokens; t += step) {
    const int64_t pos = __ldg(p.positions + t);
    if (pos < 0 || pos >= p.max_position) continue;
    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const T*>(p.query) + t * p.query_stride) + at;
    uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(p.query_out) + t * p.query_out_stride) + at;
    float c[M], s[M];
    if (j < rot) {
      const float* cs = p.table + pos * p.rotary_dim + j * M;
      load_table<M>(cs, c);
      load_table<M>(cs + (p.rotary_dim >> 1), s);
    }
    for (int h = h0; h < p.heads; h += kAhead * per) {
      // (plain loads: the rows may be rewritten in place)
      Piece<T, N> a[kAhead], b[kRope == kHalf ? kAhead : 1];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int64_t off = static_cast<int64_t>(h + u * per) * (D / N);
        if (h + u * per < p.heads) {
          a[u].v[0] = src[off];
          if (kRope == kHalf && j < rot) b[u].v[0] = src[off + rot];
        }
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        if (h + u * per >= p.heads) break;
        uint4* out = dst + static_cast<int64_t>(h + u * per) * (D / N);
        auto store = [&](uint4* to, const float (&y)[N]) {
          if constexpr (sizeof(T) == 4)
            *to = make_uint4(__float_as_uint(y[0]), __float_as_uint(y[1]), __float_as_uint(y[2]), __float_as_uint(y[3]));
          else
            *to = make_uint4(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]), pack_bf16(y[4], y[5]), pack_bf16(y[6], y[7]));
        };
        if (j >= rot) {
          *out = a[u].v[0];
          continue;
        }
        float y[N];
        if constexpr (kRope == kHalf) {
#pragma unroll
          for (int k = 0; k < N; ++k) y[k] = a[u].at(k) * c[k] - b[u].at(k) * s[k];
          store(out, y);
#pragma unroll
          for (int k = 0; k < N; ++k) y[k] = b[u].at(k) * c[k] + a[u].at(k) * s[k];
          store(out + rot, y);
        } else {
#pragma unroll
          for (int k = 0; k < N; k += 2) {
            y[k] = a[u].at(k) * c[k / 2] - a[u].at(k + 1) * s[k / 2];
            y[k + 1] = a[u].at(k + 1) * c[k / 2] + a[u].at(k) * s[k / 2];
          }
          store(out, y);
        }
      }
    }
  }
}

template <typename T, int D, Rope kRope>
__global__ void __launch_bounds__(write_threads<kRope>(), (sizeof(T) == 2 ? 1024 : 512) / write_threads<kRope>())
    reshape_and_cache_fp8_kernel(const WriteParams p) {
  constexpr int kThreads = write_threads<kRope>();
  // a programmatic dependent of the kernel before it, which may still read the cache or
  // write the new rows
  grid_dependency_wait();
  if (threadIdx.x == 0) grid_launch_dependents();
  if constexpr (kRope != kNone) {
    if (static_cast<int>(blockIdx.x) >= p.cache_ctas) {
      rotate_queries<T, D, kRope>(
          p, static_cast<int64_t>(blockIdx.x - p.cache_ctas) * (kThreads / 32) + (threadIdx.x >> 5),
          static_cast<int64_t>(gridDim.x - p.cache_ctas) * (kThreads / 32), threadIdx.x & 31);
      return;
    }
  }
  __shared__ int block_of[kWriteWindow], first_of[kWriteWindow], taken[kWriteWindow];
  __shared__ int rows[kWriteWindow][kF8Block];
  __shared__ int found;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int win = blockIdx.x / p.splits, split = blockIdx.x - win * p.splits;
  const int T0 = win * p.window, n = min(p.window, p.num_tokens - T0);
  // the rows are wanted once the search below is through
  {
    const int lines = p.hkv * D * static_cast<int>(sizeof(T)) / 128;  // of a row
    for (int i = threadIdx.x; i < 2 * n * lines; i += kThreads) {
      const int k = i / lines, t = T0 + (k >> 1);
      const char* row = (k & 1) ? static_cast<const char*>(p.value) + t * p.value_stride * static_cast<int64_t>(sizeof(T))
                                : static_cast<const char*>(p.key) + t * p.key_stride * static_cast<int64_t>(sizeof(T));
      asm volatile("prefetch.global.L2 [%0];" ::"l"(row + (i - k * lines) * 128));
    }
  }
  // the block of token t, or -1 where it is not written
  auto block_at = [&](int t, bool report) -> int {
    const int64_t slot = __ldg(p.slot_mapping + t);
    bool ok = slot >= 0 && slot < p.num_slots;
    if constexpr (kRope != kNone) {
      const int64_t pos = __ldg(p.positions + t);
      if (pos < 0 || pos >= p.max_position) {
        if (report && p.err) atomicOr(p.err, PKV_ERR_POSITION);
        return -1;
      }
    }
    if (report && slot >= p.num_slots && p.err) atomicOr(p.err, PKV_ERR_SLOT);
    return ok ? static_cast<int>(slot / kF8Block) : -1;
  };
  if (warp == 0) {
    int b = -1;
    bool first = false;
    if (lane < n) {
      b = block_at(T0 + lane, split == 0);
      first = b >= 0 && (T0 + lane == 0 || block_at(T0 + lane - 1, false) != b);
    }
    const unsigned leads = __ballot_sync(0xffffffffu, first);
    const unsigned before = __match_any_sync(0xffffffffu, b) & leads & ((1u << lane) - 1u);
    if (first) {
      const int k = __popc(leads & ((1u << lane) - 1u));
      block_of[k] = b;
      first_of[k] = T0 + lane;
      taken[k] = before != 0u ? 1 : 0;
    }
    if (lane == 0) found = __popc(leads);
  }
  for (int i = threadIdx.x; i < kWriteWindow * kF8Block; i += kThreads) rows[i / kF8Block][i % kF8Block] = -1;
  __syncthreads();
  const int leads = found;
  if (leads == 0) return;
  // so are the scales and codes of blocks that have rows already
  // (8192 tokens 19.3 us without, 18.4 with; of 64 tokens with RoPE 5.5 and 6.2)
  for (int k = 0; k < leads && p.window > 1; ++k) {
    if (__ldg(p.slot_mapping + first_of[k]) % kF8Block == 0) continue;
    constexpr int kLines = f8_chunk_bytes(D) / 128 + 1;
    const int64_t blk = static_cast<int64_t>(block_of[k]) * p.hkv * f8_chunk_bytes(D);
    for (int i = threadIdx.x; i < 2 * p.hkv * kLines; i += kThreads) {
      const int item = i / kLines;
      const int64_t at = static_cast<int64_t>(item >> 1) * f8_chunk_bytes(D) + min((i - item * kLines) * 128, f8_code_bytes(D));
      asm volatile("prefetch.global.L2 [%0];" ::"l"(((item & 1) ? p.value_cache : p.key_cache) + blk + at));
    }
  }
  // ---- the other tokens of those blocks, two blocks at a time (in the order of the requests
  // a window has hardly more) ----
  for (int k = 0; k < leads; k += 2) {
    const uint32_t b0 = block_of[k], b1 = block_of[min(k + 1, leads - 1)];
    auto look = [&](int64_t slot, int t) {
      const uint32_t b = static_cast<uint32_t>(slot >> 4);
      if (b != b0 && b != b1) return;
      if (block_at(t, false) < 0) return;  // (a slot past 2^36 may look like another)
      const int i = b == b0 ? k : k + 1;
      if (t < first_of[i]) taken[i] = 1;
      atomicMax(&rows[i][slot % kF8Block], t);
    };
    // eight slots a thread at a time, where there are as many and they are aligned
    constexpr int kAhead = 4;
    int t = 0;
    if ((reinterpret_cast<uintptr_t>(p.slot_mapping) & 15u) == 0) {
      const longlong2* pairs = reinterpret_cast<const longlong2*>(p.slot_mapping);
      for (; t + 2 * kThreads * kAhead <= p.num_tokens; t += 2 * kThreads * kAhead) {
        longlong2 s[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) s[u] = __ldg(pairs + t / 2 + u * kThreads + threadIdx.x);
        bool any = false;
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          const uint32_t x = static_cast<uint32_t>(s[u].x >> 4), y = static_cast<uint32_t>(s[u].y >> 4);
          any |= x == b0 || x == b1 || y == b0 || y == b1;
        }
        if (any) {
#pragma unroll
          for (int u = 0; u < kAhead; ++u) {
            const int at = t + 2 * (u * kThreads + static_cast<int>(threadIdx.x));
            look(s[u].x, at);
            look(s[u].y, at + 1);
          }
        }
      }
    }
    for (t += threadIdx.x; t < p.num_tokens; t += kThreads) look(__ldg(p.slot_mapping + t), t);
  }
  __syncthreads();
  const int per = 2 * p.hkv;
  for (int i = split * (kThreads / 32) + warp; i < leads * per; i += p.splits * (kThreads / 32)) {
    const int k = i / per, item = i - k * per;
    if (taken[k]) continue;
    if (item & 1) write_values<T, D>(p, block_of[k], item >> 1, rows[k], lane);
    else write_keys<T, D, kRope>(p, block_of[k], item >> 1, rows[k], lane);
  }
}

// Stores eight (four) values of an output row.
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&x)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float (&x)[4]) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
}
__device__ __forceinline__ void store4(float* p, const float (&x)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
}

__device__ __forceinline__ float scale_of(const uint8_t* chunk, int d) {
  return f8_pow2(f8_scale(__ldg(chunk + f8_code_bytes(d))) - 127);
}

struct GatherParams {
  const uint8_t* key_cache;
  const uint8_t* value_cache;
  const int64_t* slot_mapping;
  void* key_out;
  void* value_out;
  int64_t key_stride;    // elements
  int64_t value_stride;
  int64_t num_tokens;
  int64_t num_slots;
  int32_t hkv;
  int32_t window;        // tokens of a CTA at a time
  uint32_t* err;
};

// One token, all heads, by a warp.  A lane takes 16 dimensions of a key at a time (a vector of
// codes), and 4 of a value: the vector that holds them has three other tokens' too.
template <typename T, int D>
__device__ __forceinline__ void gather_token(const GatherParams& p, int64_t t, int64_t slot, bool in, int lane) {
  constexpr int P = D / 8, kAhead = 4;
  const int nk = p.hkv * D / 16, nv = p.hkv * D / 4;
  const int row = static_cast<int>(slot & (kF8Block - 1));
  const int64_t blk = (in ? slot / kF8Block : 0) * p.hkv * f8_chunk_bytes(D);
  const uint8_t* kblk = p.key_cache + blk;
  const uint8_t* vblk = p.value_cache + blk;
  T* ko = static_cast<T*>(p.key_out) + t * p.key_stride;
  T* vo = static_cast<T*>(p.value_out) + t * p.value_stride;
  for (int i = lane; i < nk; i += 32) {
    const int h = i / (D / 16), c = i % (D / 16);
    uint4 w = make_uint4(0u, 0u, 0u, 0u);
    float scale = 0.f;
    if (in) {
      const uint8_t* chunk = kblk + static_cast<int64_t>(h) * f8_chunk_bytes(D);
      w = __ldg(reinterpret_cast<const uint4*>(chunk + f8_key_at<D>(row, 16 * c)));
      scale = scale_of(chunk, D);
    }
    const uint32_t words[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float a[4], b[4];
      e4m3x4_to_f32(words[2 * k], a);
      e4m3x4_to_f32(words[2 * k + 1], b);
      const float x[8] = {a[0] * scale, a[1] * scale, a[2] * scale, a[3] * scale,
                          b[0] * scale, b[1] * scale, b[2] * scale, b[3] * scale};
      store8(ko + 16 * i + 8 * k, x);
    }
  }
  const uint32_t low = 0x0040u + 0x0011u * ((row >> 3) * 2 + (row & 1));  // the token's bytes of two words, side by side
  for (int base = lane; base < nv; base += 32 * kAhead) {
    uint4 w[kAhead];
    float scale[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int i = base + 32 * u;
      const int h = i / (D / 4), c = i % (D / 4);  // dims 4 c .. + 3: lane group c / (P / 4), vector c % (P / 4)
      w[u] = make_uint4(0u, 0u, 0u, 0u);
      scale[u] = 0.f;
      if (in && i < nv) {
        const uint8_t* chunk = vblk + static_cast<int64_t>(h) * f8_chunk_bytes(D);
        w[u] = __ldg(reinterpret_cast<const uint4*>(chunk + c % (P / 4) * 512 + (c / (P / 4) * 4 + (row & 7) / 2) * 16));
        scale[u] = scale_of(chunk, D);
      }
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int i = base + 32 * u;
      if (i >= nv) break;
      float x[4];
      e4m3x4_to_f32(__byte_perm(__byte_perm(w[u].x, w[u].y, low), __byte_perm(w[u].z, w[u].w, low), 0x5410), x);
#pragma unroll
      for (int k = 0; k < 4; ++k) x[k] *= scale[u];
      store4(vo + 4 * i, x);
    }
  }
}

// One block's keys, or values, of a head by a warp: row r goes to token rows[r], if any.
template <typename T, int D, bool kIsV>
__device__ __forceinline__ void gather_block(const GatherParams& p, int64_t blk, bool in, int h, const int64_t* rows, int lane) {
  constexpr int NV = D / 32, P = D / 8;
  const uint8_t* chunk = (kIsV ? p.value_cache : p.key_cache) + (blk * p.hkv + h) * f8_chunk_bytes(D);
  uint4 w[NV];
  float scale = 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j) w[j] = in ? __ldg(reinterpret_cast<const uint4*>(chunk + j * 512) + lane) : make_uint4(0u, 0u, 0u, 0u);
  if (in) scale = scale_of(chunk, D);
  T* out = static_cast<T*>(kIsV ? p.value_out : p.key_out) + static_cast<int64_t>(h) * D;
  const int64_t stride = kIsV ? p.value_stride : p.key_stride;
  if constexpr (!kIsV) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int64_t t = rows[(lane >> 2) + 8 * (j / (D / 64))];
      if (t < 0) continue;
      T* to = out + t * stride + 64 * (j % (D / 64)) + 16 * (lane & 3);
      const uint32_t words[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float a[4], b[4];
        e4m3x4_to_f32(words[2 * k], a);
        e4m3x4_to_f32(words[2 * k + 1], b);
        const float x[8] = {a[0] * scale, a[1] * scale, a[2] * scale, a[3] * scale,
                            b[0] * scale, b[1] * scale, b[2] * scale, b[3] * scale};
        store8(to + 8 * k, x);
      }
    }
  } else {
    int64_t t[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) t[i] = rows[2 * (lane & 3) + (i & 1) + 8 * (i >> 1)];
#pragma unroll
    for (int k = 0; k < P / 8; ++k) {  // eight dimensions
      const uint32_t words[8] = {w[2 * k].x, w[2 * k].y, w[2 * k].z, w[2 * k].w,
                                 w[2 * k + 1].x, w[2 * k + 1].y, w[2 * k + 1].z, w[2 * k + 1].w};
      float x[4][8];
#pragma unroll
      for (int d = 0; d < 8; ++d) {
        float a[4];
        e4m3x4_to_f32(words[d], a);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i][d] = a[i] * scale;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (t[i] >= 0) store8(out + t[i] * stride + P * (lane >> 2) + 8 * k, x[i]);
    }
  }
}

// Every value is exact in either output type.  A CTA takes a window of tokens.  Runs of them
// that follow one another in a block are read by block, a warp a head and K or V; where the
// window has more than a run in four tokens, a warp takes a token.  (8192 tokens in order, 8
// heads of 128, bfloat16: by token 16.5 us, by block 14.2.  7777 in random order, 5 heads of 64,
// float32: by token 8.3.)
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) gather_cache_fp8_kernel(const GatherParams p) {
  grid_dependency_wait();  // the kernel before it may write the cache
  if (threadIdx.x == 0) grid_launch_dependents();
  __shared__ int64_t rows[kWindow][kF8Block];  // by run: the tokens of a block's rows
  __shared__ int64_t slots[kWindow];
  __shared__ int first[kWindow];               // tokens (of the window) that begin a run
  __shared__ int count[2];                     // of runs, and of tokens
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int64_t T0 = static_cast<int64_t>(blockIdx.x) * p.window; T0 < p.num_tokens;
       T0 += static_cast<int64_t>(gridDim.x) * p.window) {
    const int n = static_cast<int>(min(static_cast<int64_t>(p.window), p.num_tokens - T0));
    for (int i = threadIdx.x; i < kWindow * kF8Block; i += kThreads) rows[i / kF8Block][i % kF8Block] = -1;
    __syncthreads();
    if (warp == 0) {
      const int64_t slot = lane < n ? __ldg(p.slot_mapping + T0 + lane) : -1;
      const int64_t prev = __shfl_up_sync(0xffffffffu, slot, 1);
      // (rows of a run ascend, so each is one token's)
      const bool leads = slot >= 0 && (lane == 0 || prev < 0 || prev / kF8Block != slot / kF8Block || prev >= slot);
      const unsigned lead = __ballot_sync(0xffffffffu, leads), live = __ballot_sync(0xffffffffu, slot >= 0);
      const int k = __popc(lead & (0xffffffffu >> (31 - lane))) - 1;
      if (lane < n) slots[lane] = slot;
      if (slot >= 0) rows[k][slot % kF8Block] = T0 + lane;
      if (leads) first[k] = lane;
      if (lane == 0) {
        count[0] = __popc(lead);
        count[1] = __popc(live);
      }
      if (slot >= p.num_slots && p.err) atomicOr(p.err, PKV_ERR_SLOT);
    }
    __syncthreads();
    const int runs = count[0], per = 2 * p.hkv;
    if (4 * runs <= count[1]) {
      for (int i = warp; i < runs * per; i += kThreads / 32) {
        const int k = i / per, item = i - k * per;
        const int64_t slot = slots[first[k]];
        const bool in = slot < p.num_slots;
        const int64_t blk = in ? slot / kF8Block : 0;
        if (item & 1) gather_block<T, D, true>(p, blk, in, item >> 1, rows[k], lane);
        else gather_block<T, D, false>(p, blk, in, item >> 1, rows[k], lane);
      }
    } else {
      for (int i = warp; i < n; i += kThreads / 32)
        if (slots[i] >= 0) gather_token<T, D>(p, T0 + i, slots[i], slots[i] < p.num_slots, lane);
    }
    __syncthreads();  // the tables are written again
  }
}

template <typename T, int D, Rope kRope>
cudaError_t write_t(const F8WriteArgs& a, cudaStream_t stream) {
  constexpr int kThreads = write_threads<kRope>();
  WriteParams p;
  p.key = a.cache.key;
  p.value = a.cache.value;
  p.key_stride = a.cache.key_stride;
  p.value_stride = a.cache.value_stride;
  p.key_cache = a.cache.key_cache;
  p.value_cache = a.cache.value_cache;
  p.slot_mapping = a.cache.slot_mapping;
  p.num_slots = a.cache.num_slots;
  p.num_tokens = static_cast<int32_t>(a.cache.num_tokens);
  p.hkv = a.cache.num_kv_heads;
  p.err = a.cache.err;
  p.positions = a.positions;
  p.table = a.cos_sin_cache;
  p.max_position = a.max_position;
  p.rotary_dim = a.rotary_dim;
  p.heads = a.num_heads;
  p.query = a.query;
  p.query_out = a.query_out;
  p.query_stride = a.query_stride;
  p.query_out_stride = a.query_out_stride;
  const int sms = current_sm_count();
  // a token a window while there are SMs for them
  const int64_t want = (a.cache.num_tokens + 4 * sms - 1) / (4 * sms);
  p.window = static_cast<int32_t>(want < kWriteWindow ? want : kWriteWindow);
  const int windows = (p.num_tokens + p.window - 1) / p.window;
  p.splits = (2 * p.hkv + kThreads / 32 - 1) / (kThreads / 32);
  const int most = 4 * sms / windows;  // (bfloat16: one wave, of CTAs of 512 threads two)
  if (p.splits > most) p.splits = most > 1 ? most : 1;
  p.cache_ctas = windows * p.splits;
  int64_t grid = p.cache_ctas;
  if (kRope != kNone) {
    const int64_t ctas = (a.cache.num_tokens + kThreads / 32 - 1) / (kThreads / 32), cap = 8 * static_cast<int64_t>(sms);
    grid += ctas < cap ? ctas : cap;
  }
  return launch_programmatic(reshape_and_cache_fp8_kernel<T, D, kRope>, dim3(static_cast<unsigned>(grid)),
                             dim3(kThreads), 0, stream, p);
}

template <typename T, int D>
cudaError_t write_d(const F8WriteArgs& a, cudaStream_t stream) {
  if (a.positions == nullptr) return write_t<T, D, kNone>(a, stream);
  return a.is_neox ? write_t<T, D, kHalf>(a, stream) : write_t<T, D, kInterleaved>(a, stream);
}

template <typename T, int D>
cudaError_t gather_t(const MxCacheArgs& a, cudaStream_t stream) {
  GatherParams p;
  p.key_cache = a.key_cache;
  p.value_cache = a.value_cache;
  p.slot_mapping = a.slot_mapping;
  p.key_out = const_cast<void*>(a.key);
  p.value_out = const_cast<void*>(a.value);
  p.key_stride = a.key_stride;
  p.value_stride = a.value_stride;
  p.num_tokens = a.num_tokens;
  p.num_slots = a.num_slots;
  p.hkv = a.num_kv_heads;
  p.err = a.err;
  const int64_t sms = current_sm_count(), want = (a.num_tokens + 4 * sms - 1) / (4 * sms);
  p.window = static_cast<int32_t>(want < kWindow ? want : kWindow);
  const int64_t windows = (a.num_tokens + p.window - 1) / p.window, cap = 64 * sms;
  return launch_programmatic(gather_cache_fp8_kernel<T, D>, dim3(static_cast<unsigned>(windows < cap ? windows : cap)),
                             dim3(kThreads), 0, stream, p);
}

}  // namespace

cudaError_t launch_write_fp8(const F8WriteArgs& a, cudaStream_t stream) {
  if (a.cache.num_tokens == 0) return cudaSuccess;
  if (a.cache.head_dim == 128)
    return a.cache.bf16 ? write_d<__nv_bfloat16, 128>(a, stream) : write_d<float, 128>(a, stream);
  if (a.cache.head_dim == 64)
    return a.cache.bf16 ? write_d<__nv_bfloat16, 64>(a, stream) : write_d<float, 64>(a, stream);
  return cudaErrorNotSupported;
}

cudaError_t launch_gather_cache_fp8(const MxCacheArgs& a, cudaStream_t stream) {
  if (a.num_tokens == 0) return cudaSuccess;
  if (a.head_dim == 128)
    return a.bf16 ? gather_t<__nv_bfloat16, 128>(a, stream) : gather_t<float, 128>(a, stream);
  if (a.head_dim == 64)
    return a.bf16 ? gather_t<__nv_bfloat16, 64>(a, stream) : gather_t<float, 64>(a, stream);
  return cudaErrorNotSupported;
}

}  // namespace pkv
