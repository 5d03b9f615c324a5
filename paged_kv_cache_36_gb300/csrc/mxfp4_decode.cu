// Split-KV decode attention (query length 1) over the 4-bit paged cache.
//
// For a decode request r, query head h of KV head g and its keys j < seq_len:
//   out = sum_j softmax_j(scale <q, K_j>) V_j,
// K and V the values that codes and power-of-two scales stand for (mxfp4.cuh).
//
// Work split.  A unit is one 16-token block of one KV head.  Units are ordered
// by request, KV head and block, and worker w of W (a worker is one warp) takes
// units [wN/W, (w+1)N/W): every warp streams the same bytes whatever the
// context lengths, and no warp waits for another.  A (request, KV head) run
// that crosses workers leaves one partial (m, l, o) per worker in the
// workspace; the warp whose count completes a group of kFan partials merges
// them, and the one that completes the groups merges those, so that even a
// run of thousands of workers costs two short merges.  The order of every sum
// is fixed by the split, not by who comes last.
//
// Data movement.  A warp keeps its own ring of stages, each two units (4.3 KiB
// at head_dim 128), filled by 16-byte cp.async: a head's chunk of a block is
// contiguous, K and V.  The fetch cursor runs ahead of the compute over
// request boundaries, so a new request costs no bubble.
//
// Compute.  S^T = K Q^T and O^T += V^T P^T are m16n8k16 f16 products with the
// query heads of the KV head as N, float32 accumulators.
//   - Codes become f16 by one conversion per pair and go straight into the A
//     fragment: the cache's byte order is the fragment's.
//   - Q is brought to f16 by an exact power of two per head.  f16 holds the 8
//     bits of a bfloat16 over 30 binades below the head's largest element, so
//     what is lost is below 2^-38 of it.
//   - K scales multiply the partial sums of each group of 32 dimensions, in
//     float32: any scale is exact.
//   - V scales go onto the weights: P^T (f16, 11 bits) times 2^(e - base) for
//     each group of dimensions, `base` a running exponent per group.  Scales
//     within 2^7 of it, which is nearly always, cost one f16x2 product per
//     group; a tile outside the window takes the slow path below, which moves
//     the base and splits the tile into windows so that no weight leaves f16's
//     range.
//   - The running maximum moves only when a score exceeds it by 2^8: the common
//     tile needs a vote, and no shuffle.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "kernels.h"
#include "mxfp4.cuh"
#include "pkv_device.cuh"

namespace pkv {

namespace {

constexpr int kFan = 16;         // partials per first-level merge, at least
constexpr int kMinUnits = 8;     // units a worker takes at least (128 tokens of one KV head)
constexpr float kMaxSlack = 8.f; // log2 units a score may exceed the running maximum by

template <int NT>
constexpr int warps_per_cta() { return NT == 1 ? 16 : 8; }

struct Params {
  const __nv_bfloat16* q;
  int64_t q_stride;
  const uint8_t* key_cache;
  const uint8_t* value_cache;
  const int32_t* block_table;
  int32_t bt_stride;
  int32_t bt_width;
  const int32_t* qsl;
  const int32_t* seq_lens;
  const int32_t* num_computed;
  __nv_bfloat16* out;
  int64_t out_stride;
  int64_t num_tokens;
  int32_t num_reqs;
  int32_t num_blocks;
  int32_t hkv;
  int32_t group;
  float scale_log2;
  uint32_t* err;
  int32_t* count1;   // [2 * workers] arrivals of a first-level group, at its first slot
  int32_t* count2;   // [2 * workers] completed groups of a run, at its first slot
  float2* part_ml;   // [2 * workers][group]
  float* part_o;     // [2 * workers][group][D]
  int32_t stages;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool real) {
  // `real` false: 16 zero bytes, nothing is read
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(real ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// D = A B + C, m16n8k16, f16 inputs, float32 accumulators.
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  const __half2 h = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&h);
}
// 2^k for k in [-126, 127]; 0 below.
__device__ __forceinline__ float pow2(int k) {
  return k < -126 ? 0.f : __uint_as_float(static_cast<uint32_t>(k + 127) << 23);
}

// A worker's position in the ordered units: block j of nb of (request r, KV
// head h), `left` units to go.
struct Cursor {
  int r, h, j, nb;
  int64_t left;
  __device__ __forceinline__ int pair() const {  // units of the next stage: 1 or 2
    int n = nb - j < 2 ? nb - j : 2;
    return left < n ? static_cast<int>(left) : n;
  }
  __device__ __forceinline__ void advance(int n, const int32_t* prefix, int hkv) {
    j += n;
    left -= n;
    if (j == nb && left > 0) {
      j = 0;
      if (++h == hkv) {
        h = 0;
        do ++r; while (prefix[r + 1] == prefix[r]);
        nb = prefix[r + 1] - prefix[r];
      }
    }
  }
};

template <int D, int NT>
__global__ void __launch_bounds__(warps_per_cta<NT>() * 32, 1)
    decode_mxfp4_kernel(const Params p) {
  constexpr int NB = D / 32;                       // groups of dimensions
  constexpr int KS = D / 16;                       // k-steps of S^T
  constexpr int NW = D / 64;                       // words of V codes of a lane and token
  constexpr uint32_t kChunk = mx_chunk_bytes(D);   // one head of one block
  constexpr uint32_t kScale = mx_scale_off(D);
  constexpr uint32_t kUnit = 2 * kChunk;           // K then V
  constexpr uint32_t kStage = 2 * kUnit;           // two units
  constexpr int kWarps = warps_per_cta<NT>();
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int32_t scan_tmp[32];
  int32_t* prefix = reinterpret_cast<int32_t*>(smem + static_cast<size_t>(p.stages) * kWarps * kStage);

  // the kernel before may write q, the cache, out or the metadata
  grid_dependency_wait();
  if (threadIdx.x == 0) grid_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gid = lane >> 2, tid = lane & 3;
  const int R = p.num_reqs;

  // ---- plan: blocks of every decode request and their prefix sum ----
  if (threadIdx.x == 0) prefix[0] = 0;
  for (int r = threadIdx.x; r < R; r += blockDim.x) {
    const int q0 = __ldg(p.qsl + r), q1 = __ldg(p.qsl + r + 1);
    const int seq = __ldg(p.seq_lens + r), nc = __ldg(p.num_computed + r);
    int nb = 0;
    if (q1 - q0 == 1) {
      nb = (seq - 1) / kMxBlock + 1;
      if (nc < 0 || nc > 0x7ffffffe || seq != nc + 1 || nb > p.bt_width || q0 < 0 ||
          q1 > p.num_tokens) {
        if (blockIdx.x == 0) atomicOr(p.err, PKV_ERR_METADATA);
        nb = 0;
      }
    }
    prefix[r + 1] = nb;
  }
  __syncthreads();
  block_inclusive_scan(prefix + 1, R, scan_tmp);
  __syncthreads();
  const int64_t N = static_cast<int64_t>(prefix[R]) * p.hkv;
  if (N == 0) return;
  const int64_t most = static_cast<int64_t>(gridDim.x) * kWarps;
  const int64_t want = (N + kMinUnits - 1) / kMinUnits;
  const int64_t W = want < most ? want : most;
  const int64_t me = static_cast<int64_t>(warp) * gridDim.x + blockIdx.x;  // spread over the SMs first
  if (me >= W) return;
  const int64_t u0 = me * N / W, u1 = (me + 1) * N / W;
  auto worker_of = [&](int64_t unit) -> int64_t { return ((unit + 1) * W - 1) / N; };

  Cursor at;
  {
    int lo = 0, hi = R;  // prefix[lo] hkv <= u0 < prefix[hi] hkv
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (static_cast<int64_t>(prefix[mid]) * p.hkv <= u0) lo = mid; else hi = mid;
    }
    at.r = lo;
    at.nb = prefix[lo + 1] - prefix[lo];
    const int64_t off = u0 - static_cast<int64_t>(prefix[lo]) * p.hkv;
    at.h = static_cast<int>(off / at.nb);
    at.j = static_cast<int>(off - static_cast<int64_t>(at.h) * at.nb);
    at.left = u1 - u0;
  }

  // ---- the ring: fetch cursor, ids of its next stage already loaded ----
  const int64_t block_bytes = static_cast<int64_t>(p.hkv) * kChunk;
  const uint32_t ring = smem_u32(smem) + static_cast<uint32_t>(warp) * p.stages * kStage;
  Cursor next = at;
  int id0 = 0, id1 = -1;
  auto load_ids = [&]() {
    if (next.left <= 0) return;
    const int32_t* row = p.block_table + static_cast<int64_t>(next.r) * p.bt_stride + next.j;
    id0 = __ldg(row);
    id1 = next.pair() == 2 ? __ldg(row + 1) : -1;
  };
  // V codes of two tokens (128 or 64 bytes) are XOR-swizzled by 16-byte chunks
  // so that the four token pairs that a quad row reads at once hit different
  // banks.
  const uint32_t v_dst = D == 128 ? (lane >> 3) * 128 + (((lane & 7) ^ (2 * ((lane >> 3) & 3))) << 4)
                                  : (lane ^ (((lane >> 3) & 1) << 1)) << 4;
  auto fetch = [&](int slot) {
    if (next.left > 0) {
      const int n = next.pair();
      const uint32_t dst = ring + slot * kStage;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int id = u == 0 ? id0 : id1;
        const bool real = id >= 0 && id < p.num_blocks;
        if (u < n && !real && lane == 0) atomicOr(p.err, PKV_ERR_BLOCK_ID);
        const int64_t off = (real ? id : 0) * block_bytes + static_cast<int64_t>(next.h) * kChunk;
        const uint8_t* k = p.key_cache + off + lane * 16;
        const uint8_t* v = p.value_cache + off + lane * 16;
        const uint32_t kd = dst + u * kUnit + lane * 16, vd = dst + u * kUnit + kChunk + v_dst;
#pragma unroll
        for (int i = 0; i < NW; ++i) {
          cp_async16(kd + i * 512, k + i * 512, real);
          cp_async16(vd + i * 512, v + i * 512, real);
        }
        // scales: NB chunks of 16 bytes each for K and V
        if (lane < 2 * NB) {
          const bool is_v = lane >= NB;
          const int c = is_v ? lane - NB : lane;
          cp_async16(dst + u * kUnit + (is_v ? kChunk : 0) + kScale + c * 16,
                     (is_v ? p.value_cache : p.key_cache) + off + kScale + c * 16, real);
        }
      }
      next.advance(n, prefix, p.hkv);
      load_ids();
    }
    cp_async_commit();
  };
  load_ids();
  const int stages = p.stages;
  for (int s = 0; s < stages - 1; ++s) fetch(s);

  const int G = p.group;
  int slot = 0;
  while (at.left > 0) {
    // ======================= one run of this worker =======================
    const int r = at.r, h = at.h;
    const int64_t run0 = static_cast<int64_t>(prefix[r]) * p.hkv + static_cast<int64_t>(h) * at.nb;
    const int64_t run1 = run0 + at.nb;
    const int64_t tok = __ldg(p.qsl + r);
    const int seq = __ldg(p.seq_lens + r);

    // B fragments of Q^T in f16: k-step 2b + s of lane tid holds dims 32 b + 8
    // tid + 4 s .. + 3, the order of the K codes
    uint32_t qb[NT][KS][2];
    float qs[NT][2];  // what undoes the power of two, times scale log2(e), of heads 2 tid, + 1
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int head = nt * 8 + gid;
      const __nv_bfloat16* qrow =
          p.q + tok * p.q_stride + static_cast<int64_t>(h * G + (head < G ? head : 0)) * D;
      uint4 w[NB];
      uint32_t mx = 0u;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        w[b] = __ldg(reinterpret_cast<const uint4*>(qrow + 32 * b + 8 * tid));
        const uint32_t x[4] = {w[b].x, w[b].y, w[b].z, w[b].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) mx = max(mx, max(x[i] & 0x7fffu, (x[i] >> 16) & 0x7fffu));
      }
      mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      // largest element to [2^14, 2^15)
      const uint32_t ex = min(max(mx >> 7, 15u), 254u);
      const int up = 141 - static_cast<int>(ex);  // in [-113, 126]
      const float f = pow2(up);
      const float undo = p.scale_log2 * pow2(-up);
      qs[nt][0] = __shfl_sync(0xffffffffu, undo, 8 * tid);
      qs[nt][1] = __shfl_sync(0xffffffffu, undo, 8 * tid + 4);
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const uint32_t x[4] = {w[b].x, w[b].y, w[b].z, w[b].w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          qb[nt][2 * b + (i >> 1)][i & 1] =
              head < G ? pack_f16(__uint_as_float(x[i] << 16) * f,
                                  __uint_as_float(x[i] & 0xffff0000u) * f)
                       : 0u;
      }
    }

    float o[2 * NB][NT][4];
    float m[NT][2], l[NT][2];
    uint32_t base[NW];  // running scale byte per group, as the V scale words have them: b0 b1 b0 b1
    uint32_t top[NW];   // the highest base so far
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < 2 * NB; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) o[i][nt][c] = 0.f;
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.f;
    }
#pragma unroll
    for (int w = 0; w < NW; ++w) base[w] = top[w] = 0u;

    bool more = true;
    while (more) {
      const int n = at.pair();
      const int j = at.j;
      // at the fewest stages one fetch may still be in flight, else two
      if (stages == 2) cp_async_wait<0>(); else cp_async_wait<1>();
      __syncwarp();
      fetch(slot == 0 ? stages - 1 : slot - 1);
      const uint8_t* st = smem + (static_cast<size_t>(warp) * stages + slot) * kStage;

      // ---- S^T = K Q^T of both units, in log2 units ----
      float s[2][NT][4];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint8_t* k = st + u * kUnit;
        uint32_t lo[NB], hi[NB], slo, shi;  // tokens gid and gid + 8
        if constexpr (D == 128) {
          const uint4 x = *reinterpret_cast<const uint4*>(k + gid * 64 + tid * 16);
          const uint4 y = *reinterpret_cast<const uint4*>(k + gid * 64 + 512 + tid * 16);
          lo[0] = x.x; lo[1] = x.y; lo[2] = x.z; lo[3] = x.w;
          hi[0] = y.x; hi[1] = y.y; hi[2] = y.z; hi[3] = y.w;
          slo = *reinterpret_cast<const uint32_t*>(k + kScale + gid * 4);
          shi = *reinterpret_cast<const uint32_t*>(k + kScale + gid * 4 + 32);
        } else {
          const uint2 x = *reinterpret_cast<const uint2*>(k + gid * 32 + tid * 8);
          const uint2 y = *reinterpret_cast<const uint2*>(k + gid * 32 + 256 + tid * 8);
          lo[0] = x.x; lo[1] = x.y;
          hi[0] = y.x; hi[1] = y.y;
          slo = *reinterpret_cast<const uint16_t*>(k + kScale + gid * 2);
          shi = *reinterpret_cast<const uint16_t*>(k + kScale + gid * 2 + 16);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 4; ++c) s[u][nt][c] = 0.f;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          uint32_t x[4], y[4];
          e2m1x8_to_f16(lo[b], x);
          e2m1x8_to_f16(hi[b], y);
          // 2^(e - 127): the scale byte in a float's exponent field (NaN's 255
          // gives infinity, and times its zero codes NaN; 0 reads as zero, below
          // the smallest scale that the cache write makes)
          const float fl = __uint_as_float((b < 3 ? slo << (23 - 8 * b) : slo >> 1) & 0x7f800000u);
          const float fh = __uint_as_float((b < 3 ? shi << (23 - 8 * b) : shi >> 1) & 0x7f800000u);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float d[4] = {0.f, 0.f, 0.f, 0.f};
            mma_f16(d, x[0], y[0], x[1], y[1], qb[nt][2 * b][0], qb[nt][2 * b][1]);
            mma_f16(d, x[2], y[2], x[3], y[3], qb[nt][2 * b + 1][0], qb[nt][2 * b + 1][1]);
            s[u][nt][0] = fmaf(d[0], fl, s[u][nt][0]);
            s[u][nt][1] = fmaf(d[1], fl, s[u][nt][1]);
            s[u][nt][2] = fmaf(d[2], fh, s[u][nt][2]);
            s[u][nt][3] = fmaf(d[3], fh, s[u][nt][3]);
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 4; ++c) s[u][nt][c] *= qs[nt][c & 1];
      }
      // tokens of this stage that the request has (a full stage: 32)
      const int valid = min(seq - j * kMxBlock, n * kMxBlock);
      if (valid < 32) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 4; ++c)
              if (u * 16 + gid + (c >> 1) * 8 >= valid) s[u][nt][c] = -INFINITY;
      }

      // ---- online softmax per head column ----
      float mx[NT][2];
      bool grow = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int cc = 0; cc < 2; ++cc) {
          mx[nt][cc] = fmaxf(fmaxf(s[0][nt][cc], s[0][nt][2 + cc]),
                             fmaxf(s[1][nt][cc], s[1][nt][2 + cc]));
          grow |= mx[nt][cc] > m[nt][cc] + kMaxSlack;
        }
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int cc = 0; cc < 2; ++cc) {
            float x = mx[nt][cc];
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
            const float mn = fmaxf(m[nt][cc], x);
            const float alpha = mn == m[nt][cc] ? 1.f : exp2_approx(m[nt][cc] - mn);
            m[nt][cc] = mn;
            l[nt][cc] *= alpha;
#pragma unroll
            for (int i = 0; i < 2 * NB; ++i) {
              o[i][nt][cc] *= alpha;
              o[i][nt][2 + cc] *= alpha;
            }
          }
      }

#pragma unroll
      for (int u = 0; u < 2; ++u) {
        if (u == 1 && valid <= 16) break;
        // P^T fragments: tokens 2 tid, + 1 (and + 8) of head gid
        uint32_t pt[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float e[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) e[c] = exp2_approx(s[u][nt][c] - m[nt][c & 1]);
          l[nt][0] += e[0] + e[2];
          l[nt][1] += e[1] + e[3];
          pt[nt][0] = movmatrix_trans(pack_f16(e[0], e[1]));
          pt[nt][1] = movmatrix_trans(pack_f16(e[2], e[3]));
        }

        // ---- V codes and scales of tokens 2 tid, + 1, + 8, + 9 ----
        const uint8_t* v = st + u * kUnit + kChunk;
        uint32_t vw[4][NW], sw[2][NW];
        if constexpr (D == 128) {
          // pair tid, halves: chunk (token parity 4 + gid / 2) ^ 2 tid, 8 bytes at gid % 2
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint2 x = *reinterpret_cast<const uint2*>(
                v + (i >> 1) * 512 + tid * 128 + (((((i & 1) << 2) + (gid >> 1)) ^ (2 * tid)) << 4) +
                (gid & 1) * 8);
            vw[i][0] = x.x;
            vw[i][1] = x.y;
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint2 x = *reinterpret_cast<const uint2*>(v + kScale + i * 32 + tid * 8);
            sw[i][0] = x.x;
            sw[i][1] = x.y;
          }
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            vw[i][0] = *reinterpret_cast<const uint32_t*>(
                v + (i >> 1) * 256 + tid * 64 + (((i & 1) ^ (tid >> 1)) << 5) + gid * 4);
#pragma unroll
          for (int i = 0; i < 2; ++i)
            sw[i][0] = *reinterpret_cast<const uint32_t*>(v + kScale + i * 16 + tid * 4);
        }
        if (valid - u * 16 < 16) {
          // bytes of tokens past the end may be anything: any scale inside the window
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int t = u * 16 + 2 * tid + 8 * i;
            const uint32_t keep = (t < valid ? 0x0000ffffu : 0u) | (t + 1 < valid ? 0xffff0000u : 0u);
#pragma unroll
            for (int w = 0; w < NW; ++w) sw[i][w] = (sw[i][w] & keep) | (base[w] & ~keep);
          }
        }
        // All scales within [base, base + 7]?  If so no byte borrows, and every
        // difference fits its low three bits.  A byte below base by 1 .. 247
        // leaves one of the tested bits set (base is at most 247, and NaN's 255
        // is above every base by 8 or more).
        uint32_t far = 0u;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int w = 0; w < NW; ++w) far |= sw[i][w] - base[w];
        // codes of a token pair side by side: byte k holds position 2k (even) or
        // 2k + 1 (odd) of both tokens
        uint32_t ev[2][NW], od[2][NW];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int w = 0; w < NW; ++w) {
            const uint32_t x = vw[2 * i][w], y = vw[2 * i + 1][w];
            ev[i][w] = (x & 0x0f0f0f0fu) | ((y << 4) & 0xf0f0f0f0u);
            od[i][w] = ((x >> 4) & 0x0f0f0f0fu) | (y & 0xf0f0f0f0u);
          }

        if (!__any_sync(0xffffffffu, (far & 0xf8f8f8f8u) != 0u)) {
#pragma unroll
          for (int w = 0; w < NW; ++w) {
            // 2^(e - base) as f16: exponent field e - base + 15 in each half
            const uint32_t c = 0x3c3c3c3cu - 4u * base[w];
            const uint32_t x0 = sw[0][w] * 4u + c, x1 = sw[1][w] * 4u + c;
            uint32_t e0[4], e1[4], o0[4], o1[4];
            e2m1x8_to_f16(ev[0][w], e0);
            e2m1x8_to_f16(od[0][w], o0);
            e2m1x8_to_f16(ev[1][w], e1);
            e2m1x8_to_f16(od[1][w], o1);
#pragma unroll
            for (int b = 0; b < 2; ++b) {  // groups 2w and 2w + 1
              const uint32_t f0 = (b == 0 ? x0 << 8 : x0) & 0xff00ff00u;
              const uint32_t f1 = (b == 0 ? x1 << 8 : x1) & 0xff00ff00u;
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                const uint32_t b0 = mul_f16x2(pt[nt][0], f0), b1 = mul_f16x2(pt[nt][1], f1);
#pragma unroll
                for (int k = 0; k < 2; ++k)
                  mma_f16(o[4 * w + 2 * b + k][nt], e0[2 * b + k], o0[2 * b + k], e1[2 * b + k],
                          o1[2 * b + k], b0, b1);
              }
            }
          }
        } else {
          // ---- slow path: scales outside the window ----
          // Tokens with no weight left in f16 (for every head) count for nothing
          // here, as they do in the product.
          uint32_t live = 0u;  // bit i: token 2 tid + (i & 1) + 8 (i >> 1)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if ((pt[nt][i >> 1] >> (16 * (i & 1))) & 0x7fffu) live |= 1u << i;
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) live |= __shfl_xor_sync(0xffffffffu, live, x);
#pragma unroll
          for (int w = 0; w < NW; ++w) {
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              int e[4];       // scale bytes of this lane's tokens in group 2 w + b
              int hi = -1;
              bool nan = false;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                e[i] = (sw[i >> 1][w] >> (16 * (i & 1) + 8 * b)) & 0xff;
                const bool in = u * 16 + 2 * tid + (i & 1) + 8 * (i >> 1) < valid;
                nan |= in && e[i] == 255;
                if (!in || e[i] == 255 || !((live >> i) & 1u)) e[i] = -1;
                hi = max(hi, e[i]);
              }
              hi = max(hi, __shfl_xor_sync(0xffffffffu, hi, 1));
              hi = max(hi, __shfl_xor_sync(0xffffffffu, hi, 2));
              nan = __any_sync(0xffffffffu, nan);
              // the base follows the largest scale, five below it; down again
              // only while what is summed up stays far from overflow
              int bs = (base[w] >> (8 * b)) & 0xff, tp = (top[w] >> (8 * b)) & 0xff;
              const int to = min(max(hi - 5, 0), 247);
              if (hi >= 0 && (to > bs || (hi < bs && tp - to <= 60))) {
                const float f = bs > to ? pow2(bs - to) : pow2(max(bs - to, -127));
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                  for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int c = 0; c < 4; ++c) o[4 * w + 2 * b + k][nt][c] *= f;
                const uint32_t hold = ~(0x00ff00ffu << (8 * b));
                base[w] = (base[w] & hold) | (static_cast<uint32_t>(to) * 0x00010001u) << (8 * b);
                tp = max(tp, to);
                top[w] = (top[w] & hold) | (static_cast<uint32_t>(tp) * 0x00010001u) << (8 * b);
                bs = to;
              }
              // windows of eight binades, from the base down
              for (int below = 0; below < 256; below += 8) {
                uint32_t f[2] = {0u, 0u};
                bool rest = false;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const int d = e[i] < 0 ? -1000 : e[i] - bs + below;
                  if (d >= 0 && d < 8) f[i >> 1] |= static_cast<uint32_t>(d + 15) << (10 + 16 * (i & 1));
                  rest |= e[i] >= 0 && d < 0;
                }
                const float back = pow2(-below);
                uint32_t a[2][4];  // fragments of the group's two m-tiles
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                  const int at8 = 8 * (2 * b + k);
                  a[k][0] = e2m1x2_to_f16x2(ev[0][w] >> at8);
                  a[k][1] = e2m1x2_to_f16x2(od[0][w] >> at8);
                  a[k][2] = e2m1x2_to_f16x2(ev[1][w] >> at8);
                  a[k][3] = e2m1x2_to_f16x2(od[1][w] >> at8);
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                  const uint32_t b0 = mul_f16x2(pt[nt][0], f[0]), b1 = mul_f16x2(pt[nt][1], f[1]);
#pragma unroll
                  for (int k = 0; k < 2; ++k) {
                    float t[4] = {0.f, 0.f, 0.f, 0.f};
                    mma_f16(t, a[k][0], a[k][1], a[k][2], a[k][3], b0, b1);
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                      o[4 * w + 2 * b + k][nt][c] = fmaf(t[c], back, o[4 * w + 2 * b + k][nt][c]);
                  }
                }
                if (!__any_sync(0xffffffffu, rest)) break;
              }
              if (nan) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                  for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                      o[4 * w + 2 * b + k][nt][c] = __uint_as_float(0x7fffffffu);
              }
            }
          }
        }
      }
      if (++slot == stages) slot = 0;
      at.advance(n, prefix, p.hkv);
      more = at.left > 0 && at.r == r && at.h == h;
    }

    // ======================= end of this worker's part of the run =======================
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int cc = 0; cc < 2; ++cc) {
        float x = l[nt][cc];
        x += __shfl_xor_sync(0xffffffffu, x, 4);
        x += __shfl_xor_sync(0xffffffffu, x, 8);
        x += __shfl_xor_sync(0xffffffffu, x, 16);
        l[nt][cc] = x;
      }
    const int64_t wf = worker_of(run0);
    const int splits = static_cast<int>(worker_of(run1 - 1) - wf) + 1;
    // slot of split k: a worker's own, except that a run which starts inside
    // the first worker's range has that worker's second slot
    const bool inside = run0 > wf * N / W;
    auto slot_of = [&](int k) -> int64_t { return 2 * (wf + k) + (k == 0 && inside ? 1 : 0); };
    const int mine = static_cast<int>(me - wf);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int cc = 0; cc < 2; ++cc) {
        const int g = nt * 8 + 2 * tid + cc;
        if (g >= G) continue;
        // o[2 b + s]: dims 32 b + 4 gid + 2 s (elements 0, 1) and + 1 (2, 3)
        const float inv = splits == 1 ? 1.f / l[nt][cc] : 1.f;
        __nv_bfloat16* dst = p.out + tok * p.out_stride + static_cast<int64_t>(h * G + g) * D + 4 * gid;
        float* po = p.part_o + (slot_of(mine) * G + g) * D + 4 * gid;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const uint32_t e = (base[b >> 1] >> (8 * (b & 1))) & 0xffu;
          const float f = mx_scale(e);
          float x[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) x[i] = o[2 * b + (i >> 1)][nt][2 * (i & 1) + cc] * f;
          if (splits == 1)
            *reinterpret_cast<uint2*>(dst + 32 * b) =
                make_uint2(pack_bf16(x[0] * inv, x[1] * inv), pack_bf16(x[2] * inv, x[3] * inv));
          else
            *reinterpret_cast<float4*>(po + 32 * b) = make_float4(x[0], x[1], x[2], x[3]);
        }
        if (splits > 1 && gid == 0)
          p.part_ml[slot_of(mine) * G + g] = make_float2(m[nt][cc], l[nt][cc]);
      }
    if (splits == 1) continue;

    // ---- join: groups of `fan` splits, then the groups ----
    int fan = kFan;
    while (fan * fan < splits) fan += 8;
    int first = mine / fan * fan, step = 1, count = min(fan, splits - first);
    int32_t* ctr = p.count1 + slot_of(first);
    const int groups = (splits + fan - 1) / fan;
    bool top_level = groups == 1;
    while (true) {
      __threadfence();
      __syncwarp();
      int last = 0;
      if (lane == 0) last = atomicAdd(ctr, 1) == count - 1;
      if (!__shfl_sync(0xffffffffu, last, 0)) break;
      __threadfence();
      if (lane == 0) *ctr = 0;  // complete: ready for the next call
      // every lane takes whole float4s of the G x D partials, four at a time
      const int vecs = G * (D / 4);
      for (int v0 = lane; v0 < vecs; v0 += 128) {
        float4 acc[4];
        float big[4], den[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
          big[i] = -INFINITY;
          den[i] = 0.f;
        }
        for (int k = 0; k < count; k += 2) {
          float4 x[2][4];
          float2 ml[2][4];
#pragma unroll
          for (int kk = 0; kk < 2; ++kk)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int v = v0 + 32 * i;
              ml[kk][i] = make_float2(-INFINITY, 0.f);
              x[kk][i] = make_float4(0.f, 0.f, 0.f, 0.f);
              if (v < vecs && k + kk < count) {
                const int64_t row = slot_of(first + (k + kk) * step) * G + v / (D / 4);
                ml[kk][i] = __ldcg(p.part_ml + row);
                x[kk][i] = __ldcg(reinterpret_cast<const float4*>(p.part_o + row * D) + v % (D / 4));
              }
            }
#pragma unroll
          for (int kk = 0; kk < 2; ++kk)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float mn = fmaxf(big[i], ml[kk][i].x);
              const float wa = big[i] == mn ? 1.f : exp2_approx(big[i] - mn);
              const float wb = ml[kk][i].x == mn ? 1.f : exp2_approx(ml[kk][i].x - mn);
              big[i] = mn;
              den[i] = den[i] * wa + ml[kk][i].y * wb;
              acc[i].x = acc[i].x * wa + x[kk][i].x * wb;
              acc[i].y = acc[i].y * wa + x[kk][i].y * wb;
              acc[i].z = acc[i].z * wa + x[kk][i].z * wb;
              acc[i].w = acc[i].w * wa + x[kk][i].w * wb;
            }
        }
        __syncwarp();  // the first split's slot, read above by every lane, takes the group's sum
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int v = v0 + 32 * i;
          if (v >= vecs) continue;
          const int g = v / (D / 4), d4 = v % (D / 4);
          if (top_level) {
            const float inv = 1.f / den[i];
            *reinterpret_cast<uint2*>(p.out + tok * p.out_stride +
                                      static_cast<int64_t>(h * G + g) * D + 4 * d4) =
                make_uint2(pack_bf16(acc[i].x * inv, acc[i].y * inv),
                           pack_bf16(acc[i].z * inv, acc[i].w * inv));
          } else {
            const int64_t row = slot_of(first) * G + g;
            reinterpret_cast<float4*>(p.part_o + row * D)[d4] = acc[i];
            if (d4 == 0) p.part_ml[row] = make_float2(big[i], den[i]);
          }
        }
      }
      if (top_level) break;
      // this warp's group is done: the groups' own count
      top_level = true;
      first = 0;
      step = fan;
      count = groups;
      ctr = p.count2 + slot_of(0);
    }
  }
}

template <int D, int NT>
cudaError_t launch_t(Params p, int sms, cudaStream_t stream) {
  constexpr int kWarps = warps_per_cta<NT>();
  constexpr size_t kRing = static_cast<size_t>(kWarps) * 4 * mx_chunk_bytes(D);  // one stage of all warps
  constexpr size_t kLimit = 232448 - 1024;                                       // static shared memory aside
  const size_t plan = 4 * (static_cast<size_t>(p.num_reqs) + 1);
  // three stages keep about 139 KB in flight on an SM; two where the plan of
  // a very large batch needs the room
  p.stages = 3 * kRing + plan <= kLimit ? 3 : 2;
  const size_t smem = p.stages * kRing + plan;
  cudaError_t e = raise_smem_limit_once<decode_mxfp4_kernel<D, NT>>(kLimit);
  if (e != cudaSuccess) return e;
  return launch_programmatic(decode_mxfp4_kernel<D, NT>, dim3(static_cast<unsigned>(sms)),
                             dim3(kWarps * 32), smem, stream, p);
}

}  // namespace

int64_t decode_mxfp4_workers(int sms) { return static_cast<int64_t>(sms) * warps_per_cta<1>(); }

cudaError_t launch_decode_mxfp4(const AttnArgs& a, const MxDecodeScratch& ws, int sms,
                                cudaStream_t stream) {
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
  p.count1 = ws.count1;
  p.count2 = ws.count2;
  p.part_ml = reinterpret_cast<float2*>(ws.part_ml);
  p.part_o = ws.part_o;
  p.stages = 0;
  const bool wide = p.group > 8;
  if (a.head_dim == 128)
    return wide ? launch_t<128, 2>(p, sms, stream) : launch_t<128, 1>(p, sms, stream);
  if (a.head_dim == 64)
    return wide ? launch_t<64, 2>(p, sms, stream) : launch_t<64, 1>(p, sms, stream);
  return cudaErrorNotSupported;
}

}  // namespace pkv
