// Split-KV decode attention (query length 1) over the 8-bit paged cache.
//
// For a decode request r, query head h of KV head g and its keys j < seq_len:
//   out = sum_j softmax_j(scale <q, K_j>) V_j,
// K and V the values that codes and power-of-two scales stand for (fp8.cuh).
//
// Work split.  As in the 4-bit decode: the decode requests' blocks form one sequence, cut
// into Q equal ranges; a range is walked by one warp per KV head, the warps of a range side
// by side in one CTA.  A block is one unit, the change to a request kF8RequestCost ahead of
// its blocks.  A request that crosses ranges leaves one partial (m, l, o / l) per range and
// head in the workspace, and a second kernel joins them,
//   M = max_s (m_s + floor(log2 l_s)),  w_s = 2^(m_s - M) l_s,  out = sum_s w_s (o_s / l_s) / sum_s w_s,
// in an order that the ranges fix: no counters, no atomics, the same bits every time.
//
// Data movement.  A warp keeps its own ring of stages, each one block of its head (4.1 KB at
// head_dim 128), filled by two bulk copies: a head's chunk of a block, codes and scale, is
// contiguous.  The fetch cursor runs ahead of the compute over request boundaries, so a new
// request costs no bubble.
//
// Compute.  S^T = K Q^T and O^T += V^T P^T are m16n8k16 bfloat16 products with the query
// heads of the KV head as N and float32 accumulators; 16 tokens are one block, so a scale is
// the same for all lanes.  The cache's byte order is the A fragments', and a code is exact in
// bfloat16.
//   - K's scale multiplies the scores in float32.  The queries of a head are brought to
//     [1, 2) by a power of two first, so that sums over codes are below 2^17 whatever q and
//     the scale are; nothing of an element is lost above 2^-126 of the head's largest.  The
//     exponents of q, of K's scale and of the softmax's are added up before they multiply.
//   - V's scale multiplies its codes, exactly, so weights and values go into the product as
//     they are: weights are bfloat16 (8 bits) over 102 binades below the largest, values have no
//     other limit than that float32 sums hold.
//   - The sums are those of the rounded weights, so what rounding does to all of a row's weights
//     cancels (64 requests: errors of 0.0018 of the result, where its own rounding is 0.0016; with
//     the unrounded sums 0.0022; weights of two bfloat16 reach 0.0016, but took 337 us for 8
//     requests of 131072 tokens where these took 326).
//   - The reference m of the weights lies 2^24 above a score that was the largest and moves when
//     one exceeds that by 2^32 (by 2 where the block's values are large, kF8Loud): the common
//     block needs a vote, and no shuffle, and sums stay finite for any values there are.
//
// What bounds it.  8 requests of 131072 tokens with 64 query and 8 KV heads of 128 take 325
// us, 6.6 TB/s, 97 to 98 % of the copy rate.  64 requests of 128 to 4096 tokens (32/8 heads of
// 128, 284 MB) take 55.3 us.  By the kernel's clocks (when blocks still made the plan together)
// the plan was there at 2.0 us, the first data at 6.9, the last block at 41 to 50.4, median 47.4:
// 7.0 TB/s in between; the start and the join are the rest.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "fp8.cuh"
#include "kernels.h"
#include "pkv_device.cuh"

namespace pkv {

namespace {

constexpr int kMinUnits = 3;     // units in a range, nearly: at least 2, more than kF8RequestCost
// Weights are 2^(score - m): a new reference m puts the largest at 2^kLargest, and m moves when
// one exceeds 2^kMost, or in a block of large values 2^kMostLoud: sums over 2^22 keys of those
// stay finite, over the others' always.
constexpr float kLargest = -24.f, kMost = 8.f, kMostLoud = -23.f;
constexpr int kMaxStages = 6;
constexpr int kWarpPlan = 32;    // requests up to which a warp makes the plan for itself

template <int NT>
constexpr int warps_per_cta() { return NT == 1 ? 16 : 8; }
// Ranges that a CTA of `warps` warps walks at once; with more KV heads than
// warps, a warp walks its one range once per head it has.
__host__ __device__ constexpr int ranges_per_cta(int warps, int hkv) {
  return warps > hkv ? warps / hkv : 1;
}

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
  float scale_m;       // scale log2(e) = scale_m 2^scale_e, scale_m zero or of magnitude [1, 2]
  int32_t scale_e;
  uint32_t* err;
  int2* plan;        // [num_reqs]: what there is to join (see slot_of)
  float2* part_ml;   // [2 * ranges][hkv][group]
  float* part_o;     // [2 * ranges][hkv][group][D], divided by l
  int32_t stages;
};

__device__ __forceinline__ void prefetch_l2(const void* p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}

// D += A B, m16n8k16, bfloat16 inputs, float32 accumulators.  Not volatile, so that
// the compiler may interleave independent products.
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 h = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                   *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&h);
}
// The four codes of a word as two bfloat16 pairs.
__device__ __forceinline__ void codes_to_bf16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  float x[4];
  e4m3x4_to_f32(w, x);
  lo = pack_bf16(x[0], x[1]);
  hi = pack_bf16(x[2], x[3]);
}

// The partial of range q of a request: slot 2q, except that a request which
// starts inside the range (after its first block) has slot 2q + 1.  A range
// leaves two partials at most, of the request it begins in and of the one it
// ends in.
__device__ __forceinline__ int slot_of(int q, bool starts_inside) {
  return 2 * q + (starts_inside ? 1 : 0);
}

// A position in a range: `run` blocks of request r to go, then `rest` more units
// of later requests.
struct Cursor {
  int r, run, rest;
  // the next request's part; run is 0 where the range ends before its blocks
  __device__ __forceinline__ void next_run(const int32_t* prefix) {
    do ++r; while (prefix[r + 1] == prefix[r]);
    const int units = prefix[r + 1] - prefix[r];
    const int take = rest < units ? rest : units;
    rest -= take;
    run = take > kF8RequestCost ? take - kF8RequestCost : 0;
  }
};

// Unit where range q of Q begins, floor(q N / Q), from N / Q and N % Q.
__device__ __forceinline__ int range_begin(int q, int Q, int quot, int rem) {
  return q * quot + static_cast<int>(static_cast<uint32_t>(q * rem) / static_cast<uint32_t>(Q));
}

template <int D, int NT>
__global__ void __launch_bounds__(warps_per_cta<NT>() * 32, 1)
    decode_fp8_kernel(const Params p) {
  constexpr int KS = D / 16;                       // k-steps of S^T, m-tiles of O^T
  constexpr int NV = D / 32;                       // vectors of codes of a lane, K or V
  constexpr int P = D / 8;                         // dimensions of a lane's V
  constexpr uint32_t kChunk = f8_chunk_bytes(D);   // one head of one block
  constexpr uint32_t kStage = 2 * kChunk;          // K then V
  constexpr int kWarps = warps_per_cta<NT>();
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t full[kWarps * kMaxStages];
  __shared__ int32_t warp_sum[kWarps];
  int32_t* prefix = reinterpret_cast<int32_t*>(smem + static_cast<size_t>(p.stages) * kWarps * kStage);

  // the kernel before may write q, the cache, out or the metadata
  grid_dependency_wait();
  if (threadIdx.x == 0) grid_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gid = lane >> 2, tid = lane & 3;
  const int R = p.num_reqs;
  const int stages = p.stages;
  uint64_t* bars = full + warp * kMaxStages;
  if (lane == 0) {
    for (int s = 0; s < stages; ++s) mbar_init(&bars[s], 1);
    fence_mbar_init();
  }

  // ---- plan: units of every decode request and their prefix sum ----
  auto units_of = [&](int r, bool report) -> int {
    const int q0 = __ldg(p.qsl + r), q1 = __ldg(p.qsl + r + 1);
    const int seq = __ldg(p.seq_lens + r), nc = __ldg(p.num_computed + r);
    // (unsigned: offsets that are garbage may be anything apart)
    if (static_cast<uint32_t>(q1) - static_cast<uint32_t>(q0) != 1u) return 0;
    const int nb = (seq - 1) / kF8Block + 1;
    if (nc < 0 || nc > 0x7ffffffe || seq != nc + 1 || nb > p.bt_width || q0 < 0 || q0 >= p.num_tokens) {
      if (report && blockIdx.x == 0) atomicOr(p.err, PKV_ERR_METADATA);
      return 0;
    }
    return nb > 0 ? nb + kF8RequestCost : 0;
  };
  if (R <= kWarpPlan) {
    // every warp makes all of it (and writes what the others write), so none waits for another.
    // Requests of 100 to 300 tokens, 32/8 heads of 128, each way and by the CTA together: 1 10.3
    // and 10.6 us, 16 11.5 and 12.3, 32 11.7 and 13.0; with up to 128 to a warp, four a lane, 33
    // 14.0 and 13.9, 64 17.1 and 16.5, 128 23.2 and 20.6.
    int inc = lane < R ? units_of(lane, warp == 0) : 0;
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, inc, x);
      if (lane >= x) inc += y;
    }
    if (lane < R) prefix[lane + 1] = inc;
    if (lane == 0) prefix[0] = 0;
    __syncwarp();
  } else {
    for (int r = threadIdx.x; r < R; r += blockDim.x) prefix[r + 1] = units_of(r, true);
    __syncthreads();
    // each thread sums its own run of requests, then the CTA scans
    const int per = (R + kWarps * 32 - 1) / (kWarps * 32);
    const int first = min(R, static_cast<int>(threadIdx.x) * per), last = min(R, first + per);
    int sum = 0;
    for (int r = first; r < last; ++r) sum += prefix[r + 1];
    int inc = sum;
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, inc, x);
      if (lane >= x) inc += y;
    }
    if (lane == 31) warp_sum[warp] = inc;
    __syncthreads();
    inc -= sum;
    for (int w = 0; w < warp; ++w) inc += warp_sum[w];
    if (threadIdx.x == 0) prefix[0] = 0;
    for (int r = first; r < last; ++r) {
      inc += prefix[r + 1];
      prefix[r + 1] = inc;
    }
    __syncthreads();
  }
  const int N = prefix[R];
  const int per_cta = ranges_per_cta(kWarps, p.hkv);
  const int Q = min((N + kMinUnits - 1) / kMinUnits, static_cast<int>(gridDim.x) * per_cta);
  const int quot = N / max(Q, 1), rem = N % max(Q, 1);
  // what the join has to do for each request: its first range, and twice the
  // number of its ranges plus whether it starts inside the first; 0: nothing
  auto write_plan = [&]() {
    for (int r = threadIdx.x * gridDim.x + blockIdx.x; r < R; r += blockDim.x * gridDim.x) {
      const int run0 = prefix[r], run1 = prefix[r + 1];
      int2 to_join = make_int2(0, 0);
      if (run1 > run0) {
        // the range of unit x: the largest q with floor(qN/Q) <= x
        auto range_of = [&](int x) {
          return static_cast<int>(((static_cast<int64_t>(x) + 1) * Q - 1) / N);
        };
        const int qf = range_of(run0 + kF8RequestCost), ql = range_of(run1 - 1);
        const bool inside = run0 > range_begin(qf, Q, quot, rem);
        if (ql > qf) to_join = make_int2(qf, 2 * (ql - qf + 1) + (inside ? 1 : 0));
      }
      p.plan[r] = to_join;
    }
  };
  // few ranges: one per SM first
  const int sub = warp / p.hkv;
  const int me = sub * static_cast<int>(gridDim.x) + static_cast<int>(blockIdx.x);
  if (sub >= per_cta || me >= Q) {
    write_plan();
    return;
  }
  const int u0 = range_begin(me, Q, quot, rem), u1 = range_begin(me + 1, Q, quot, rem);

  const uint64_t block_bytes = static_cast<uint64_t>(p.hkv) * kChunk;
  uint8_t* ring = smem + static_cast<size_t>(warp) * stages * kStage;
  const uint32_t num_blocks = static_cast<uint32_t>(p.num_blocks);
  const int G = p.group;
  // the ring: the stages filled and read next, the parity of the latter, and which hold a
  // block that is not in the pool
  int fill = 0, stage = 0;
  uint32_t parity = 0u, missing = 0u;
  bool alive = true;
  // one pass, or with more KV heads than warps one for each head of this warp
  for (int h = warp - sub * p.hkv; h < p.hkv && alive; h += kWarps) {
  const uint8_t* k_src = p.key_cache + static_cast<uint64_t>(h) * kChunk;
  const uint8_t* v_src = p.value_cache + static_cast<uint64_t>(h) * kChunk;
  // the fetch cursor, the table entries after it, and the next stage's id
  Cursor next;
  const int32_t* row;
  uint32_t id = 0u;
  int first_j;  // the block of its request that the run begins with
  {
    int lo = 0, hi = R;  // prefix[lo] <= u0 < prefix[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (prefix[mid] <= u0) lo = mid; else hi = mid;
    }
    next.r = lo;
    // a range has more units than a request's cost: at least one block comes
    const int end = min(u1, prefix[lo + 1]);
    first_j = max(u0 - prefix[lo] - kF8RequestCost, 0);
    next.run = end - prefix[lo] - kF8RequestCost - first_j;
    next.rest = u1 - end;
    row = p.block_table + static_cast<int64_t>(lo) * p.bt_stride + first_j;
  }
  Cursor at = next;
  int ahead = 0;  // stages that are filled and not read
  // the query heads of the request that the cursor has come to are wanted some stages on
  auto want_queries = [&]() {
    if (lane * 128 < 2 * G * D)
      prefetch_l2(p.q + static_cast<int64_t>(__ldg(p.qsl + next.r)) * p.q_stride +
                  static_cast<int64_t>(h * G) * D + lane * 64);
  };
  auto fetch = [&]() {
    if (next.run <= 0) return;
    const bool in = id < num_blocks;
    if (lane == 0) {
      if (in) {
        uint8_t* dst = ring + fill * kStage;
        mbar_arrive_expect_tx(&bars[fill], kStage);
        bulk_load(dst, k_src + id * block_bytes, kChunk, &bars[fill]);
        bulk_load(dst + kChunk, v_src + id * block_bytes, kChunk, &bars[fill]);
      } else {
        atomicOr(p.err, PKV_ERR_BLOCK_ID);
        mbar_arrive(&bars[fill]);
      }
    }
    missing = in ? missing & ~(1u << fill) : missing | (1u << fill);
    fill = fill + 1 == stages ? 0 : fill + 1;
    ++ahead;
    ++row;
    if (--next.run == 0 && next.rest > 0) {
      next.next_run(prefix);
      row = p.block_table + static_cast<int64_t>(next.r) * p.bt_stride;
      want_queries();
    }
    if (next.run > 0) id = static_cast<uint32_t>(__ldg(row));
  };
  id = static_cast<uint32_t>(__ldg(row));
  want_queries();
  __syncwarp();
  for (int s = 0; s < stages - 1; ++s) fetch();
  if (h < kWarps) write_plan();  // with the first bytes on their way
  while (true) {
    // ======================= the range's part of one request =======================
    const int r = at.r;

    // B fragments of Q^T: k-step 4 a + i of lane tid holds dims 64 a + 16 tid + 4 i .. + 3, the
    // order of the K codes
    uint32_t qb[NT][KS][2];
    int qe[NT][2];  // of heads 2 tid, + 1: the exponent that undoes the power of two, and the scale's
    bool far = false;  // whether with some scale of K 2^qe may be no normal float32
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int head = nt * 8 + gid;
      const __nv_bfloat16* qrow =
          p.q + static_cast<int64_t>(__ldg(p.qsl + r)) * p.q_stride + static_cast<int64_t>(h * G + (head < G ? head : 0)) * D;
      uint32_t mx = 0u;
#pragma unroll
      for (int a = 0; a < D / 64; ++a)
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const uint4 w = __ldg(reinterpret_cast<const uint4*>(qrow + 64 * a + 16 * tid + 8 * b));
          const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            mx = max(mx, max(x[i] & 0x7fffu, (x[i] >> 16) & 0x7fffu));
            qb[nt][4 * a + 2 * b + (i >> 1)][i & 1] = head < G ? x[i] : 0u;
          }
        }
      mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      // largest element to [1, 2)
      const int ex = static_cast<int>(min(max(mx >> 7, 1u), 253u));
      const uint32_t up = static_cast<uint32_t>(254 - ex) << 7;  // 2^(127 - ex)
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int i = 0; i < 2; ++i) qb[nt][k][i] = mul_bf16x2(qb[nt][k][i], up * 0x00010001u);
      qe[nt][0] = __shfl_sync(0xffffffffu, ex - 127, 8 * tid) + p.scale_e;
      qe[nt][1] = __shfl_sync(0xffffffffu, ex - 127, 8 * tid + 4) + p.scale_e;
      far |= max(qe[nt][0], qe[nt][1]) > 253 - kF8MaxScale || min(qe[nt][0], qe[nt][1]) < 1 - kF8MinScale;
    }
    far = __any_sync(0xffffffffu, far);

    float o[KS][NT][4];
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < KS; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) o[i][nt][c] = 0.f;
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.f;
    }

    int left = at.run;             // blocks of the run to go
    // tokens the request has from the block's first on
    int valid = __ldg(p.seq_lens + r) - first_j * kF8Block;
    for (; left > 0; --left, valid -= kF8Block) {
      if (!mbar_wait(&bars[stage], parity, p.err)) {
        alive = false;
        break;
      }
      // the stage read last is free: every lane has its values
      __syncwarp();
      fetch();
      const uint8_t* st = ring + stage * kStage;
      const bool zeros = (missing >> stage) & 1u;
      if (++stage == stages) {
        stage = 0;
        parity ^= 1u;
      }
      --ahead;
      const int tokens = min(valid, kF8Block);

      // ---- S^T = K Q^T of the block ----
      uint4 kw[NV], vw[NV];
#pragma unroll
      for (int j = 0; j < NV; ++j) kw[j] = *reinterpret_cast<const uint4*>(st + j * 512 + lane * 16);
#pragma unroll
      for (int j = 0; j < NV; ++j) vw[j] = *reinterpret_cast<const uint4*>(st + kChunk + j * 512 + lane * 16);
      const int ke = f8_scale(st[f8_code_bytes(D)]);
      int ve = f8_scale(st[kChunk + f8_code_bytes(D)]);
      if (zeros) {
        ve = 127;
#pragma unroll
        for (int j = 0; j < NV; ++j) kw[j] = vw[j] = make_uint4(0u, 0u, 0u, 0u);
      }
      float s[NT][4], s2[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 4; ++c) s[nt][c] = s2[nt][c] = 0.f;
#pragma unroll
      for (int a = 0; a < D / 64; ++a) {
        const uint4 x = kw[a], y = kw[a + D / 64];  // tokens gid and gid + 8
        const uint32_t lo[4] = {x.x, x.y, x.z, x.w}, hi[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t a0, a1, a2, a3;
          codes_to_bf16(lo[i], a0, a2);
          codes_to_bf16(hi[i], a1, a3);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma_bf16((i & 1) ? s2[nt] : s[nt], a0, a1, a2, a3, qb[nt][4 * a + i][0], qb[nt][4 * a + i][1]);
        }
      }
      float f[NT][2];  // what brings the sums to log2 units
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int c = 0; c < 4; ++c) s[nt][c] += s2[nt][c];
#pragma unroll
        for (int cc = 0; cc < 2; ++cc) f[nt][cc] = __uint_as_float(static_cast<uint32_t>(qe[nt][cc] + ke) << 23) * p.scale_m;
      }
      if (far) {
        // of q, K and the scale maybe only the product is within float32: the sums take what one
        // power of two does not hold, so what they become lies between them and the scores
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int cc = 0; cc < 2; ++cc) {
            const int e = qe[nt][cc] + ke - 127, last = min(max(e, -126), 126);
            const int first = min(max(e - last, -126), 126), then = min(max(e - last - first, -126), 126);
            f[nt][cc] = f8_pow2(last) * p.scale_m;
            s[nt][cc] = s[nt][cc] * f8_pow2(first) * f8_pow2(then);
            s[nt][2 + cc] = s[nt][2 + cc] * f8_pow2(first) * f8_pow2(then);
          }
      }
      if (tokens < kF8Block) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (gid + (c >> 1) * 8 >= tokens) s[nt][c] = -INFINITY;
        // (codes of tokens past the end may be NaN)
        uint32_t keep = 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (2 * tid + (i >> 1) * 8 + (i & 1) < tokens) keep |= 0xffu << (8 * i);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          vw[j].x &= keep;
          vw[j].y &= keep;
          vw[j].z &= keep;
          vw[j].w &= keep;
        }
      }

      // ---- online softmax per head column ----
      float mx[NT][2];
      const float most = ve > kF8Loud ? kMostLoud : kMost;
      bool grow = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (!(tokens < kF8Block && gid + (c >> 1) * 8 >= tokens)) s[nt][c] *= f[nt][c & 1];
#pragma unroll
        for (int cc = 0; cc < 2; ++cc) {
          mx[nt][cc] = fmaxf(s[nt][cc], s[nt][2 + cc]);
          grow |= mx[nt][cc] > m[nt][cc] + most;
        }
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
            const float mn = fmaxf(m[nt][cc], x - kLargest);
            const float alpha = mn == m[nt][cc] ? 1.f : exp2_approx(m[nt][cc] - mn);
            m[nt][cc] = mn;
            l[nt][cc] *= alpha;
#pragma unroll
            for (int i = 0; i < KS; ++i) {
              o[i][nt][cc] *= alpha;
              o[i][nt][2 + cc] *= alpha;
            }
          }
      }
      // P^T fragments: the weights of tokens 2 tid, + 1 (and + 8) for head gid, and their sums
      uint32_t pt[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float e[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) e[c] = exp2_approx(s[nt][c] - m[nt][c & 1]);
        const uint32_t w0 = pack_bf16(e[0], e[1]), w1 = pack_bf16(e[2], e[3]);
        // (the rounded ones: what rounding does to all of a row's weights cancels)
        l[nt][0] += __uint_as_float(w0 << 16) + __uint_as_float(w1 << 16);
        l[nt][1] += __uint_as_float(w0 & 0xffff0000u) + __uint_as_float(w1 & 0xffff0000u);
        pt[nt][0] = transpose_8x8(w0);
        pt[nt][1] = transpose_8x8(w1);
      }
      // ---- O^T += V^T P^T ----
      const uint32_t vs = static_cast<uint32_t>(ve << 7) * 0x00010001u;  // 2^(ve - 127)
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const uint32_t w[4] = {vw[j].x, vw[j].y, vw[j].z, vw[j].w};
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          uint32_t a0, a1, a2, a3;  // dims 4 j + 2 x and + 1 of the lane's
          codes_to_bf16(w[2 * x], a0, a2);
          codes_to_bf16(w[2 * x + 1], a1, a3);
          a0 = mul_bf16x2(a0, vs);
          a1 = mul_bf16x2(a1, vs);
          a2 = mul_bf16x2(a2, vs);
          a3 = mul_bf16x2(a3, vs);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma_bf16(o[2 * j + x][nt], a0, a1, a2, a3, pt[nt][0], pt[nt][1]);
        }
      }
    }
    if (!alive) break;

    // ======================= end of the range's part of the request =======================
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
    const bool inside = prefix[r] > u0;
    const bool whole = prefix[r] + kF8RequestCost >= u0 && prefix[r + 1] <= u1;
    const int64_t mine = static_cast<int64_t>(slot_of(me, inside)) * p.hkv + h;
    const int64_t tok = __ldg(p.qsl + r);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int cc = 0; cc < 2; ++cc) {
        const int g = nt * 8 + 2 * tid + cc;
        if (g >= G) continue;
        // o[i]: dims P gid + 2 i (elements 0, 1) and + 1 (2, 3)
        const float inv = 1.f / l[nt][cc];
        __nv_bfloat16* dst = p.out + tok * p.out_stride + static_cast<int64_t>(h * G + g) * D + P * gid;
        float* po = p.part_o + (mine * G + g) * D + P * gid;
#pragma unroll
        for (int b = 0; b < KS / 4; ++b) {
          float x[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = o[4 * b + (i >> 1)][nt][2 * (i & 1) + cc] * inv;
          if (whole) {
            *reinterpret_cast<uint4*>(dst + 8 * b) = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]),
                                                                pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
          } else {
            *reinterpret_cast<float4*>(po + 8 * b) = make_float4(x[0], x[1], x[2], x[3]);
            *reinterpret_cast<float4*>(po + 8 * b + 4) = make_float4(x[4], x[5], x[6], x[7]);
          }
        }
        if (!whole && gid == 0) p.part_ml[mine * G + g] = make_float2(m[nt][cc], l[nt][cc]);
      }
    if (at.rest == 0) break;
    at.next_run(prefix);
    if (at.run == 0) break;
    first_j = 0;
  }
  // a wait that gave up leaves copies in flight: they land before the CTA exits
  if (!alive)
    for (; ahead > 0; --ahead) {
      mbar_wait(&bars[stage], parity, nullptr);
      if (++stage == stages) {
        stage = 0;
        parity ^= 1u;
      }
    }
  }
}

// log2 of a range's weight 2^m l, to the binade.
__device__ __forceinline__ float range_weight(float2 ml) {
  return ml.x + static_cast<float>(static_cast<int>(__float_as_uint(ml.y) >> 23) - 127);
}

// Joins the partials of every request that crosses ranges.  kLanes lanes take 4 kLanes
// dimensions of one (request, query head); the groups of a warp, or with kTogether of all
// warps of the CTA, take the ranges in turn, kBatch loads of a lane in flight, and add up at
// the end.
template <int D, int kLanes, bool kTogether>
__global__ void __launch_bounds__(256, 4) join_fp8_kernel(const Params p) {
  grid_dependency_wait();  // the decode's partials
  if (threadIdx.x == 0) grid_launch_dependents();
  constexpr int kBatch = 4, kItems = D / (4 * kLanes), kGroups = 32 / kLanes;
  constexpr int kParts = kTogether ? 8 * kGroups : kGroups;
  __shared__ float4 part_acc[kTogether ? 8 : 1][kLanes];
  __shared__ float2 part_sum[kTogether ? 8 : 1];
  const int G = p.group, H = p.hkv * G;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, part = (kTogether ? warp * kGroups : 0) + lane / kLanes;
  const int per_req = H * kItems;  // items of a request
  const int64_t total = static_cast<int64_t>(p.num_reqs) * per_req;
  const int64_t first = kTogether ? blockIdx.x : static_cast<int64_t>(blockIdx.x) * 8 + warp;
  for (int64_t i = first; i < total; i += static_cast<int64_t>(gridDim.x) * (kTogether ? 1 : 8)) {
    const int r = static_cast<int>(i / per_req);
    const int item = static_cast<int>(i - static_cast<int64_t>(r) * per_req);
    const int2 to_join = __ldcg(p.plan + r);
    if (to_join.y == 0) continue;  // written by the decode itself, or no decode row
    const int splits = to_join.y >> 1;
    const bool inside = to_join.y & 1;
    const int head = item / kItems, d4 = (item % kItems) * kLanes + (lane & (kLanes - 1));
    const int h = head / G, g = head - h * G;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float big = -INFINITY, den = 0.f;
    for (int k0 = part; k0 < splits; k0 += kParts * kBatch) {
      float2 ml[kBatch];
      float4 x[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int q = k0 + kParts * k;
        ml[k] = make_float2(-INFINITY, 0.f);
        x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (q < splits) {
          const int64_t at =
              (static_cast<int64_t>(slot_of(to_join.x + q, q == 0 && inside)) * p.hkv + h) * G + g;
          ml[k] = __ldcg(p.part_ml + at);
          x[k] = __ldcg(reinterpret_cast<const float4*>(p.part_o + at * D) + d4);
        }
      }
      float mx = big;
#pragma unroll
      for (int k = 0; k < kBatch; ++k) mx = fmaxf(mx, range_weight(ml[k]));
      const float keep = big == mx ? 1.f : exp2_approx(big - mx);
      big = mx;
      den *= keep;
      acc.x *= keep;
      acc.y *= keep;
      acc.z *= keep;
      acc.w *= keep;
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        if (k0 + kParts * k >= splits) break;
        // 2^-13 at most: values near float32's end of as many ranges as there are, 16 an SM, may
        // be added up
        const float w = exp2_approx(ml[k].x - mx - 14.f) * ml[k].y;
        den += w;
        acc.x = fmaf(x[k].x, w, acc.x);
        acc.y = fmaf(x[k].y, w, acc.y);
        acc.z = fmaf(x[k].z, w, acc.z);
        acc.w = fmaf(x[k].w, w, acc.w);
      }
    }
#pragma unroll
    for (int x = kLanes; x < 32; x <<= 1) {
      const float mx = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, x));
      const float w = big == mx ? 1.f : exp2_approx(big - mx);
      big = mx;
      den *= w;
      den += __shfl_xor_sync(0xffffffffu, den, x);
      float* a = &acc.x;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        a[c] *= w;
        a[c] += __shfl_xor_sync(0xffffffffu, a[c], x);
      }
    }
    if constexpr (kTogether) {
      __syncthreads();  // the item before is read
      if (lane < kLanes) part_acc[warp][lane] = acc;
      if (lane == 0) part_sum[warp] = make_float2(big, den);
      __syncthreads();
      if (warp == 0) {
        float mx = -INFINITY;
#pragma unroll
        for (int w = 0; w < 8; ++w) mx = fmaxf(mx, part_sum[w].x);
        den = 0.f;
        acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < 8; ++w) {
          const float2 sum = part_sum[w];
          const float f = sum.x == mx ? 1.f : exp2_approx(sum.x - mx);
          const float4 x = part_acc[w][lane & (kLanes - 1)];
          den = fmaf(sum.y, f, den);
          acc.x = fmaf(x.x, f, acc.x);
          acc.y = fmaf(x.y, f, acc.y);
          acc.z = fmaf(x.z, f, acc.z);
          acc.w = fmaf(x.w, f, acc.w);
        }
      }
    }
    if (part == 0) {
      const float inv = 1.f / den;
      const int64_t tok = __ldg(p.qsl + r);
      *reinterpret_cast<uint2*>(p.out + tok * p.out_stride + static_cast<int64_t>(head) * D + 4 * d4) =
          make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
    }
  }
}

template <int D, int NT>
cudaError_t launch_t(Params p, int sms, cudaStream_t stream) {
  constexpr int kWarps = warps_per_cta<NT>();
  constexpr size_t kRing = static_cast<size_t>(kWarps) * 2 * f8_chunk_bytes(D);  // one stage of all warps
  constexpr size_t kLimit = 232448 - 2048;                                       // static shared memory aside
  const size_t plan = 4 * (static_cast<size_t>(p.num_reqs) + 1);
  // as many stages as there is room for: 3 of 66 KB at head_dim 128, 6 at 64
  p.stages = kMaxStages;
  while (p.stages > 2 && p.stages * kRing + plan > kLimit) --p.stages;
  const size_t smem = p.stages * kRing + plan;
  if (smem > kLimit) return cudaErrorInvalidValue;
  cudaError_t e = raise_smem_limit_once<decode_fp8_kernel<D, NT>>(kLimit);
  if (e != cudaSuccess) return e;
  e = launch_programmatic(decode_fp8_kernel<D, NT>, dim3(static_cast<unsigned>(sms)),
                          dim3(kWarps * 32), smem, stream, p);
  if (e != cudaSuccess) return e;
  // Few requests have many ranges each: eight lanes take 32 dimensions, and the warps of a CTA
  // an item together (one request of 30000 tokens, 16/4 heads of 64: 36 us with a warp an
  // item) or, where that is more than a wave of warps, each its own, four ranges at a time;
  // where that is too, more lanes and fewer ranges.
  const int64_t heads = static_cast<int64_t>(p.num_reqs) * p.hkv * p.group;
  const int64_t wave = 32 * static_cast<int64_t>(sms);
  constexpr int kWide = D / 4;
  const int lanes = heads * (D / 32) <= wave ? 8 : heads * (D / 64) <= wave ? 16 : kWide;
  const int64_t items = heads * (D / (4 * lanes));
  const bool together = lanes == 8 && 8 * items <= wave;
  const int64_t grid = together ? items : (items + 7) / 8;
  return launch_programmatic(together      ? join_fp8_kernel<D, 8, true>
                             : lanes == 8  ? join_fp8_kernel<D, 8, false>
                             : lanes == 16 ? join_fp8_kernel<D, 16, false>
                                           : join_fp8_kernel<D, kWide, false>,
                             dim3(static_cast<unsigned>(grid < wave / 4 ? grid : wave / 4)),
                             dim3(256), 0, stream, p);
}

}  // namespace

int64_t decode_fp8_slots(int sms, int num_kv_heads) {
  return 2 * static_cast<int64_t>(sms) * ranges_per_cta(warps_per_cta<1>(), num_kv_heads) * num_kv_heads;
}

cudaError_t launch_decode_fp8(const AttnArgs& a, const MxDecodeScratch& ws, int sms,
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
  int e;
  p.scale_m = static_cast<float>(2.0 * std::frexp(static_cast<double>(a.scale) * 1.4426950408889634, &e));
  p.scale_e = e - 1;
  p.err = a.err;
  p.plan = reinterpret_cast<int2*>(ws.plan);
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
