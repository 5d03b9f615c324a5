// Split-KV decode attention (query length 1) over the 4-bit paged cache.
//
// For a decode request r, query head h of KV head g and its keys j < seq_len:
//   out = sum_j softmax_j(scale <q, K_j>) V_j,
// K and V the values that codes and power-of-two scales stand for (mxfp4.cuh).
//
// Work split.  The decode requests' blocks form one sequence, cut into Q equal
// ranges; a range is walked by one warp per KV head, the warps of a range side by
// side in one CTA, so that every warp has the same work whatever the context
// lengths, no warp waits for another, and a block's heads are fetched together.
// Work is counted in units: a block is one, and the change to a request
// kMxRequestCost, ahead of its blocks, so N = sum (blocks + kMxRequestCost) and
// range q is the units [floor(qN/Q), floor((q+1)N/Q)).  (64 requests of some 2000
// tokens, 8 KV heads of 128: counting blocks alone, warps with no change were
// through after 31.5 us, those with one after 34.3, with two after 37.1.)  A request that crosses ranges leaves one
// partial (m, l, o / l) per range and head in the workspace, and a second kernel
// joins them,
//   M = max_s (m_s + floor(log2 l_s)),  w_s = 2^(m_s - M) l_s,  out = sum_s w_s (o_s / l_s) / sum_s w_s,
// in an order that the ranges fix: no counters, no atomics, the same bits every
// time.  (Joining in this kernel, by the warp that
// came last, took about 18 us of a 230 us call: one warp reads the partials of
// a request at the latency of L2.)
//
// Data movement.  A warp keeps its own ring of stages, each two blocks' worth of
// its head (4.3 KiB at head_dim 128), filled by 16-byte cp.async: a head's
// chunk of a block is contiguous, K and V.  The fetch cursor runs ahead of the
// compute over request boundaries, so a new request costs no bubble.
//
// Compute.  S^T = K Q^T and O^T += V^T P^T are m16n8k16 f16 products with the
// query heads of the KV head as N, float32 accumulators.
//   - Codes become f16 by one conversion per pair and go straight into the A
//     fragment: the cache's byte order is the fragment's.
//   - Q is brought to f16 by an exact power of two per head.  f16 holds the 8
//     bits of a bfloat16 over 30 binades below the head's largest element, so
//     what is lost is below 2^-38 of it.
//   - K scales multiply the partial sums of each group of 32 dimensions, in
//     float32.  Those sums are up to 2^22, so the scales go 2^24 down first, unless
//     a query is above 2^20 (then keys that this keeps in range have scores beyond it).
//   - V scales go onto the weights: P^T (f16, 11 bits) times 2^(e - base) for
//     each group of dimensions, `base` a running exponent per group.  Scales
//     in the 16 binades from it up, which is nearly always, cost one f16x2
//     product per group; a tile outside the window takes the slow path below,
//     which brings each product of weight and scale to f16 as a whole, relative to
//     the largest of its 16 tokens, group and head.
//   - The reference m of the weights lies 2^11 below a score that was the largest
//     and moves when one exceeds it by 2^14: the common tile needs a vote, and no
//     shuffle.
//
// What bounds it.  8 requests of 131072 tokens with 64 query and 8 KV heads of 128
// take 201 us, 5.7 TB/s, where the copies alone (the same ring, nothing computed)
// reach 6.9: the warps' issue slots are half full, mostly with the conversion of
// codes, and a warp that computes late asks for its next bytes late.  64 requests of
// 128 to 4096 tokens take 42.0 us (150 MB): 2.5 us for the plan, 4.5 until the first
// bytes are there, 27 at 4.8 TB/s, 4 for the join with its launch.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "kernels.h"
#include "mxfp4.cuh"
#include "pkv_device.cuh"

namespace pkv {

namespace {

constexpr int kMinUnits = 8;     // units in a range, nearly: at least 4
// The weights 2^(s - m) of a head: m moves when a weight exceeds 2^kMaxWeight, to where
// it is 2^kLargest.  A V scale multiplies them by 2^(e - base + kLow) with e - base in
// [0, 15]: 2^(14 + 1) at most, inside f16.  Each rounding to f16 is off by 2^-25 at most
// where it is below f16's normal numbers, 2^-36 of the largest weight before the scale
// and, at the window's lower end (where that weight's product is 2^-3), 2^-22 of it
// after: n keys that count for less lose n 2^-21 of the largest product, at worst.
constexpr float kLargest = 11.f;
constexpr float kMaxWeight = 14.f;
constexpr int kLow = -14;
constexpr int kBelow = 11;       // where a new base goes below the largest scale of its tile
constexpr int kTopBase = 239;
// A product of weight and scale, of 16 tokens, that the slow path lets the sums grow by
// (log2), and what it leaves them below when it lowers a base.
constexpr float kMostProduct = 60.f;
constexpr float kMostSum = 1.2379400e27f;  // 2^90

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
  float scale_log2;
  uint32_t* err;
  int2* plan;        // [num_reqs]: what there is to join (see slot_of)
  float2* part_ml;   // [2 * ranges][hkv][group]
  float* part_o;     // [2 * ranges][hkv][group][D], divided by l
  int32_t stages;
};

// 16 bytes from src + kSrc to shared dst + kDst; with `bytes` 0 nothing is read
// and zeros are written.
template <int kDst, int kSrc>
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0 + %2], [%1 + %3], 16;" ::"r"(dst), "l"(src), "n"(kDst),
               "n"(kSrc)
               : "memory");
}
template <int kDst, int kSrc>
__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0 + %2], [%1 + %3], 16, %4;" ::"r"(dst), "l"(src),
               "n"(kDst), "n"(kSrc), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void prefetch_l2(const void* p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// D += A B, m16n8k16, f16 inputs, float32 accumulators.  Not volatile, so that
// the compiler may interleave independent products.
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// D = A B.
__device__ __forceinline__ void mma_f16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                              uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// NaN for NaN.
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 h = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                   *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
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
    run = take > kMxRequestCost ? take - kMxRequestCost : 0;
  }
};

// Unit where range q of Q begins, floor(q N / Q), from N / Q and N % Q.
__device__ __forceinline__ int range_begin(int q, int Q, int quot, int rem) {
  return q * quot + static_cast<int>(static_cast<uint32_t>(q * rem) / static_cast<uint32_t>(Q));
}

// base + a b, 64-bit.
__device__ __forceinline__ const uint8_t* at_offset(const uint8_t* base, uint32_t a, uint32_t b) {
  uint64_t r;
  asm("mad.wide.u32 %0, %1, %2, %3;" : "=l"(r) : "r"(a), "r"(b), "l"(base));
  return reinterpret_cast<const uint8_t*>(r);
}

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
  __shared__ int32_t warp_sum[kWarps];
  int32_t* prefix = reinterpret_cast<int32_t*>(smem + static_cast<size_t>(p.stages) * kWarps * kStage);

  // the kernel before may write q, the cache, out or the metadata
  grid_dependency_wait();
  if (threadIdx.x == 0) grid_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gid = lane >> 2, tid = lane & 3;
  const int R = p.num_reqs;

  // ---- plan: units of every decode request and their prefix sum ----
  for (int r = threadIdx.x; r < R; r += blockDim.x) {
    const int q0 = __ldg(p.qsl + r), q1 = __ldg(p.qsl + r + 1);
    const int seq = __ldg(p.seq_lens + r), nc = __ldg(p.num_computed + r);
    int nb = 0;
    // (unsigned: offsets that are garbage may be anything apart)
    if (static_cast<uint32_t>(q1) - static_cast<uint32_t>(q0) == 1u) {
      nb = (seq - 1) / kMxBlock + 1;
      if (nc < 0 || nc > 0x7ffffffe || seq != nc + 1 || nb > p.bt_width || q0 < 0 ||
          q0 >= p.num_tokens) {
        if (blockIdx.x == 0) atomicOr(p.err, PKV_ERR_METADATA);
        nb = 0;
      }
    }
    prefix[r + 1] = nb > 0 ? nb + kMxRequestCost : 0;
  }
  __syncthreads();
  {
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
        const int qf = range_of(run0 + kMxRequestCost), ql = range_of(run1 - 1);
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

  // ---- the ring ----
  // A lane copies the same 16-byte pieces of every unit: NW of the K codes, NW
  // of the V codes, and (lanes below 2 NB) one of the scales.  V codes of two
  // tokens (128 or 64 bytes) are XOR-swizzled by 16-byte pieces, so that the
  // four token pairs that a quad reads at once hit different banks.
  const uint32_t block_bytes = static_cast<uint32_t>(p.hkv) * kChunk;
  const int stages = p.stages;
  const uint32_t ring = smem_u32(smem) + static_cast<uint32_t>(warp) * stages * kStage;
  const uint32_t ring_end = stages * kStage;
  const bool scale_v = lane >= NB, has_scale = lane < 2 * NB;
  const uint32_t k_dst = ring + lane * 16;
  const uint32_t v_dst =
      ring + kChunk +
      (D == 128 ? (lane >> 3) * 128 + (((lane & 7) ^ (2 * ((lane >> 3) & 3))) << 4)
                : (lane ^ (((lane >> 3) & 1) << 1)) << 4);
  const uint32_t s_dst = ring + kScale + (scale_v ? kChunk + (lane - NB) * 16 : lane * 16);
  const uint32_t num_blocks = static_cast<uint32_t>(p.num_blocks);
  // where this lane finds the V codes of tokens 2 tid and 2 tid + 1 (2 tid + 8
  // and + 9: four pairs on)
  int v_at[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    v_at[i] = D == 128 ? tid * 128 + (((4 * i + (gid >> 1)) ^ (2 * tid)) << 4) + (gid & 1) * 8
                       : tid * 64 + ((i ^ (tid >> 1)) << 5) + gid * 4;
  const int G = p.group;
  // one pass, or with more KV heads than warps one for each head of this warp
  for (int h = warp - sub * p.hkv; h < p.hkv; h += kWarps) {
  const int64_t head_off = static_cast<int64_t>(h) * kChunk;
  const uint8_t* k_src = p.key_cache + head_off + lane * 16;
  const uint8_t* v_src = p.value_cache + head_off + lane * 16;
  const uint8_t* s_src =
      (scale_v ? p.value_cache + (lane - NB) * 16 : p.key_cache + lane * 16) + head_off + kScale;
  // the fetch cursor, the table entries after it, and the next stage's two ids
  Cursor next;
  const int32_t* row;
  uint32_t id0 = 0u, id1 = 0u;
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
    first_j = max(u0 - prefix[lo] - kMxRequestCost, 0);
    next.run = end - prefix[lo] - kMxRequestCost - first_j;
    next.rest = u1 - end;
    row = p.block_table + static_cast<int64_t>(lo) * p.bt_stride + first_j;
  }
  Cursor at = next;
  auto load_ids = [&]() {
    id0 = static_cast<uint32_t>(__ldg(row));
    id1 = next.run > 1 ? static_cast<uint32_t>(__ldg(row + 1)) : 0u;
  };
  auto fetch = [&](uint32_t stage) {
    if (next.run > 0) {
      const uint32_t kd = k_dst + stage, vd = v_dst + stage, sd = s_dst + stage;
      const bool two = next.run > 1;
      if (id0 < num_blocks && id1 < num_blocks) {
        const uint8_t* k = at_offset(k_src, id0, block_bytes);
        const uint8_t* v = at_offset(v_src, id0, block_bytes);
        cp_async16<0, 0>(kd, k);
        cp_async16<0, 0>(vd, v);
        if constexpr (NW == 2) {
          cp_async16<512, 512>(kd, k);
          cp_async16<512, 512>(vd, v);
        }
        if (has_scale) cp_async16<0, 0>(sd, at_offset(s_src, id0, block_bytes));
        if (two) {
          k = at_offset(k_src, id1, block_bytes);
          v = at_offset(v_src, id1, block_bytes);
          cp_async16<kUnit, 0>(kd, k);
          cp_async16<kUnit, 0>(vd, v);
          if constexpr (NW == 2) {
            cp_async16<kUnit + 512, 512>(kd, k);
            cp_async16<kUnit + 512, 512>(vd, v);
          }
          if (has_scale) cp_async16<kUnit, 0>(sd, at_offset(s_src, id1, block_bytes));
        }
      } else {
        // a block id outside the pool: its block reads as zeros
        if (lane == 0) atomicOr(p.err, PKV_ERR_BLOCK_ID);
        for (int u = 0; u < (two ? 2 : 1); ++u) {
          const uint32_t id = u == 0 ? id0 : id1;
          const int n = id < num_blocks ? 16 : 0;
          const uint64_t off = static_cast<uint64_t>(n ? id : 0u) * block_bytes;
          cp_async16_or_zero<0, 0>(kd + u * kUnit, k_src + off, n);
          cp_async16_or_zero<0, 0>(vd + u * kUnit, v_src + off, n);
          if constexpr (NW == 2) {
            cp_async16_or_zero<512, 512>(kd + u * kUnit, k_src + off, n);
            cp_async16_or_zero<512, 512>(vd + u * kUnit, v_src + off, n);
          }
          if (has_scale) cp_async16_or_zero<0, 0>(sd + u * kUnit, s_src + off, n);
        }
      }
      row += 2;
      next.run -= 2;
      if (next.run <= 0 && next.rest > 0) {
        next.next_run(prefix);
        row = p.block_table + static_cast<int64_t>(next.r) * p.bt_stride;
        // its query heads are wanted two stages on
        if (lane * 128 < 2 * G * D)
          prefetch_l2(p.q + static_cast<int64_t>(__ldg(p.qsl + next.r)) * p.q_stride +
                      static_cast<int64_t>(h * G) * D + lane * 64);
      }
      if (next.run > 0) load_ids();
    }
    cp_async_commit();
  };
  load_ids();
  for (int s = 0; s < stages - 1; ++s) fetch(s * kStage);
  if (h < kWarps) write_plan();  // with the first bytes on their way
  uint32_t stage = 0;                          // the stage to compute on
  uint32_t refill = (stages - 1) * kStage;     // the one it takes the next fetch
  while (true) {
    // ======================= the range's part of one request =======================
    const int r = at.r;

    // B fragments of Q^T in f16: k-step 2b + s of lane tid holds dims 32 b + 8
    // tid + 4 s .. + 3, the order of the K codes
    uint32_t qb[NT][KS][2];
    float qs[NT][2];  // what undoes the powers of two, times scale log2(e), of heads 2 tid, + 1
    uint32_t key_down = 0x33803380u;  // 2^-24, bfloat16
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int head = nt * 8 + gid;
      const __nv_bfloat16* qrow =
          p.q + static_cast<int64_t>(__ldg(p.qsl + r)) * p.q_stride + static_cast<int64_t>(h * G + (head < G ? head : 0)) * D;
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
      const float f = copysignf(pow2(up), p.scale_log2);  // the scale's sign is Q's
      if (__any_sync(0xffffffffu, ex > 147u)) key_down = 0x3f803f80u;  // 1
      qs[nt][0] = __int_as_float(__shfl_sync(0xffffffffu, up, 8 * tid));
      qs[nt][1] = __int_as_float(__shfl_sync(0xffffffffu, up, 8 * tid + 4));
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

#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int cc = 0; cc < 2; ++cc) {
        const float undo =
            fabsf(p.scale_log2) * pow2((key_down == 0x3f803f80u ? 0 : 24) - __float_as_int(qs[nt][cc]));
        // (never zero, for the masked scores' infinities)
        qs[nt][cc] = undo < 1.17549435e-38f ? 1.17549435e-38f : undo;
      }
    float o[2 * NB][NT][4];
    float m[NT][2], l[NT][2];
    uint32_t base[NW];  // running scale byte per group, as the V scale words have them: b0 b1 b0 b1
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
    for (int w = 0; w < NW; ++w) base[w] = 0u;

    int left = at.run;             // units of the run to go
    // tokens the request has from the stage's first on
    int valid = __ldg(p.seq_lens + r) - first_j * kMxBlock;
    for (; left > 0; left -= 2, valid -= 32,
                     stage = stage + kStage == ring_end ? 0u : stage + kStage) {
      // at the fewest stages one fetch may still be in flight, else two
      if (stages == 2) cp_async_wait<0>(); else cp_async_wait<1>();
      __syncwarp();
      fetch(refill);
      const uint8_t* st = smem + static_cast<uint32_t>(warp) * ring_end + stage;
      refill = stage;
      // tokens of this stage: below 32 in a run's last one only
      const int tokens = min(valid, left * kMxBlock);

      // ---- S^T = K Q^T of both units; times qs they are in log2 units ----
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
        uint32_t ks[2][NW];  // K scales as bfloat16 pairs, NaN for 255
#pragma unroll
        for (int w = 0; w < NW; ++w) {
          ks[0][w] = mul_bf16x2(e8m0x2_to_bf16x2(slo >> (16 * w)), key_down);
          ks[1][w] = mul_bf16x2(e8m0x2_to_bf16x2(shi >> (16 * w)), key_down);
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
          const float fl = (b & 1) ? __uint_as_float(ks[0][b >> 1] & 0xffff0000u)
                                   : __uint_as_float(ks[0][b >> 1] << 16);
          const float fh = (b & 1) ? __uint_as_float(ks[1][b >> 1] & 0xffff0000u)
                                   : __uint_as_float(ks[1][b >> 1] << 16);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float d[4];
            mma_f16_first(d, x[0], y[0], x[1], y[1], qb[nt][2 * b][0], qb[nt][2 * b][1]);
            mma_f16(d, x[2], y[2], x[3], y[3], qb[nt][2 * b + 1][0], qb[nt][2 * b + 1][1]);
            s[u][nt][0] = fmaf(d[0], fl, s[u][nt][0]);
            s[u][nt][1] = fmaf(d[1], fl, s[u][nt][1]);
            s[u][nt][2] = fmaf(d[2], fh, s[u][nt][2]);
            s[u][nt][3] = fmaf(d[3], fh, s[u][nt][3]);
          }
        }
      }
      if (tokens < 32) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 4; ++c)
              if (u * 16 + gid + (c >> 1) * 8 >= tokens) s[u][nt][c] = -INFINITY;
      }

      // ---- V scales of token pairs tid and tid + 4 of each unit ----
      uint32_t sw[2][2][NW];
      uint32_t far[2] = {0u, 0u};
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint8_t* v = st + u * kUnit + kChunk + kScale;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if constexpr (D == 128) {
            const uint2 x = *reinterpret_cast<const uint2*>(v + i * 32 + tid * 8);
            sw[u][i][0] = x.x;
            sw[u][i][1] = x.y;
          } else {
            sw[u][i][0] = *reinterpret_cast<const uint32_t*>(v + i * 16 + tid * 4);
          }
        }
        if (tokens < 32) {
          // bytes of tokens past the end may be anything: any scale inside the window
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int t = u * 16 + 2 * tid + 8 * i;
            const uint32_t keep = (t < tokens ? 0x0000ffffu : 0u) | (t + 1 < tokens ? 0xffff0000u : 0u);
#pragma unroll
            for (int w = 0; w < NW; ++w) sw[u][i][w] = (sw[u][i][w] & keep) | (base[w] & ~keep);
          }
        }
        // All scales within [base, base + 15]?  If so no byte borrows, and every
        // difference fits its low four bits.  A byte below base by 1 .. 239
        // leaves one of the tested bits set (base is at most 239, and NaN's 255
        // is above every base by 16 or more).
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int w = 0; w < NW; ++w) far[u] |= sw[u][i][w] - base[w];
      }

      // ---- online softmax per head column ----
      float mx[NT][2];
      bool grow = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int cc = 0; cc < 2; ++cc) {
          mx[nt][cc] = fmaxf(fmaxf(s[0][nt][cc], s[0][nt][2 + cc]),
                             fmaxf(s[1][nt][cc], s[1][nt][2 + cc])) * qs[nt][cc];
          grow |= mx[nt][cc] > m[nt][cc] + kMaxWeight;
        }
      // P^T fragments of a unit: the weights of tokens 2 tid, + 1 (and + 8) for
      // head gid, and their sums
      auto weights = [&](int u, uint32_t (&pt)[NT][2]) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float e[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) e[c] = exp2_approx(fmaf(s[u][nt][c], qs[nt][c & 1], -m[nt][c & 1]));
          l[nt][0] += e[0] + e[2];
          l[nt][1] += e[1] + e[3];
          pt[nt][0] = transpose_8x8(pack_f16(e[0], e[1]));
          pt[nt][1] = transpose_8x8(pack_f16(e[2], e[3]));
        }
      };
      // V codes of tokens 2 tid, + 1 (index 0), + 8, + 9 (index 1), a token pair
      // side by side: byte k holds position 2k (ev) or 2k + 1 (od) of both
      auto codes = [&](int u, uint32_t (&ev)[2][NW], uint32_t (&od)[2][NW]) {
        const uint8_t* v = st + u * kUnit + kChunk;
        uint32_t vw[4][NW];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (D == 128) {
            const uint2 x = *reinterpret_cast<const uint2*>(v + (i >> 1) * 512 + v_at[i & 1]);
            vw[i][0] = x.x;
            vw[i][1] = x.y;
          } else {
            vw[i][0] = *reinterpret_cast<const uint32_t*>(v + (i >> 1) * 256 + v_at[i & 1]);
          }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int w = 0; w < NW; ++w) {
            const uint32_t x = vw[2 * i][w], y = vw[2 * i + 1][w];
            ev[i][w] = (x & 0x0f0f0f0fu) | ((y << 4) & 0xf0f0f0f0u);
            od[i][w] = ((x >> 4) & 0x0f0f0f0fu) | (y & 0xf0f0f0f0u);
          }
      };
      // one vote for everything that is rare
      if (__any_sync(0xffffffffu, grow || ((far[0] | far[1]) & 0xf0f0f0f0u) != 0u)) {
        if (left == at.run) {
          // the first stage: nothing is summed up yet, so the base is free to go
          // where this stage's largest scales want it
#pragma unroll
          for (int w = 0; w < NW; ++w) {
            uint32_t x = __vmaxu4(__vmaxu4(sw[0][0][w], sw[0][1][w]), __vmaxu4(sw[1][0][w], sw[1][1][w]));
            x = __vmaxu4(x, __byte_perm(x, 0u, 0x1032));  // both tokens of a pair
            x = __vmaxu4(x, __shfl_xor_sync(0xffffffffu, x, 1));
            x = __vmaxu4(x, __shfl_xor_sync(0xffffffffu, x, 2));
            const uint32_t to = __vminu4(__vsubus4(x, kBelow * 0x01010101u), kTopBase * 0x01010101u);
            if (tokens < 32) {  // bytes past the end follow the base
#pragma unroll
              for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  const int t = u * 16 + 2 * tid + 8 * i;
                  const uint32_t keep = (t < tokens ? 0x0000ffffu : 0u) | (t + 1 < tokens ? 0xffff0000u : 0u);
                  sw[u][i][w] = (sw[u][i][w] & keep) | (to & ~keep);
                }
            }
            base[w] = to;
          }
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            far[u] = 0u;
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int w = 0; w < NW; ++w) far[u] |= sw[u][i][w] - base[w];
          }
        }
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
            for (int i = 0; i < 2 * NB; ++i) {
              o[i][nt][cc] *= alpha;
              o[i][nt][2 + cc] *= alpha;
            }
          }
        if (__any_sync(0xffffffffu, ((far[0] | far[1]) & 0xf0f0f0f0u) != 0u)) {
          // ---- slow path: scales outside the window ----
          // The weight and the scale of a token make one power of two before anything is
          // rounded: for 16 tokens, a group and a head, 2^(z - zm + 12) goes into the product
          // as f16, z = s - m + e - base, zm the largest of them, and the result comes
          // back by 2^(zm - 12 + kLow) in float32.  What is further below goes into products
          // of its own, so a key's precision depends on no other key's score or scale.
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            if (u == 1 && tokens <= 16) break;
            uint32_t ev[2][NW], od[2][NW];
            codes(u, ev, od);
            // This lane has the scores of tokens gid and gid + 8 (i = 0, 1) and heads 2 tid, + 1.
            // The largest weight of each token (log2), of any head there is:
            float live[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                const float x = fmaf(s[u][nt][c], qs[nt][c & 1], -m[nt][c & 1]);
                l[nt][c & 1] += exp2_approx(x);
                if (nt * 8 + 2 * tid + (c & 1) < G) live[c >> 1] = fmaxf(live[c >> 1], x);
              }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              live[i] = fmaxf(live[i], __shfl_xor_sync(0xffffffffu, live[i], 1));
              live[i] = fmaxf(live[i], __shfl_xor_sync(0xffffffffu, live[i], 2));
            }
#pragma unroll
            for (int w = 0; w < NW; ++w) {
#pragma unroll
              for (int b = 0; b < 2; ++b) {
                const uint8_t* scales = st + u * kUnit + kChunk + mx_vscale_off<D>(gid, 2 * w + b);
                int bs = (base[w] >> (8 * b)) & 0xff, hi = -1;
                bool nan = false;
                float e[2];  // of the tokens, above the base; -inf where there is nothing to add
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  const int byte = scales[i * (D / 4)];  // 8 tokens on: four pairs
                  const bool in = u * 16 + gid + 8 * i < tokens;
                  nan |= in && byte == 255;
                  e[i] = in && byte != 255 ? static_cast<float>(byte - bs) : -INFINITY;
                  if (in && byte != 255 && live[i] > -25.f) hi = max(hi, byte);
                }
                nan = __any_sync(0xffffffffu, nan);
                float most = -INFINITY;  // of z, any token and head
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                  for (int c = 0; c < 4; ++c)
                    most = fmaxf(most, fmaf(s[u][nt][c], qs[nt][c & 1], -m[nt][c & 1]) + e[c >> 1]);
#pragma unroll
                for (int x = 1; x < 32; x <<= 1) {
                  hi = max(hi, __shfl_xor_sync(0xffffffffu, hi, x));
                  most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, x));
                }
                // the base follows the largest scale that f16 weights still count for; down
                // only while what is summed up stays far from overflow, up too for the sake
                // of the sums
                int to = hi < 0 ? bs : min(max(hi - kBelow, 0), kTopBase);
                if (to < bs) {
                  to = hi < bs ? max(to, bs - 100) : bs;
                  float sum = 0.f;
#pragma unroll
                  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int k = 0; k < 2; ++k)
#pragma unroll
                      for (int c = 0; c < 4; ++c) sum = fmaxf(sum, fabsf(o[4 * w + 2 * b + k][nt][c]));
                  if (__any_sync(0xffffffffu, sum * pow2(bs - to) > kMostSum)) to = bs;
                }
                if (most - static_cast<float>(to - bs) > kMostProduct)
                  to = min(bs + static_cast<int>(most - kMostProduct) + 1, kTopBase);
                if (to != bs) {
                  const float f = pow2(bs - to);
#pragma unroll
                  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int k = 0; k < 2; ++k)
#pragma unroll
                      for (int c = 0; c < 4; ++c) o[4 * w + 2 * b + k][nt][c] *= f;
                  const uint32_t hold = ~(0x00ff00ffu << (8 * b));
                  base[w] = (base[w] & hold) | (static_cast<uint32_t>(to) * 0x00010001u) << (8 * b);
                  e[0] += static_cast<float>(bs - to);
                  e[1] += static_cast<float>(bs - to);
                }
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
                  float z[4];  // below the head's largest
                  float zm[2];
#pragma unroll
                  for (int cc = 0; cc < 2; ++cc) {
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                      z[2 * i + cc] = fmaf(s[u][nt][2 * i + cc], qs[nt][cc], -m[nt][cc]) + e[i];
                    float x = fmaxf(fmaxf(z[cc], z[2 + cc]), -1e30f);
#pragma unroll
                    for (int k = 4; k < 32; k <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, k));
                    // (above the largest: not in any product)
                    z[cc] = z[cc] < -1e29f ? 1.f : z[cc] - x;
                    z[2 + cc] = z[2 + cc] < -1e29f ? 1.f : z[2 + cc] - x;
                    zm[cc] = x;
                  }
                  // 26 binades of them at a time: f16's normal numbers below 2^13
                  bool more = true;
                  for (float down = 0.f; more && down < 120.f; down += 26.f) {
                    float p16[4];
                    more = false;
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                      const float y = z[c] + down;  // (NaN goes on)
                      more |= y <= -26.f;
                      p16[c] = y > 0.f || y <= -26.f ? 0.f : exp2_approx(y + 12.f);
                    }
                    const uint32_t b0 = transpose_8x8(pack_f16(p16[0], p16[1]));
                    const uint32_t b1 = transpose_8x8(pack_f16(p16[2], p16[3]));
                    const float back[2] = {exp2_approx(zm[0] - down + (kLow - 12)),
                                           exp2_approx(zm[1] - down + (kLow - 12))};
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                      float t[4];
                      mma_f16_first(t, a[k][0], a[k][1], a[k][2], a[k][3], b0, b1);
#pragma unroll
                      for (int c = 0; c < 4; ++c)
                        o[4 * w + 2 * b + k][nt][c] = fmaf(t[c], back[c & 1], o[4 * w + 2 * b + k][nt][c]);
                    }
                    more = __any_sync(0xffffffffu, more);
                  }
                  if (nan) {
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
          continue;
        }
      }

#pragma unroll
      for (int u = 0; u < 2; ++u) {
        if (u == 1 && tokens <= 16) break;
        uint32_t pt[NT][2], ev[2][NW], od[2][NW];
        weights(u, pt);
        codes(u, ev, od);
#pragma unroll
        for (int w = 0; w < NW; ++w) {
          // 2^(e - base + kLow) as f16: the exponent field in each half's high byte
          const uint32_t c = 4u * (15 + kLow) * 0x01010101u - 4u * base[w];
          const uint32_t x0 = sw[u][0][w] * 4u + c, x1 = sw[u][1][w] * 4u + c;
          uint32_t e0[4], e1[4], o0[4], o1[4];
          e2m1x8_to_f16(ev[0][w], e0);
          e2m1x8_to_f16(od[0][w], o0);
          e2m1x8_to_f16(ev[1][w], e1);
          e2m1x8_to_f16(od[1][w], o1);
#pragma unroll
          for (int b = 0; b < 2; ++b) {  // groups 2w and 2w + 1
            // bytes b and b + 2 to the halves' high bytes
            const uint32_t f0 = __byte_perm(x0, 0u, b == 0 ? 0x2404 : 0x3414);
            const uint32_t f1 = __byte_perm(x1, 0u, b == 0 ? 0x2404 : 0x3414);
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
      }
    }

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
    const bool whole = prefix[r] + kMxRequestCost >= u0 && prefix[r + 1] <= u1;
    const int64_t mine = static_cast<int64_t>(slot_of(me, inside)) * p.hkv + h;
    const int64_t tok = __ldg(p.qsl + r);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int cc = 0; cc < 2; ++cc) {
        const int g = nt * 8 + 2 * tid + cc;
        if (g >= G) continue;
        // o[2 b + s]: dims 32 b + 4 gid + 2 s (elements 0, 1) and + 1 (2, 3)
        const float inv = 1.f / l[nt][cc];
        __nv_bfloat16* dst = p.out + tok * p.out_stride + static_cast<int64_t>(h * G + g) * D + 4 * gid;
        float* po = p.part_o + (mine * G + g) * D + 4 * gid;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          // what the weights' scales left out: 2^(base - kLow - 127)
          const float f = mx_scale((base[b >> 1] >> (8 * (b & 1))) & 0xffu) * pow2(-kLow);
          float x[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) x[i] = o[2 * b + (i >> 1)][nt][2 * (i & 1) + cc] * inv * f;
          if (whole)
            *reinterpret_cast<uint2*>(dst + 32 * b) =
                make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
          else
            *reinterpret_cast<float4*>(po + 32 * b) = make_float4(x[0], x[1], x[2], x[3]);
        }
        if (!whole && gid == 0) p.part_ml[mine * G + g] = make_float2(m[nt][cc], l[nt][cc]);
      }
    if (at.rest == 0) break;
    at.next_run(prefix);
    if (at.run == 0) break;
    first_j = 0;
  }
  // every copy of this pass has been waited for by its stage; none is in flight
  }
}

// log2 of a range's weight 2^m l, to the binade.
__device__ __forceinline__ float range_weight(float2 ml) {
  return ml.x + static_cast<float>(static_cast<int>(__float_as_uint(ml.y) >> 23) - 127);
}

// Joins the partials of every request that crosses ranges.  kLanes lanes take 4
// kLanes dimensions of one (request, query head); the groups of a warp take the
// ranges in turn, kBatch loads of a lane in flight, and add up at the end.
template <int D, int kLanes>
__global__ void __launch_bounds__(256, 4) join_mxfp4_kernel(const Params p) {
  grid_dependency_wait();  // the decode's partials
  if (threadIdx.x == 0) grid_launch_dependents();
  constexpr int kBatch = 4, kParts = 32 / kLanes, kItems = D / (4 * kLanes);
  const int G = p.group, H = p.hkv * G;
  const int lane = threadIdx.x & 31, part = lane / kLanes;
  const int per_req = H * kItems;  // warps' items of a request
  const int64_t total = static_cast<int64_t>(p.num_reqs) * per_req;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5); i < total;
       i += static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5)) {
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
        // 2^-9 at most: some hundred values near float32's end may be added up
        const float w = exp2_approx(ml[k].x - mx - 10.f) * ml[k].y;
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
  constexpr size_t kRing = static_cast<size_t>(kWarps) * 4 * mx_chunk_bytes(D);  // one stage of all warps
  constexpr size_t kLimit = 232448 - 1024;                                       // static shared memory aside
  const size_t plan = 4 * (static_cast<size_t>(p.num_reqs) + 1);
  // three stages keep about 139 KB in flight on an SM; two where the plan of
  // a very large batch needs the room
  p.stages = 3 * kRing + plan <= kLimit ? 3 : 2;
  const size_t smem = p.stages * kRing + plan;
  cudaError_t e = raise_smem_limit_once<decode_mxfp4_kernel<D, NT>>(kLimit);
  if (e != cudaSuccess) return e;
  e = launch_programmatic(decode_mxfp4_kernel<D, NT>, dim3(static_cast<unsigned>(sms)),
                          dim3(kWarps * 32), smem, stream, p);
  if (e != cudaSuccess) return e;
  // Few requests have many ranges each: eight lanes take 32 dimensions, four ranges at
  // a time.  Where that is more than a wave of warps, more lanes and fewer ranges (64
  // requests with 32 heads of 128: sixteen take 0.8 us less than thirty-two, 1.1 less than eight).
  const int64_t heads = static_cast<int64_t>(p.num_reqs) * p.hkv * p.group;
  const int64_t wave = 32 * static_cast<int64_t>(sms);
  constexpr int kWide = D / 4;
  const int lanes = heads * (D / 32) <= wave ? 8 : heads * (D / 64) <= wave ? 16 : kWide;
  const int64_t grid = (heads * (D / (4 * lanes)) + 7) / 8;
  return launch_programmatic(lanes == 8    ? join_mxfp4_kernel<D, 8>
                             : lanes == 16 ? join_mxfp4_kernel<D, 16>
                                           : join_mxfp4_kernel<D, kWide>,
                             dim3(static_cast<unsigned>(grid < wave / 4 ? grid : wave / 4)),
                             dim3(256), 0, stream, p);
}

}  // namespace

int64_t decode_mxfp4_slots(int sms, int num_kv_heads) {
  return 2 * static_cast<int64_t>(sms) * ranges_per_cta(warps_per_cta<1>(), num_kv_heads) * num_kv_heads;
}

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
