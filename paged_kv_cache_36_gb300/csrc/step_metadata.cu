// A step's metadata built on the device from request lengths: new cache blocks
// from a ring of free ones, block_table entries, query_start_loc, seq_lens,
// positions and slot_mapping.
//
// "显存与调度", section "分配是词元计划的一部分": request i with T_i tokens held and
// s_i new ones needs delta_i = ceil((T_i + s_i) / B) - ceil(T_i / B) new blocks;
// a plan takes all of its blocks, from the front of the free list in plan order,
// or none.  "AI Infra入门干货总结：大模型是如何高效推理的", section "Paged Attention":
// slot = block_table[pos / B] B + pos % B.  The same results as the host
// allocator's reserve and the scheduler's metadata, for a step whose lengths
// are known on the device only.
//
// One launch, no waiting between CTAs.  The lengths are few (8 bytes a
// request) and the outputs many (16 bytes a token), so every CTA scans all
// requests itself, from L2, and then writes its share of blocks and tokens:
// both prefix sums in shared memory turn a block or token index into its
// request by a binary search.  A token's block comes from the ring by
// arithmetic, not from the table row that another CTA may be writing.  All CTAs
// reach the same verdict (enough blocks, lengths in range), so a refused step
// is refused everywhere.  With free_state updated in place the last CTA to
// finish writes it, after every CTA has read it.
#include <cuda_runtime.h>

#include <cstdint>

#include "kernels.h"
#include "pkv_device.cuh"

namespace pkv {

namespace {

constexpr int kThreads = 512;
constexpr int kBlock = 16;

// The largest r with start(r) <= x, where ends[] holds inclusive sums and
// start(r) = r ? ends[r - 1] : 0; x is below ends[n - 1].
__device__ __forceinline__ int request_of(const int32_t* ends, int n, int x) {
  int lo = 0, hi = n - 1;  // the first r with ends[r] > x
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (ends[mid] > x) hi = mid; else lo = mid + 1;
  }
  return lo;
}

__global__ void __launch_bounds__(kThreads) step_metadata_kernel(const StepMetadataArgs a) {
  extern __shared__ int32_t smem[];
  int32_t* tok_end = smem;              // [R] inclusive sums of new tokens
  int32_t* blk_end = smem + a.num_reqs; // [R] inclusive sums of new blocks
  __shared__ long long warp_tok[kThreads / 32], warp_blk[kThreads / 32];
  grid_dependency_wait();  // the lengths may be the kernel before's
  const int R = a.num_reqs, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const long long head = a.free_state[0], tail = a.free_state[1];

  // ---- each thread sums its own run of requests, then the CTA scans ----
  bool bad = head < 0 || tail < head || tail - head > a.ring_size;
  for (int r = tid; r < R; r += kThreads) {
    const int nw = __ldg(a.query_lens + r), nc = __ldg(a.num_computed + r);
    const long long seq = static_cast<long long>(nw) + nc;
    int need = 0;
    if (nw < 0 || nc < 0 || seq > 0x7fffffffLL - kBlock ||
        (seq + kBlock - 1) / kBlock > a.bt_width) {
      bad = true;
    } else {
      need = static_cast<int>((seq + kBlock - 1) / kBlock - (nc + kBlock - 1) / kBlock);
    }
    tok_end[r] = nw;
    blk_end[r] = need;
  }
  const bool any_bad = __syncthreads_or(bad);
  const int per = (R + kThreads - 1) / kThreads;
  const int first = min(R, tid * per), last = min(R, first + per);
  long long tsum = 0, bsum = 0;
  for (int r = first; r < last; ++r) {
    tsum += tok_end[r];
    bsum += blk_end[r];
  }
  long long tinc = tsum, binc = bsum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, tinc, o);
    const long long y = __shfl_up_sync(0xffffffffu, binc, o);
    if (lane >= o) {
      tinc += x;
      binc += y;
    }
  }
  if (lane == 31) {
    warp_tok[warp] = tinc;
    warp_blk[warp] = binc;
  }
  __syncthreads();
  long long total_tok = 0, total_blk = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) {
      tinc += warp_tok[w];
      binc += warp_blk[w];
    }
    total_tok += warp_tok[w];
    total_blk += warp_blk[w];
  }
  const bool fits = total_tok <= a.num_tokens;
  const bool enough = total_blk <= tail - head;
  const bool ok = !any_bad && fits && enough;
  // sums that do not fit 31 bits belong to a refused step and are not used
  long long t = tinc - tsum, b = binc - bsum;
  for (int r = first; r < last; ++r) {
    t += tok_end[r];
    b += blk_end[r];
    tok_end[r] = static_cast<int32_t>(t);
    blk_end[r] = static_cast<int32_t>(b);
  }
  __syncthreads();
  if (!ok && blockIdx.x == 0 && tid == 0 && a.err)
    atomicOr(a.err, (any_bad || !fits ? PKV_ERR_METADATA : 0u) |
                        (!any_bad && fits && !enough ? PKV_ERR_NO_BLOCKS : 0u));

  const int hm = a.ring_size > 0 ? static_cast<int>(head % a.ring_size) : 0;
  auto ring_entry = [&](int k) -> int32_t {  // the k-th block of this step, k < total_blk
    int i = hm + k;
    if (i >= a.ring_size) i -= a.ring_size;
    return __ldg(a.free_ring + i);
  };
  const int gtid = blockIdx.x * kThreads + tid, gstep = gridDim.x * kThreads;
  // ---- per request ----
  for (int r = gtid; r < R; r += gstep) {
    const int nc = __ldg(a.num_computed + r);
    const int end = ok ? tok_end[r] : 0, begin = ok && r > 0 ? tok_end[r - 1] : 0;
    a.query_start_loc[r + 1] = end;
    a.seq_lens[r] = nc + (end - begin);
  }
  if (gtid == 0) a.query_start_loc[0] = 0;
  // ---- new blocks into their table rows ----
  const int nblk = ok ? static_cast<int>(total_blk) : 0;
  for (int k = gtid; k < nblk; k += gstep) {
    const int r = request_of(blk_end, R, k);
    const int nc = __ldg(a.num_computed + r);
    const int col = (nc + kBlock - 1) / kBlock + (k - (r > 0 ? blk_end[r - 1] : 0));
    a.block_table[static_cast<int64_t>(r) * a.bt_stride + col] = ring_entry(k);
  }
  // ---- tokens ----
  const int ntok = ok ? static_cast<int>(total_tok) : 0;
  for (int64_t x = gtid; x < a.num_tokens; x += gstep) {
    int64_t slot = -1, pos = 0;  // padding behind the last request
    if (x < ntok) {
      const int i = static_cast<int>(x);
      const int r = request_of(tok_end, R, i);
      const int nc = __ldg(a.num_computed + r);
      const int p = nc + (i - (r > 0 ? tok_end[r - 1] : 0));
      const int col = p / kBlock, have = (nc + kBlock - 1) / kBlock;
      const int32_t blk =
          col < have ? a.block_table[static_cast<int64_t>(r) * a.bt_stride + col]
                     : ring_entry((r > 0 ? blk_end[r - 1] : 0) + (col - have));
      pos = p;
      if (blk >= 0) slot = static_cast<int64_t>(blk) * kBlock + p % kBlock;
      else if (a.err) atomicOr(a.err, PKV_ERR_BLOCK_ID);
    }
    a.slot_mapping[x] = slot;
    if (a.positions) a.positions[x] = pos;
  }
  // ---- the ring's state ----
  if (a.free_state_out != a.free_state) {
    if (gtid == 0) {
      a.free_state_out[0] = head + nblk;
      a.free_state_out[1] = tail;
    }
    return;
  }
  __syncthreads();
  if (tid == 0) {
    // every CTA has read free_state before it counts itself here
    unsigned long long* ticket = reinterpret_cast<unsigned long long*>(a.free_state + 2);
    __threadfence();
    if (atomicAdd(ticket, 1ull) == gridDim.x - 1) {
      *ticket = 0;
      a.free_state[0] = head + nblk;
    }
  }
}

}  // namespace

int step_metadata_max_reqs() { return 8192; }

cudaError_t launch_step_metadata(const StepMetadataArgs& a, cudaStream_t stream) {
  const size_t smem = 8 * static_cast<size_t>(a.num_reqs);
  const cudaError_t e =
      raise_smem_limit_once<step_metadata_kernel>(8 * static_cast<size_t>(step_metadata_max_reqs()));
  if (e != cudaSuccess) return e;
  const int sms = current_sm_count();
  const int64_t items = a.num_tokens > a.num_reqs ? a.num_tokens : a.num_reqs;
  int64_t grid = (items + kThreads - 1) / kThreads;
  if (grid > sms) grid = sms;
  if (grid < 1) grid = 1;
  return launch_programmatic(step_metadata_kernel, dim3(static_cast<unsigned>(grid)),
                             dim3(kThreads), smem, stream, a);
}

}  // namespace pkv
