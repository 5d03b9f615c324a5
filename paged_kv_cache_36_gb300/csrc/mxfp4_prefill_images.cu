// Chunked-prefill attention over the 4-bit paged cache on the 5th-generation tensor
// cores, for requests with many query tiles: their key tiles are converted to f16 once,
// to images in the workspace, and a kernel without any conversion of K and V reads
// those.
//
// For a query row at position p and KV head g, out = softmax_{j <= p}(scale <q, K_j>)
// V_j with K, V the values that codes and power-of-two scales stand for (mxfp4.cuh).
//
// An image is a key tile of one KV head in the layout that the tensor core reads: K and
// V as 128-byte swizzled rows of f16, and a Meta with the tile's base exponents.  It is
// made once for all query tiles of the request, so the conversion, which in the direct
// kernel takes issue slots and instruction cache from the softmax for every query tile,
// costs a few microseconds, and loading a tile is one bulk copy of 16 or 32 KB from L2.
//
// Tiling is that of the bfloat16 prefill: 128 rows = floor(128 / G) query tokens x the G
// query heads of a KV head against key tiles of 128, S = Q K^T and O += P V as tcgen05
// products, S and O in tensor memory, P written over S.
//
// What bounds it: the chain of a key tile, S from tensor memory, its maximum, the
// exchange between the two warps of a row, exponentials, P back, at eight softmax warps
// an SM; the tensor core is busy 40 % of the time.  A prompt of 4096 tokens with 32
// query and 8 KV heads of 128 takes 158 us, 870 TFLOP/s, about 8 us of them for the images; of
// 16384 tokens 1662 us, 1323 TFLOP/s.  (bfloat16 caches: 116 and 1455 us.)
//
// Warp roles (16 warps): warp 0 copies K and Meta, warp 1 V; warp 2 owns the tensor
// memory and issues Q K^T, warp 3 issues P V; warps 4-11 run the softmax and the
// epilogue, two per 32-lane quadrant of tensor memory, each with half of the key tile's
// columns; warps 12-15 bring Q to f16.
// Every wait is bounded; a timeout sets PKV_ERR_TIMEOUT and an abort flag that stops all
// roles.
#include "mxfp4_prefill.cuh"

namespace pkv {

using namespace mxprefill;

namespace {

constexpr int kKStages = 3;
constexpr int kVStages = 2;
constexpr int kSBufs = 3;
constexpr int kMetas = 4;            // key tiles whose scales are in shared memory
constexpr int kQfs = kSBufs + 1;     // query tiles whose factors are (see kQf0)
constexpr int kThreads = 512;
// Registers a thread by role (setmaxnreg; four warpgroups of 128 at launch): the
// softmax holds 64 scores and 32 words of weights.
constexpr int kLaunchRegs = 128, kIssueRegs = 40, kSoftmaxRegs = 184, kConvertRegs = 80;
static_assert(kIssueRegs + 2 * kSoftmaxRegs + kConvertRegs <= 4 * kLaunchRegs,
              "the roles' registers fit in what the block is launched with");
static_assert(kThreads * kLaunchRegs <= 65536, "and those in an SM");

enum Bar {
  kQFull, kQEmpty,
  kKFull0, kKEmpty0 = kKFull0 + kKStages,
  kVFull0 = kKEmpty0 + kKStages, kVEmpty0 = kVFull0 + kVStages,
  kSFull0 = kVEmpty0 + kVStages, kSFree0 = kSFull0 + kSBufs,
  kPFull0 = kSFree0 + kSBufs, kODone0 = kPFull0 + kSBufs,
  kOFinal = kODone0 + kSBufs, kPair0,
  kMFull0 = kPair0 + 4, kMFree0 = kMFull0 + kMetas,
  // Factors of query tile n are in buffer n % kQfs.  They are written once all S of tile
  // n - 1 are issued, the last of which took a buffer that the softmax of tile n - 1 -
  // kSBufs, or a later one, had given back: the reader of the buffer is through.
  kQf0 = kMFree0 + kMetas,
  kNumBars = kQf0 + kQfs
};

// What the softmax has to know of a key tile, at the end of its image.
struct alignas(16) Meta {
  float kf;            // K base: 2^(base - 127 - kUp)
  float vb;            // V base: base - 127 - kUp, log2 units
  uint32_t flags;      // 1: K by key, 2: V by key, 4: NaN in V, 8: V of uneven groups, 16: loose V
  uint32_t unused;
  int32_t nan_pos[4];  // first key position with a NaN V group, by group
  float key_kf[kKeys];
  float key_vb[kKeys];
};

template <int D>
__host__ __device__ constexpr uint32_t image_bytes() {
  return 2 * (D / 64) * kRegion + (sizeof(Meta) + 127) / 128 * 128;
}

template <int D>
struct Layout {
  static constexpr int NDH = D / 64;
  static constexpr uint32_t kHalf = NDH * kRegion;  // one K (or V or Q) tile
  static constexpr uint32_t kQ = 0;
  static constexpr uint32_t kK = kQ + kHalf;
  static constexpr uint32_t kV = kK + kKStages * kHalf;
  static constexpr uint32_t kBars = kV + kVStages * kHalf;
  static constexpr uint32_t kXch = (kBars + 8 * kNumBars + 15) / 16 * 16;  // [2 parity][2 half][128 rows] floats
  static constexpr uint32_t kQf = kXch + 2 * 2 * 128 * 4;                  // [kQfs][128 rows] floats
  static constexpr uint32_t kMeta = kQf + kQfs * kRows * 4;
  static constexpr uint32_t kMisc = kMeta + kMetas * sizeof(Meta);  // tensor memory slot, abort flag
  static constexpr uint32_t kPrefix = kMisc + 16;
  static_assert(kMeta % 16 == 0 && sizeof(Meta) % 16 == 0 && kBars % 8 == 0, "copies to Meta, and the barriers");
};

// Copies the K tiles and Metas, or the V tiles, of this CTA's query tiles (one thread).
template <int D, bool kIsV>
__device__ __forceinline__ void copy_role(const Params& p, uint8_t* smem, const int32_t* prefix, int entries,
                                          int total, int tpt) {
  using L = Layout<D>;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMisc + 4);
  constexpr int kStages = kIsV ? kVStages : kKStages;
  constexpr int kFull0 = kIsV ? kVFull0 : kKFull0, kEmpty0 = kIsV ? kVEmpty0 : kKEmpty0;
  const int cid = blockIdx.x, ncta = gridDim.x;
  const int64_t step = static_cast<int64_t>(p.hkv) * image_bytes<D>();
  uint32_t count = 0, metas = 0;
  bool ok = true;
  fence_proxy_async_global();  // the Metas were written with plain stores
  for (int it = 0, ct = cta_tile(0, cid, ncta, total); ct >= 0 && ok && !*abort_flag;
       ct = cta_tile(++it, cid, ncta, total)) {
    const Tile t = find_tile<true>(ct, prefix, entries, p, tpt);
    const uint8_t* image = p.images + __ldcg(p.image_base + t.r) * step +
                           t.h * static_cast<int64_t>(image_bytes<D>());
    for (int j = 0; j < t.nkt; ++j, ++count, image += step) {
      if constexpr (!kIsV) {
        const int ms = count % kMetas;
        ok = count < kMetas ||
             held_wait(&bars[kMFree0 + ms], (count / kMetas - 1) & 1, p.err, abort_flag);
        if (!ok) break;
        mbar_arrive_expect_tx(&bars[kMFull0 + ms], sizeof(Meta));
        bulk_load(smem + L::kMeta + ms * sizeof(Meta), image + 2 * L::kHalf, sizeof(Meta), &bars[kMFull0 + ms]);
        ++metas;
      }
      const int st = count % kStages;
      ok = count < kStages ||
           held_wait(&bars[kEmpty0 + st], (count / kStages - 1) & 1, p.err, abort_flag);
      if (!ok) break;
      mbar_arrive_expect_tx(&bars[kFull0 + st], L::kHalf);
      bulk_load(smem + (kIsV ? L::kV : L::kK) + st * L::kHalf, image + (kIsV ? L::kHalf : 0u), L::kHalf,
                &bars[kFull0 + st]);
    }
  }
  // drain: every copy has landed before the CTA may exit
  for (uint32_t back = 1; back <= kStages && back <= count; ++back)
    mbar_wait(&bars[kFull0 + (count - back) % kStages], ((count - back) / kStages) & 1, p.err);
  for (uint32_t back = 1; back <= kMetas && back <= metas; ++back)
    mbar_wait(&bars[kMFull0 + (metas - back) % kMetas], ((metas - back) / kMetas) & 1, p.err);
}

}  // namespace

template <int D>
__global__ void __launch_bounds__(kThreads, 1) prefill_mxfp4_images_kernel(const Params p) {
  using L = Layout<D>;
  constexpr int NDH = L::NDH;
  constexpr int NB = D / 32;
  constexpr uint32_t kColS = 0;
  constexpr uint32_t kColO = kSBufs * kKeys;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBars);
  float* xch = reinterpret_cast<float*>(smem + L::kXch);
  float* qfs = reinterpret_cast<float*>(smem + L::kQf);
  const Meta* metas = reinterpret_cast<const Meta*>(smem + L::kMeta);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMisc + 4);
  int32_t* prefix = reinterpret_cast<int32_t*>(smem + L::kPrefix);

  grid_dependency_wait();  // the images
  if (threadIdx.x == 0) grid_launch_dependents();
  if (__ldcg(p.any + 1) == 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int R = p.num_reqs;
  const int entries = (R + (1 << p.entry_shift) - 1) >> p.entry_shift;
  int32_t* scan_tmp = prefix + entries + 1;
  const int cid = blockIdx.x, ncta = gridDim.x;
  const int G = p.group;
  const int tpt = kRows / G;  // query tokens per tile

  // ---- plan: tiles per entry and their prefix sum ----
  if (threadIdx.x == 0) {
    *abort_flag = 0;
    prefix[0] = 0;
    for (int b = 0; b < kNumBars; ++b) {
      uint32_t n = 1;
      if (b == kQFull || (b >= kQf0 && b < kQf0 + kQfs)) n = 4;  // the warps that convert Q
      if ((b >= kPFull0 && b < kPFull0 + kSBufs) || (b >= kMFree0 && b < kMFree0 + kMetas))
        n = 8;  // softmax warps
      if (b >= kPair0 && b < kPair0 + 4) n = 2;  // the two warps sharing a quadrant
      mbar_init(&bars[b], n);
    }
    fence_mbar_init();
  }
  for (int i = threadIdx.x; i < entries; i += blockDim.x) {
    int n = 0;
    bool bad = false;  // reported by the conversion
    for (int k = 0; k < (1 << p.entry_shift); ++k) {
      const int r = (i << p.entry_shift) + k;
      if (r < R) n += own_tiles<true>(p, r, tpt, &bad);
    }
    prefix[i + 1] = n;
  }
  __syncthreads();
  block_inclusive_scan(prefix + 1, entries, scan_tmp);
  __syncthreads();
  const int total = prefix[entries];
  if (cid >= total) return;  // no tile for this CTA, and no tensor memory held
  if (warp == 2) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp < 4) {
    set_registers<kIssueRegs, false>();
    if (warp == 0) {
      if (lane == 0) copy_role<D, false>(p, smem, prefix, entries, total, tpt);
    } else if (warp == 1) {
      if (lane == 0) copy_role<D, true>(p, smem, prefix, entries, total, tpt);
    } else if (warp == 2) {
      // ============================ QK^T issuer ============================
      if (lane == 0) {
        constexpr uint32_t idesc_s = idesc_f16_f32(kRows, kKeys, 0);
        const uint64_t q_desc = smem_desc_sw128(smem_u32(smem + L::kQ), 16, 1024);
        // K stage: groups of 8 keys every NDH KiB, dim half dh at +dh KiB
        const uint64_t k_desc0 = smem_desc_sw128(smem_u32(smem + L::kK), 16, NDH * 1024);
        uint32_t q_count = 0, count = 0;
        bool ok = true;
        for (int it = 0, ct = cta_tile(0, cid, ncta, total); ct >= 0 && ok && !*abort_flag;
             ct = cta_tile(++it, cid, ncta, total)) {
          const Tile t = find_tile<true>(ct, prefix, entries, p, tpt);
          ok = held_wait(&bars[kQFull], q_count & 1, p.err, abort_flag);
          ++q_count;
          for (int j = 0; j < t.nkt && ok; ++j, ++count) {
            const int ks = count % kKStages, b = count % kSBufs;
            ok = held_wait(&bars[kKFull0 + ks], (count / kKStages) & 1, p.err, abort_flag);
            // S/P buffer b is free once PV of the key tile that last used it is done
            if (ok && count >= kSBufs)
              ok = held_wait(&bars[kSFree0 + b], (count / kSBufs - 1) & 1, p.err, abort_flag);
            if (!ok) break;
            tc_fence_after();
            const uint64_t kd = k_desc0 + ((ks * L::kHalf) >> 4);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint64_t q_off = ((kk >> 2) * kRegion + (kk & 3) * 32) >> 4;
              const uint64_t k_off = ((kk >> 2) * 1024 + (kk & 3) * 32) >> 4;
              tc_mma_ss(tmem + kColS + b * kKeys, q_desc + q_off, kd + k_off, idesc_s, kk > 0);
            }
            tc_commit(&bars[kSFull0 + b]);
            tc_commit(&bars[kKEmpty0 + ks]);
            if (j == t.nkt - 1) tc_commit(&bars[kQEmpty]);
          }
        }
      }
    } else if (lane == 0) {
      // ============================ PV issuer ============================
      constexpr uint32_t idesc_o = idesc_f16_f32(kRows, D, 1);
      // V stage, MN-major: 64-dim atoms of a group of 8 keys 1 KiB apart, groups
      // of 8 keys NDH KiB apart
      const uint64_t v_desc0 = smem_desc_sw128(smem_u32(smem + L::kV), 1024, NDH * 1024);
      uint32_t count = 0;
      bool ok = true;
      for (int it = 0, ct = cta_tile(0, cid, ncta, total); ct >= 0 && ok && !*abort_flag;
           ct = cta_tile(++it, cid, ncta, total)) {
        const Tile t = find_tile<true>(ct, prefix, entries, p, tpt);
        for (int j = 0; j < t.nkt && ok; ++j, ++count) {
          const int vs = count % kVStages, b = count % kSBufs;
          ok = held_wait(&bars[kPFull0 + b], (count / kSBufs) & 1, p.err, abort_flag) &&
               held_wait(&bars[kVFull0 + vs], (count / kVStages) & 1, p.err, abort_flag);
          if (!ok) break;
          tc_fence_after();
          const uint64_t vd = v_desc0 + ((vs * L::kHalf) >> 4);
          const uint32_t a_p = tmem + kColS + b * kKeys;
          // P columns hold the keys of each softmax half in their first 32 (f16
          // pairs), V rows [64 half, 64 half + 64)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              tc_mma_ts(tmem + kColO, a_p + half * 64 + kk * 8,
                        vd + ((((half * 64 + kk * 16) / 8) * NDH * 1024) >> 4), idesc_o,
                        (j > 0 || half > 0 || kk > 0) ? 1u : 0u);
          }
          tc_commit(&bars[kODone0 + b]);
          if (j == t.nkt - 1) tc_commit(&bars[kOFinal]);
          tc_commit(&bars[kSFree0 + b]);
          tc_commit(&bars[kVEmpty0 + vs]);
        }
      }
    }
  } else if (warp >= 12) {
    // ============================ Q to f16 ============================
    set_registers<kConvertRegs, false>();
    const int row = (warp - 12) * 32 + lane;
    uint32_t tiles = 0;
    for (int it = 0, ct = cta_tile(0, cid, ncta, total); ct >= 0;
         ct = cta_tile(++it, cid, ncta, total), ++tiles) {
      if (__shfl_sync(0xffffffffu, *abort_flag, 0)) break;
      const Tile t = find_tile<true>(ct, prefix, entries, p, tpt);
      float qf;
      // the tile before is done with the buffer
      const bool ok = convert_q_row<D, 2, 1>(p, t, row, smem + L::kQ, qf, [&]() {
        return tiles == 0 || held_warp_wait(&bars[kQEmpty], (tiles - 1) & 1, p.err, abort_flag);
      });
      if (!ok) break;
      qfs[tiles % kQfs * kRows + row] = qf;
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&bars[kQFull]);
        mbar_arrive(&bars[kQf0 + tiles % kQfs]);
      }
    }
  } else {
    // ============================ softmax warps ============================
    set_registers<kSoftmaxRegs, true>();
    // Two warps share each 32-lane quadrant of tensor memory (the same 32 rows):
    // warp half h reads S columns [64 h, 64 h + 64).  They agree on the row maximum
    // every key tile, so one O serves the row; each keeps the partial sum l of its own
    // columns.
    const int quad = warp & 3;
    const int half = (warp - 4) >> 2;
    const int row = quad * 32 + lane;    // tile row = tensor-memory lane
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const uint32_t o_cols = lane_addr + kColO + half * (D / 2);
    uint64_t* pair_bar = &bars[kPair0 + quad];
    uint32_t count = 0, pair_uses = 0, tiles_done = 0;
    auto exchange = [&](float mine) -> float {
      float* slot = xch + (pair_uses & 1) * 256;
      slot[half * 128 + row] = mine;
      __syncwarp();
      if (lane == 0) mbar_arrive(pair_bar);
      const bool done = warp_wait(pair_bar, pair_uses & 1, p.err, abort_flag);
      ++pair_uses;
      return done ? slot[(half ^ 1) * 128 + row] : mine;
    };
    for (int it = 0, ct = cta_tile(0, cid, ncta, total); ct >= 0;
         ct = cta_tile(++it, cid, ncta, total)) {
      if (__shfl_sync(0xffffffffu, *abort_flag, 0)) break;
      const Tile t = find_tile<true>(ct, prefix, entries, p, tpt);
      const int u = row / G;
      const int pos = t.nc + t.u0 + (u < t.ntok ? u : t.ntok - 1);
      const int pos_min = t.nc + t.u0;
      float m_used = -INFINITY, ml = kNoScore, l = 0.f;
      uint32_t nan_groups = 0u;  // V groups that are NaN for this row
      bool ok = warp_wait(&bars[kQf0 + tiles_done % kQfs], (tiles_done / kQfs) & 1, p.err, abort_flag);
      const float qf = qfs[tiles_done % kQfs * kRows + row];
      for (int j = 0; j < t.nkt && ok; ++j, ++count) {
        const int b = count % kSBufs, ms = count % kMetas;
        if (!warp_wait(&bars[kMFull0 + ms], (count / kMetas) & 1, p.err, abort_flag)) {
          ok = false;
          break;
        }
        const Meta& meta = metas[ms];
        const uint4 head = *reinterpret_cast<const uint4*>(&meta);
        // never zero, for the masked scores' infinities
        float f = qf * __uint_as_float(head.x), vb = __uint_as_float(head.y);
        f = f < 1.17549435e-38f ? 1.17549435e-38f : f;
        const uint32_t flags = head.z;
        if (!warp_wait(&bars[kSFull0 + b], (count / kSBufs) & 1, p.err, abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t s_cols = lane_addr + kColS + b * kKeys + half * 64;
        if (__builtin_expect(flags != 0u, 0)) {
          if ((flags & 8u) && warp == 4 && lane == 0) {
            p.uneven[t.r] = 1;  // for the direct kernel
            p.any[0] = 1;
          }
          if (flags & 3u) {  // bases by key
            scale_scores<64>(s_cols, qf, (flags & 1u) ? meta.key_kf + half * 64 : nullptr, f,
                             (flags & 2u) ? meta.key_vb + half * 64 : nullptr, vb);
            f = 1.f;
            vb = 0.f;
          }
          if (flags & 4u)
            for (int g = 0; g < NB; ++g)
              if (meta.nan_pos[g] <= pos) nan_groups |= 1u << g;
        }
        // causal mask (only tiles reaching past the tile's first row)
        const int key0 = j * kKeys + half * 64;
        if (key0 + 63 > pos_min) mask_scores(s_cols, pos_min + 1 - key0, pos + 1 - key0);
        float sv[64];
        {
          uint32_t (&r)[64] = *reinterpret_cast<uint32_t(*)[64]>(&sv);
          tmem_ld32(s_cols, *reinterpret_cast<uint32_t(*)[32]>(&r[0]));
          tmem_ld32(s_cols + 32, *reinterpret_cast<uint32_t(*)[32]>(&r[32]));
          tmem_wait_ld();
        }
        // row max: four chains of three-input maxima
        float m4[4] = {sv[0], sv[1], sv[2], sv[3]};
#pragma unroll
        for (int c = 4; c < 60; c += 8)
#pragma unroll
          for (int k = 0; k < 4; ++k) m4[k] = fmax3(m4[k], sv[c + k], sv[c + 4 + k]);
#pragma unroll
        for (int k = 0; k < 4; ++k) m4[k] = fmaxf(m4[k], sv[60 + k]);
        const float x_max = fmax3(m4[0], m4[1], fmaxf(m4[2], m4[3]));
        const float m_mine = fmaf(x_max, f, vb);
        const float mx = fmaxf(m_mine, exchange(m_mine));  // row max of the key tile
        const bool keyed = (flags & 3u) != 0u;
        float mw = x_max * f;
        if (j == 0) m_used = mx - ((flags & 16u) ? kMoved : kFirst);  // key 0 is visible to every row
        float up = m_used - vb;
        // both warps of the quadrant see the same mx and m_used
        const bool grow = mx > m_used + kRescaleThreshold;
        bool summed = false;
        // one vote for everything that is rare
        if (__any_sync(0xffffffffu, grow || keyed || mw > ml + kRescaleThreshold || up - ml > kApart)) {
          if (__any_sync(0xffffffffu, grow)) {
            // O must hold PV of the previous key tile before it is rescaled
            const uint32_t prev = count - 1;
            if (!warp_wait(&bars[kODone0 + prev % kSBufs], (prev / kSBufs) & 1, p.err, abort_flag)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const float alpha = grow ? exp2_approx(m_used - mx + kMoved) : 1.f;
            if (grow) m_used = mx - kMoved;
            rescale<D / 2>(o_cols, alpha);
            up = m_used - vb;
          }
          const float* key_vb = (flags & 2u) ? meta.key_vb + half * 64 : nullptr;
          if (keyed) mw = max_scores<64>(s_cols, key_vb, __uint_as_float(head.y));
          move_reference(mw, ml, l);
          summed = __any_sync(0xffffffffu, keyed || weights_lost(mw, vb, m_used, ml));
          if (summed)
            l += sum_scores<64>(s_cols, f, keyed ? key_vb : nullptr, keyed ? __uint_as_float(head.y) : 0.f, ml);
        }
        const float lw = summed ? 0.f : weight_factor(up, ml);
        // P = 2^(s f + vb - m_used) as f16 pairs over the first 32 of this warp's 64 S
        // columns
        const float2 f2 = make_float2(f, f), c2 = make_float2(-up, -up);
        float2 l2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        uint32_t w[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const float2 x = __ffma2_rn(make_float2(sv[2 * e], sv[2 * e + 1]), f2, c2);
          const float2 pe = make_float2(exp2_approx(x.x), exp2_approx(x.y));
          l2[e & 1] = __fadd2_rn(l2[e & 1], pe);
          w[e] = pack_f16(pe.x, pe.y);
        }
        tmem_st32(s_cols, w);
        l = fmaf((l2[0].x + l2[1].x) + (l2[0].y + l2[1].y), lw, l);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&bars[kPFull0 + b]);
          mbar_arrive(&bars[kMFree0 + ms]);
        }
      }
      if (!ok) break;
      // ---- epilogue: O 2^m / (l_0 2^ml_0 + l_1 2^ml_1) -> out ----
      if (!warp_wait(&bars[kOFinal], tiles_done & 1, p.err, abort_flag)) break;
      ++tiles_done;
      tc_fence_after();
      const float ml_other = exchange(ml), l_other = exchange(l);
      const float top = fmaxf(ml, ml_other);  // a score: key 0 is visible to every row
      const float inv = 1.f / fmaf(l, exp2_approx(ml - top), l_other * exp2_approx(ml_other - top));
      const float root = exp2_approx(0.5f * (m_used - top));  // its square may be too small for a float
      // This warp holds output dims [half * D/2, half * D/2 + D/2) of its 32
      // rows: NV 16-byte pieces per row, transposed among groups of NV lanes so
      // that every store instruction writes whole rows' segments.
      constexpr int NV = D / 16;
      uint4 seg[NV];
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        uint32_t r0[32];
        tmem_ld32(lane_addr + kColO + half * (D / 2) + c * 32, r0);
        tmem_wait_ld();
        // these 32 dimensions are one scale group of V
        const float s = (nan_groups >> (half * (D / 64) + c)) & 1u ? __uint_as_float(0x7fffffffu) : inv;
#pragma unroll
        for (int q4 = 0; q4 < 4; ++q4) {
          uint4& v = seg[c * 4 + q4];
          float x[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = __uint_as_float(r0[q4 * 8 + e]) * s * root * root;
          v.x = pack_bf16(x[0], x[1]);
          v.y = pack_bf16(x[2], x[3]);
          v.z = pack_bf16(x[4], x[5]);
          v.w = pack_bf16(x[6], x[7]);
        }
      }
      transpose_lane_groups<NV>(seg, lane);
      // lane NV g + j now holds piece j of rows NV g + k (k < NV) of the warp
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int trow = quad * 32 + (lane & ~(NV - 1)) + k;  // tile row
        if (trow / G < t.ntok) {
          __nv_bfloat16* dst = p.out + (t.qs + t.u0 + trow / G) * p.out_stride +
                               static_cast<int64_t>(t.h * G + trow % G) * D + half * (D / 2) +
                               (lane & (NV - 1)) * 8;
          *reinterpret_cast<uint4*>(dst) = seg[k];
        }
      }
      tc_fence_before();
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 2) tmem_dealloc(tmem, kTmemCols);
}

// Makes the images: a CTA takes one at a time, warps 0-3 its K rows and 4-7 its V rows,
// 32 each, to shared memory in the tile's layout and from there in one copy a warp.
// Also decides which requests have images, and reports bad metadata.
template <int D>
__global__ void __launch_bounds__(256) expand_mxfp4_kernel(const Params p) {
  constexpr int NB = D / 32, NDH = D / 64;
  constexpr uint32_t kHalf = Layout<D>::kHalf, kPart = kHalf / 4;
  extern __shared__ __align__(128) uint8_t parts[];  // [8 warps][kPart]
  int32_t* prefix = reinterpret_cast<int32_t*>(parts + 8 * kPart);  // [R + 1]: key tiles
  struct Found {
    int most, least;  // of the warp's rows' largest scales (least: as unsigned, -1 none)
    int uneven;       // whether a row of V has uneven groups
    int nan_pos[4];   // by group; 0x7fffffff: none
  };
  __shared__ Found found[2][8];
  // the kernel before may write the cache or the metadata, or read the images
  grid_dependency_wait();
  if (threadIdx.x == 0) grid_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int R = p.num_reqs, tpt = kRows / p.group;
  bool bad = false;
  for (int r = threadIdx.x; r < R; r += blockDim.x) {
    const int tiles = request_tiles(p, r, tpt, &bad) / p.hkv;
    const int keys = tiles < kImageQueryTiles ? 0 : (__ldg(p.seq_lens + r) - 1) / kKeys + 1;
    prefix[r + 1] = keys < kImageKeyTiles ? 0 : keys;
  }
  if (threadIdx.x == 0) prefix[0] = 0;
  if (bad && blockIdx.x == 0) atomicOr(p.err, PKV_ERR_METADATA);
  __syncthreads();
  block_inclusive_scan(prefix + 1, R, prefix + R + 1);
  __syncthreads();
  if (blockIdx.x == 0) {
    bool direct = false, images = false;
    for (int r = threadIdx.x; r < R; r += blockDim.x) {
      const bool has = prefix[r + 1] > prefix[r] && prefix[r + 1] <= p.image_tiles;
      p.image_base[r] = has ? prefix[r] : -1;
      p.uneven[r] = 0;
      images |= has;
      direct |= !has && request_tiles(p, r, tpt, &bad) > 0;
    }
    direct = __syncthreads_or(direct);
    images = __syncthreads_or(images);
    if (threadIdx.x == 0) {
      p.any[0] = direct ? 1 : 0;
      p.any[1] = images ? 1 : 0;
    }
  }

  const bool is_v = warp >= 4;
  const int cw = warp & 3, key = cw * 32 + lane, sw = key % 8, tk = key % kMxBlock;
  const int64_t block_bytes = static_cast<int64_t>(p.hkv) * mx_chunk_bytes(D);
  uint8_t* part = parts + warp * kPart;
  uint8_t* dst = part + (lane / 8) * NDH * 1024 + (key % 8) * 128;
  int turn = 0;
  for (int64_t i = blockIdx.x;; i += gridDim.x, turn ^= 1) {
    const int64_t tile = i / p.hkv;
    if (tile >= prefix[R]) break;
    const int h = static_cast<int>(i - tile * p.hkv);
    int lo = 0, hi = R;  // prefix[lo] <= tile < prefix[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (prefix[mid] <= tile) lo = mid; else hi = mid;
    }
    if (prefix[lo + 1] > p.image_tiles) break;  // and so are the requests after it
    const int pos = static_cast<int>(tile - prefix[lo]) * kKeys + key;
    bool real = pos < __ldg(p.seq_lens + lo);
    int id = real ? __ldg(p.block_table + static_cast<int64_t>(lo) * p.bt_stride + pos / kMxBlock) : 0;
    if (static_cast<uint32_t>(id) >= static_cast<uint32_t>(p.num_blocks)) {
      atomicOr(p.err, PKV_ERR_BLOCK_ID);
      real = false;
      id = 0;
    }
    const uint8_t* chunk = (is_v ? p.value_cache : p.key_cache) +
                           static_cast<uint32_t>(id) * static_cast<uint64_t>(block_bytes) +
                           static_cast<int64_t>(h) * mx_chunk_bytes(D);
    uint4 c[NB];
#pragma unroll
    for (int k = 0; k < NB; ++k) c[k] = __ldg(reinterpret_cast<const uint4*>(chunk + tk * (D / 2)) + k);
    const uint32_t scales =
        is_v ? load_scale_bytes<D, true>(chunk + mx_vscale_off<D>(tk, 0))
             : load_scale_bytes<D, false>(chunk + mx_scale_off(D) + tk * (D / 32));
    // ---- the tile's bases, and the NaN of its V ----
    const int mine = real ? largest_scale<D>(scales) : -1;
    const int most = __reduce_max_sync(0xffffffffu, mine);
    const int least = __reduce_min_sync(0xffffffffu, static_cast<unsigned>(mine));  // -1: largest
    bool uneven = is_v && real && uneven_groups<D>(scales);
    if (__any_sync(0xffffffffu, uneven))
      uneven = __any_sync(0xffffffffu, uneven && uneven_groups<D>(without_zeros<D>(scales, c)));
    Found* mates = found[turn] + (is_v ? 4 : 0);
    if (lane == 0) {
      mates[cw].most = most;
      mates[cw].least = least;
      mates[cw].uneven = uneven ? 1 : 0;
    }
    if (__any_sync(0xffffffffu, is_v && real && nan_scale(scales))) {
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const bool nan = real && ((scales >> (8 * b)) & 0xffu) == 255u;
        const int first = __reduce_min_sync(0xffffffffu, nan ? pos : 0x7fffffff);
        if (lane == 0) mates[cw].nan_pos[b] = first;
      }
    } else if (lane < 4) {
      mates[cw].nan_pos[lane] = 0x7fffffff;
    }
    // (the next turn writes the other half, so one barrier does)
    __syncthreads();
    int base = -1;
    unsigned low = 0xffffffffu;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      base = max(base, mates[w].most);
      low = min(low, static_cast<unsigned>(mates[w].least));
    }
    const bool wide = low != 0xffffffffu && base - static_cast<int>(low) > kWide;
    if (base < 0) base = 127;
    uint8_t* image = p.images + i * static_cast<int64_t>(image_bytes<D>());
    Meta* meta = reinterpret_cast<Meta*>(image + 2 * kHalf);
    if (key == 0) {
      // the V half's thread writes what both know: the K half's by its own reading
      if (is_v) {
        int k_base = -1;
        unsigned k_low = 0xffffffffu, flags = wide ? 2u : 0u;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          k_base = max(k_base, found[turn][w].most);
          k_low = min(k_low, static_cast<unsigned>(found[turn][w].least));
        }
        if (k_low != 0xffffffffu && k_base - static_cast<int>(k_low) > kWide) flags |= 1u;
        if (low != 0xffffffffu && base - static_cast<int>(low) > kLoose) flags |= 16u;
#pragma unroll
        for (int w = 0; w < 4; ++w)
          if (mates[w].uneven) flags |= 8u;
        if (k_base < 0) k_base = 127;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          int first = mates[0].nan_pos[b];
#pragma unroll
          for (int w = 1; w < 4; ++w) first = min(first, mates[w].nan_pos[b]);
          if (first != 0x7fffffff) flags |= 4u;
          meta->nan_pos[b] = first;
        }
        meta->kf = pow2(k_base - 127 - kUp);
        meta->vb = static_cast<float>(base - 127 - kUp);
        meta->flags = flags;
      }
    }
    if (wide) {
      if (mine >= 0) base = mine;
      if (is_v) meta->key_vb[key] = static_cast<float>(base - 127 - kUp);
      else meta->key_kf[key] = pow2(base - 127 - kUp);
    }
    // ---- the rows ----
    uint32_t f[NB];
    if (is_v) row_factors<D, true>(scales, real, base, f); else row_factors<D, false>(scales, real, base, f);
    if (lane == 0) bulk_wait_read<0>();  // the copy before has left shared memory
    __syncwarp();
#pragma unroll
    for (int k = 0; k < NB; ++k) {
      if (is_v) store_piece<D, true>(dst, k, c[k], f, sw); else store_piece<D, false>(dst, k, c[k], f, sw);
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      bulk_store(image + (is_v ? kHalf : 0u) + cw * kPart, part, kPart);
      bulk_commit();
    }
  }
  fence_proxy_async_global();  // the Metas, which the next kernel's copies read
  if (lane == 0) bulk_wait_all();
}

template <int D>
static cudaError_t launch_images_t(Params p, int sms, cudaStream_t stream) {
  const size_t expand_smem = 2 * Layout<D>::kHalf + 4 * (static_cast<size_t>(p.num_reqs) + 1 + 32);
  int entries = p.num_reqs;
  p.entry_shift = 0;
  while (entries > kPrefixMax) {
    ++p.entry_shift;
    entries = (p.num_reqs + (1 << p.entry_shift) - 1) >> p.entry_shift;
  }
  const size_t smem = 1024 + Layout<D>::kPrefix + 4 * (static_cast<size_t>(entries) + 1) + 4 * 32;
  if (smem > kSmemLimit || expand_smem > kSmemLimit) return cudaErrorInvalidValue;
  cudaError_t e = raise_smem_limit_once<expand_mxfp4_kernel<D>>(kSmemLimit - 1024);
  if (e != cudaSuccess) return e;
  e = raise_smem_limit_once<prefill_mxfp4_images_kernel<D>>(kSmemLimit);
  if (e != cudaSuccess) return e;
  e = launch_programmatic(expand_mxfp4_kernel<D>, dim3(static_cast<unsigned>(3 * sms)), dim3(256),
                          expand_smem, stream, p);
  if (e != cudaSuccess) return e;
  return launch_programmatic(prefill_mxfp4_images_kernel<D>, dim3(static_cast<unsigned>(sms)),
                             dim3(kThreads), smem, stream, p);
}

static cudaError_t launch_images(Params p, int head_dim, int sms, cudaStream_t stream) {
  if (head_dim == 128) return launch_images_t<128>(p, sms, stream);
  if (head_dim == 64) return launch_images_t<64>(p, sms, stream);
  return cudaErrorNotSupported;
}

int64_t prefill_mxfp4_image_bytes(int num_kv_heads, int head_dim) {
  return static_cast<int64_t>(num_kv_heads) * (head_dim == 128 ? image_bytes<128>() : image_bytes<64>());
}

cudaError_t launch_prefill_mxfp4(const AttnArgs& a, const MxPrefillScratch& ws, int max_query_len,
                                 int sms, cudaStream_t stream) {
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
  p.entry_shift = 0;
  p.images = nullptr;
  p.image_base = nullptr;
  p.uneven = nullptr;
  p.any = nullptr;
  p.image_tiles = ws.image_tiles;
  // where the longest query, the room or the table's width says that no request can have
  // images, nothing looks for them
  if (ws.image_tiles >= kImageKeyTiles && p.bt_width > (kImageKeyTiles - 1) * (kKeys / kMxBlock) &&
      (max_query_len == 0 || max_query_len > (kImageQueryTiles - 1) * (kRows / p.group))) {
    p.images = ws.images;
    p.any = ws.image_base;
    p.image_base = ws.image_base + 2;
    p.uneven = p.image_base + a.num_reqs;
    const cudaError_t e = launch_images(p, a.head_dim, sms, stream);
    if (e != cudaSuccess) return e;
  }
  return launch_prefill_mxfp4_direct(p, a.head_dim, sms, stream);
}

}  // namespace pkv
