// Chunked-prefill attention over the 4-bit paged cache on the 5th-generation tensor
// cores, with the conversion of keys and values inside: rows of requests with query
// length > 1 whose key tiles are not converted ahead (mxfp4_prefill_images.cu).
//
// For a query row at position p and KV head g, out = softmax_{j <= p}(scale <q, K_j>)
// V_j with K, V the values that codes and power-of-two scales stand for (mxfp4.cuh).
//
// Tiling is that of the bfloat16 prefill: 128 rows = floor(128 / G) query tokens x the G
// query heads of a KV head against key tiles of 128, S = Q K^T and O += P V as tcgen05
// products, S and O in tensor memory, P written over S.  The operands are f16, and the
// copies are made by eight warps that convert:
//   - Thread t of four warps takes key t of every key tile, 64 code bytes of K (the
//     other four: of V; head_dim 128): one conversion a pair, one f16x2 product by its
//     group's scale, one 16-byte store per 8 dimensions, in the 128-byte swizzled layout
//     that both operands read.  Codes of the next tile are loaded while this one is
//     converted.  Each warp's 32 keys share the base exponents of mxfp4_prefill.cuh.
//   - Q is brought to f16 by a power of two per row, as in the decode.
//   - A V group that is NaN is stored as zeros, and its position noted; a row at or
//     behind it gets NaN in that group's dimensions.  (0 times NaN would poison the rows
//     before it.)
//
// Two sweeps.  The warps that convert V note a key whose groups are too far apart for f16
// (mxfp4_prefill.cuh); a CTA that has met one goes through its query tiles again, V and P in
// bfloat16, and writes their rows again.  Also here, in the second sweep alone, are the rows
// of requests in whose images such a key was found.  The sweeps are code of their own: the
// roles share the instruction cache, and with one loop for both a prompt of 4096 tokens took
// 168 us in place of 159.  Normal rows of 32 query and 8 KV heads of 128 with one group 2^20 times
// the others: 512 tokens 48 us (23 without), behind 2048 138 (43), 4096 tokens 756 (147).
//
// What bounds it: the conversion, which runs again for every query tile and takes issue
// slots and instruction cache from the softmax.  32 query and 8 KV heads of 128, in a graph:
// 512 tokens 23 us, 2048 75 us, 4096 242 us; converted ahead 2048 62 and 4096 161.
//
// Warp roles (20 warps): warp 0 owns the tensor memory and issues Q K^T; warp 1 issues P
// V; warps 4-11 run the softmax and the epilogue, two per 32-lane quadrant of tensor
// memory, each with half of the key tile's columns; warps 12-15 convert Q and K, warps
// 16-19 V.
// Every wait is bounded; a timeout sets PKV_ERR_TIMEOUT and an abort flag that stops all
// roles.
#include "mxfp4_prefill.cuh"

namespace pkv {

using namespace mxprefill;

namespace {

constexpr int kKStages = 3;
constexpr int kVStages = 2;
constexpr int kSBufs = 3;
constexpr int kMetas = 4;            // key tiles whose scales are in flight
constexpr int kThreads = 640;
// Registers a thread by role (setmaxnreg; five warpgroups of 96 at launch): the
// softmax holds 64 scores, the converting warps two rows of codes.
constexpr int kLaunchRegs = 96, kIssueRegs = 32, kSoftmaxRegs = 152, kConvertRegs = 72;
static_assert(kIssueRegs + 2 * kSoftmaxRegs + 2 * kConvertRegs <= 5 * kLaunchRegs,
              "the roles' registers fit in what the block is launched with");
static_assert(kThreads * kLaunchRegs <= 65536, "and those in an SM");
constexpr uint32_t kColS = 0;
constexpr uint32_t kColO = kSBufs * kKeys;

enum Bar {
  kQFull, kQEmpty,
  kKFull0, kKEmpty0 = kKFull0 + kKStages,
  kVFull0 = kKEmpty0 + kKStages, kVEmpty0 = kVFull0 + kVStages,
  kSFull0 = kVEmpty0 + kVStages, kSFree0 = kSFull0 + kSBufs,
  kPFull0 = kSFree0 + kSBufs, kODone0 = kPFull0 + kSBufs,
  kOFinal = kODone0 + kSBufs, kPair0,
  kMFull0 = kPair0 + 4, kMFree0 = kMFull0 + kMetas,
  kNumBars = kMFree0 + kMetas
};

// What the softmax has to know of one key tile: by converting warp (32 keys), and
// by key where a warp's keys are far apart.  The K warps write kf, k_flags, key_kf
// and qf, the V warps the rest.
struct alignas(16) Meta {
  float kf[4];           // K base: 2^(base - 127 - kUp)
  float vb[4];           // V base: base - 127 - kUp, log2 units
  uint32_t k_flags[4];   // 1: K by key
  uint32_t v_flags[4];   // 2: V by key (always, in the second sweep), 4: NaN in V, 16: loose V
  int32_t nan_pos[4][4]; // first key position with a NaN V group, by warp and group
  float key_kf[kKeys];
  float key_vb[kKeys];
  float qf[kRows];       // per row, with the query tile's first key tile
};

template <int D>
struct Layout {
  static constexpr int NDH = D / 64;
  static constexpr uint32_t kHalf = NDH * kRegion;  // one K (or V or Q) tile
  static constexpr uint32_t kQ = 0;
  static constexpr uint32_t kK = kQ + kHalf;
  static constexpr uint32_t kV = kK + kKStages * kHalf;
  static constexpr uint32_t kBars = kV + kVStages * kHalf;
  static constexpr uint32_t kXch = (kBars + 8 * kNumBars + 15) / 16 * 16;  // [2 parity][2 half][128 rows] floats
  static constexpr uint32_t kMeta = kXch + 2 * 2 * 128 * 4;
  // tensor memory slot, abort flag, whether there is a second sweep, and whether that alone
  static constexpr uint32_t kMisc = kMeta + kMetas * sizeof(Meta);
  static constexpr uint32_t kPrefix = kMisc + 16;
  static_assert(kMeta % alignof(Meta) == 0 && kBars % 8 == 0, "vector loads of Meta, and the barriers");
};

// Whether this CTA's first sweep is left out: requests are among its that are known to be
// uneven.
template <int D>
__device__ __forceinline__ bool only_second_sweep(const uint8_t* smem) {
  return *reinterpret_cast<const volatile int*>(smem + Layout<D>::kMisc + 12) != 0;
}

// Between the sweeps: all warps are through with the first one, and whether there is a
// second.  (Every role comes here, whatever ended its loop.)
template <int D>
__device__ __forceinline__ bool second_sweep(uint8_t* smem) {
  __syncwarp();
  asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory");
  const volatile int* flags = reinterpret_cast<const volatile int*>(smem + Layout<D>::kMisc + 4);
  return flags[0] == 0 && flags[1] != 0;
}

// The converting warps of K (and Q), or of V: warp cw of the four takes keys
// [32 cw, 32 cw + 32) of every key tile.  kBf16 (the second sweep): V as bfloat16, every key
// with a base of its own.  `count` and `tiles` are the key and query tiles so far.
template <int D, bool kIsV, bool kBf16>
__device__ __forceinline__ void convert_sweep(const Params& p, uint8_t* smem, const int32_t* prefix,
                                              int entries, int total, int tpt, int cw, uint32_t& count,
                                              uint32_t& tiles) {
  using L = Layout<D>;
  constexpr int NDH = L::NDH;
  constexpr int NB = D / 32;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBars);
  Meta* metas = reinterpret_cast<Meta*>(smem + L::kMeta);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMisc + 4);
  const int lane = threadIdx.x & 31, cid = blockIdx.x, ncta = gridDim.x;
  const int key = cw * 32 + lane;
  const int64_t block_bytes = static_cast<int64_t>(p.hkv) * mx_chunk_bytes(D);
  // where this thread's row starts in a stage, and its swizzle
  const uint32_t row_off = (key / 8) * NDH * 1024 + (key % 8) * 128;
  const int sw = key % 8, tk = key % kMxBlock;
  bool ok = true;
  for (int it = 0, ct = cta_tile(0, cid, ncta, total); ct >= 0 && ok;
       ct = cta_tile(++it, cid, ncta, total), ++tiles) {
    if (__shfl_sync(0xffffffffu, *abort_flag, 0)) break;
    const Tile t = find_tile<false>(ct, prefix, entries, p, tpt);
    // This thread's block of the next key tile, and where a block's row of it is;
    // `left` keys of the request from this thread's on (none: not a key, block 0
    // is read and its factors are 0).
    const int32_t* ids = p.block_table + static_cast<int64_t>(t.r) * p.bt_stride + key / kMxBlock;
    int left = t.nkeys - key;
    const uint8_t* head =
        (kIsV ? p.value_cache : p.key_cache) + static_cast<int64_t>(t.h) * mx_chunk_bytes(D);
    const uint8_t* codes_at = head + tk * (D / 2);
    const uint8_t* scales_at = head + (kIsV ? mx_vscale_off<D>(tk, 0) : mx_scale_off(D) + tk * (D / 32));
    auto load_id = [&](int ahead) -> int { return left > ahead * kKeys ? __ldg(ids + 8 * ahead) : 0; };
    auto load_scales = [&](int id) -> uint32_t {
      return load_scale_bytes<D, kIsV>(scales_at + static_cast<uint32_t>(id) * static_cast<uint64_t>(block_bytes));
    };
    // id of a key tile this thread has a key in, checked; 0 where it is not in the pool
    auto checked = [&](int id, int ahead, bool& real) -> int {
      real = left > ahead * kKeys;
      if (static_cast<uint32_t>(id) >= static_cast<uint32_t>(p.num_blocks)) {
        atomicOr(p.err, PKV_ERR_BLOCK_ID);
        real = false;
        id = 0;
      }
      return id;
    };
    bool real, next_real = false;
    const int id = checked(load_id(0), 0, real);
    int next_id = load_id(1);
    const uint4* codes = reinterpret_cast<const uint4*>(
        codes_at + static_cast<uint32_t>(id) * static_cast<uint64_t>(block_bytes));
    uint4 c[NB];  // this key's codes: of the current tile, piece by piece replaced by the next's
#pragma unroll
    for (int i = 0; i < NB; ++i) c[i] = __ldg(codes + i);
    uint32_t scales = load_scales(id), next_scales = 0u;
    float qf = 0.f;

    // ---- Q: thread t of the K warps brings row t to f16 ----
    if constexpr (!kIsV) {
      // the tile before is done with the buffer
      ok = convert_q_row<D, 8, 4>(p, t, key, smem + L::kQ, qf, [&]() {
        return tiles == 0 || held_warp_wait(&bars[kQEmpty], (tiles - 1) & 1, p.err, abort_flag);
      });
      if (!ok) break;
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[kQFull]);
    }
    constexpr int kStages = kIsV ? kVStages : kKStages;
    constexpr int kFull0 = kIsV ? kVFull0 : kKFull0, kEmpty0 = kIsV ? kVEmpty0 : kKEmpty0;
    constexpr uint32_t kTiles = kIsV ? L::kV : L::kK;
    for (int j = 0; j < t.nkt && ok; ++j, ++count) {
      // the next tile's block, its scales, and the block after it
      next_id = checked(next_id, 1, next_real);
      codes = reinterpret_cast<const uint4*>(
          codes_at + static_cast<uint32_t>(next_id) * static_cast<uint64_t>(block_bytes));
      next_scales = load_scales(next_id);
      next_id = load_id(2);
      // ---- base of the warp's 32 keys ----
      const int mine = real ? largest_scale<D>(scales) : -1;
      int apart;
      int base = common_base(mine, apart);
      const bool wide = kBf16 || apart > kWide;
      const int ms = count % kMetas;
      Meta& meta = metas[ms];
      if (count >= kMetas) {
        ok = held_warp_wait(&bars[kMFree0 + ms], (count / kMetas - 1) & 1, p.err, abort_flag);
        if (!ok) break;
      }
      if constexpr (kIsV) {
        const bool any_nan = __any_sync(0xffffffffu, real && nan_scale(scales));
        if (!kBf16 && real && uneven_groups<D>(scales) && uneven_groups<D>(without_zeros<D>(scales, c)))
          abort_flag[1] = 1;  // there is a second sweep
        if (lane == 0) {
          meta.vb[cw] = static_cast<float>(base - 127 - kUp);
          meta.v_flags[cw] = (wide ? 2u : 0u) | (any_nan ? 4u : 0u) | (apart > kLoose ? 16u : 0u);
        }
        if (wide) {
          if (mine >= 0) base = mine;
          meta.key_vb[key] = static_cast<float>(base - 127 - (kBf16 ? 0 : kUp));
        }
        if (any_nan) {
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            const bool nan = real && ((scales >> (8 * b)) & 0xffu) == 255u;
            const int first = __reduce_min_sync(0xffffffffu, nan ? j * kKeys + key : 0x7fffffff);
            if (lane == 0) meta.nan_pos[cw][b] = first;
          }
        }
      } else {
        if (lane == 0) {
          meta.kf[cw] = pow2(base - 127 - kUp);
          meta.k_flags[cw] = wide ? 1u : 0u;
        }
        if (wide) {
          if (mine >= 0) base = mine;
          meta.key_kf[key] = pow2(base - 127 - kUp);
        }
        if (j == 0) meta.qf[key] = qf;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[kMFull0 + ms]);

      // ---- the row, to its stage ----
      uint32_t f[NB];
      if constexpr (kBf16) row_factors_bf16<D>(scales, real, base, f);
      else row_factors<D, kIsV>(scales, real, base, f);
      const int st = count % kStages;
      if (count >= kStages) {
        ok = held_warp_wait(&bars[kEmpty0 + st], (count / kStages - 1) & 1, p.err, abort_flag);
        if (!ok) break;
      }
      uint8_t* dst = smem + kTiles + st * L::kHalf + row_off;
      // One piece of the row at a time, the next tile's taking its place behind the
      // others: a short loop, because the roles' code shares the instruction cache
      // (unrolled, the kernel took longer by a tenth).
#pragma unroll 1
      for (int i = 0; i < NB; ++i) {
        const uint4 piece = c[0];
#pragma unroll
        for (int e = 0; e < NB - 1; ++e) c[e] = c[e + 1];
        c[NB - 1] = __ldg(codes + i);
        store_piece<D, kIsV, kBf16>(dst, i, piece, f, sw);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[kFull0 + st]);
      scales = next_scales;
      real = next_real;
      ids += 8;
      left -= kKeys;
    }
  }
}

// Issues the products P V of this CTA's query tiles (one thread).  kPairs (the second
// sweep): P and V are bfloat16, and what P rounds off is a product of its own.
template <int D, bool kPairs>
__device__ __forceinline__ void weights_sweep(const Params& p, uint8_t* smem, const int32_t* prefix, int entries,
                                              int total, int tpt, uint32_t tmem, uint32_t& count) {
  using L = Layout<D>;
  constexpr int NDH = L::NDH;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMisc + 4);
  const int cid = blockIdx.x, ncta = gridDim.x;
  constexpr uint32_t idesc_o = kPairs ? idesc_bf16_f32(kRows, D, 1) : idesc_f16_f32(kRows, D, 1);
  // V stage, MN-major: 64-dim atoms of a group of 8 keys 1 KiB apart, groups
  // of 8 keys NDH KiB apart
  const uint64_t v_desc0 = smem_desc_sw128(smem_u32(smem + L::kV), 1024, NDH * 1024);
  bool ok = true;
  for (int it = 0, ct = cta_tile(0, cid, ncta, total); ct >= 0 && ok && !*abort_flag;
       ct = cta_tile(++it, cid, ncta, total)) {
    const Tile t = find_tile<false>(ct, prefix, entries, p, tpt);
    for (int j = 0; j < t.nkt && ok; ++j, ++count) {
      const int vs = count % kVStages, b = count % kSBufs;
      ok = held_wait(&bars[kPFull0 + b], (count / kSBufs) & 1, p.err, abort_flag) &&
           held_wait(&bars[kVFull0 + vs], (count / kVStages) & 1, p.err, abort_flag);
      if (!ok) break;
      tc_fence_after();
      const uint64_t vd = v_desc0 + ((vs * L::kHalf) >> 4);
      const uint32_t a_p = tmem + kColS + b * kKeys;
      // P columns hold the keys of each softmax half in their first 32 (pairs; what those
      // round off in the others), V rows [64 half, 64 half + 64)
#pragma unroll
      for (int low = 0; low < (kPairs ? 2 : 1); ++low) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            tc_mma_ts(tmem + kColO, a_p + half * 64 + low * 32 + kk * 8,
                      vd + ((((half * 64 + kk * 16) / 8) * NDH * 1024) >> 4), idesc_o,
                      (j > 0 || low > 0 || half > 0 || kk > 0) ? 1u : 0u);
        }
      }
      tc_commit(&bars[kODone0 + b]);
      if (j == t.nkt - 1) tc_commit(&bars[kOFinal]);
      tc_commit(&bars[kSFree0 + b]);
      tc_commit(&bars[kVEmpty0 + vs]);
    }
  }
}

// The softmax and the epilogue of this CTA's query tiles (eight warps).  kPairs (the second
// sweep): V is bfloat16 with a base by key, and so are the weights, two each.
template <int D, bool kPairs>
__device__ __forceinline__ void softmax_sweep(const Params& p, uint8_t* smem, const int32_t* prefix, int entries,
                                              int total, uint32_t tmem, uint32_t& count, uint32_t& pair_uses,
                                              uint32_t& tiles_done) {
  using L = Layout<D>;
  constexpr int NB = D / 32;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBars);
  float* xch = reinterpret_cast<float*>(smem + L::kXch);
  const Meta* metas = reinterpret_cast<const Meta*>(smem + L::kMeta);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMisc + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, cid = blockIdx.x, ncta = gridDim.x;
  const int G = p.group, tpt = kRows / G;
  // Two warps share each 32-lane quadrant of tensor memory (the same 32 rows):
  // warp half h reads S columns [64 h, 64 h + 64), the keys of converting warps
  // 2h and 2h + 1.  They agree on the row maximum every key tile, so one O
  // serves the row; each keeps the partial sum l of its own columns.
  const int quad = warp & 3;
  const int half = (warp - 4) >> 2;
  const int row = quad * 32 + lane;    // tile row = tensor-memory lane
  const uint32_t lane_addr = tmem + (static_cast<uint32_t>(quad * 32) << 16);
  const uint32_t o_cols = lane_addr + kColO + half * (D / 2);
  uint64_t* pair_bar = &bars[kPair0 + quad];
  auto exchange = [&](float mine) -> float {
    float* slot = xch + (pair_uses & 1) * 256;
    slot[half * 128 + row] = mine;
    __syncwarp();
    if (lane == 0) mbar_arrive(pair_bar);
    const bool done = held_warp_wait(pair_bar, pair_uses & 1, p.err, abort_flag);
    ++pair_uses;
    return done ? slot[(half ^ 1) * 128 + row] : mine;
  };
  for (int it = 0, ct = cta_tile(0, cid, ncta, total); ct >= 0;
       ct = cta_tile(++it, cid, ncta, total)) {
    if (__shfl_sync(0xffffffffu, *abort_flag, 0)) break;
    const Tile t = find_tile<false>(ct, prefix, entries, p, tpt);
    const int u = row / G;
    const int pos = t.nc + t.u0 + (u < t.ntok ? u : t.ntok - 1);
    const int pos_min = t.nc + t.u0;
    float m_used = -INFINITY, ml = kNoScore, l = 0.f, qf = 0.f;
    uint32_t nan_groups = 0u;  // V groups that are NaN for this row
    bool ok = true;
    for (int j = 0; j < t.nkt && ok; ++j, ++count) {
      const int b = count % kSBufs, ms = count % kMetas;
      if (!held_warp_wait(&bars[kMFull0 + ms], (count / kMetas) & 1, p.err, abort_flag)) {
        ok = false;
        break;
      }
      const Meta& meta = metas[ms];
      if (j == 0) qf = meta.qf[row];
      float f[2], vb[2];
      const uint4 kfl = *reinterpret_cast<const uint4*>(meta.k_flags);
      const uint4 vfl = *reinterpret_cast<const uint4*>(meta.v_flags);
      const uint32_t flags =  // of anything rare in the key tile
          kfl.x | kfl.y | kfl.z | kfl.w | vfl.x | vfl.y | vfl.z | vfl.w;
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        // never zero, for the masked scores' infinities
        f[g] = qf * meta.kf[2 * half + g];
        f[g] = f[g] < 1.17549435e-38f ? 1.17549435e-38f : f[g];
        vb[g] = meta.vb[2 * half + g];
      }
      if (!held_warp_wait(&bars[kSFull0 + b], (count / kSBufs) & 1, p.err, abort_flag)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t s_cols = lane_addr + kColS + b * kKeys + half * 64;
      uint32_t keyed = 0u;  // this warp's groups of 32 keys with bases by key
      if (__builtin_expect(flags != 0u, 0)) {
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const bool by_k = meta.k_flags[2 * half + g] != 0u;
          const bool by_v = (meta.v_flags[2 * half + g] & 2u) != 0u;
          if (by_k || by_v) {
            keyed |= 1u << g;
            const int key = half * 64 + g * 32;
            scale_scores<32>(s_cols + 32 * g, qf, by_k ? meta.key_kf + key : nullptr, f[g],
                             by_v ? meta.key_vb + key : nullptr, vb[g]);
            f[g] = 1.f;
            vb[g] = 0.f;
          }
        }
        for (int c = 0; c < 4; ++c)
          if (meta.v_flags[c] & 4u)
            for (int g = 0; g < NB; ++g)
              if (meta.nan_pos[c][g] <= pos) nan_groups |= 1u << g;
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
      float mg[2], mw[2];  // the groups' largest s + v, and s
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        float m4[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) m4[c] = sv[32 * g + c];
#pragma unroll
        for (int c = 4; c < 28; c += 8)
#pragma unroll
          for (int k = 0; k < 4; ++k) m4[k] = fmax3(m4[k], sv[32 * g + c + k], sv[32 * g + c + 4 + k]);
        float x = fmax3(m4[0], m4[1], fmax3(m4[2], m4[3], sv[32 * g + 28]));
        x = fmax3(x, sv[32 * g + 29], fmax3(sv[32 * g + 30], sv[32 * g + 31], x));
        mg[g] = fmaf(x, f[g], vb[g]);
        mw[g] = x * f[g];
      }
      const float m_mine = fmaxf(mg[0], mg[1]);
      const float mx = fmaxf(m_mine, exchange(m_mine));  // row max of the key tile
      if (j == 0) m_used = mx - ((flags & 16u) ? kMoved : kFirst);  // key 0 is visible to every row
      float up[2] = {m_used - vb[0], m_used - vb[1]};
      // both warps of the quadrant see the same mx and m_used
      const bool grow = mx > m_used + kRescaleThreshold;
      uint32_t summed = 0u;  // groups whose weights are summed already
      // one vote for everything that is rare
      if (__any_sync(0xffffffffu, grow || keyed != 0u || fmaxf(mw[0], mw[1]) > ml + kRescaleThreshold ||
                                      fmaxf(up[0], up[1]) - ml > kApart)) {
        if (__any_sync(0xffffffffu, grow)) {
          // O must hold PV of the previous key tile before it is rescaled
          const uint32_t prev = count - 1;
          if (!held_warp_wait(&bars[kODone0 + prev % kSBufs], (prev / kSBufs) & 1, p.err, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const float alpha = grow ? exp2_approx(m_used - mx + kMoved) : 1.f;
          if (grow) m_used = mx - kMoved;
          rescale<D / 2>(o_cols, alpha);
        }
        const float* key_vb[2];
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          up[g] = m_used - vb[g];
          key_vb[g] = (meta.v_flags[2 * half + g] & 2u) ? meta.key_vb + half * 64 + g * 32 : nullptr;
          if ((keyed >> g) & 1u) mw[g] = max_scores<32>(s_cols + 32 * g, key_vb[g], meta.vb[2 * half + g]);
        }
        move_reference(fmaxf(mw[0], mw[1]), ml, l);
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const bool by_key = (keyed >> g) & 1u;
          if (!__any_sync(0xffffffffu, by_key || weights_lost(mw[g], vb[g], m_used, ml))) continue;
          l += sum_scores<32>(s_cols + 32 * g, f[g], by_key ? key_vb[g] : nullptr,
                              by_key ? meta.vb[2 * half + g] : 0.f, ml);
          summed |= 1u << g;
        }
      }
      if constexpr (kPairs) {  // (every group's weights are summed already)
        split_weights(s_cols, m_used);
      } else {
        float lw[2];
#pragma unroll
        for (int g = 0; g < 2; ++g) lw[g] = (summed >> g) & 1u ? 0.f : weight_factor(up[g], ml);
        // P = 2^(s f + vb - m_used) as f16 pairs over the first 32 of this
        // warp's 64 S columns
        uint32_t w[32];
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const float2 f2 = make_float2(f[g], f[g]);
          const float2 c2 = make_float2(-up[g], -up[g]);
          float2 l2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float2 x = __ffma2_rn(make_float2(sv[32 * g + 2 * e], sv[32 * g + 2 * e + 1]), f2, c2);
            const float2 pe = make_float2(exp2_approx(x.x), exp2_approx(x.y));
            l2[e & 1] = __fadd2_rn(l2[e & 1], pe);
            w[16 * g + e] = pack_f16(pe.x, pe.y);
          }
          l = fmaf((l2[0].x + l2[1].x) + (l2[0].y + l2[1].y), lw[g], l);
        }
        tmem_st32(s_cols, w);
      }
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
    if (!held_warp_wait(&bars[kOFinal], tiles_done & 1, p.err, abort_flag)) break;
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

// Out of the way of the code that always runs, for head_dim 64: 512 tokens of 16/4 heads take
// 18.4 us instead of 18.9, 128 behind 23190 243 instead of 274.  (128: 41.0 instead of 35.6
// for 64 tokens behind 2048.)
__device__ __noinline__ void convert_again_64(const Params& p, uint8_t* smem, const int32_t* prefix, int entries,
                                              int total, int tpt, int cw, uint32_t count, uint32_t tiles) {
  convert_sweep<64, true, true>(p, smem, prefix, entries, total, tpt, cw, count, tiles);
}

}  // namespace

template <int D>
__global__ void __launch_bounds__(kThreads, 1) prefill_mxfp4_kernel(const Params p) {
  using L = Layout<D>;
  constexpr int NDH = L::NDH;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBars);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMisc + 4);
  int32_t* prefix = reinterpret_cast<int32_t*>(smem + L::kPrefix);

  // the kernel before may write q, the cache, out or the metadata
  grid_dependency_wait();
  if (threadIdx.x == 0) grid_launch_dependents();
  if (p.images != nullptr && __ldcg(p.any) == 0) return;  // images serve every row
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int R = p.num_reqs;
  const int entries = (R + (1 << p.entry_shift) - 1) >> p.entry_shift;
  int32_t* scan_tmp = prefix + entries + 1;
  const int cid = blockIdx.x, ncta = gridDim.x;
  const int tpt = kRows / p.group;  // query tokens per tile

  // ---- plan: tiles per entry and their prefix sum ----
  if (threadIdx.x == 0) {
    abort_flag[0] = 0;
    prefix[0] = 0;
    for (int b = 0; b < kNumBars; ++b) {
      uint32_t n = 1;
      if (b == kQFull || (b >= kKFull0 && b < kKFull0 + kKStages) ||
          (b >= kVFull0 && b < kVFull0 + kVStages))
        n = 4;  // the converting warps of K (Q too) or V
      if (b >= kMFull0 && b < kMFull0 + kMetas) n = 8;  // all converting warps
      if ((b >= kPFull0 && b < kPFull0 + kSBufs) || (b >= kMFree0 && b < kMFree0 + kMetas))
        n = 8;  // softmax warps
      if (b >= kPair0 && b < kPair0 + 4) n = 2;  // the two warps sharing a quadrant
      mbar_init(&bars[b], n);
    }
    fence_mbar_init();
  }
  bool bad = false;
  for (int i = threadIdx.x; i < entries; i += blockDim.x) {
    int n = 0;
    for (int k = 0; k < (1 << p.entry_shift); ++k) {
      const int r = (i << p.entry_shift) + k;
      if (r < R) n += own_tiles<false>(p, r, tpt, &bad);
    }
    prefix[i + 1] = n;
  }
  if (bad && cid == 0) atomicOr(p.err, PKV_ERR_METADATA);
  bool uneven = false;
  if (p.images != nullptr)
    for (int r = threadIdx.x; r < R; r += blockDim.x) uneven |= __ldcg(p.uneven + r) != 0;
  uneven = __syncthreads_or(uneven);
  if (threadIdx.x == 0) abort_flag[1] = abort_flag[2] = uneven ? 1 : 0;
  block_inclusive_scan(prefix + 1, entries, scan_tmp);
  __syncthreads();
  const int total = prefix[entries];
  if (cid >= total) return;  // no tile for this CTA, and no tensor memory held
  if (warp == 0) {
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
      // ============================ QK^T issuer ============================
      constexpr uint32_t idesc_s = idesc_f16_f32(kRows, kKeys, 0);
      const uint64_t q_desc = smem_desc_sw128(smem_u32(smem + L::kQ), 16, 1024);
      // K stage: groups of 8 keys every NDH KiB, dim half dh at +dh KiB
      const uint64_t k_desc0 = smem_desc_sw128(smem_u32(smem + L::kK), 16, NDH * 1024);
      uint32_t q_count = 0, count = 0;
#pragma unroll 1
      for (int sweep = 0; sweep < 2; ++sweep) {
        if (lane == 0 && !(sweep == 0 && only_second_sweep<D>(smem))) {
          bool ok = true;
          for (int it = 0, ct = cta_tile(0, cid, ncta, total); ct >= 0 && ok && !*abort_flag;
               ct = cta_tile(++it, cid, ncta, total)) {
            const Tile t = find_tile<false>(ct, prefix, entries, p, tpt);
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
              // (a loop: unrolled, 4096 tokens of 32/8 heads of 128 took 254 us instead of 240)
#pragma unroll 1
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
        if (sweep == 0 && !second_sweep<D>(smem)) break;
      }
    } else if (warp == 1) {
      // ============================ PV issuer ============================
      uint32_t count = 0;
      if (lane == 0 && !only_second_sweep<D>(smem))
        weights_sweep<D, false>(p, smem, prefix, entries, total, tpt, tmem, count);
      if (second_sweep<D>(smem) && lane == 0)
        weights_sweep<D, true>(p, smem, prefix, entries, total, tpt, tmem, count);
    } else {
      second_sweep<D>(smem);
    }
  } else if (warp >= 16) {
    set_registers<kConvertRegs, false>();
    uint32_t count = 0, tiles = 0;
    if (!only_second_sweep<D>(smem))
      convert_sweep<D, true, false>(p, smem, prefix, entries, total, tpt, warp - 16, count, tiles);
    if (second_sweep<D>(smem)) {
      if constexpr (D == 64) convert_again_64(p, smem, prefix, entries, total, tpt, warp - 16, count, tiles);
      else convert_sweep<D, true, true>(p, smem, prefix, entries, total, tpt, warp - 16, count, tiles);
    }
  } else if (warp >= 12) {
    set_registers<kConvertRegs, false>();
    uint32_t count = 0, tiles = 0;
#pragma unroll 1
    for (int sweep = 0; sweep < 2; ++sweep) {
      if (sweep == 1 || !only_second_sweep<D>(smem))
        convert_sweep<D, false, false>(p, smem, prefix, entries, total, tpt, warp - 12, count, tiles);
      if (sweep == 0 && !second_sweep<D>(smem)) break;
    }
  } else if (warp >= 4) {
    // ============================ softmax warps ============================
    set_registers<kSoftmaxRegs, true>();
    uint32_t count = 0, pair_uses = 0, tiles_done = 0;
    if (!only_second_sweep<D>(smem))
      softmax_sweep<D, false>(p, smem, prefix, entries, total, tmem, count, pair_uses, tiles_done);
    if (second_sweep<D>(smem))
      softmax_sweep<D, true>(p, smem, prefix, entries, total, tmem, count, pair_uses, tiles_done);
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem, kTmemCols);
}

template <int D>
static cudaError_t launch_prefill_t(Params p, int sms, cudaStream_t stream) {
  int entries = p.num_reqs;
  p.entry_shift = 0;
  while (entries > kPrefixMax) {
    ++p.entry_shift;
    entries = (p.num_reqs + (1 << p.entry_shift) - 1) >> p.entry_shift;
  }
  const size_t smem = 1024 + Layout<D>::kPrefix + 4 * (static_cast<size_t>(entries) + 1) + 4 * 32;
  if (smem > kSmemLimit) return cudaErrorInvalidValue;
  const cudaError_t e = raise_smem_limit_once<prefill_mxfp4_kernel<D>>(kSmemLimit);
  if (e != cudaSuccess) return e;
  return launch_programmatic(prefill_mxfp4_kernel<D>, dim3(static_cast<unsigned>(sms)), dim3(kThreads),
                             smem, stream, p);
}

cudaError_t launch_prefill_mxfp4_direct(Params p, int head_dim, int sms, cudaStream_t stream) {
  if (head_dim == 128) return launch_prefill_t<128>(p, sms, stream);
  if (head_dim == 64) return launch_prefill_t<64>(p, sms, stream);
  return cudaErrorNotSupported;
}

}  // namespace pkv
