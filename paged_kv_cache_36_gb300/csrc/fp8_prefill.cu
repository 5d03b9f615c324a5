// Chunked-prefill attention over the 8-bit paged cache on the 5th-generation tensor cores,
// for the rows of requests with query length > 1.
//
// For a query row at position p and KV head g, out = softmax_{j <= p}(scale <q, K_j>) V_j
// with K, V the values that codes and power-of-two scales stand for (fp8.cuh).  Those are
// exact in bfloat16, so both products are the bfloat16 prefill's: 128 rows = floor(128 / G)
// query tokens x the G query heads of a KV head against key tiles of 128, S = Q K^T and O +=
// P V as tcgen05 products, S and O in tensor memory, P (bfloat16) written over S.
//
// Where K and V tiles come from.
//   - Requests with enough of them have their key tiles converted once, by expand_fp8_kernel,
//     to images in the workspace: K and V as the 128-byte swizzled rows
//     that the tensor core reads, so that a tile is one bulk copy of 16 or 32 KB from L2.
//   - For the others eight warps convert as they go: a warp takes whole blocks, whose codes
//     it reads as D / 32 coalesced vectors, and writes rows to the stage.
//
// Large values.  The reference of a row's weights moves at once in key tiles that hold some
// (kF8Loud), so that sums stay finite; without images a warp notes which.  Over images it does
// so in all key tiles if one of the call's holds some (with a word read for each of them a
// prompt of 16384 tokens took 1434 us instead of 1407).
//
// NaN.  Zero times NaN would poison rows that do not see a NaN in V, so one is stored as
// zero and its position noted by dimension; a row at or behind it gets NaN there.  (In a tile
// that every row sees it is left in V.)
//
// Warp roles: warp 0 owns the tensor memory and issues Q K^T, warp 1 issues P V; over images
// warps 2 and 3 copy K and V; warps 4-11 run the softmax and the epilogue, two per 32-lane
// quadrant of tensor memory, each with half of the key tile's columns; warps 12-15 bring the
// query rows in, and without images they convert K, warps 16-19 V, and warp 2 notes large
// values.
//
// What bounds it.  A prompt of 4096 tokens with 32 query and 8 KV heads of 128 takes 129 us,
// 1065 TFLOP/s, 56 % of the bf16 rate; of 16384 tokens 1400 us, 1571 TFLOP/s, 83 %.  Neither the
// products nor memory bound it, but the chain from S to P: when 16384 tokens took 1489 us they
// took 7 % less without exponentials, 9 without maxima, 6 with an eighth of Q K^T, 5 with a
// quarter of P V.
// Measured and not kept, with what it was measured against (us, a prompt of 4096): two softmax
// groups with key tiles in turn and an S and an O each 150 (136), with P in halves 142 (136);
// rows written by the warps that bring Q 130 (129), with two O and two S 137 (129); two S
// instead of three 137 (129); spinning instead of suspended waits in the issuing warps 147.5
// (146); copies split in 4 KB 150 (146); weights made before the maxima are exchanged 139
// (134); a query tile ended after the next one's first scores 130.6 (128.4).
//
// Every wait is bounded; a timeout sets PKV_ERR_TIMEOUT and an abort flag that stops all
// roles.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "fp8.cuh"
#include "kernels.h"
#include "pkv_device.cuh"
#include "prefill_common.cuh"
#include "tcgen05.cuh"

namespace pkv {

namespace {

constexpr int kRows = 128;
constexpr int kKeys = 128;
constexpr int kTileBlocks = kKeys / kF8Block;
constexpr uint32_t kRegion = 16384;  // 128 rows x 128 bytes
constexpr int kKStages = 3;
constexpr int kVStages = 2;
constexpr int kSBufs = 3;
// Query tiles whose NaN positions are in shared memory (no images).  V of query tile n + 4 is
// converted after P V of n + 2, and so after the epilogue of n + 1.
constexpr int kNanBufs = 4;
// Key tiles of which shared memory says whether they hold large values (no images).  It does of
// tile n after the Q K^T of n - 3, and so after the P V of n - 6.
constexpr int kLoudBufs = 8;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 0;
constexpr uint32_t kColO = kSBufs * kKeys;
// Weights are 2^(score - m): a new reference m puts the largest at 2^kLargest, and m moves when
// 64 of a row add up to more than kMost.  So O is rescaled once a row's maximum has grown by
// 2^26 to 2^32 (2^8, as for bfloat16 caches: a prompt of 4096 tokens 146 us instead of 134), and
// weights vanish (at 2^-126) 102 binades below the largest.  In a key tile of large values
// (kF8Loud) the sum may be kMostLoud, twice that of 64 of the largest: sums over 2^22 of those
// keys stay finite, and over others always.  Only a row's first key tile, and one that moves m,
// needs the maximum itself (found in every tile: a prompt of 16384 tokens 1475 us instead of 1430).
constexpr float kLargest = -24.f, kMost = 256.f, kMostLoud = 1.f / 131072;
constexpr int kPrefixMax = 4096;           // entries of the plan in shared memory
constexpr int kMaxKeys = 0x7fffff00;       // a whole key tile more is still an int
constexpr size_t kSmemLimit = 232448;
constexpr int kNone = 0x7fffffff;          // no NaN
// Which requests have images, by what both ways cost (see expand_fp8_kernel).  In a graph a
// CTA takes some 2.0 us for a key tile of head_dim 128 that it converts and 1.1 over images, of
// 64 1.0 and 0.6; images cost two kernels, 6 to 7 us, and for each key tile and KV head what they
// write and read again.  us over images / converted as they go, without those kernels, 32 query
// and 8 KV heads of 128:
//   tokens 4096 130 / 256, 2048 56 / 79, 1024 30.8 / 31.1, 512 behind 1223 30 / 32, behind 11539
//   80 / 145, 128 behind 3874 34 / 43, 64 behind 2048 31 / 35, 4 behind 8000 65 / 108, 4 behind
//   1000 25 / 23; 8 requests of 256 behind 1000 66 / 80, of 256 40 / 42; 16 of 4 behind 4000 125 /
//   87, 64 of 4 behind 2000 227 / 160 (so 0.014 a key tile and KV head).
//   16 query and 4 KV heads of 64: tokens 4096 61 / 81, 2048 30 / 29, 512 behind 1069 24 / 21, 64
//   behind 4096 38 / 45.
// The host weighs the two kernels, by the most that the batch may be; once they are launched the
// device compares the rest (1024 tokens: 31 us, with the two weighed again 37; 2048 of 16/4
// heads of 64 31 and 35).
constexpr float kImageFixed = 6.5f;
template <int D>
constexpr float image_gain() { return D == 128 ? 0.9f : 0.4f; }     // of a key tile, a CTA
template <int D>
constexpr float image_cost() { return D == 128 ? 0.014f : 0.012f; }  // of a key tile and KV head
constexpr int kManyTiles = 4;  // query tiles from which on reading images often pays for writing them

// Threads, and registers a thread by role (setmaxnreg), over images and without.
template <bool kImages>
struct Shape {
  static constexpr int kThreads = kImages ? 512 : 640;
  static constexpr int kLaunch = kImages ? 128 : 96;
  static constexpr int kIssue = kImages ? 40 : 32, kSoftmax = kImages ? 192 : 152, kConvert = kImages ? 88 : 72;
  static_assert(kIssue + 2 * kSoftmax + (kImages ? 1 : 2) * kConvert <= kThreads / 128 * kLaunch,
                "the roles' registers fit in what the block is launched with");
  static_assert(kThreads * kLaunch <= 65536, "and those in an SM");
};

enum Bar {
  kQFull, kQEmpty,
  kKFull0, kKEmpty0 = kKFull0 + kKStages,
  kVFull0 = kKEmpty0 + kKStages, kVEmpty0 = kVFull0 + kVStages,
  kSFull0 = kVEmpty0 + kVStages, kSFree0 = kSFull0 + kSBufs,
  kPFull0 = kSFree0 + kSBufs, kODone0 = kPFull0 + kSBufs,
  kOFinal = kODone0 + kSBufs, kNanRead, kPair0,
  kNumBars = kPair0 + 4
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
  static constexpr uint32_t kNan = kXch + 2 * 2 * 128 * 4;                 // [kNanBufs][D] positions, [kNanBufs] any
  static constexpr uint32_t kLoud = kNan + kNanBufs * (D + 1) * 4;         // [kLoudBufs]
  static constexpr uint32_t kMisc = kLoud + kLoudBufs * 4;                 // tensor memory slot, abort flag
  static constexpr uint32_t kPrefix = kMisc + 16;
  static_assert(kBars % 8 == 0 && kMisc % 4 == 0, "barriers, and words");
};

// An image: K, V, then the first position of a NaN in V by dimension (where there is one).
template <int D>
__host__ __device__ constexpr uint32_t image_bytes() { return 2 * Layout<D>::kHalf + D * 4; }

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
  int32_t entry_shift;  // requests per plan entry, as a power of two
  // Key tiles converted ahead (null: none): request r's are images image_base[r] hkv on, its
  // key tiles in order, KV head fastest; -1: none, its rows are converted as they are needed.
  // any[0]: whether there are such; any[1]: whether there are images.  image_nan: by image,
  // whether V has a NaN; flags_seen: whether one of this call's has (1), and whether one has
  // large values (2) (zero between calls).
  uint8_t* images;
  int32_t* image_base;
  int32_t* image_nan;
  uint32_t* flags_seen;
  int32_t* any;
  int32_t image_tiles;  // key tiles (of all KV heads) there is room for
  int32_t sms;
};

struct Tile {
  int r, h, u0, ntok;
  int nkeys;   // keys any of the tile's rows sees
  int nkt;     // key tiles
  int64_t qs;
  int nc;
};

// Query tiles of request r (all KV heads); 0 where it has no rows of length > 1 or its
// metadata is wrong (*bad).
__device__ __forceinline__ int request_tiles(const Params& p, int r, int tpt, bool* bad) {
  const int q0 = __ldg(p.qsl + r), q1 = __ldg(p.qsl + r + 1);
  // (offsets that are garbage may be anything apart: those that wrap fail q1 < q0)
  const int qlen = static_cast<int>(static_cast<uint32_t>(q1) - static_cast<uint32_t>(q0));
  if (qlen <= 1) return 0;
  const int seq = __ldg(p.seq_lens + r), nc = __ldg(p.num_computed + r);
  if (q0 < 0 || q1 < q0 || q1 > p.num_tokens || nc < 0 || nc > kMaxKeys - qlen ||
      seq != nc + qlen || (seq - 1) / kF8Block >= p.bt_width) {
    *bad = true;
    return 0;
  }
  return (qlen + tpt - 1) / tpt * p.hkv;
}

// Those of them that are computed from images (kImages), or without.
template <bool kImages>
__device__ __forceinline__ int own_tiles(const Params& p, int r, int tpt, bool* bad) {
  const int n = request_tiles(p, r, tpt, bad);
  if (n == 0 || p.images == nullptr) return kImages ? 0 : n;
  return (__ldcg(p.image_base + r) >= 0) == kImages ? n : 0;
}

// Tile `ct` -> (request, KV head, query rows).  prefix[i] counts the tiles before
// plan entry i; within a request tiles run KV head fastest, then query tiles.
template <bool kImages>
__device__ __forceinline__ Tile find_tile(int ct, const int32_t* prefix, int entries,
                                          const Params& p, int tpt) {
  int lo = 0, hi = entries;  // prefix[lo] <= ct < prefix[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (prefix[mid] <= ct) lo = mid; else hi = mid;
  }
  Tile t;
  t.r = lo << p.entry_shift;
  int rem = ct - prefix[lo];
  if (p.entry_shift > 0) {  // an entry of several requests
    bool bad = false;
    for (int n = own_tiles<kImages>(p, t.r, tpt, &bad); rem >= n;
         n = own_tiles<kImages>(p, t.r, tpt, &bad)) {
      rem -= n;
      ++t.r;
    }
  }
  const int qt = rem / p.hkv;
  t.h = rem - qt * p.hkv;
  t.qs = __ldg(p.qsl + t.r);
  const int qlen = __ldg(p.qsl + t.r + 1) - static_cast<int>(t.qs);
  t.nc = __ldg(p.num_computed + t.r);
  t.u0 = qt * tpt;
  t.ntok = min(tpt, qlen - t.u0);
  t.nkeys = t.nc + t.u0 + t.ntok;
  t.nkt = (t.nkeys - 1) / kKeys + 1;
  return t;
}

// ------------------------------------------------------------------ conversion
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 h = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                   *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&h);
}
// The power of two of a scale byte as a bfloat16 pair.
__device__ __forceinline__ uint32_t scale_pair(int e) { return static_cast<uint32_t>(e << 7) * 0x00010001u; }

// The two of a bfloat16 pair to two sums.  (The rounded weights, so that what rounding does to
// all of a row's cancels: errors of 1.1 of the result's own rounding instead of 1.4.  Adding
// them as they are instead of as two floats: a prompt of 16384 tokens 1406 us instead of 1430.)
__device__ __forceinline__ void add_pair(float2& sum, uint32_t w) {
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "add.rn.f32.bf16 %0, a, %0;\n\t"
      "add.rn.f32.bf16 %1, b, %1;\n\t}"
      : "+f"(sum.x), "+f"(sum.y)
      : "r"(w));
}

// Eight codes times their scale.
__device__ __forceinline__ uint4 eight_values(uint32_t w0, uint32_t w1, uint32_t scale) {
  float x[4], y[4];
  e4m3x4_to_f32(w0, x);
  e4m3x4_to_f32(w1, y);
  return make_uint4(mul_bf16x2(pack_bf16(x[0], x[1]), scale), mul_bf16x2(pack_bf16(x[2], x[3]), scale),
                    mul_bf16x2(pack_bf16(y[0], y[1]), scale), mul_bf16x2(pack_bf16(y[2], y[3]), scale));
}

// One block's codes of a KV head, this lane's vectors, and the scale.
template <int D>
struct Codes {
  uint4 v[D / 32];
  int e;
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int j = 0; j < D / 32; ++j) v[j] = make_uint4(0u, 0u, 0u, 0u);
    e = 127;
  }
  __device__ __forceinline__ void load(const uint8_t* chunk, int lane) {
#pragma unroll
    for (int j = 0; j < D / 32; ++j) v[j] = __ldg(reinterpret_cast<const uint4*>(chunk + j * 512) + lane);
    e = f8_scale(__ldg(chunk + f8_code_bytes(D)));
  }
};

// Rows [16 block, + 16) of a swizzled tile at `tile` from the keys' codes.
template <int D>
__device__ __forceinline__ void store_keys(uint8_t* tile, int block, const Codes<D>& c, int lane) {
  constexpr int NDH = D / 64;
  const int gid = lane >> 2, tid = lane & 3;
  const uint32_t scale = scale_pair(c.e);
#pragma unroll
  for (int j = 0; j < D / 32; ++j) {
    uint8_t* row = tile + ((2 * block + j / NDH) * NDH + j % NDH) * 1024 + gid * 128;
    const uint4& w = c.v[j];
    *reinterpret_cast<uint4*>(row + (((2 * tid) ^ gid) << 4)) = eight_values(w.x, w.y, scale);
    *reinterpret_cast<uint4*>(row + (((2 * tid + 1) ^ gid) << 4)) = eight_values(w.z, w.w, scale);
  }
}

// The same of the values' codes: this lane's vectors are 4 dimensions by 4 tokens.
template <int D>
__device__ __forceinline__ void store_values(uint8_t* tile, int block, const Codes<D>& c, int lane) {
  constexpr int NDH = D / 64, P = D / 8;
  const int gid = lane >> 2, tid = lane & 3;
  const uint32_t scale = scale_pair(c.e);
#pragma unroll
  for (int k = 0; k < P / 8; ++k) {  // eight dimensions, P gid + 8 k on
    const uint32_t w[8] = {c.v[2 * k].x, c.v[2 * k].y, c.v[2 * k].z, c.v[2 * k].w,
                           c.v[2 * k + 1].x, c.v[2 * k + 1].y, c.v[2 * k + 1].z, c.v[2 * k + 1].w};
    uint32_t y[4][4];  // by token, pairs of dimensions
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float a[4], b[4];
      e4m3x4_to_f32(w[2 * i], a);
      e4m3x4_to_f32(w[2 * i + 1], b);
#pragma unroll
      for (int t = 0; t < 4; ++t) y[t][i] = mul_bf16x2(pack_bf16(a[t], b[t]), scale);
    }
    const int d = P * gid + 8 * k;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int in8 = 2 * tid + (t & 1);
      uint8_t* row = tile + ((2 * block + (t >> 1)) * NDH + d / 64) * 1024 + in8 * 128;
      *reinterpret_cast<uint4*>(row + (((d % 64 / 8) ^ in8) << 4)) = make_uint4(y[t][0], y[t][1], y[t][2], y[t][3]);
    }
  }
}

// Whether a word holds a code for NaN; NaN codes made zero, the first position of each
// dimension noted (`first` is the position of the block's row 0).
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }
template <int D>
__device__ __forceinline__ bool has_nan(const Codes<D>& c) {
  uint32_t any = 0u;
#pragma unroll
  for (int j = 0; j < D / 32; ++j) any |= nan_codes(c.v[j].x) | nan_codes(c.v[j].y) | nan_codes(c.v[j].z) | nan_codes(c.v[j].w);
  return any != 0u;
}
template <int D>
__device__ __forceinline__ void note_nan(Codes<D>& c, int32_t* nan, int first, int lane) {
#pragma unroll
  for (int j = 0; j < D / 32; ++j) {
    uint32_t* w = &c.v[j].x;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll 1
      for (uint32_t m = nan_codes(w[i]); m != 0u; m &= m - 1u) {
        const int t = (__ffs(m) - 1) >> 3;
        w[i] &= ~(0xffu << (8 * t));
        atomicMin(&nan[D / 8 * (lane >> 2) + 4 * j + i], first + 2 * (lane & 3) + (t & 1) + 8 * (t >> 1));
      }
  }
}
// Bytes of a V word whose tokens are among a block's first n.
__device__ __forceinline__ uint32_t keep_tokens(int n, int lane) {
  uint32_t keep = 0u;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (2 * (lane & 3) + (i >> 1) * 8 + (i & 1) < n) keep |= 0xffu << (8 * i);
  return keep;
}
template <int D>
__device__ __forceinline__ void keep_codes(Codes<D>& c, uint32_t keep) {
#pragma unroll
  for (int j = 0; j < D / 32; ++j) {
    c.v[j].x &= keep;
    c.v[j].y &= keep;
    c.v[j].z &= keep;
    c.v[j].w &= keep;
  }
}

// ------------------------------------------------------------------ roles
// Copies the K tiles, or the V tiles, of this CTA's query tiles from their images (one thread).
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
  uint32_t count = 0;
  bool ok = true;
  fence_proxy_async_global();  // the images were written with plain stores
  for (int it = 0, ct = cta_tile(0, cid, ncta, total); ct >= 0 && ok && !*abort_flag;
       ct = cta_tile(++it, cid, ncta, total)) {
    const Tile t = find_tile<true>(ct, prefix, entries, p, tpt);
    const uint8_t* image = p.images + __ldcg(p.image_base + t.r) * step +
                           t.h * static_cast<int64_t>(image_bytes<D>()) + (kIsV ? L::kHalf : 0u);
    for (int j = 0; j < t.nkt; ++j, ++count, image += step) {
      const int st = count % kStages;
      ok = count < kStages ||
           held_wait(&bars[kEmpty0 + st], (count / kStages - 1) & 1, p.err, abort_flag);
      if (!ok) break;
      mbar_arrive_expect_tx(&bars[kFull0 + st], L::kHalf);
      bulk_load(smem + (kIsV ? L::kV : L::kK) + st * L::kHalf, image, L::kHalf, &bars[kFull0 + st]);
    }
  }
  // drain: every copy has landed before the CTA may exit
  for (uint32_t back = 1; back <= kStages && back <= count; ++back)
    mbar_wait(&bars[kFull0 + (count - back) % kStages], ((count - back) / kStages) & 1, p.err);
}

// One row of Q, as it is (the scale's sign on it), zeros where there is no row.  kHalves of
// the row are read before the wait for the buffer, the rest after.
template <int D, int kHalves>
__device__ __forceinline__ bool copy_q_row(const Params& p, const Tile& t, int row, uint8_t* smem, uint32_t tiles) {
  using L = Layout<D>;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMisc + 4);
  const int G = p.group, u = row / G;
  const bool real = u < t.ntok;
  const uint32_t sign = p.scale_log2 < 0.f ? 0x80008000u : 0u;
  const uint4* src = reinterpret_cast<const uint4*>(
      p.q + (t.qs + t.u0 + (real ? u : 0)) * p.q_stride +
      static_cast<int64_t>(t.h * G + (real ? row % G : 0)) * D);
  uint8_t* dst = smem + L::kQ + row * 128;
#pragma unroll
  for (int half = 0; half < L::NDH; half += kHalves) {
    uint4 x[8 * kHalves];
#pragma unroll
    for (int i = 0; i < 8 * kHalves; ++i) x[i] = real ? __ldg(src + 8 * half + i) : make_uint4(0u, 0u, 0u, 0u);
    // the tile before is done with the buffer
    if (half == 0 && tiles > 0 && !held_warp_wait(&bars[kQEmpty], (tiles - 1) & 1, p.err, abort_flag)) return false;
#pragma unroll
    for (int i = 0; i < 8 * kHalves; ++i)
      *reinterpret_cast<uint4*>(dst + (half + i / 8) * kRegion + (((i & 7) ^ (row & 7)) << 4)) =
          make_uint4(x[i].x ^ sign, x[i].y ^ sign, x[i].z ^ sign, x[i].w ^ sign);
  }
  fence_proxy_async_smem();
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(&bars[kQFull]);
  return true;
}

// The warps that convert K (and bring Q), or V: warp cw of the four takes blocks 2 cw and 2 cw
// + 1 of every key tile.
template <int D, bool kIsV>
__device__ __forceinline__ void convert_role(const Params& p, uint8_t* smem, const int32_t* prefix, int entries,
                                             int total, int tpt, int cw) {
  using L = Layout<D>;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMisc + 4);
  int32_t* nans = reinterpret_cast<int32_t*>(smem + L::kNan);
  int32_t* any_nan = nans + kNanBufs * D;
  const int lane = threadIdx.x & 31, cid = blockIdx.x, ncta = gridDim.x;
  const uint64_t block_bytes = static_cast<uint64_t>(p.hkv) * f8_chunk_bytes(D);
  constexpr int kStages = kIsV ? kVStages : kKStages;
  constexpr int kFull0 = kIsV ? kVFull0 : kKFull0, kEmpty0 = kIsV ? kVEmpty0 : kKEmpty0;
  constexpr uint32_t kTiles = kIsV ? L::kV : L::kK;
  uint32_t count = 0, tiles = 0;
  bool ok = true;
  for (int it = 0, ct = cta_tile(0, cid, ncta, total); ct >= 0 && ok;
       ct = cta_tile(++it, cid, ncta, total), ++tiles) {
    if (__shfl_sync(0xffffffffu, *abort_flag, 0)) break;
    const Tile t = find_tile<false>(ct, prefix, entries, p, tpt);
    // this warp's blocks of the request in turn: 2 cw, 2 cw + 1, 2 cw + 8, ...
    const int nblk = (t.nkeys - 1) / kF8Block + 1;
    const int32_t* ids = p.block_table + static_cast<int64_t>(t.r) * p.bt_stride;
    const uint8_t* head = (kIsV ? p.value_cache : p.key_cache) + static_cast<uint64_t>(t.h) * f8_chunk_bytes(D);
    auto block_of = [&](int n) { return (n >> 1) * kTileBlocks + 2 * cw + (n & 1); };
    auto load_id = [&](int n) -> int { return block_of(n) < nblk ? __ldg(ids + block_of(n)) : -1; };
    auto load = [&](Codes<D>& c, int n, int id) {
      if (static_cast<uint32_t>(id) < static_cast<uint32_t>(p.num_blocks)) {
        c.load(head + static_cast<uint32_t>(id) * block_bytes, lane);
      } else {
        if (block_of(n) < nblk && lane == 0) atomicOr(p.err, PKV_ERR_BLOCK_ID);
        c.zero();
      }
    };
    Codes<D> next;
    load(next, 0, load_id(0));
    int id = load_id(1);
    if constexpr (!kIsV) {
      ok = copy_q_row<D, 1>(p, t, cw * 32 + lane, smem, tiles);
      if (!ok) break;
    }
    for (int j = 0; j < t.nkt && ok; ++j, ++count) {
      const int st = count % kStages;
      if (count >= kStages) {
        ok = held_warp_wait(&bars[kEmpty0 + st], (count / kStages - 1) & 1, p.err, abort_flag);
        if (!ok) break;
      }
#pragma unroll 1
      for (int b = 0; b < 2; ++b) {
        const int n = 2 * j + b, at = block_of(n) * kF8Block;
        Codes<D> c = next;
        load(next, n + 1, id);
        id = load_id(n + 2);
        if constexpr (kIsV) {
          // (bytes of tokens that no row sees may be NaN)
          if (at + kF8Block > t.nkeys) keep_codes<D>(c, keep_tokens(t.nkeys - at, lane));
          // keys that not every row sees
          if (at + kF8Block - 1 > t.nc + t.u0 && has_nan<D>(c)) {
            any_nan[tiles % kNanBufs] = 1;
            note_nan<D>(c, nans + tiles % kNanBufs * D, at, lane);
          }
          store_values<D>(smem + kTiles + st * L::kHalf, 2 * cw + b, c, lane);
        } else {
          store_keys<D>(smem + kTiles + st * L::kHalf, 2 * cw + b, c, lane);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[kFull0 + st]);
    }
  }
}

// Notes which key tiles hold large values (a warp; no images), with the stages of K.
template <int D>
__device__ __forceinline__ void loud_role(const Params& p, uint8_t* smem, const int32_t* prefix, int entries,
                                          int total, int tpt) {
  using L = Layout<D>;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMisc + 4);
  volatile uint32_t* loud = reinterpret_cast<volatile uint32_t*>(smem + L::kLoud);
  const int lane = threadIdx.x & 31, cid = blockIdx.x, ncta = gridDim.x;
  const uint64_t block_bytes = static_cast<uint64_t>(p.hkv) * f8_chunk_bytes(D);
  uint32_t count = 0;
  bool ok = true;
  for (int it = 0, ct = cta_tile(0, cid, ncta, total); ct >= 0 && ok; ct = cta_tile(++it, cid, ncta, total)) {
    if (__shfl_sync(0xffffffffu, *abort_flag, 0)) break;
    const Tile t = find_tile<false>(ct, prefix, entries, p, tpt);
    const int nblk = (t.nkeys - 1) / kF8Block + 1;
    const int32_t* ids = p.block_table + static_cast<int64_t>(t.r) * p.bt_stride;
    const uint8_t* scale = p.value_cache + static_cast<uint64_t>(t.h) * f8_chunk_bytes(D) + f8_code_bytes(D);
    auto load = [&](int j) -> uint32_t {  // a block a lane
      const int b = j * kTileBlocks + lane;
      if (lane >= kTileBlocks || b >= nblk) return 0u;
      const uint32_t id = static_cast<uint32_t>(__ldg(ids + b));
      return id < static_cast<uint32_t>(p.num_blocks) ? __ldg(scale + id * block_bytes) : 0u;
    };
    uint32_t next = 0u;  // (of a row's first key tile nothing asks)
    for (int j = 0; j < t.nkt; ++j, ++count) {
      const int st = count % kKStages;
      ok = count < kKStages || held_warp_wait(&bars[kKEmpty0 + st], (count / kKStages - 1) & 1, p.err, abort_flag);
      if (!ok) break;
      const bool any = __any_sync(0xffffffffu, next > kF8Loud);
      if (lane == 0) {
        loud[count % kLoudBufs] = any ? 1u : 0u;
        mbar_arrive(&bars[kKFull0 + st]);
      }
      if (j + 1 < t.nkt) next = load(j + 1);
    }
  }
}

template <int D, bool kImages>
__global__ void __launch_bounds__(Shape<kImages>::kThreads, 1) prefill_fp8_kernel(const Params p) {
  using L = Layout<D>;
  using S = Shape<kImages>;
  constexpr int NDH = L::NDH;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBars);
  float* xch = reinterpret_cast<float*>(smem + L::kXch);
  int32_t* nans = reinterpret_cast<int32_t*>(smem + L::kNan);
  int32_t* any_nan = nans + kNanBufs * D;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMisc + 4);
  int32_t* prefix = reinterpret_cast<int32_t*>(smem + L::kPrefix);

  // the kernel before may write the images, q, the cache, out or the metadata
  grid_dependency_wait();
  if (threadIdx.x == 0) grid_launch_dependents();
  // (the kernel over images is through)
  if (!kImages && p.images != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *p.flags_seen = 0u;
  if (kImages ? __ldcg(p.any + 1) == 0 : p.images != nullptr && __ldcg(p.any) == 0) return;
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
      if (b == kQFull) n = 4;  // the warps that bring Q
      // the warps that convert, and with K the one that notes large values
      if (!kImages && b >= kKFull0 && b < kKFull0 + kKStages) n = 5;
      if (!kImages && b >= kVFull0 && b < kVFull0 + kVStages) n = 4;
      if ((b >= kPFull0 && b < kPFull0 + kSBufs) || b == kNanRead) n = 8;  // softmax warps
      if (b >= kPair0 && b < kPair0 + 4) n = 2;         // the two warps sharing a quadrant
      mbar_init(&bars[b], n);
    }
    fence_mbar_init();
  }
  if (!kImages)
    for (int i = threadIdx.x; i < kNanBufs * (D + 1); i += S::kThreads) nans[i] = i < kNanBufs * D ? kNone : 0;
  bool bad = false;
  for (int i = threadIdx.x; i < entries; i += S::kThreads) {
    int n = 0;
    for (int k = 0; k < (1 << p.entry_shift); ++k) {
      const int r = (i << p.entry_shift) + k;
      if (r < R) n += own_tiles<kImages>(p, r, tpt, &bad);
    }
    prefix[i + 1] = n;
  }
  if (!kImages && bad && cid == 0) atomicOr(p.err, PKV_ERR_METADATA);
  __syncthreads();
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
    set_registers<S::kIssue, false>();
    if (warp == 0) {
      // ============================ QK^T issuer ============================
      if (lane == 0) {
        constexpr uint32_t idesc_s = idesc_bf16_f32(kRows, kKeys, 0);
        const uint64_t q_desc = smem_desc_sw128(smem_u32(smem + L::kQ), 16, 1024);
        // K stage: groups of 8 keys every NDH KiB, dim half dh at +dh KiB
        const uint64_t k_desc0 = smem_desc_sw128(smem_u32(smem + L::kK), 16, NDH * 1024);
        uint32_t q_count = 0, count = 0;
        bool ok = true;
        for (int it = 0, ct = cta_tile(0, cid, ncta, total); ct >= 0 && ok && !*abort_flag;
             ct = cta_tile(++it, cid, ncta, total)) {
          const Tile t = find_tile<kImages>(ct, prefix, entries, p, tpt);
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
    } else if (warp == 1) {
      // ============================ PV issuer ============================
      if (lane == 0) {
        constexpr uint32_t idesc_o = idesc_bf16_f32(kRows, D, 1);
        // V stage, MN-major: 64-dim atoms of a group of 8 keys 1 KiB apart, groups
        // of 8 keys NDH KiB apart
        const uint64_t v_desc0 = smem_desc_sw128(smem_u32(smem + L::kV), 1024, NDH * 1024);
        uint32_t count = 0;
        bool ok = true;
        for (int it = 0, ct = cta_tile(0, cid, ncta, total); ct >= 0 && ok && !*abort_flag;
             ct = cta_tile(++it, cid, ncta, total)) {
          const Tile t = find_tile<kImages>(ct, prefix, entries, p, tpt);
          for (int j = 0; j < t.nkt && ok; ++j, ++count) {
            const int vs = count % kVStages, b = count % kSBufs;
            ok = held_wait(&bars[kPFull0 + b], (count / kSBufs) & 1, p.err, abort_flag) &&
                 held_wait(&bars[kVFull0 + vs], (count / kVStages) & 1, p.err, abort_flag);
            if (!ok) break;
            tc_fence_after();
            const uint64_t vd = v_desc0 + ((vs * L::kHalf) >> 4);
            const uint32_t a_p = tmem + kColS + b * kKeys;
            // P columns hold the keys of each softmax half in their first 32 (pairs), V rows
            // [64 half, 64 half + 64)
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
    } else if constexpr (kImages) {
      if (lane == 0) {
        if (warp == 2) copy_role<D, false>(p, smem, prefix, entries, total, tpt);
        else copy_role<D, true>(p, smem, prefix, entries, total, tpt);
      }
    } else if (warp == 2) {
      loud_role<D>(p, smem, prefix, entries, total, tpt);
    }
  } else if (warp >= 12) {
    set_registers<S::kConvert, false>();
    if constexpr (kImages) {
      uint32_t tiles = 0;
      for (int it = 0, ct = cta_tile(0, cid, ncta, total); ct >= 0;
           ct = cta_tile(++it, cid, ncta, total), ++tiles) {
        if (__shfl_sync(0xffffffffu, *abort_flag, 0)) break;
        const Tile t = find_tile<true>(ct, prefix, entries, p, tpt);
        if (!copy_q_row<D, L::NDH>(p, t, (warp - 12) * 32 + lane, smem, tiles)) break;
      }
    } else {
      if (warp < 16) convert_role<D, false>(p, smem, prefix, entries, total, tpt, warp - 12);
      else convert_role<D, true>(p, smem, prefix, entries, total, tpt, warp - 16);
    }
  } else {
    // ============================ softmax warps ============================
    set_registers<S::kSoftmax, true>();
    // Two warps share each 32-lane quadrant of tensor memory (the same 32 rows): warp half h
    // reads S columns [64 h, 64 h + 64).  They agree on the row maximum every key tile, so
    // one O serves the row; each keeps the partial sum l of its own columns.
    const int quad = warp & 3;
    const int half = (warp - 4) >> 2;
    const int row = quad * 32 + lane;    // tile row = tensor-memory lane
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const uint32_t o_cols = lane_addr + kColO + half * (D / 2);
    uint64_t* pair_bar = &bars[kPair0 + quad];
    // never zero, for the masked scores' infinities (2^-149 leaves 2^-21 of the largest sums);
    // the scale's sign is on Q
    const float f = fmaxf(fabsf(p.scale_log2), 1.4e-45f);
    const uint32_t flags_seen = kImages ? __ldcg(p.flags_seen) : 0u;
    const bool nan_seen = (flags_seen & 1u) != 0u;
    const volatile uint32_t* loud = reinterpret_cast<volatile uint32_t*>(smem + L::kLoud);
    float most = (flags_seen & 2u) ? kMostLoud : kMost;
    uint32_t count = 0, pair_uses = 0, tiles_done = 0, nan_tiles = 0;
    auto exchange = [&](float mine) -> float {
      float* slot = xch + (pair_uses & 1) * 256;
      slot[half * 128 + row] = mine;
      __syncwarp();
      if (lane == 0) mbar_arrive(pair_bar);
      const bool done = warp_wait(pair_bar, pair_uses & 1, p.err, abort_flag);
      ++pair_uses;
      return done ? slot[(half ^ 1) * 128 + row] : mine;
    };
    const int u = row / G;
    int ct = cta_tile(0, cid, ncta, total);
    Tile t = find_tile<kImages>(ct, prefix, entries, p, tpt);
    for (int it = 0; ct >= 0;) {
      if (__shfl_sync(0xffffffffu, *abort_flag, 0)) break;
      const int pos = t.nc + t.u0 + (u < t.ntok ? u : t.ntok - 1);
      const int pos_min = t.nc + t.u0;
      float m_used = -INFINITY, l = 0.f;
      bool ok = true;
      for (int j = 0; j < t.nkt && ok; ++j, ++count) {
        const int b = count % kSBufs;
        if (!warp_wait(&bars[kSFull0 + b], (count / kSBufs) & 1, p.err, abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t s_cols = lane_addr + kColS + b * kKeys + half * 64;
        if (!kImages) most = loud[count % kLoudBufs] != 0u ? kMostLoud : kMost;
        // causal mask (only tiles reaching past the tile's first row)
        const int key0 = j * kKeys + half * 64;
        if (key0 + 63 > pos_min) mask_scores(s_cols, pos_min + 1 - key0, pos + 1 - key0);
        // the largest of the row's scores in the key tile
        auto row_max = [&]() -> float {
          float mine = -INFINITY;
#pragma unroll 1
          for (int c = 0; c < 64; c += 32) {
            float sv[32];
            tmem_ld32(s_cols + c, *reinterpret_cast<uint32_t(*)[32]>(&sv));
            tmem_wait_ld();
            float m4[4] = {sv[0], sv[1], sv[2], sv[3]};  // four chains of three-input maxima
#pragma unroll
            for (int i = 4; i < 28; i += 8)
#pragma unroll
              for (int k = 0; k < 4; ++k) m4[k] = fmax3(m4[k], sv[i + k], sv[i + 4 + k]);
#pragma unroll
            for (int k = 0; k < 4; ++k) m4[k] = fmaxf(m4[k], sv[28 + k]);
            mine = fmax3(mine, fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
          }
          mine *= f;
          return fmaxf(mine, exchange(mine));
        };
        if (j == 0) m_used = row_max() - kLargest;  // key 0 is visible to every row
        // P = 2^(s f - m_used) as bf16 pairs over the first 32 of this warp's 64 S columns
        uint32_t w[32];
        float sv[64];
        {
          uint32_t (&r)[64] = *reinterpret_cast<uint32_t(*)[64]>(&sv);
          tmem_ld32(s_cols, *reinterpret_cast<uint32_t(*)[32]>(&r[0]));
          tmem_ld32(s_cols + 32, *reinterpret_cast<uint32_t(*)[32]>(&r[32]));
          tmem_wait_ld();
        }
        const float2 f2 = make_float2(f, f), c2 = make_float2(-m_used, -m_used);
        float2 l2 = make_float2(0.f, 0.f);
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const float2 x = __ffma2_rn(make_float2(sv[2 * e], sv[2 * e + 1]), f2, c2);
          w[e] = pack_bf16(exp2_approx(x.x), exp2_approx(x.y));
          add_pair(l2, w[e]);
        }
        // Whether the reference has to move the sums tell; both warps of the quadrant see the
        // same.  (Not in the first key tile: 64 weights of 2^kLargest at most.)
        const float sum = l2.x + l2.y;
        const bool grow = j > 0 && fmaxf(sum, exchange(sum)) > most;
        if (!__any_sync(0xffffffffu, grow)) {
          l += sum;
          tmem_st32(s_cols, w);
        } else {
          // (rare: in short loops, from S once more)
          const float mx = row_max();
          // O must hold PV of the previous key tile before it is rescaled
          const uint32_t prev = count - 1;
          if (!warp_wait(&bars[kODone0 + prev % kSBufs], (prev / kSBufs) & 1, p.err, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const float alpha = grow ? exp2_approx(m_used - mx + kLargest) : 1.f;
          if (grow) m_used = mx - kLargest;
          l *= alpha;
          rescale<D / 2>(o_cols, alpha);
          l2 = make_float2(0.f, 0.f);
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t r[16], y[8];
            tmem_ld8(s_cols + 16 * c, *reinterpret_cast<uint32_t(*)[8]>(&r[0]));
            tmem_ld8(s_cols + 16 * c + 8, *reinterpret_cast<uint32_t(*)[8]>(&r[8]));
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              y[e] = pack_bf16(exp2_approx(fmaf(__uint_as_float(r[2 * e]), f, -m_used)),
                               exp2_approx(fmaf(__uint_as_float(r[2 * e + 1]), f, -m_used)));
              add_pair(l2, y[e]);
            }
            tmem_st8(s_cols + 8 * c, y);
          }
          l += l2.x + l2.y;
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[kPFull0 + b]);
      }
      if (!ok) break;
      // (the next query tile is looked up while P V ends)
      ct = cta_tile(++it, cid, ncta, total);
      Tile next = t;
      if (ct >= 0) next = find_tile<kImages>(ct, prefix, entries, p, tpt);
      // ---- epilogue: O / (l_0 + l_1) -> out ----
      if (!warp_wait(&bars[kOFinal], tiles_done & 1, p.err, abort_flag)) break;
      tc_fence_after();
      const float inv = 1.f / (l + exchange(l));
      // dimensions of this warp's half in which the row sees a NaN
      uint64_t nan_dims = 0u;
      if constexpr (kImages) {
        if (nan_seen) {
          const int64_t first = static_cast<int64_t>(__ldcg(p.image_base + t.r)) * p.hkv + t.h;
          for (int j = 0; j < t.nkt; ++j) {
            const int64_t i = first + static_cast<int64_t>(j) * p.hkv;
            if (__ldcg(p.image_nan + i) == 0) continue;
            const int32_t* at = reinterpret_cast<const int32_t*>(p.images + i * image_bytes<D>() + 2 * L::kHalf) + half * (D / 2);
            for (int d = 0; d < D / 2; ++d)
              if (__ldcg(at + d) <= pos) nan_dims |= 1ull << d;
          }
        }
      } else if (any_nan[tiles_done % kNanBufs] != 0) {
        const int32_t* at = nans + tiles_done % kNanBufs * D + half * (D / 2);
        for (int d = 0; d < D / 2; ++d)
          if (at[d] <= pos) nan_dims |= 1ull << d;
        // once every softmax warp has read them they are ready for another query tile
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[kNanRead]);
        if (warp == 4) {
          if (!warp_wait(&bars[kNanRead], nan_tiles & 1, p.err, abort_flag)) break;
          for (int d = lane; d < D; d += 32) nans[tiles_done % kNanBufs * D + d] = kNone;
          if (lane == 0) any_nan[tiles_done % kNanBufs] = 0;
        }
        ++nan_tiles;
      }
      ++tiles_done;
      // This warp holds output dims [half * D/2, half * D/2 + D/2) of its 32
      // rows: NV 16-byte pieces per row, transposed among groups of NV lanes so
      // that every store instruction writes whole rows' segments.
      constexpr int NV = D / 16;
      uint4 seg[NV];
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        uint32_t r0[32];
        tmem_ld32(o_cols + c * 32, r0);
        tmem_wait_ld();
        if (__any_sync(0xffffffffu, nan_dims != 0u)) {
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if ((nan_dims >> (c * 32 + e)) & 1u) r0[e] = 0x7fffffffu;
        }
#pragma unroll
        for (int q4 = 0; q4 < 4; ++q4) {
          uint4& v = seg[c * 4 + q4];
          float x[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = __uint_as_float(r0[q4 * 8 + e]) * inv;
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
      t = next;
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem, kTmemCols);
}

// Makes the images: a CTA takes the K or the V of one at a time, a block each of its eight
// warps.  Also decides which requests have images, and reports bad metadata.
template <int D>
__global__ void __launch_bounds__(256, 4) expand_fp8_kernel(const Params p) {
  constexpr uint32_t kHalf = Layout<D>::kHalf;
  extern __shared__ int32_t prefix[];  // [R + 1]: key tiles; then the scan's
  __shared__ int32_t nans[D];
  // the kernel before may write the cache or the metadata, or read the images
  grid_dependency_wait();
  if (threadIdx.x == 0) grid_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int R = p.num_reqs, tpt = kRows / p.group;
  bool bad = false;
  // Requests of many query tiles, and of few: their most key tiles, all key tiles, and visits
  // of query tiles to key tiles.  Each kind has images if that takes longer without.
  float longest[2] = {0.f, 0.f}, all[2] = {0.f, 0.f}, visits[2] = {0.f, 0.f};
  for (int r = threadIdx.x; r < R; r += blockDim.x) {
    const int tiles = request_tiles(p, r, tpt, &bad) / p.hkv;
    const int keys = tiles == 0 ? 0 : (__ldg(p.seq_lens + r) - 1) / kKeys + 1;
    const int few = tiles < kManyTiles ? 1 : 0;
    longest[few] = fmaxf(longest[few], static_cast<float>(keys));
    all[few] += static_cast<float>(keys);
    visits[few] += tiles * (static_cast<float>(__ldg(p.num_computed + r)) / kKeys + keys) * 0.5f;
    prefix[r + 1] = few ? -keys : keys;
  }
#pragma unroll
  for (int x = 1; x < 32; x <<= 1)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      longest[k] = fmaxf(longest[k], __shfl_xor_sync(0xffffffffu, longest[k], x));
      all[k] += __shfl_xor_sync(0xffffffffu, all[k], x);
      visits[k] += __shfl_xor_sync(0xffffffffu, visits[k], x);
    }
  __shared__ float sums[8][2][3];
  if (lane == 0)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      sums[warp][k][0] = longest[k];
      sums[warp][k][1] = all[k];
      sums[warp][k][2] = visits[k];
    }
  __syncthreads();
  bool ahead[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    float most = 0.f, n = 0.f, v = 0.f;
    for (int w = 0; w < 8; ++w) {
      most = fmaxf(most, sums[w][k][0]);
      n += sums[w][k][1];
      v += sums[w][k][2];
    }
    most = fmaxf(most, v * p.hkv / p.sms);  // key tiles of the CTA that has most
    ahead[k] = image_gain<D>() * most > image_cost<D>() * n * p.hkv;
  }
  for (int r = threadIdx.x; r < R; r += blockDim.x) {
    const int keys = prefix[r + 1];
    prefix[r + 1] = keys < 0 ? (ahead[1] ? -keys : 0) : ahead[0] ? keys : 0;
  }
  if (threadIdx.x == 0) prefix[0] = 0;
  if (threadIdx.x < D) nans[threadIdx.x] = kNone;
  if (bad && blockIdx.x == 0) atomicOr(p.err, PKV_ERR_METADATA);
  __syncthreads();
  block_inclusive_scan(prefix + 1, R, prefix + R + 1);
  __syncthreads();
  if (blockIdx.x == 0) {
    bool direct = false, images = false;
    for (int r = threadIdx.x; r < R; r += blockDim.x) {
      const bool has = prefix[r + 1] > prefix[r] && prefix[r + 1] <= p.image_tiles;
      p.image_base[r] = has ? prefix[r] : -1;
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
  const uint64_t block_bytes = static_cast<uint64_t>(p.hkv) * f8_chunk_bytes(D);
  for (int64_t x = blockIdx.x;; x += gridDim.x) {
    const int64_t i = x >> 1, tile = i / p.hkv;
    const bool is_v = x & 1;
    if (tile >= prefix[R]) break;
    const int h = static_cast<int>(i - tile * p.hkv);
    int lo = 0, hi = R;  // prefix[lo] <= tile < prefix[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (prefix[mid] <= tile) lo = mid; else hi = mid;
    }
    if (prefix[lo + 1] > p.image_tiles) break;  // and so are the requests after it
    const int at = static_cast<int>(tile - prefix[lo]) * kKeys + warp * kF8Block;
    const int seq = __ldg(p.seq_lens + lo);
    Codes<D> c;
    c.zero();
    if (at < seq) {
      const int id = __ldg(p.block_table + static_cast<int64_t>(lo) * p.bt_stride + at / kF8Block);
      if (static_cast<uint32_t>(id) < static_cast<uint32_t>(p.num_blocks))
        c.load((is_v ? p.value_cache : p.key_cache) + static_cast<uint32_t>(id) * block_bytes +
                   static_cast<uint64_t>(h) * f8_chunk_bytes(D), lane);
      else if (lane == 0)
        atomicOr(p.err, PKV_ERR_BLOCK_ID);
    }
    uint8_t* image = p.images + i * static_cast<int64_t>(image_bytes<D>());
    if (!is_v) {
      store_keys<D>(image, warp, c, lane);
      continue;
    }
    if (at + kF8Block > seq) keep_codes<D>(c, keep_tokens(seq - at, lane));
    const bool nan = has_nan<D>(c);
    if (nan) note_nan<D>(c, nans, at, lane);
    store_values<D>(image + kHalf, warp, c, lane);
    const bool loud = c.e > kF8Loud;
    if (!__syncthreads_or(nan || loud)) {
      if (threadIdx.x == 0) p.image_nan[i] = 0;
    } else {
      const bool nan_here = __syncthreads_or(nan), loud_here = __syncthreads_or(loud);
      if (threadIdx.x == 0) {
        p.image_nan[i] = nan_here ? 1 : 0;
        atomicOr(p.flags_seen, (nan_here ? 1u : 0u) | (loud_here ? 2u : 0u));
      }
      if (threadIdx.x < D) {
        reinterpret_cast<int32_t*>(image + 2 * kHalf)[threadIdx.x] = nans[threadIdx.x];
        nans[threadIdx.x] = kNone;
      }
      __syncthreads();
    }
  }
  fence_proxy_async_global();  // the next kernel's copies read what was stored
}

template <int D, bool kImages>
cudaError_t launch_tiles(Params p, int sms, cudaStream_t stream) {
  int entries = p.num_reqs;
  p.entry_shift = 0;
  while (entries > kPrefixMax) {
    ++p.entry_shift;
    entries = (p.num_reqs + (1 << p.entry_shift) - 1) >> p.entry_shift;
  }
  const size_t smem = 1024 + Layout<D>::kPrefix + 4 * (static_cast<size_t>(entries) + 1) + 4 * 32;
  if (smem > kSmemLimit) return cudaErrorInvalidValue;
  const cudaError_t e = raise_smem_limit_once<prefill_fp8_kernel<D, kImages>>(kSmemLimit);
  if (e != cudaSuccess) return e;
  return launch_programmatic(prefill_fp8_kernel<D, kImages>, dim3(static_cast<unsigned>(sms)),
                             dim3(Shape<kImages>::kThreads), smem, stream, p);
}

template <int D>
cudaError_t launch_t(const Params& p, int sms, cudaStream_t stream) {
  if (p.images != nullptr) {
    const size_t smem = 4 * (static_cast<size_t>(p.num_reqs) + 1 + 32);
    cudaError_t e = launch_programmatic(expand_fp8_kernel<D>, dim3(static_cast<unsigned>(4 * sms)), dim3(256),
                                        smem, stream, p);
    if (e == cudaSuccess) e = launch_tiles<D, true>(p, sms, stream);
    if (e != cudaSuccess) return e;
  }
  return launch_tiles<D, false>(p, sms, stream);
}

}  // namespace

int64_t prefill_fp8_image_bytes(int num_kv_heads, int head_dim) {
  // (and the word that says whether V has a NaN)
  return static_cast<int64_t>(num_kv_heads) * ((head_dim == 128 ? image_bytes<128>() : image_bytes<64>()) + 4);
}

cudaError_t launch_prefill_fp8(const AttnArgs& a, const MxPrefillScratch& ws, int sms,
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
  p.flags_seen = a.err + 1;
  p.entry_shift = 0;
  p.images = nullptr;
  p.image_base = p.image_nan = p.any = nullptr;
  p.image_tiles = ws.image_tiles;
  p.sms = sms;
  // where the room, the table's width or the number of tokens says that no request can have
  // images, nothing looks for them
  const int tpt = kRows / p.group;
  const float keys = static_cast<float>((a.bt_width + kTileBlocks - 1) / kTileBlocks);
  const float tiles = static_cast<float>((a.num_tokens + tpt - 1) / tpt + a.num_reqs) * p.hkv / sms;
  const float gain = a.head_dim == 128 ? image_gain<128>() : image_gain<64>();
  const float cost = a.head_dim == 128 ? image_cost<128>() : image_cost<64>();
  if (ws.image_tiles > 0 && gain * keys * (tiles > 1.f ? tiles : 1.f) > kImageFixed + cost * keys * p.hkv) {
    p.images = ws.images;
    p.image_nan = reinterpret_cast<int32_t*>(
        ws.images + static_cast<int64_t>(ws.image_tiles) * p.hkv * (a.head_dim == 128 ? image_bytes<128>() : image_bytes<64>()));
    p.any = ws.image_base;
    p.image_base = ws.image_base + 2;
  }
  if (a.head_dim == 128) return launch_t<128>(p, sms, stream);
  if (a.head_dim == 64) return launch_t<64>(p, sms, stream);
  return cudaErrorNotSupported;
}

}  // namespace pkv
