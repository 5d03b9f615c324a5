// What the 4-bit prefill kernels share: query tiles and their plan, bounded waits that
// leave the issue slots to others, and the conversion of cache rows to f16 tiles.
//
// Scales.  Keys that are converted together share a base exponent for K and one for
// V: a value is code 2^(e - base + kUp) in f16, exact for scales down to 2^-26 of the
// base's and then rounded at f16's 2^-25.  The softmax puts the bases back for free:
// x = s f + (v - M), with f = 2^(K base) times the query's factor and v the V base in
// log2 units, so that P carries 2^v and the running reference M follows s + v (see
// move_reference for the sum of the weights).  Where those keys differ by more than 2^kWide
// (an outlier, perhaps one that the row may not even see), every key gets a base of its own,
// that of its largest group, and the softmax a factor and an offset per column.
//
// What f16 loses: a weight below 2^-14 keeps fewer than 11 bits, off by 2^-25 at most, where
// the largest s + v has 2 or more.  A base that keys share may be 2^8 above a key's own (2^14,
// but then M starts lower), and a group's scale is 2^-kUneven of its key's largest at least:
// n keys that count for little lose n 2^-26 2^(8 + 8) of a group's largest product, at worst.
//
// Groups of one key further apart than that (a reference M that one of them sets says
// nothing about another) take another way: the direct kernel goes through such query tiles
// again with V as bfloat16 below a base by key (a code has two bits and is exact) and P as
// two bfloat16, the second what the first rounds off: 16 bits, and 2^-126 below M before
// anything is lost, at the cost of a second product and of the slower path by key.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "kernels.h"
#include "mxfp4.cuh"
#include "pkv_device.cuh"
#include "prefill_common.cuh"
#include "tcgen05.cuh"

namespace pkv {

namespace mxprefill {

constexpr int kRows = 128;
constexpr int kKeys = 128;
constexpr uint32_t kRegion = 16384;  // 128 rows x 128 bytes
constexpr uint32_t kTmemCols = 512;
constexpr float kRescaleThreshold = 15.9f;  // log2 units: weights up to 2^15.9 are inside f16
constexpr float kFirst = 1.0f;       // where a row's first M puts its largest weight: room to grow
constexpr float kMoved = 8.0f;       // and where a later one does: hardly any row needs a third
constexpr int kUp = 12;              // a base's scale becomes 2^kUp: 6 2^12 is inside f16
constexpr int kWide = 14;            // binades between keys before each has its base
constexpr int kLoose = 8;            // and before their V lets M start at kMoved
constexpr int kUneven = 8;           // binades between the groups of one key's V in f16
constexpr int kPrefixMax = 4096;     // entries of the plan in shared memory
constexpr int kMaxKeys = 0x7fffff00;  // a whole key tile more is still an int
// Query tiles (of a KV head) and key tiles from which on a request has its key tiles
// converted ahead.  That saves the conversion for every query tile but one, and costs two
// kernels more, which also run, for 5 us, where no request turns out to have enough.  In a
// graph, us ahead / directly:
//   32 query and 8 KV heads of 128: 128 new tokens (4 query tiles) behind 3874 54 / 64, behind
//   17513 157 / 228; 512 behind 1223 37 / 39, behind 11539 115 / 164; 1024 (8 key tiles)
//   behind 0 36 / 35, behind 914 49 / 58; 2048 and 4096 behind 0 62 / 75 and 161 / 242.
//   16 query and 4 KV heads of 64: 128 behind 3789 44 / 58; 512 behind 1069 29 / 34; 1024 and
//   4096 behind 0 25 / 25 and 74 / 122.
constexpr int kImageQueryTiles = 4;
constexpr int kImageKeyTiles = 8;
constexpr size_t kSmemLimit = 232448;

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
  // Key tiles converted ahead (null: none): request r's are images image_base[r] hkv
  // on, its key tiles in order, KV head fastest; -1: none, its rows are the direct
  // kernel's.  uneven[r]: the images' kernel has found V that is not for f16, and leaves its
  // rows to the direct kernel too.  any[0]: whether there are such; any[1]: whether there are
  // images.
  uint8_t* images;
  int32_t* image_base;
  int32_t* uneven;
  int32_t* any;
  int32_t image_tiles;  // key tiles (of all KV heads) there is room for
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
      seq != nc + qlen || (seq - 1) / kMxBlock >= p.bt_width) {
    *bad = true;
    return 0;
  }
  return (qlen + tpt - 1) / tpt * p.hkv;
}

// The query tiles of request r that are computed from images (kImages), or directly.
template <bool kImages>
__device__ __forceinline__ int own_tiles(const Params& p, int r, int tpt, bool* bad) {
  const int n = request_tiles(p, r, tpt, bad);
  if (n == 0 || p.images == nullptr) return kImages ? 0 : n;
  const bool has = __ldcg(p.image_base + r) >= 0;
  if (kImages) return has ? n : 0;
  return !has || __ldcg(p.uneven + r) != 0 ? n : 0;
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

// 2^k, subnormal or zero below 2^-126.
__device__ __forceinline__ float pow2(int k) {
  if (k >= -126) return __uint_as_float(static_cast<uint32_t>(min(k, 127) + 127) << 23);
  return k < -149 ? 0.f : __uint_as_float(1u << (k + 149));
}

// 2^x as f16, gradually down to 2^-24, then 0.
__device__ __forceinline__ uint32_t f16_pow2(int x) {
  return x >= -14 ? static_cast<uint32_t>(x + 15) << 10 : x >= -24 ? 1u << (x + 24) : 0u;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  const __half2 h = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Like mbar_wait_or_abort, but the hardware may hold the warp for a while before
// it answers "not yet", so that waiting warps leave the issue slots to the
// others (they wake when the phase completes).
__device__ __forceinline__ bool held_wait(uint64_t* bar, uint32_t parity, uint32_t* err,
                                          volatile int* abort) {
  const uint32_t addr = smem_u32(bar);
  auto ready = [&]() {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(addr), "r"(parity), "r"(20000u)  // nanoseconds, at most
        : "memory");
    return done != 0;
  };
  if (ready()) return true;
  const long long t0 = clock64();
  while (!ready()) {
    if (*abort) return false;
    if (clock64() - t0 > kWaitLimitCycles) {
      atomicOr(err, PKV_ERR_TIMEOUT);
      *abort = 1;
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ bool held_warp_wait(uint64_t* bar, uint32_t parity, uint32_t* err,
                                               volatile int* abort) {
  return __all_sync(0xffffffffu, held_wait(bar, parity, err, abort));
}

// Instruction descriptor of kind::f16 with f16 A and B, float32 D.
__host__ __device__ constexpr uint32_t idesc_f16_f32(int m, int n, int b_mn_major) {
  return idesc_bf16_f32(m, n, b_mn_major) & ~((1u << 7) | (1u << 10));
}

template <int kRegs, bool kMore>
__device__ __forceinline__ void set_registers() {
  if constexpr (kMore)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
  else
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

// Eight codes times their group's scale as bfloat16.
__device__ __forceinline__ uint4 convert8_bf16(uint32_t w, uint32_t f) {
  uint32_t x[4];
  e2m1x8_to_f16(w, x);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&x[i]));
    const uint32_t code = pack_bf16(v.x, v.y);
    const __nv_bfloat162 y = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&code),
                                     *reinterpret_cast<const __nv_bfloat162*>(&f));
    x[i] = *reinterpret_cast<const uint32_t*>(&y);
  }
  return make_uint4(x[0], x[1], x[2], x[3]);
}

// Eight codes times their group's scale, to one 16-byte piece of a tile row.
__device__ __forceinline__ uint4 convert8(uint32_t w, uint32_t f) {
  uint32_t x[4];
  e2m1x8_to_f16(w, x);
  return make_uint4(mul_f16x2(x[0], f), mul_f16x2(x[1], f), mul_f16x2(x[2], f), mul_f16x2(x[3], f));
}

// The largest scale byte of a row that is not NaN, or -1.
template <int D>
__device__ __forceinline__ int largest_scale(uint32_t e) {
  const uint32_t b0 = e & 0xffu, b1 = (e >> 8) & 0xffu, b2 = (e >> 16) & 0xffu, b3 = e >> 24;
  const uint32_t m = D == 128 ? max(max(b0, b1), max(b2, b3)) : max(b0, b1);
  if (m < 255u) return static_cast<int>(m);
  int x = -1;
  if (b0 != 255u) x = max(x, static_cast<int>(b0));
  if (b1 != 255u) x = max(x, static_cast<int>(b1));
  if (D == 128 && b2 != 255u) x = max(x, static_cast<int>(b2));
  if (D == 128 && b3 != 255u) x = max(x, static_cast<int>(b3));
  return x;
}

// The scale bytes of a row, group by group; `at` is its first group's.
template <int D, bool kIsV>
__device__ __forceinline__ uint32_t load_scale_bytes(const uint8_t* at) {
  if constexpr (kIsV) {
    uint32_t e = __ldg(reinterpret_cast<const uint16_t*>(at));
    if constexpr (D == 128) e |= static_cast<uint32_t>(__ldg(reinterpret_cast<const uint16_t*>(at + 4))) << 16;
    return e;
  } else if constexpr (D == 128) {
    return __ldg(reinterpret_cast<const uint32_t*>(at));
  } else {
    return __ldg(reinterpret_cast<const uint16_t*>(at));
  }
}

// Scale bytes of a row of V with 255 for the groups whose codes are all zero.
template <int D>
__device__ __forceinline__ uint32_t without_zeros(uint32_t e, const uint4 (&c)[D / 32]) {
  uint32_t even = 0u, odd = 0u;  // of the words of codes
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    even |= c[i].x | c[i].z;
    odd |= c[i].y | c[i].w;
  }
  if (D == 64) even |= odd;
  if ((even & 0x00007777u) == 0u) e |= 0xffu;
  if ((even & 0x77770000u) == 0u) e |= 0xff00u;
  if (D == 128 && (odd & 0x00007777u) == 0u) e |= 0xff0000u;
  if (D == 128 && (odd & 0x77770000u) == 0u) e |= 0xff000000u;
  return e;
}

// Whether a row's groups, NaN aside, are more than 2^kUneven apart.
template <int D>
__device__ __forceinline__ bool uneven_groups(uint32_t e) {
  const uint32_t b0 = e & 0xffu, b1 = (e >> 8) & 0xffu, b2 = (e >> 16) & 0xffu, b3 = e >> 24;
  const uint32_t least = D == 128 ? min(min(b0, b1), min(b2, b3)) : min(b0, b1);
  return largest_scale<D>(e) - static_cast<int>(least) > kUneven;  // (-1 - 255 where all are NaN)
}

// The groups' factors 2^(e - base) as bfloat16, in both halves, down to 2^-133 (V).
template <int D>
__device__ __forceinline__ void row_factors_bf16(uint32_t scales, bool real, int base, uint32_t (&f)[D / 32]) {
#pragma unroll
  for (int b = 0; b < D / 32; ++b) {
    const int e = (scales >> (8 * b)) & 0xff, x = e - base;
    const uint32_t power = x >= -126 ? static_cast<uint32_t>(x + 127) << 7 : x >= -133 ? 1u << (x + 133) : 0u;
    f[b] = !real || e == 255 ? 0u : power * 0x00010001u;
  }
}

// The groups' factors 2^(e - base + kUp) as f16, in both halves.
template <int D, bool kIsV>
__device__ __forceinline__ void row_factors(uint32_t scales, bool real, int base, uint32_t (&f)[D / 32]) {
  // All scales in [base - 26, base + 5]: the exponent fields by arithmetic.  (A byte
  // below by at most 223, or NaN's 255, leaves a tested bit set.)
  const uint32_t low = static_cast<uint32_t>(max(base - 26, 0)) * 0x01010101u;
  const uint32_t tested = D == 128 ? 0xe0e0e0e0u : 0x0000e0e0u;
  if (((scales - low) & tested) == 0u && real && base <= 249) {
    const uint32_t add = static_cast<uint32_t>((kUp + 15 - base) * 1024) * 0x00010001u;
#pragma unroll
    for (int b = 0; b < D / 32; ++b)
      f[b] = __byte_perm(scales, 0u, 0x4040 + 0x0101 * b) * 1024u + add;
  } else {
#pragma unroll
    for (int b = 0; b < D / 32; ++b) {
      const int e = (scales >> (8 * b)) & 0xff;
      f[b] = !real ? 0u : e == 255 ? (kIsV ? 0u : 0x7fff7fffu) : f16_pow2(e - base + kUp) * 0x00010001u;
    }
  }
}

// The i-th 16 bytes of a row's codes times the groups' factors, to the row at dst of
// a swizzled tile (sw: the row's index modulo 8).
// K: a word is 8 dimensions.  head_dim 128: word e is (lane c = i, group e); 64: (c =
// 2i + e / 2, group e % 2).  V: the half-words of two words are 8 dimensions; 128:
// words (group / 2) of lane groups 2i and 2i + 1; 64: of lane groups 4i + 2 (e / 2)
// and + 1.
template <int D, bool kIsV, bool kBf16 = false>
__device__ __forceinline__ void store_piece(uint8_t* dst, int i, const uint4& codes,
                                            const uint32_t (&f)[D / 32], int sw) {
  const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int b = D == 128 ? e : e & 1;
    const int q = D == 128 ? i : 2 * i + (e >> 1);  // below 4
    uint32_t eight = w[e];
    if constexpr (kIsV) {
      const uint32_t lo = D == 128 ? w[b >> 1] : w[2 * (e >> 1)];
      const uint32_t hi = D == 128 ? w[2 + (b >> 1)] : w[2 * (e >> 1) + 1];
      eight = __byte_perm(lo, hi, (b & 1) ? 0x7632 : 0x5410);
    }
    // dims 32 b + 8 q .. + 7: piece 4 b + q of the row
    const uint32_t at = (static_cast<uint32_t>(q ^ sw) << 4) ^ ((b & 1) << 6);
    *reinterpret_cast<uint4*>(dst + (b >> 1) * 1024 + at) =
        kBf16 ? convert8_bf16(eight, f[b]) : convert8(eight, f[b]);
  }
}

// The base exponent of a warp's 32 keys, `mine` being each lane's largest scale (-1:
// none), and how far (binades) the keys are apart.
__device__ __forceinline__ int common_base(int mine, int& apart) {
  const int base = __reduce_max_sync(0xffffffffu, mine);
  const int least = __reduce_min_sync(0xffffffffu, static_cast<unsigned>(mine));  // -1: largest
  apart = least >= 0 ? base - least : 0;
  return base < 0 ? 127 : base;
}

// A byte of 255 among a row's scales?
__device__ __forceinline__ bool nan_scale(uint32_t scales) {
  return ((~scales - 0x01010101u) & scales & 0x80808080u) != 0u;
}

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// What only some key tiles need is done to the scores in tensor memory, in short loops:
// unrolled over the registers, code that hardly ever runs took instruction cache from
// the code that always does (a prompt of 4096 tokens: 177 us, in loops 167).

// Scores of N columns from `cols` on times a factor plus an offset by key: qf kf[c] (f
// where kf is null) and kv[c] (v).
template <int N>
__device__ __forceinline__ void scale_scores(uint32_t cols, float qf, const float* kf, float f,
                                             const float* kv, float v) {
#pragma unroll 1
  for (int c = 0; c < N; c += 8) {
    uint32_t r[8];
    tmem_ld8(cols + c, r);
    tmem_wait_ld();
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float fk = kf != nullptr ? qf * kf[c + e] : f;
      fk = fk < 1.17549435e-38f ? 1.17549435e-38f : fk;
      r[e] = __float_as_uint(fmaf(__uint_as_float(r[e]), fk, kv != nullptr ? kv[c + e] : v));
    }
    tmem_st8(cols + c, r);
  }
  tmem_wait_st();
}

// Over N columns of scores x f - kv[c] (v where kv is null): the largest, and the sum of
// 2^(score - ml).
template <int N>
__device__ __forceinline__ float max_scores(uint32_t cols, const float* kv, float v) {
  float mx = -INFINITY;
#pragma unroll 1
  for (int c = 0; c < N; c += 8) {
    uint32_t r[8];
    tmem_ld8(cols + c, r);
    tmem_wait_ld();
#pragma unroll
    for (int e = 0; e < 8; ++e)
      mx = fmaxf(mx, __uint_as_float(r[e]) - (kv != nullptr ? kv[c + e] : v));
  }
  return mx;
}
template <int N>
__device__ __forceinline__ float sum_scores(uint32_t cols, float f, const float* kv, float v, float ml) {
  float sum = 0.f;
#pragma unroll 1
  for (int c = 0; c < N; c += 8) {
    uint32_t r[8];
    tmem_ld8(cols + c, r);
    tmem_wait_ld();
#pragma unroll
    for (int e = 0; e < 8; ++e)
      // (fused as in the products' weights: large scores must not round differently here)
      sum += exp2_approx(fmaf(__uint_as_float(r[e]), f, -(ml + (kv != nullptr ? kv[c + e] : v))));
  }
  return sum;
}

// The sum of the weights, l = sum 2^(s - ml), has a reference of its own beside O's, M,
// because values may be further apart than float32's exponents: M follows s + v, ml
// follows s (both only when that grows by 2^15).  From the products' weights P = 2^(s +
// vb - M) a group of keys with largest score mw adds sum(P) 2^(M - vb - ml).  Where P has
// underflowed although the keys count, the sum is made from the scores: P below 2^-90
// (its lesser ones would be lost), and weights above 2^-45 (n keys below that are n 2^-45
// at most, less than n float32 additions round off).  Then M - vb - ml is above kApart.
constexpr float kNoScore = -1e30f;  // ml before the first key
constexpr float kApart = 45.f;
__device__ __forceinline__ void move_reference(float mw, float& ml, float& l) {
  const float to = mw > ml + kRescaleThreshold ? mw : ml;
  l *= exp2_approx(ml - to);
  ml = to;
}
__device__ __forceinline__ bool weights_lost(float mw, float vb, float m, float ml) {
  return mw + vb - m < -90.f && mw - ml > -45.f;
}
// 2^(up - ml), up = M - vb.  (The limit: above it only weights that do not count.)
__device__ __forceinline__ float weight_factor(float up, float ml) { return exp2_approx(fminf(up - ml, 110.f)); }

// Weights 2^(x - up) of the 64 scores x from `cols` on, over their columns: as pairs of
// bfloat16 in the first 32, and what those round off in the others.
__device__ __forceinline__ void split_weights(uint32_t cols, float up) {
  uint32_t r[32], w[32];
#pragma unroll 1
  for (int c = 0; c < 64; c += 32) {
    tmem_ld32(cols + c, r);
    tmem_wait_ld();
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const float x = exp2_approx(__uint_as_float(r[2 * e]) - up);
      const float y = exp2_approx(__uint_as_float(r[2 * e + 1]) - up);
      w[e] = pack_bf16(x, y);
      w[16 + e] = pack_bf16(x - __uint_as_float(w[e] << 16), y - __uint_as_float(w[e] & 0xffff0000u));
    }
    tmem_st32(cols + c, w);
  }
  tmem_wait_st();
  // the second 16 columns and the third change places
  tmem_ld32(cols + 16, r);
  tmem_wait_ld();
#pragma unroll
  for (int e = 0; e < 32; ++e) w[e] = r[e ^ 16];
  tmem_st32(cols + 16, w);
}

// -inf into this row's columns from `visible` on, of 64; `first` is the smallest such
// column of the warp's rows.
__device__ __forceinline__ void mask_scores(uint32_t cols, int first, int visible) {
#pragma unroll 1
  for (int c = max(first, 0) & ~7; c < 64; c += 8) {
    uint32_t r[8];
    tmem_ld8(cols + c, r);
    tmem_wait_ld();
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (c + e >= visible) r[e] = 0xff800000u;
    tmem_st8(cols + c, r);
  }
  tmem_wait_st();
}

// Rescales N columns of O from `cols` on.
template <int N>
__device__ __forceinline__ void rescale(uint32_t cols, float alpha) {
#pragma unroll 1
  for (int c = 0; c < N; c += 32) {
    uint32_t r32[32];
    tmem_ld32(cols + c, r32);
    tmem_wait_ld();
#pragma unroll
    for (int e = 0; e < 32; ++e) r32[e] = __float_as_uint(__uint_as_float(r32[e]) * alpha);
    tmem_st32(cols + c, r32);
  }
  tmem_wait_st();
}

// A row of Q (row `key` of the tile at dst_tile, one region of 128 bytes a row per 64
// dimensions) brought to f16: its largest element to [2^14, 2^15), the scale's sign on
// it; zeros where there is no row.  qf is what undoes that, times the scale in log2
// units.  `ready` is waited with before the tile is written; false if it gave up.  The
// loops are unrolled kRead and kWrite times: a prompt of 4096 tokens takes 162 us with 2
// and 1 over images, where the warps have time and 8 and 4 cost 167; directly, where
// they convert K besides, 227 with 2 and 1 and 213 with 8 and 4.
template <int D, int kRead, int kWrite, typename F>
__device__ __forceinline__ bool convert_q_row(const Params& p, const Tile& t, int row, uint8_t* q_tile,
                                              float& qf, F&& ready) {
  const int G = p.group, u = row / G, sw = row % 8;
  const bool real = u < t.ntok;
  const uint4* src = reinterpret_cast<const uint4*>(
      p.q + (t.qs + t.u0 + (real ? u : 0)) * p.q_stride +
      static_cast<int64_t>(t.h * G + (real ? row % G : 0)) * D);
  uint32_t mx = 0u;
#pragma unroll kRead
  for (int i = 0; i < D / 8; ++i) {
    const uint4 x = __ldg(src + i);
    mx = max(mx, max(max(x.x & 0x7fffu, (x.x >> 16) & 0x7fffu),
                     max(x.y & 0x7fffu, (x.y >> 16) & 0x7fffu)));
    mx = max(mx, max(max(x.z & 0x7fffu, (x.z >> 16) & 0x7fffu),
                     max(x.w & 0x7fffu, (x.w >> 16) & 0x7fffu)));
  }
  const int ex = static_cast<int>(min(max(mx >> 7, 15u), 254u));
  const float f = copysignf(pow2(141 - ex), p.scale_log2);
  qf = fabsf(p.scale_log2) * pow2(ex - 141);
  if (!ready()) return false;
  uint8_t* dst = q_tile + row * 128;
#pragma unroll kWrite
  for (int i = 0; i < D / 8; ++i) {
    const uint4 x = __ldg(src + i);
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t y[4];
#pragma unroll
    for (int c = 0; c < 4; ++c)
      y[c] = real ? pack_f16(__uint_as_float(w[c] << 16) * f,
                             __uint_as_float(w[c] & 0xffff0000u) * f)
                  : 0u;
    *reinterpret_cast<uint4*>(dst + (i >> 3) * kRegion + (((i & 7) ^ sw) << 4)) =
        make_uint4(y[0], y[1], y[2], y[3]);
  }
  return true;
}

}  // namespace mxprefill

// The prefill without images; rows of requests that have images are left out.
cudaError_t launch_prefill_mxfp4_direct(mxprefill::Params p, int head_dim, int sms, cudaStream_t stream);

}  // namespace pkv
