// C ABI of the 8-bit paged cache and of the rotary table: argument checks, workspace layout
// and launches.  See include/pkv.h for the contract.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "api.h"
#include "fp8.cuh"
#include "kernels.h"
#include "pkv_error.h"

namespace pkv {
namespace {

constexpr int kMaxGroup = 16;
constexpr int64_t kMaxTokens = int64_t{1} << 30;  // of an attention: the kernels count on from them in 32 bits
constexpr int64_t kMaxWritten = int64_t{1} << 20;  // of a write, whose search takes their square
constexpr int64_t kMaxPosition = int64_t{1} << 26;  // the table's frequencies are good to 2^-26 of a radian below it

// Whether some of T rows of na bytes, sa apart, share a byte with rows of nb bytes, sb apart.
// (Of rows whose strides differ, whether their extents overlap.)
bool rows_overlap(const void* a, int64_t sa, int64_t na, const void* b, int64_t sb, int64_t nb, int64_t T) {
  if (!overlap(a, static_cast<size_t>((T - 1) * sa + na), b, static_cast<size_t>((T - 1) * sb + nb))) return false;
  if (sa != sb) return true;
  const int64_t d = static_cast<const char*>(b) - static_cast<const char*>(a);
  const int64_t m = (d % sa + sa) % sa;  // where b's rows begin between a's
  return m < na || m + nb > sa;
}

constexpr double kTau = 6.283185307179586476925;
constexpr double kTauLow = 2.4492935982947064e-16;  // what kTau lacks of 2 pi

// w radians, w in [0, 1], as turns of 64 bits behind the point, to the nearest.
uint64_t turns_of(double w) {
  const double q = w / kTau;
  const double q_low = (std::fma(-q, kTau, w) - q * kTauLow) / kTau;
  const double whole = std::floor(std::ldexp(q, 64));
  const double rest = std::ldexp(q, 64) - whole + std::ldexp(q_low, 64);
  return static_cast<uint64_t>(whole) + static_cast<uint64_t>(static_cast<int64_t>(std::nearbyint(rest)));
}

// The series of a finite float32's factor (Taylor's).
RotarySeries series_of(double factor) {
  int e;
  const double f = 2.0 * std::frexp(factor, &e);
  RotarySeries s;
  s.unit = static_cast<float>(std::ldexp(1.0, e - 1));
  double term = f;  // f (2 pi)^k / k!
  for (int k = 0; k <= 10; ++k) {
    const double x = (k & 2) ? -term : term;
    float& to = k % 2 ? s.s[k / 2] : s.c[k / 2];
    to = static_cast<float>(x);
    if (k == 0) s.c_low = static_cast<float>(x - to);
    if (k == 1) s.s_low = static_cast<float>(x - to);
    if (k == 2) s.c1_low = static_cast<float>(x - to);
    term *= kTau / (k + 1);
  }
  return s;
}

struct F8Workspace {
  size_t plan, ml, o, image_base, images, tile, total;
};

// Room for the prefill's converted key tiles: 508 of 8 KV heads of 128, 65024 tokens.
constexpr size_t kImageRoom = 256u << 20;

// The error word's 256 bytes, then the decode's plan (for the largest batch) and partials,
// then where each request has the prefill's images, and those.
F8Workspace f8_workspace(int sms, int32_t num_heads, int32_t num_kv_heads, int32_t head_dim) {
  const size_t slots = static_cast<size_t>(decode_fp8_slots(sms, num_kv_heads));
  const size_t group = static_cast<size_t>(num_heads / num_kv_heads);
  auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
  F8Workspace w;
  w.plan = 256;
  w.ml = w.plan + up(static_cast<size_t>(step_metadata_max_reqs()) * 8);
  w.o = w.ml + up(slots * group * 8);
  w.image_base = w.o + up(slots * group * head_dim * 4);
  w.images = w.image_base + up(static_cast<size_t>(step_metadata_max_reqs() + 2) * 4);
  w.tile = static_cast<size_t>(prefill_fp8_image_bytes(num_kv_heads, head_dim));
  w.total = w.images + kImageRoom / w.tile * w.tile;
  return w;
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" {

int64_t pkv_fp8_block_bytes(int32_t block_size, int32_t num_kv_heads, int32_t head_dim) {
  if (block_size != kF8Block || num_kv_heads <= 0 || num_kv_heads > (1 << 20) ||
      (head_dim != 64 && head_dim != 128))
    return 0;
  return static_cast<int64_t>(num_kv_heads) * f8_chunk_bytes(head_dim);
}

int pkv_reshape_and_cache_fp8(const void* key, const void* value, int64_t key_stride,
                              int64_t value_stride, void* key_cache, void* value_cache,
                              const int64_t* slot_mapping, int64_t num_tokens, int64_t num_blocks,
                              int32_t block_size, int32_t num_kv_heads, int32_t head_dim,
                              int32_t dtype, uint32_t* error_word, void* stream) {
  const char* where = "pkv_reshape_and_cache_fp8";
  F8WriteArgs a = {};
  const int rc = cache_args(where, key, value, key_stride, value_stride, key_cache, value_cache,
                            slot_mapping, num_tokens, num_blocks, block_size, num_kv_heads,
                            head_dim, dtype, error_word, &a.cache);
  if (rc != PKV_OK || num_tokens == 0) return rc;
  if (num_tokens > kMaxWritten) return fail(PKV_E_UNSUPPORTED, "%s: more than 2^20 tokens", where);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = launch_write_fp8(a, st);
  if (e != cudaSuccess) return cuda_fail(e, "reshape_and_cache_fp8 launch");
  return validate_error_word(error_word, st, "reshape_and_cache_fp8");
}

int pkv_rope_reshape_and_cache_fp8(const int64_t* positions, const void* query, int64_t query_stride,
                                   void* query_out, int64_t query_out_stride, int32_t num_heads,
                                   const void* key, int64_t key_stride, const void* value,
                                   int64_t value_stride, void* key_cache, void* value_cache,
                                   const int64_t* slot_mapping, const float* cos_sin_cache,
                                   int64_t max_position, int32_t rotary_dim, int32_t is_neox,
                                   int64_t num_tokens, int64_t num_blocks, int32_t block_size,
                                   int32_t num_kv_heads, int32_t head_dim, int32_t dtype,
                                   uint32_t* error_word, void* stream) {
  const char* where = "pkv_rope_reshape_and_cache_fp8";
  F8WriteArgs a = {};
  const int rc = cache_args(where, key, value, key_stride, value_stride, key_cache, value_cache,
                            slot_mapping, num_tokens, num_blocks, block_size, num_kv_heads,
                            head_dim, dtype, error_word, &a.cache);
  if (rc != PKV_OK) return rc;
  if (num_tokens > kMaxWritten) return fail(PKV_E_UNSUPPORTED, "%s: more than 2^20 tokens", where);
  if (num_heads <= 0 || num_heads > (1 << 20) || max_position < 0)
    return fail(PKV_E_INVALID, "%s: bad sizes", where);
  const int64_t es = dtype == PKV_F32 ? 4 : 2;
  if (rotary_dim <= 0 || rotary_dim > head_dim || rotary_dim % 2 ||
      (is_neox ? rotary_dim / 2 : rotary_dim) * es % 16)
    return fail(PKV_E_UNSUPPORTED, "%s: rotary_dim %d of %d (whole 16-byte vectors)", where, rotary_dim, head_dim);
  if (num_tokens == 0) return PKV_OK;
  if (!positions || !query || !query_out || !cos_sin_cache)
    return fail(PKV_E_INVALID, "%s: null pointer", where);
  const int64_t row = static_cast<int64_t>(num_heads) * head_dim, kv_row = static_cast<int64_t>(num_kv_heads) * head_dim;
  if (query_stride < row || query_out_stride < row || query_stride * es % 16 || query_out_stride * es % 16 ||
      !aligned16(query) || !aligned16(query_out) || !aligned16(cos_sin_cache))
    return fail(PKV_E_INVALID, "%s: query strides and bases, and the table, must be 16-byte aligned, token "
                "strides not shorter than a row", where);
  if (query_out == query ? query_out_stride != query_stride
                         : rows_overlap(query, query_stride * es, row * es, query_out, query_out_stride * es, row * es, num_tokens))
    return fail(PKV_E_INVALID, "%s: query_out must be query itself or apart from it", where);
  if (rows_overlap(key, key_stride * es, kv_row * es, query_out, query_out_stride * es, row * es, num_tokens) ||
      rows_overlap(value, value_stride * es, kv_row * es, query_out, query_out_stride * es, row * es, num_tokens))
    return fail(PKV_E_INVALID, "%s: query_out overlaps key or value", where);
  a.positions = positions;
  a.cos_sin_cache = cos_sin_cache;
  a.max_position = max_position;
  a.rotary_dim = rotary_dim;
  a.is_neox = is_neox != 0;
  a.num_heads = num_heads;
  a.query = query;
  a.query_out = query_out;
  a.query_stride = query_stride;
  a.query_out_stride = query_out_stride;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = launch_write_fp8(a, st);
  if (e != cudaSuccess) return cuda_fail(e, "rope_reshape_and_cache_fp8 launch");
  return validate_error_word(error_word, st, "rope_reshape_and_cache_fp8");
}

int pkv_gather_cache_fp8(const void* key_cache, const void* value_cache,
                         const int64_t* slot_mapping, void* key_out, void* value_out,
                         int64_t key_out_stride, int64_t value_out_stride, int64_t num_tokens,
                         int64_t num_blocks, int32_t block_size, int32_t num_kv_heads,
                         int32_t head_dim, int32_t dtype, uint32_t* error_word, void* stream) {
  MxCacheArgs a;
  const int rc = cache_args("pkv_gather_cache_fp8", key_out, value_out, key_out_stride,
                            value_out_stride, key_cache, value_cache, slot_mapping, num_tokens,
                            num_blocks, block_size, num_kv_heads, head_dim, dtype, error_word, &a);
  if (rc != PKV_OK || num_tokens == 0) return rc;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = launch_gather_cache_fp8(a, st);
  if (e != cudaSuccess) return cuda_fail(e, "gather_cache_fp8 launch");
  return validate_error_word(error_word, st, "gather_cache_fp8");
}

size_t pkv_fp8_attention_workspace_bytes(int32_t num_heads, int32_t num_kv_heads, int32_t head_dim) {
  if (num_heads <= 0 || num_kv_heads <= 0 || num_heads % num_kv_heads ||
      num_heads / num_kv_heads > kMaxGroup || (head_dim != 64 && head_dim != 128))
    return 0;
  return f8_workspace(current_sm_count(), num_heads, num_kv_heads, head_dim).total;
}

int pkv_paged_attention_varlen_fp8(const void* q, int64_t q_stride, const void* key_cache,
                                   const void* value_cache, const int32_t* block_table,
                                   int32_t block_table_stride, int32_t max_blocks_per_req,
                                   const int32_t* query_start_loc, const int32_t* seq_lens,
                                   const int32_t* num_computed_tokens, float scale, void* out,
                                   int64_t out_stride, int64_t num_tokens, int32_t num_reqs,
                                   int64_t num_blocks, int32_t block_size, int32_t num_heads,
                                   int32_t num_kv_heads, int32_t head_dim, int32_t max_query_len,
                                   void* workspace, size_t workspace_bytes, void* stream) {
  const char* where = "pkv_paged_attention_varlen_fp8";
  if (num_tokens < 0 || num_reqs < 0 || num_heads <= 0 || max_query_len < 0)
    return fail(PKV_E_INVALID, "%s: bad sizes", where);
  if (!std::isfinite(static_cast<float>(scale * 1.4426950408889634)))
    return fail(PKV_E_INVALID, "%s: scale must be finite", where);
  const int rc = check_cache_shape(where, num_blocks, block_size, num_kv_heads, head_dim);
  if (rc != PKV_OK) return rc;
  if (num_heads % num_kv_heads) return fail(PKV_E_INVALID, "%s: num_heads %% num_kv_heads != 0", where);
  if (num_heads / num_kv_heads > kMaxGroup)
    return fail(PKV_E_UNSUPPORTED, "%s: more than %d query heads per KV head", where, kMaxGroup);
  if (num_reqs > step_metadata_max_reqs() || num_tokens > kMaxTokens)
    return fail(PKV_E_UNSUPPORTED, "%s: at most %d requests and 2^30 tokens", where,
                step_metadata_max_reqs());
  if (!workspace) return fail(PKV_E_WORKSPACE, "%s: workspace is required", where);
  const int sms = current_sm_count();
  const F8Workspace w = f8_workspace(sms, num_heads, num_kv_heads, head_dim);
  if (workspace_bytes < w.images || !aligned16(workspace))
    return fail(PKV_E_WORKSPACE, "%s: workspace of %zu bytes, %zu needed, 16-byte aligned", where,
                workspace_bytes, w.images);
  if (num_tokens == 0 || num_reqs == 0) return PKV_OK;
  if (!q || !key_cache || !value_cache || !block_table || !query_start_loc || !seq_lens ||
      !num_computed_tokens || !out)
    return fail(PKV_E_INVALID, "%s: null pointer", where);
  const int64_t row = static_cast<int64_t>(num_heads) * head_dim;
  if (q_stride < row || out_stride < row || q_stride % 8 || out_stride % 8 || !aligned16(q) ||
      !aligned16(out) || !aligned16(key_cache) || !aligned16(value_cache))
    return fail(PKV_E_INVALID,
                "%s: q, out and caches must be 16-byte aligned, token strides >= heads * dim and "
                "multiples of 8", where);
  if (max_blocks_per_req <= 0 || (num_reqs > 1 && block_table_stride < max_blocks_per_req))
    return fail(PKV_E_INVALID, "%s: block_table rows of %d entries, %d apart", where,
                max_blocks_per_req, block_table_stride);
  // (the decode counts these units in 32 bits, and some more)
  if (num_reqs * (static_cast<int64_t>(max_blocks_per_req) + kF8RequestCost) > 0x7fffffffLL - 15)
    return fail(PKV_E_UNSUPPORTED, "%s: a block table of more than 2^31 - 16 entries, with one for each request", where);
  // (offsets that are garbage may give every request the same rows)
  const int64_t tile = 128 / (num_heads / num_kv_heads);
  if (max_query_len != 1 && (num_tokens + tile - 1) / tile * num_kv_heads > 0x7fffffffLL / num_reqs)
    return fail(PKV_E_UNSUPPORTED, "%s: %d requests of %lld tokens may have 2^31 query tiles", where, num_reqs,
                static_cast<long long>(num_tokens));
  AttnArgs a;
  a.q = q;
  a.q_stride = q_stride;
  a.key_cache = key_cache;
  a.value_cache = value_cache;
  a.block_table = block_table;
  a.bt_stride = block_table_stride;
  a.bt_width = max_blocks_per_req;
  a.qsl = query_start_loc;
  a.seq_lens = seq_lens;
  a.num_computed = num_computed_tokens;
  a.out = out;
  a.out_stride = out_stride;
  a.num_tokens = num_tokens;
  a.num_reqs = num_reqs;
  a.num_blocks = num_blocks;
  a.block_size = block_size;
  a.num_heads = num_heads;
  a.num_kv_heads = num_kv_heads;
  a.head_dim = head_dim;
  a.scale = scale;
  a.err = static_cast<uint32_t*>(workspace);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  MxDecodeScratch ds;
  ds.plan = reinterpret_cast<int32_t*>(ws + w.plan);
  ds.part_ml = reinterpret_cast<float*>(ws + w.ml);
  ds.part_o = reinterpret_cast<float*>(ws + w.o);
  cudaError_t e = cudaSuccess;
  if (max_query_len != 1) {
    MxPrefillScratch ps;
    ps.images = ws + w.images;
    ps.image_base = reinterpret_cast<int32_t*>(ws + w.image_base);
    ps.image_tiles = static_cast<int32_t>((std::min(workspace_bytes, w.total) - w.images) / w.tile);
    e = launch_prefill_fp8(a, ps, sms, st);
  }
  if (e == cudaSuccess) e = launch_decode_fp8(a, ds, sms, st);
  if (e != cudaSuccess) return cuda_fail(e, "paged_attention_varlen_fp8 launch");
  return validate_error_word(a.err, st, "paged_attention_varlen_fp8");
}

int pkv_build_cos_sin_cache(float* out, int64_t num_positions, int64_t start, int32_t rotary_dim,
                            double base, int32_t scaling, double factor,
                            int64_t original_max_position, double low, double high,
                            double attention_factor, void* stream) {
  const char* where = "pkv_build_cos_sin_cache";
  if (num_positions < 0 || start < 0 || rotary_dim <= 0 || rotary_dim % 2)
    return fail(PKV_E_INVALID, "%s: positions must not be negative, rotary_dim positive and even", where);
  if (rotary_dim > 2 * kMaxRotaryPairs)
    return fail(PKV_E_UNSUPPORTED, "%s: rotary_dim of at most %d", where, 2 * kMaxRotaryPairs);
  if (num_positions > kMaxPosition || start > kMaxPosition - num_positions)
    return fail(PKV_E_UNSUPPORTED, "%s: positions past 2^26", where);
  if (!(base > 1.0) || !std::isfinite(base) || !std::isfinite(static_cast<float>(attention_factor)))
    return fail(PKV_E_INVALID, "%s: base must be above 1, and attention_factor a finite float32", where);
  if (scaling < PKV_ROPE_NONE || scaling > PKV_ROPE_YARN)
    return fail(PKV_E_INVALID, "%s: scaling %d", where, scaling);
  if (scaling != PKV_ROPE_NONE && (!(factor >= 1.0) || !std::isfinite(factor)))
    return fail(PKV_E_INVALID, "%s: factor must be at least 1", where);
  if (scaling == PKV_ROPE_NTK && rotary_dim < 4)
    return fail(PKV_E_INVALID, "%s: a changed base needs a rotary_dim of 4 or more", where);
  const bool banded = scaling == PKV_ROPE_PARTS || scaling == PKV_ROPE_YARN;
  if (banded && (original_max_position <= 0 || !(low > 0.0) || !(high > low) || !std::isfinite(high)))
    return fail(PKV_E_INVALID, "%s: original_max_position must be positive, and 0 < low < high", where);
  if (num_positions == 0) return PKV_OK;
  if (!out || !aligned16(out)) return fail(PKV_E_INVALID, "%s: the table must be 16-byte aligned", where);
  const double rd = rotary_dim;
  const double b = scaling == PKV_ROPE_NTK ? base * std::pow(factor, rd / (rd - 2)) : base;
  // the pair that makes `turns` turns within the original length
  auto pair = [&](double turns) {
    return rd * std::log(static_cast<double>(original_max_position) / (kTau * turns)) / (2 * std::log(base));
  };
  const double first = banded ? std::max(std::floor(pair(high)), 0.0) : 0.0;
  const double last = banded ? std::min(std::ceil(pair(low)), rd - 1) : 0.0;
  RotaryFrequencies f;
  for (int i = 0; i < rotary_dim / 2; ++i) {
    double w = std::pow(b, -2.0 * i / rd), keep = 1.0;
    if (scaling == PKV_ROPE_LINEAR) keep = 0.0;
    if (scaling == PKV_ROPE_PARTS)
      keep = (static_cast<double>(original_max_position) * w / kTau - low) / (high - low);
    if (scaling == PKV_ROPE_YARN) keep = 1.0 - (i - first) / std::max(last - first, 0.001);
    keep = std::min(std::max(keep, 0.0), 1.0);
    w = keep == 1.0 ? w : keep * w + (1.0 - keep) * w / factor;
    f.turns[i] = turns_of(w);  // (below a sixth of a turn)
  }
  const cudaError_t e = launch_rotary_table(f, out, num_positions, start, rotary_dim,
                                            series_of(attention_factor), static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "build_cos_sin_cache launch");
  return PKV_OK;
}

}  // extern "C"
