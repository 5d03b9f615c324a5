// C ABI of the 4-bit paged cache and of the device-built step metadata:
// argument checks, workspace layout and launches.  See include/pkv.h for the
// contract.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "api.h"
#include "kernels.h"
#include "mxfp4.cuh"
#include "pkv_error.h"

namespace pkv {
namespace {

constexpr int kMaxGroup = 16;

struct MxWorkspace {
  size_t plan, ml, o, image_base, images, tile, total;
};

// Room for the prefill's converted key tiles: 503 of 8 KV heads of 128, 64384 tokens.
constexpr size_t kImageRoom = 256u << 20;

// The error word's 256 bytes, then the decode's plan (for the largest batch) and
// partials, then the prefill's images and where each request has them.
MxWorkspace mx_workspace(int sms, int32_t num_heads, int32_t num_kv_heads, int32_t head_dim) {
  const size_t slots = static_cast<size_t>(decode_mxfp4_slots(sms, num_kv_heads));
  const size_t group = static_cast<size_t>(num_heads / num_kv_heads);
  auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
  MxWorkspace w;
  w.plan = 256;
  w.ml = w.plan + up(static_cast<size_t>(step_metadata_max_reqs()) * 8);
  w.o = w.ml + up(slots * group * 8);
  w.image_base = w.o + up(slots * group * head_dim * 4);
  w.images = w.image_base + up(static_cast<size_t>(2 * step_metadata_max_reqs() + 2) * 4);
  w.tile = static_cast<size_t>(prefill_mxfp4_image_bytes(num_kv_heads, head_dim));
  w.total = w.images + kImageRoom / w.tile * w.tile;
  return w;
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" {

int64_t pkv_mxfp4_block_bytes(int32_t block_size, int32_t num_kv_heads, int32_t head_dim) {
  if (block_size != kMxBlock || num_kv_heads <= 0 || num_kv_heads > (1 << 20) ||
      (head_dim != 64 && head_dim != 128))
    return 0;
  return static_cast<int64_t>(num_kv_heads) * mx_chunk_bytes(head_dim);
}

int pkv_reshape_and_cache_mxfp4(const void* key, const void* value, int64_t key_stride,
                                int64_t value_stride, void* key_cache, void* value_cache,
                                const int64_t* slot_mapping, int64_t num_tokens,
                                int64_t num_blocks, int32_t block_size, int32_t num_kv_heads,
                                int32_t head_dim, int32_t dtype, uint32_t* error_word,
                                void* stream) {
  MxCacheArgs a;
  const int rc = cache_args("pkv_reshape_and_cache_mxfp4", key, value, key_stride, value_stride,
                            key_cache, value_cache, slot_mapping, num_tokens, num_blocks,
                            block_size, num_kv_heads, head_dim, dtype, error_word, &a);
  if (rc != PKV_OK || num_tokens == 0) return rc;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = launch_reshape_and_cache_mxfp4(a, st);
  if (e != cudaSuccess) return cuda_fail(e, "reshape_and_cache_mxfp4 launch");
  return validate_error_word(error_word, st, "reshape_and_cache_mxfp4");
}

int pkv_gather_cache_mxfp4(const void* key_cache, const void* value_cache,
                           const int64_t* slot_mapping, void* key_out, void* value_out,
                           int64_t key_out_stride, int64_t value_out_stride, int64_t num_tokens,
                           int64_t num_blocks, int32_t block_size, int32_t num_kv_heads,
                           int32_t head_dim, int32_t dtype, uint32_t* error_word, void* stream) {
  MxCacheArgs a;
  const int rc = cache_args("pkv_gather_cache_mxfp4", key_out, value_out, key_out_stride,
                            value_out_stride, key_cache, value_cache, slot_mapping, num_tokens,
                            num_blocks, block_size, num_kv_heads, head_dim, dtype, error_word, &a);
  if (rc != PKV_OK || num_tokens == 0) return rc;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = launch_gather_cache_mxfp4(a, st);
  if (e != cudaSuccess) return cuda_fail(e, "gather_cache_mxfp4 launch");
  return validate_error_word(error_word, st, "gather_cache_mxfp4");
}

size_t pkv_mxfp4_attention_workspace_bytes(int32_t num_heads, int32_t num_kv_heads,
                                           int32_t head_dim) {
  if (num_heads <= 0 || num_kv_heads <= 0 || num_heads % num_kv_heads ||
      num_heads / num_kv_heads > kMaxGroup || (head_dim != 64 && head_dim != 128))
    return 0;
  return mx_workspace(current_sm_count(), num_heads, num_kv_heads, head_dim).total;
}

int pkv_paged_attention_varlen_mxfp4(const void* q, int64_t q_stride, const void* key_cache,
                                     const void* value_cache, const int32_t* block_table,
                                     int32_t block_table_stride, int32_t max_blocks_per_req,
                                     const int32_t* query_start_loc,
                                     const int32_t* seq_lens, const int32_t* num_computed_tokens,
                                     float scale, void* out, int64_t out_stride,
                                     int64_t num_tokens, int32_t num_reqs, int64_t num_blocks,
                                     int32_t block_size, int32_t num_heads, int32_t num_kv_heads,
                                     int32_t head_dim, int32_t max_query_len, void* workspace,
                                     size_t workspace_bytes, void* stream) {
  const char* where = "pkv_paged_attention_varlen_mxfp4";
  if (num_tokens < 0 || num_reqs < 0 || num_heads <= 0 || max_query_len < 0)
    return fail(PKV_E_INVALID, "%s: bad sizes", where);
  const int rc = check_cache_shape(where, num_blocks, block_size, num_kv_heads, head_dim);
  if (rc != PKV_OK) return rc;
  if (num_heads % num_kv_heads) return fail(PKV_E_INVALID, "%s: num_heads %% num_kv_heads != 0", where);
  if (num_heads / num_kv_heads > kMaxGroup)
    return fail(PKV_E_UNSUPPORTED, "%s: more than %d query heads per KV head", where, kMaxGroup);
  if (num_reqs > step_metadata_max_reqs() || num_tokens > 0x7fffffffLL)
    return fail(PKV_E_UNSUPPORTED, "%s: at most %d requests and 2^31 - 1 tokens", where,
                step_metadata_max_reqs());
  if (!workspace) return fail(PKV_E_WORKSPACE, "%s: workspace is required", where);
  const int sms = current_sm_count();
  const MxWorkspace w = mx_workspace(sms, num_heads, num_kv_heads, head_dim);
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
  if (num_reqs * (static_cast<int64_t>(max_blocks_per_req) + kMxRequestCost) > 0x7fffffffLL - 15)
    return fail(PKV_E_UNSUPPORTED, "%s: a block table of more than 2^31 - 16 entries, with %d for each request",
                where, kMxRequestCost);
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
    e = launch_prefill_mxfp4(a, ps, max_query_len, sms, st);
  }
  if (e == cudaSuccess) e = launch_decode_mxfp4(a, ds, sms, st);
  if (e != cudaSuccess) return cuda_fail(e, "paged_attention_varlen_mxfp4 launch");
  return validate_error_word(a.err, st, "paged_attention_varlen_mxfp4");
}

int pkv_build_step_metadata(const int32_t* query_lens, const int32_t* num_computed_tokens,
                            int32_t num_reqs, int32_t* block_table, int32_t block_table_stride,
                            int32_t max_blocks_per_req, const int32_t* free_ring, int64_t ring_size, int64_t* free_state,
                            int64_t* free_state_out, int32_t block_size, int64_t num_tokens,
                            int32_t* query_start_loc, int32_t* seq_lens, int64_t* slot_mapping,
                            int64_t* positions, uint32_t* error_word, void* stream) {
  const char* where = "pkv_build_step_metadata";
  if (num_reqs < 0 || num_tokens < 0 || ring_size < 0 || max_blocks_per_req < 0)
    return fail(PKV_E_INVALID, "%s: sizes must not be negative", where);
  if (num_reqs > 1 && block_table_stride < max_blocks_per_req)
    return fail(PKV_E_INVALID, "%s: block_table rows of %d entries, %d apart", where,
                max_blocks_per_req, block_table_stride);
  if (block_size != kMxBlock)
    return fail(PKV_E_UNSUPPORTED, "%s: block_size must be 16 (got %d)", where, block_size);
  if (num_reqs > step_metadata_max_reqs() || num_tokens > 0x7fffffffLL || ring_size > 0x3fffffffLL)
    return fail(PKV_E_UNSUPPORTED, "%s: at most %d requests, 2^31 - 1 tokens and 2^30 - 1 ring entries",
                where, step_metadata_max_reqs());
  const size_t R = static_cast<size_t>(num_reqs), T = static_cast<size_t>(num_tokens);
  // from the first row's start to the last row's end
  const size_t table = R == 0 || max_blocks_per_req == 0 ? 0
      : 4 * ((R - 1) * static_cast<size_t>(block_table_stride) + max_blocks_per_req);
  if ((R && (!query_lens || !num_computed_tokens || !seq_lens)) || (table && !block_table) ||
      (ring_size && !free_ring) || !free_state || !free_state_out || !query_start_loc ||
      (T && !slot_mapping))
    return fail(PKV_E_INVALID, "%s: null pointer", where);
  // every CTA reads the inputs while others already write
  const struct { const void* p; size_t n; } in[] = {{query_lens, R * 4},
                                                    {num_computed_tokens, R * 4},
                                                    {free_ring, static_cast<size_t>(ring_size) * 4},
                                                    {free_state, 32}};
  const struct { const void* p; size_t n; } out[] = {{block_table, table},
                                                     {query_start_loc, (R + 1) * 4},
                                                     {seq_lens, R * 4},
                                                     {slot_mapping, T * 8},
                                                     {positions, T * 8},
                                                     {free_state_out, 16}};
  for (int i = 0; i < 6; ++i) {
    for (int j = 0; j < 4; ++j)
      if (!(i == 5 && j == 3 && out[i].p == in[j].p) && overlap(out[i].p, out[i].n, in[j].p, in[j].n))
        return fail(PKV_E_INVALID, "%s: an output overlaps an input", where);
    for (int j = 0; j < i; ++j)
      if (overlap(out[i].p, out[i].n, out[j].p, out[j].n))
        return fail(PKV_E_INVALID, "%s: two outputs overlap", where);
  }
  StepMetadataArgs a;
  a.query_lens = query_lens;
  a.num_computed = num_computed_tokens;
  a.block_table = block_table;
  a.bt_stride = block_table_stride;
  a.bt_width = max_blocks_per_req;
  a.free_ring = free_ring;
  a.ring_size = ring_size;
  a.free_state = free_state;
  a.free_state_out = free_state_out;
  a.query_start_loc = query_start_loc;
  a.seq_lens = seq_lens;
  a.slot_mapping = slot_mapping;
  a.positions = positions;
  a.num_tokens = num_tokens;
  a.num_reqs = num_reqs;
  a.err = error_word;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = launch_step_metadata(a, st);
  if (e != cudaSuccess) return cuda_fail(e, "build_step_metadata launch");
  return validate_error_word(error_word, st, "build_step_metadata");
}

}  // extern "C"
