// Argument checks and error reporting shared by the C ABI's device entry points.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "kernels.h"
#include "pkv.h"
#include "pkv_error.h"

namespace pkv {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Records the CUDA error and returns PKV_E_CUDA.
int cuda_fail(cudaError_t e, const char* what);

// With PKV_VALIDATE=1 in the environment: waits for the stream, reads the error
// word and returns PKV_E_INVALID if any bit is set (PKV_OK otherwise, and
// always when word is NULL or validation is off).
int validate_error_word(const uint32_t* word, cudaStream_t stream, const char* where);

// Whether [p, p + np) and [q, q + nq) share a byte.
inline bool overlap(const void* p, size_t np, const void* q, size_t nq) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return p && q && np && nq && a < b + nq && b < a + np;
}

inline int check_cache_shape(const char* where, int64_t num_blocks, int32_t block_size,
                      int32_t num_kv_heads, int32_t head_dim) {
  if (num_blocks <= 0 || num_kv_heads <= 0)
    return fail(PKV_E_INVALID, "%s: sizes must be positive", where);
  if (block_size != 16)
    return fail(PKV_E_UNSUPPORTED, "%s: block_size must be 16 (got %d)", where, block_size);
  if (head_dim != 64 && head_dim != 128)
    return fail(PKV_E_UNSUPPORTED, "%s: head_dim must be 64 or 128 (got %d)", where, head_dim);
  if (num_kv_heads > (1 << 20) || num_blocks > 0x7fffffffLL)
    return fail(PKV_E_UNSUPPORTED, "%s: pool too large", where);
  return PKV_OK;
}

// The arguments of the cache write and of the gather.
inline int cache_args(const char* where, const void* rows_k, const void* rows_v, int64_t k_stride,
               int64_t v_stride, const void* key_cache, const void* value_cache,
               const int64_t* slot_mapping, int64_t num_tokens, int64_t num_blocks,
               int32_t block_size, int32_t num_kv_heads, int32_t head_dim, int32_t dtype,
               uint32_t* error_word, MxCacheArgs* a) {
  if (num_tokens < 0) return fail(PKV_E_INVALID, "%s: num_tokens is negative", where);
  const int rc = check_cache_shape(where, num_blocks, block_size, num_kv_heads, head_dim);
  if (rc != PKV_OK) return rc;
  if (dtype != PKV_F32 && dtype != PKV_BF16)
    return fail(PKV_E_UNSUPPORTED, "%s: dtype %d", where, dtype);
  if (num_tokens > 0) {
    if (!rows_k || !rows_v || !key_cache || !value_cache || !slot_mapping)
      return fail(PKV_E_INVALID, "%s: null pointer", where);
    const int64_t esize = dtype == PKV_F32 ? 4 : 2;
    if ((k_stride * esize) % 16 || (v_stride * esize) % 16 || !aligned16(rows_k) ||
        !aligned16(rows_v) || !aligned16(key_cache) || !aligned16(value_cache))
      return fail(PKV_E_INVALID, "%s: strides and bases must be 16-byte aligned", where);
    const int64_t row = static_cast<int64_t>(num_kv_heads) * head_dim;
    if (k_stride < row || v_stride < row)
      return fail(PKV_E_INVALID, "%s: token stride shorter than a row", where);
  }
  a->key = rows_k;
  a->value = rows_v;
  a->key_stride = k_stride;
  a->value_stride = v_stride;
  a->key_cache = static_cast<uint8_t*>(const_cast<void*>(key_cache));
  a->value_cache = static_cast<uint8_t*>(const_cast<void*>(value_cache));
  a->slot_mapping = slot_mapping;
  a->num_tokens = num_tokens;
  a->num_slots = num_blocks * block_size;
  a->num_kv_heads = num_kv_heads;
  a->head_dim = head_dim;
  a->bf16 = dtype == PKV_BF16;
  a->err = error_word;
  return PKV_OK;
}

}  // namespace pkv
