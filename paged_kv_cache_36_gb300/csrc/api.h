// Argument checks and error reporting shared by the C ABI's device entry points.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace pkv {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Records the CUDA error and returns PKV_E_CUDA.
int cuda_fail(cudaError_t e, const char* what);

// With PKV_VALIDATE=1 in the environment: waits for the stream, reads the error
// word and returns PKV_E_INVALID if any bit is set (PKV_OK otherwise, and
// always when word is NULL or validation is off).
int validate_error_word(const uint32_t* word, cudaStream_t stream, const char* where);

}  // namespace pkv
