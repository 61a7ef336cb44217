// Shared by the C-ABI files: the calling thread's error text and small checks.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace chord {

// Records the description that chord_last_error_string() returns on this
// thread; returns `code`.
int fail(int code, const char* fmt, ...);
int cuda_fail(cudaError_t e, const char* what);

// Whether chord_debug_force_timeout is on.
bool force_timeout();

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline bool valid_block_m(int bm) { return bm == 8 || bm == 16 || bm == 32 || bm == 64 || bm == 128; }

}  // namespace chord
