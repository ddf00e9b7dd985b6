// Status and argument helpers shared by the files that implement the C ABI.
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

#include "../../include/q1.h"

namespace q1 {

// Sets the thread's error text and returns `s`.
q1_status fail(q1_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
// Clears the error text and returns Q1_OK.
q1_status ok();
// Q1_OK if the current device is a gfx950 (cached per device).
q1_status check_current_device();
q1_status hip_status(hipError_t e, const char* what);

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }
inline bool valid_out_dtype(int32_t d) { return d == Q1_F32 || d == Q1_F16 || d == Q1_BF16; }
inline size_t dtype_size(int32_t d) { return d == Q1_F32 ? 4 : 2; }

}  // namespace q1
