// Codes of the paged keys and values (q1_memory.h): conversions shared by the
// kernels that write, read and attend to them.
//
// gfx950 converts pairs of E2M1 or E4M3 codes to bf16 or fp32, times a power of two
// given as a float: one instruction a pair, exact for the scale bytes that are used
// (2^(byte - 127); a NaN scale gives NaN for every E2M1 code).  The other way, E2M1 is
// rounded to nearest even and saturates; E4M3 does not saturate, so its operands
// are clamped first.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "q1_device.h"
#include "q1_memory.h"
#include "q1_memory_device.h"

namespace q1 {

typedef uint32_t kv_u32x4 __attribute__((ext_vector_type(4)));
typedef float kv_f32x2 __attribute__((ext_vector_type(2)));
typedef short kv_s16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 kv_bf16x2 __attribute__((ext_vector_type(2)));

// The scale of a byte as the conversions take it: 255 is a NaN.
__device__ __forceinline__ float kv_scale(uint32_t byte) {
  return __uint_as_float(byte == 255u ? 0x7fc00000u : byte << 23);
}

// 8 elements (a dword of 4-bit codes, two of 8-bit ones) as 4 dwords of bf16 pairs.
template <int BITS>
__device__ __forceinline__ kv_u32x4 kv_bf16(const uint32_t* w, float scale) {
  kv_bf16x2 r[4];
  if constexpr (BITS == 4) {
    r[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[0], scale, 0);
    r[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[0], scale, 1);
    r[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[0], scale, 2);
    r[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[0], scale, 3);
  } else {
    r[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[0], scale, false);
    r[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[0], scale, true);
    r[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[1], scale, false);
    r[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[1], scale, true);
  }
  return kv_u32x4{__builtin_bit_cast(uint32_t, r[0]), __builtin_bit_cast(uint32_t, r[1]),
                  __builtin_bit_cast(uint32_t, r[2]), __builtin_bit_cast(uint32_t, r[3])};
}

}  // namespace q1
