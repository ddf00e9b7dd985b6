// Parts of an attention tile shared by the kernels over 16-bit (q1_attn.hip) and
// quantised (q1_kv_attn.hip) keys and values: 32 tokens times blocks of 16 queries of
// one wave on the matrix cores.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace q1 {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

constexpr int kWaves = 4;
constexpr int kTile = 32;               // tokens of a wave's tile
constexpr int kStep = kWaves * kTile;   // tokens of a workgroup's iteration
constexpr float kLog2e = 1.44269504088896340736f;

template <bool F16>
__device__ __forceinline__ f32x4 mma(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (F16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// Two floats rounded to the operand type, and what the rounding left.
template <bool F16>
__device__ __forceinline__ uint32_t round2(float x, float y, float* rx, float* ry) {
  if constexpr (F16) {
    const f16x2 h = __builtin_convertvector(f32x2{x, y}, f16x2);
    *rx = x - (float)h[0];
    *ry = y - (float)h[1];
    return __builtin_bit_cast(uint32_t, h);
  } else {
    const bf16x2 h = __builtin_convertvector(f32x2{x, y}, bf16x2);
    *rx = x - (float)h[0];
    *ry = y - (float)h[1];
    return __builtin_bit_cast(uint32_t, h);
  }
}

// Maximum / sum over the four lanes that differ in bits 4 and 5 of the lane id.
__device__ __forceinline__ float max_groups(float v) {
  float w = v;
  asm("" : "+v"(w));
  auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(w), false, false);
  v = fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
  w = v;
  asm("" : "+v"(w));
  auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(w), false, false);
  return fmaxf(__uint_as_float(s[0]), __uint_as_float(s[1]));
}

__device__ __forceinline__ float sum_groups(float v) {
  float w = v;
  asm("" : "+v"(w));
  auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(w), false, false);
  v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  w = v;
  asm("" : "+v"(w));
  auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(w), false, false);
  return __uint_as_float(s[0]) + __uint_as_float(s[1]);
}

// Weights are taken relative to 2^kLift of the maximum, so that an fp16 remainder
// of a small one is still a normal number; bf16 has fp32's range.
template <bool F16>
constexpr float kLift = F16 ? 12.0f : 0.0f;

// The softmax of one tile for a block of 16 queries: scores of this lane's 8 tokens
// (those of `mine`) in, weights out as two operands; m, l and the output so far
// are brought to the new maximum.
template <bool F16, int DT>
__device__ __forceinline__ void weigh(const f32x4* S, uint32_t mine, float sc, float& m, float& l, f32x4* O, int stride,
                                      u32x4& hi, u32x4& lo) {
  float s[8], top = -INFINITY;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    s[j] = (mine >> j) & 1u ? S[j >> 2][j & 3] * sc : -INFINITY;
    top = fmaxf(top, s[j]);
  }
  const float mn = fmaxf(m, max_groups(top));
  const float base = mn == -INFINITY ? 0.f : mn;  // no token yet: every exponent below is -infinity
  if (__any(mn != m)) {
    const float keep = __builtin_amdgcn_exp2f(m - base);
    l *= keep;
#pragma unroll
    for (int d = 0; d < DT; ++d) O[d * stride] *= keep;
    m = mn;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    s[j] = __builtin_amdgcn_exp2f(s[j] - base + kLift<F16>);
    l += s[j];
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float rx, ry, r0, r1;
    hi[j] = round2<F16>(s[2 * j], s[2 * j + 1], &rx, &ry);
    lo[j] = round2<F16>(rx, ry, &r0, &r1);
  }
}

// 16 columns of 32 value rows as the A operand V^T; `at`: this lane's place in rows
// 4 (l/16) .. +3 (of 16), `next16`: bytes to the other 16 rows.
__device__ __forceinline__ u32x4 transposed(const unsigned char* at, int next16) {
  const s16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)at);
  const s16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(at + next16));
  const uint2 xw = __builtin_bit_cast(uint2, x), yw = __builtin_bit_cast(uint2, y);
  return u32x4{xw.x, xw.y, yw.x, yw.y};
}

}  // namespace
}  // namespace q1
