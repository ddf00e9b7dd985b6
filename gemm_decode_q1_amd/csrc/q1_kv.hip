// Keys and values quantised into their pages, and read back (q1_memory.h).
//
// A lane has 8 elements of a key row and the same 8 of the value row (16 bytes of
// each), so four lanes share a block: its largest magnitude is a maximum over the
// raw 16-bit patterns (ordered as the magnitudes are, NaN and infinity on top), then
// over the four lanes.  From its fp32 bits the scale's byte is
//   e + 127 = ((bits + 0x1fffff) >> 23) - p:
// the sum carries into the exponent where the significand is above 1.75.
//
// Bound by bytes: 16384 tokens of 8 heads of 128, written in 4 bits and read back (170 MB), take
// 34.8 us, 4.9 TB/s, 94 % of a copy's rate.  8 tokens of 4 heads of 256 the same way 4.7: two launches.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "q1_internal.h"
#include "q1_kv_device.h"
#include "q1_memory.h"

namespace q1 {
namespace {

typedef kv_u32x4 u32x4;
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));

constexpr int kThreads = 256;

struct KvRows {
  q1_kv c;
  const int32_t* slots;
  uint32_t n;         // lanes in all: rows * Hkv * D / 8
  Divider per_row;    // by Hkv * D / 8
  Divider page;       // by page_size
  uint32_t lanes;     // Hkv * D / 8
};

// Where a lane's 8 elements are: row and first element in the operands, and the
// index of the (page, head, token) row in the pages, -1 for a slot outside.
struct Place {
  uint32_t row, elem, piece;
  int64_t at;
};

__device__ __forceinline__ Place place(const KvRows& a, uint32_t i) {
  Place p;
  p.row = divide(i, a.per_row);
  const uint32_t w = i - p.row * a.lanes, per_head = (uint32_t)a.c.D / 8;
  p.elem = w * 8;
  const uint32_t head = w / per_head;  // (per_head is 8, 16 or 32)
  p.piece = w - head * per_head;
  const int32_t slot = a.slots[p.row];
  if (slot < 0 || slot >= a.c.pages * a.c.page_size) {
    p.at = -1;
    return p;
  }
  const uint32_t page = divide((uint32_t)slot, a.page);
  p.at = ((int64_t)page * a.c.Hkv + head) * a.c.page_size + ((uint32_t)slot - page * (uint32_t)a.c.page_size);
  return p;
}

__device__ __forceinline__ uint32_t max2(uint32_t x, uint32_t y) {
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, x), __builtin_bit_cast(u16x2, y)));
}

// The largest of four neighbouring lanes' values.
__device__ __forceinline__ uint32_t max_quad(uint32_t v) {
  uint32_t w = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xb1, 0xf, 0xf, false);  // lanes 1 0 3 2
  v = v > w ? v : w;
  w = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4e, 0xf, 0xf, false);           // lanes 2 3 0 1
  return v > w ? v : w;
}

// Quantises a lane's 8 elements; its four lanes get the same scale byte.
template <bool F16, int BITS>
__device__ __forceinline__ uint32_t encode(u32x4 x, uint32_t* codes) {
  uint32_t m = max2(max2(x[0] & 0x7fff7fffu, x[1] & 0x7fff7fffu), max2(x[2] & 0x7fff7fffu, x[3] & 0x7fff7fffu));
  m = max_quad(m >> 16 > (m & 0xffffu) ? m >> 16 : m & 0xffffu);
  const bool finite = m < (F16 ? 0x7c00u : 0x7f80u);
  const uint32_t bits = __float_as_uint(F16 ? f16_bits_to_f32(m) : bf16_bits_to_f32(m));
  constexpr int low = BITS == 4 ? 2 : 10, high = F16 ? (BITS == 4 ? 140 : 134) : (BITS == 4 ? 252 : 246);
  int e = (int)((bits + 0x1fffffu) >> 23) - (BITS == 4 ? 2 : 8);
  e = e < low ? low : e > high ? high : e;
  const float scale = __uint_as_float((uint32_t)e << 23);
  float f[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = elem16<F16>(x[j >> 1], j & 1);
  if constexpr (BITS == 4) {
    uint32_t c = 0;
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, f[0], f[1], scale, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, f[2], f[3], scale, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, f[4], f[5], scale, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, f[6], f[7], scale, 3);
    codes[0] = finite ? c : 0u;
  } else {
    const float top = __uint_as_float(((uint32_t)e + 8) << 23 | 0x600000u);  // 448 * scale
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = __builtin_amdgcn_fmed3f(f[j], -top, top);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      kv_s16x2 c = {0, 0};
      c = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(c, f[4 * j], f[4 * j + 1], scale, false);
      c = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(c, f[4 * j + 2], f[4 * j + 3], scale, true);
      codes[j] = finite ? __builtin_bit_cast(uint32_t, c) : 0u;
    }
  }
  return finite ? (uint32_t)e : 255u;
}

template <int BITS>
__device__ __forceinline__ void put(void* pages, void* scales, const Place& p, int D, const uint32_t* codes, uint32_t e) {
  unsigned char* row = static_cast<unsigned char*>(pages) + p.at * (D * BITS / 8);
  if constexpr (BITS == 4) reinterpret_cast<uint32_t*>(row)[p.piece] = codes[0];
  else reinterpret_cast<uint2*>(row)[p.piece] = uint2{codes[0], codes[1]};
  if ((p.piece & 3) == 0) static_cast<unsigned char*>(scales)[p.at * (D / kKvBlock) + p.piece / 4] = (unsigned char)e;
}

template <bool F16, int BITS>
__global__ __launch_bounds__(kThreads) void q1_kv_write_kernel(const KvRows a, const uint16_t* k, const uint16_t* v,
                                                               int64_t k_ld, int64_t v_ld) {
  // (lanes of a block are neighbours in one wave: n and the stride are multiples of 4)
  for (uint32_t i = blockIdx.x * kThreads + threadIdx.x; i < a.n; i += gridDim.x * kThreads) {
    const Place p = place(a, i);
    const u32x4 x = *reinterpret_cast<const u32x4*>(k + p.row * k_ld + p.elem);
    const u32x4 y = *reinterpret_cast<const u32x4*>(v + p.row * v_ld + p.elem);
    uint32_t ck[2], cv[2];
    const uint32_t ek = encode<F16, BITS>(x, ck), ev = encode<F16, BITS>(y, cv);
    if (p.at >= 0) {
      put<BITS>(a.c.k, a.c.k_scales, p, a.c.D, ck, ek);
      put<BITS>(a.c.v, a.c.v_scales, p, a.c.D, cv, ev);
    }
  }
}

template <int BITS, int OUT>
__device__ __forceinline__ void get(const void* pages, const void* scales, const Place& p, int D, void* out, int64_t at) {
  uint32_t w[2] = {0u, 0u}, e = 2;
  if (p.at >= 0) {
    const unsigned char* row = static_cast<const unsigned char*>(pages) + p.at * (D * BITS / 8);
    if constexpr (BITS == 4) {
      w[0] = reinterpret_cast<const uint32_t*>(row)[p.piece];
    } else {
      const uint2 c = reinterpret_cast<const uint2*>(row)[p.piece];
      w[0] = c.x;
      w[1] = c.y;
    }
    e = static_cast<const unsigned char*>(scales)[p.at * (D / kKvBlock) + p.piece / 4];
  }
  const u32x4 b = kv_bf16<BITS>(w, kv_scale(e));
  if constexpr (OUT == BF16) {
    *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(out) + at) = b;
  } else {
    float f[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = elem16<false>(b[j >> 1], j & 1);
    if constexpr (OUT == F32) {
      float4* o = reinterpret_cast<float4*>(static_cast<float*>(out) + at);
      o[0] = float4{f[0], f[1], f[2], f[3]};
      o[1] = float4{f[4], f[5], f[6], f[7]};
    } else {
      u32x4 h;
#pragma unroll
      for (int j = 0; j < 4; ++j) h[j] = f32_to_f16_bits(f[2 * j]) | f32_to_f16_bits(f[2 * j + 1]) << 16;
      *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(out) + at) = h;
    }
  }
}

template <int BITS, int OUT>
__global__ __launch_bounds__(kThreads) void q1_kv_read_kernel(const KvRows a, void* k, void* v) {
  for (uint32_t i = blockIdx.x * kThreads + threadIdx.x; i < a.n; i += gridDim.x * kThreads) {
    const Place p = place(a, i);
    get<BITS, OUT>(a.c.k, a.c.k_scales, p, a.c.D, k, (int64_t)i * 8);
    get<BITS, OUT>(a.c.v, a.c.v_scales, p, a.c.D, v, (int64_t)i * 8);
  }
}

KvRows rows_of(const q1_kv& c, const int32_t* slots, int64_t rows) {
  KvRows a;
  a.c = c;
  a.slots = slots;
  a.lanes = (uint32_t)(c.Hkv * c.D / 8);
  a.n = (uint32_t)(rows * a.lanes);
  a.per_row = divider(a.lanes);
  a.page = divider((uint32_t)c.page_size);
  return a;
}

dim3 grid_of(const KvRows& a) {
  const uint32_t wgs = (a.n + kThreads - 1) / kThreads, most = (uint32_t)device_cus() * 64;
  return dim3(wgs < most ? wgs : most);
}

}  // namespace

hipError_t launch_kv_write(const q1_kv& c, const void* k, const void* v, bool f16, int64_t k_ld, int64_t v_ld,
                           int64_t tokens, const int32_t* slots, hipStream_t s) {
  const KvRows a = rows_of(c, slots, tokens);
#define Q1_KW(H, N)                                                                              \
  hipLaunchKernelGGL((q1_kv_write_kernel<H, N>), grid_of(a), dim3(kThreads), 0, s, a,             \
                     static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v), k_ld, v_ld)
  if (f16) {
    if (c.bits == 4) Q1_KW(true, 4);
    else Q1_KW(true, 8);
  } else {
    if (c.bits == 4) Q1_KW(false, 4);
    else Q1_KW(false, 8);
  }
#undef Q1_KW
  return hipGetLastError();
}

hipError_t launch_kv_read(const q1_kv& c, const int32_t* slots, int64_t rows, void* k, void* v, int32_t out_dtype,
                          hipStream_t s) {
  const KvRows a = rows_of(c, slots, rows);
#define Q1_KR(N, O) hipLaunchKernelGGL((q1_kv_read_kernel<N, O>), grid_of(a), dim3(kThreads), 0, s, a, k, v)
  if (c.bits == 4) {
    if (out_dtype == BF16) Q1_KR(4, BF16);
    else if (out_dtype == F16) Q1_KR(4, F16);
    else Q1_KR(4, F32);
  } else {
    if (out_dtype == BF16) Q1_KR(8, BF16);
    else if (out_dtype == F16) Q1_KR(8, F16);
    else Q1_KR(8, F32);
  }
#undef Q1_KR
  return hipGetLastError();
}

}  // namespace q1
