// Gated delta rule, recurrent form: the state stays in registers over the
// tokens of a call.
//
// Per token, with a = exp(g), p = S^T k, r = S^T q (both over the old state):
//   d = beta (v - a p),  o = scale (a r + (q.k) d),  S = a S + k (x) d,
// which is the rule of the header with its two products over the state taken
// together: S_t^T q = a S^T q + (k.q) d.  So a token needs one pass over the
// state and one reduction over Dk.
//
// A wave owns 32 columns of one head's state (columns are independent) and
// holds all Dk rows of them: lane l has columns 4 (l % 8) .. +3 of rows
// (l / 8) Dk/8 .. +Dk/8-1, so a load instruction reads whole 128-byte pieces
// and the reduction over Dk is a sum over registers, then over 8 lanes.
//
// Bound by the state's bytes, read and written once whatever the number of tokens:
// 61 sequences of 48 heads of 128x128 with 3 tokens each (390 MB) take 82 us, 4.75
// TB/s, where a copy of 2 GiB reaches 4.86; 8 sequences (51 MB) 11.7 us; one (6 MB)
// 5.2 us (4.6 in a replayed graph), which is a launch, two dependent reads and a write.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "q1_decode.h"
#include "q1_device.h"
#include "q1_internal.h"

namespace q1 {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

template <bool F16>
__device__ __forceinline__ float elem(uint32_t word, int hi) {
  const uint32_t b = hi ? word >> 16 : word & 0xffffu;
  return F16 ? f16_bits_to_f32(b) : bf16_bits_to_f32(b);
}

// Lane exchanges: after swap16(v, w) the pair holds, in every lane, a row of 16
// lanes' value and that of the row 16 lanes away (swap32: 32 lanes away).  The
// second operand has to be a register of its own, which the empty asm makes it.
__device__ __forceinline__ float add_xor16(float v) {
  float w = v;
  asm("" : "+v"(w));
  auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(w), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

__device__ __forceinline__ float add_xor32(float v) {
  float w = v;
  asm("" : "+v"(w));
  auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(w), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Sum over the lanes that differ in bits 3..5 of the lane id (every lane gets it).
__device__ __forceinline__ float sum_rows(float v) {
  v += __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), 0x128, 0xf, 0xf, false));
  return add_xor32(add_xor16(v));
}

constexpr int kStepWaves = 4;

template <bool F16, int DK>
__global__ __launch_bounds__(64 * kStepWaves) void q1_delta_recurrent_kernel(const DeltaArgs a) {
  constexpr int R = DK / 8;  // rows of the state per lane
  const int lane = threadIdx.x & 63;
  const int slices = (a.Dv + 31) / 32;
  const int64_t unit = (int64_t)blockIdx.x * (blockDim.x >> 6) + (threadIdx.x >> 6);
  const int64_t sh = unit / slices;
  if (sh >= a.nseq * a.Hv) return;
  const int64_t seq = sh / a.Hv;
  const int h = (int)(sh - seq * a.Hv), hk = h / (a.Hv / a.Hk);
  const int col = (int)(unit - sh * slices) * 32 + 4 * (lane & 7), rg = lane >> 3;
  const bool live = col < a.Dv;
  const int64_t first = seq * a.T;
  const int64_t slot = a.slot_ids ? a.slot_ids[seq] : seq;
  const bool have = slot >= 0 && slot < a.slots;
  const int esz = a.out_dtype == F32 ? 4 : 2;
  f32x4 S[R];
  float* st = a.state + ((have ? slot : 0) * a.Hv + h) * (int64_t)DK * a.Dv + (int64_t)rg * R * a.Dv + col;
#pragma unroll
  for (int i = 0; i < R; ++i)
    S[i] = have && live ? *reinterpret_cast<const f32x4*>(st + (int64_t)i * a.Dv) : f32x4{0.f, 0.f, 0.f, 0.f};

  for (int64_t t = first; t < first + a.T; ++t) {
    f32x4 o = {0.f, 0.f, 0.f, 0.f};
    if (have) {
      const uint16_t* kp = a.k + t * a.k_ld + hk * DK + rg * R;
      const uint16_t* qp = a.q + t * a.q_ld + hk * DK + rg * R;
      float kf[R], qf[R];
#pragma unroll
      for (int c = 0; c < R / 8; ++c) {
        const u32x4 kw = *reinterpret_cast<const u32x4*>(kp + 8 * c);
        const u32x4 qw = *reinterpret_cast<const u32x4*>(qp + 8 * c);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          kf[8 * c + e] = elem<F16>(kw[e >> 1], e & 1);
          qf[8 * c + e] = elem<F16>(qw[e >> 1], e & 1);
        }
      }
      f32x4 v = {0.f, 0.f, 0.f, 0.f};
      if (live) {
        const uint2 w = *reinterpret_cast<const uint2*>(a.v + t * a.v_ld + (int64_t)h * a.Dv + col);
        v = f32x4{elem<F16>(w.x, 0), elem<F16>(w.x, 1), elem<F16>(w.y, 0), elem<F16>(w.y, 1)};
      }
      const float decay = expf(a.g[t * a.Hv + h]), beta = a.beta[t * a.Hv + h];
      f32x4 p = {0.f, 0.f, 0.f, 0.f}, r = p;
      float kk = 0.f, qq = 0.f, qk = 0.f;
#pragma unroll
      for (int i = 0; i < R; ++i) {
        kk = __builtin_fmaf(kf[i], kf[i], kk);
        qq = __builtin_fmaf(qf[i], qf[i], qq);
        qk = __builtin_fmaf(qf[i], kf[i], qk);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          p[j] = __builtin_fmaf(S[i][j], kf[i], p[j]);
          r[j] = __builtin_fmaf(S[i][j], qf[i], r[j]);
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        p[j] = sum_rows(p[j]);
        r[j] = sum_rows(r[j]);
      }
      kk = sum_rows(kk);
      qq = sum_rows(qq);
      qk = sum_rows(qk);
      const float rk = a.l2norm ? 1.0f / sqrtf(kk + 1e-6f) : 1.0f, rq = a.l2norm ? 1.0f / sqrtf(qq + 1e-6f) : 1.0f;
      f32x4 d;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        d[j] = beta * (v[j] - decay * (rk * p[j]));
        o[j] = a.scale * (decay * (rq * r[j]) + (qk * rk * rq) * d[j]);
      }
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const float kn = kf[i] * rk;
#pragma unroll
        for (int j = 0; j < 4; ++j) S[i][j] = __builtin_fmaf(kn, d[j], decay * S[i][j]);
      }
    }
    if (rg == 0 && live) {
      unsigned char* op = static_cast<unsigned char*>(a.out) + ((t * a.Hv + h) * a.Dv + col) * esz;
      if (a.out_dtype == F32) {
        *reinterpret_cast<f32x4*>(op) = o;
      } else {
        uint32_t b[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) b[j] = a.out_dtype == BF16 ? f32_to_bf16_bits(o[j]) : f32_to_f16_bits(o[j]);
        *reinterpret_cast<uint2*>(op) = uint2{b[0] | b[1] << 16, b[2] | b[3] << 16};
      }
    }
  }
  if (have && live) {
#pragma unroll
    for (int i = 0; i < R; ++i) *reinterpret_cast<f32x4*>(st + (int64_t)i * a.Dv) = S[i];
  }
}

}  // namespace

hipError_t launch_delta_recurrent(const DeltaArgs& a, bool f16, int Dk, hipStream_t s) {
  const int64_t units = a.nseq * a.Hv * ((a.Dv + 31) / 32);
  // A workgroup of its own for each wave where they then still have a compute unit each (one
  // sequence of 48 heads: 5.2 us, with four to a workgroup 5.8); more waves by four (one by one,
  // 8 such sequences took 2 % longer, 61 with 3 tokens each 4 %).
  const int waves = units <= device_cus() ? 1 : kStepWaves;
  const dim3 grid((unsigned)((units + waves - 1) / waves)), block(64 * waves);
#define Q1_DR(H, D) hipLaunchKernelGGL((q1_delta_recurrent_kernel<H, D>), grid, block, 0, s, a)
  if (f16) {
    if (Dk == 128) Q1_DR(true, 128);
    else Q1_DR(true, 64);
  } else {
    if (Dk == 128) Q1_DR(false, 128);
    else Q1_DR(false, 64);
  }
#undef Q1_DR
  return hipGetLastError();
}

}  // namespace q1
