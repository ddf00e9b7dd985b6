// Selective state space scan (q1_memory.h), single tokens and prompts.
//
// Single tokens: four lanes have a channel, a quarter of its states each, so that a
// state is read and written in whole lines and one sequence fills some hundred waves.
//
// Prompts: a lane has a channel and all of its states in registers; B and C are the
// same for all channels and come through scalar loads.  Per token, channel and state
// that is a product, an exponential (a quarter of the rate of the others), a product
// and two multiply-adds.  A long prompt is cut into pieces so that the waves fill the
// chip, in three launches:
//   q1_scan_state  the state at the end of each piece from a zero state, and the sum
//                  of its deltas (the decay over the piece is exp(A * sum));
//   q1_scan_join   each piece's first state, one after the other;
//   q1_scan_out    the outputs, and from a sequence's last piece its final state.
// A sequence's last piece needs no q1_scan_state, so short sequences have none.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "q1_internal.h"
#include "q1_memory.h"
#include "q1_memory_device.h"

namespace q1 {
namespace {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr int kThreads = 256;

typedef const __attribute__((address_space(4))) uint32_t* scalar_words;  // read through scalar loads

template <bool F16>
__device__ __forceinline__ float elem(uint32_t b) {
  return elem16<F16>(b, 0);
}

// log(1 + exp(s)) = max(s, 0) + log1p(u), u = exp(-|s|) <= 1, and with w = u / (2 + u) <= 1/3
// log1p(u) = 2 artanh w = 2 w (1 + w^2/3 + .. + w^14/15), off by less than w^16/17 < 2^-29 of it.
// The rounding of s log2(e), which would be |s| units of u, is made good to first order.
__device__ __forceinline__ float softplus(float s) {
  const float v = -fabsf(s), r = v * kLog2e;
  const float low = __builtin_fmaf(v, kLog2e, -r) + v * 1.92596299e-8f;  // log2(e) - kLog2e
  float u = __builtin_amdgcn_exp2f(r);
  u = u > 0.f ? __builtin_fmaf(u, low * 0.693147181f, u) : u;  // (past its range low may be anything)
  const float w = u * __builtin_amdgcn_rcpf(2.0f + u), q = w * w;
  float p = 1.0f / 15;
  p = __builtin_fmaf(p, q, 1.0f / 13);
  p = __builtin_fmaf(p, q, 1.0f / 11);
  p = __builtin_fmaf(p, q, 1.0f / 9);
  p = __builtin_fmaf(p, q, 1.0f / 7);
  p = __builtin_fmaf(p, q, 1.0f / 5);
  p = __builtin_fmaf(p, q, 1.0f / 3);
  p = __builtin_fmaf(p, q, 1.0f);
  return fmaxf(s, 0.f) + 2.0f * w * p;
}

// Raw bits of dt, and its value.
__device__ __forceinline__ uint32_t load_dt(const q1_scan& d, int64_t at) {
  if (d.dt_dtype == F32) return static_cast<const uint32_t*>(d.dt)[at];
  return static_cast<const uint16_t*>(d.dt)[at];
}
template <bool F16>
__device__ __forceinline__ float delta_of(const q1_scan& d, uint32_t raw, float bias) {
  const float s = (d.dt_dtype == F32 ? __uint_as_float(raw) : elem<F16>(raw)) + bias;
  return d.softplus ? softplus(s) : s;
}

// The sum of four neighbouring lanes' values.
__device__ __forceinline__ float sum_quad(float v) {
  v += __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), 0xb1, 0xf, 0xf, false));
  v += __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), 0x4e, 0xf, 0xf, false));
  return v;
}

struct StepArgs {
  q1_scan d;
  int64_t T;
  uint32_t n, lanes;  // lanes in all, and of a sequence: 4 * Di
  Divider per_seq;
};

template <bool F16, int N>
__global__ __launch_bounds__(kThreads) void q1_scan_step_kernel(const StepArgs a) {
  constexpr int M = N / 4;  // states of a lane
  const q1_scan& d = a.d;
  const uint32_t i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= a.n) return;  // (n is a multiple of 32: the four lanes of a channel stay together)
  const int64_t seq = divide(i, a.per_seq);
  const uint32_t w = i - (uint32_t)seq * a.lanes, ch = w >> 2, part = w & 3;
  const int64_t slot = d.slot_ids ? d.slot_ids[seq] : seq;
  const bool have = slot >= 0 && slot < d.slots;
  float A[M], h[M];
  float* st = d.state + ((have ? slot : 0) * d.Di + ch) * N + part * M;
#pragma unroll
  for (int j = 0; j < M; ++j) {
    A[j] = d.A[(int64_t)ch * N + part * M + j] * kLog2e;
    h[j] = have ? st[j] : 0.f;
  }
  const float bias = d.dt_bias ? d.dt_bias[ch] : 0.f, skip = d.D ? d.D[ch] : 0.f;
  for (int64_t t = seq * a.T; t < (seq + 1) * a.T; ++t) {
    float out = 0.f;
    if (have) {
      const float x = elem<F16>(static_cast<const uint16_t*>(d.x)[t * d.x_ld + ch]);
      const float delta = delta_of<F16>(d, load_dt(d, t * d.dt_ld + ch), bias), dx = delta * x;
      const uint32_t* b = reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(d.B) + t * d.b_ld) + part * (M / 2);
      const uint32_t* c = reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(d.C) + t * d.c_ld) + part * (M / 2);
      float y = 0.f;
#pragma unroll
      for (int j = 0; j < M; ++j) {
        h[j] = __builtin_fmaf(__builtin_amdgcn_exp2f(delta * A[j]), h[j], dx * elem16<F16>(b[j >> 1], j & 1));
        y = __builtin_fmaf(elem16<F16>(c[j >> 1], j & 1), h[j], y);
      }
      out = __builtin_fmaf(skip, x, sum_quad(y));
      if (d.z != nullptr) out *= silu_fast(elem<F16>(static_cast<const uint16_t*>(d.z)[t * d.z_ld + ch]));
    }
    if (part == 0) store_out(d.out, d.out_dtype, t * d.Di + ch, out);
  }
  if (have) {
#pragma unroll
    for (int j = 0; j < M; ++j) st[j] = h[j];
  }
}

struct PromptArgs {
  q1_scan d;
  Ragged r;
  int64_t per;     // tokens of a piece
  int64_t blocks;  // of 64 channels
  float* h;        // [pieces, N, Di]: behind piece p, of which its sequence has a next one
  float* sum;      // [pieces, Di]
};

constexpr int kAhead = 8;  // tokens whose rows are in flight

// One lane's walk over the rows [t0, t1): h is advanced, sum gets the deltas, and
// with OUT the outputs are written.
template <bool F16, int N, bool OUT>
__device__ __forceinline__ void walk(const q1_scan& d, int64_t t0, int64_t t1, int64_t ch, bool live, float* h, float& sum) {
  float A[N];
#pragma unroll
  for (int n = 0; n < N; ++n) A[n] = d.A[ch * N + n] * kLog2e;
  const float bias = d.dt_bias ? d.dt_bias[ch] : 0.f, skip = OUT && d.D ? d.D[ch] : 0.f;
  const auto* xp = static_cast<const uint16_t*>(d.x) + ch;
  const auto* zp = static_cast<const uint16_t*>(d.z) + ch;
  const bool gate = OUT && d.z != nullptr;
  const int64_t last = t1 - 1;
  uint32_t xr[kAhead], dr[kAhead], zr[kAhead];
  auto load = [&](int64_t t) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int64_t at = t + u < last ? t + u : last;
      xr[u] = xp[at * d.x_ld];
      dr[u] = load_dt(d, at * d.dt_ld + ch);
      zr[u] = gate ? zp[at * d.z_ld] : 0u;
    }
  };
  load(t0);
  for (int64_t t = t0; t < t1; t += kAhead) {
    uint32_t xc[kAhead], dc[kAhead], zc[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) xc[u] = xr[u], dc[u] = dr[u], zc[u] = zr[u];
    load(t + kAhead);
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (t + u >= t1) break;
      const scalar_words b = (scalar_words)(uintptr_t)(static_cast<const uint16_t*>(d.B) + (t + u) * d.b_ld);
      const scalar_words c = (scalar_words)(uintptr_t)(static_cast<const uint16_t*>(d.C) + (t + u) * d.c_ld);
      const float x = elem<F16>(xc[u]), delta = delta_of<F16>(d, dc[u], bias), dx = delta * x;
      sum += delta;
      float y0 = 0.f, y1 = 0.f;
#pragma unroll
      for (int n = 0; n < N; n += 2) {
        const uint32_t bw = b[n / 2];
        h[n] = __builtin_fmaf(__builtin_amdgcn_exp2f(delta * A[n]), h[n], dx * elem16<F16>(bw, 0));
        h[n + 1] = __builtin_fmaf(__builtin_amdgcn_exp2f(delta * A[n + 1]), h[n + 1], dx * elem16<F16>(bw, 1));
        if constexpr (OUT) {
          const uint32_t cw = c[n / 2];
          y0 = __builtin_fmaf(elem16<F16>(cw, 0), h[n], y0);
          y1 = __builtin_fmaf(elem16<F16>(cw, 1), h[n + 1], y1);
        }
      }
      if constexpr (OUT) {
        float out = __builtin_fmaf(skip, x, y0 + y1);
        if (gate) out *= silu_fast(elem<F16>(zc[u]));
        if (live) store_out(d.out, d.out_dtype, (t + u) * d.Di + ch, out);
      }
    }
  }
}

__device__ __forceinline__ int64_t slot_of(const q1_scan& d, int64_t seq) {
  const int64_t slot = d.slot_ids ? d.slot_ids[seq] : seq;
  return slot >= 0 && slot < d.slots ? slot : -1;
}

template <bool F16, int N, bool OUT>
__global__ __launch_bounds__(64) void q1_scan_kernel(const PromptArgs a) {
  const q1_scan& d = a.d;
  const int64_t piece = blockIdx.x / a.blocks, c0 = (blockIdx.x - piece * a.blocks) * 64 + threadIdx.x;
  const Piece p = find_piece(a.r, piece, a.per);
  if (p.t0 >= p.t1) return;
  if (!OUT && p.last()) return;
  const bool live = c0 < d.Di;
  const int64_t ch = live ? c0 : d.Di - 1, slot = slot_of(d, p.seq);
  if (slot < 0) {
    if (OUT && live)
      for (int64_t t = p.t0; t < p.t1; ++t) store_out(d.out, d.out_dtype, t * d.Di + ch, 0.f);
    return;
  }
  float h[N], sum = 0.f;
  if constexpr (!OUT) {
#pragma unroll
    for (int n = 0; n < N; ++n) h[n] = 0.f;
  } else if (p.first()) {
#pragma unroll
    for (int n = 0; n < N; ++n) h[n] = d.state[(slot * d.Di + ch) * N + n];
  } else {
#pragma unroll
    for (int n = 0; n < N; ++n) h[n] = a.h[((piece - 1) * N + n) * d.Di + ch];
  }
  walk<F16, N, OUT>(d, p.t0, p.t1, ch, live, h, sum);
  if (!live) return;
  if constexpr (!OUT) {
#pragma unroll
    for (int n = 0; n < N; ++n) a.h[(piece * N + n) * d.Di + ch] = h[n];
    a.sum[piece * d.Di + ch] = sum;
  } else if (p.last()) {
#pragma unroll
    for (int n = 0; n < N; ++n) d.state[(slot * d.Di + ch) * N + n] = h[n];
  }
}

// A lane has one state of one channel of a sequence: from the ends of its pieces to
// their first states, in place.
__global__ __launch_bounds__(kThreads) void q1_scan_join(const PromptArgs a) {
  constexpr int U = 4;  // pieces in flight
  const q1_scan& d = a.d;
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x, per = d.Di * d.N, seq = i / per;
  if (seq >= a.r.nseq) return;
  const int n = (int)((i - seq * per) / d.Di);
  const int64_t ch = i - seq * per - n * d.Di, slot = slot_of(d, seq);
  const int64_t begin = cu_at(a.r, seq), end = cu_at(a.r, seq + 1);
  const int64_t pieces = (end - begin + a.per - 1) / a.per, first = begin / a.per + seq;
  if (slot < 0 || pieces < 2) return;
  const float A = d.A[ch * d.N + n] * kLog2e;
  float h = d.state[(slot * d.Di + ch) * d.N + n];
  float* hp = a.h + (first * d.N + n) * d.Di + ch;
  const float* sp = a.sum + first * d.Di + ch;
  for (int64_t j = 0; j < pieces - 1; j += U) {
    float e[U], s[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t at = j + u < pieces - 1 ? j + u : pieces - 2;
      e[u] = hp[at * d.N * d.Di];
      s[u] = sp[at * d.Di];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (j + u >= pieces - 1) break;
      h = __builtin_fmaf(__builtin_amdgcn_exp2f(A * s[u]), h, e[u]);
      hp[(j + u) * d.N * d.Di] = h;
    }
  }
}

template <bool F16, int N>
hipError_t launch_prompt(const PromptArgs& a, int64_t pieces, hipStream_t s) {
  const dim3 grid((unsigned)(pieces * a.blocks));
  if (a.h != nullptr) {
    hipLaunchKernelGGL((q1_scan_kernel<F16, N, false>), grid, dim3(64), 0, s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t n = a.r.nseq * a.d.Di * N;
    hipLaunchKernelGGL(q1_scan_join, dim3((unsigned)((n + kThreads - 1) / kThreads)), dim3(kThreads), 0, s, a);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((q1_scan_kernel<F16, N, true>), grid, dim3(64), 0, s, a);
  return hipGetLastError();
}

template <bool F16>
hipError_t launch_n(const PromptArgs& a, int64_t pieces, hipStream_t s) {
  return a.d.N == 8    ? launch_prompt<F16, 8>(a, pieces, s)
         : a.d.N == 16 ? launch_prompt<F16, 16>(a, pieces, s)
         : a.d.N == 32 ? launch_prompt<F16, 32>(a, pieces, s)
                       : launch_prompt<F16, 64>(a, pieces, s);
}

size_t sums_at(const q1_scan& d, int64_t pieces) { return ((size_t)pieces * d.N * d.Di * 4 + 255) / 256 * 256; }

}  // namespace

int64_t scan_chunk(const q1_scan& d, int64_t tokens, int64_t nseq) {
  const int64_t blocks = (d.Di + 63) / 64, slots = (int64_t)device_cus() * 4 * 4;
  if (nseq * blocks >= slots) return 0;
  const int64_t per = (tokens * blocks + slots - 1) / slots;
  return per < 32 ? 32 : per;
}

int64_t scan_pieces(const q1_scan& d, int64_t tokens, int64_t nseq) {
  const int64_t per = scan_chunk(d, tokens, nseq);
  return ragged_pieces(tokens, nseq, per == 0 ? tokens : per);
}

size_t scan_ws_bytes(const q1_scan& d, int64_t tokens, int64_t nseq) {
  if (scan_chunk(d, tokens, nseq) == 0) return 0;
  const int64_t pieces = scan_pieces(d, tokens, nseq);
  return sums_at(d, pieces) + ((size_t)pieces * d.Di * 4 + 255) / 256 * 256;
}

hipError_t launch_scan_step(const q1_scan& d, int64_t B, int64_t T, hipStream_t s) {
  StepArgs a = {};
  a.d = d;
  a.T = T;
  a.lanes = (uint32_t)(4 * d.Di);
  a.n = (uint32_t)(B * a.lanes);
  a.per_seq = divider(a.lanes);
  const dim3 grid((a.n + kThreads - 1) / kThreads), block(kThreads);
#define Q1_SS(H, N) hipLaunchKernelGGL((q1_scan_step_kernel<H, N>), grid, block, 0, s, a)
  if (d.dtype == Q1_F16) {
    if (d.N == 8) Q1_SS(true, 8);
    else if (d.N == 16) Q1_SS(true, 16);
    else if (d.N == 32) Q1_SS(true, 32);
    else Q1_SS(true, 64);
  } else {
    if (d.N == 8) Q1_SS(false, 8);
    else if (d.N == 16) Q1_SS(false, 16);
    else if (d.N == 32) Q1_SS(false, 32);
    else Q1_SS(false, 64);
  }
#undef Q1_SS
  return hipGetLastError();
}

hipError_t launch_scan_prefill(const q1_scan& d, const Ragged& r, unsigned char* ws, hipStream_t s) {
  PromptArgs a = {};
  a.d = d;
  a.r = r;
  const int64_t per = scan_chunk(d, r.tokens, r.nseq), pieces = scan_pieces(d, r.tokens, r.nseq);
  a.per = per == 0 ? r.tokens : per;
  a.blocks = (d.Di + 63) / 64;
  if (per != 0) {
    a.h = reinterpret_cast<float*>(ws);
    a.sum = reinterpret_cast<float*>(ws + sums_at(d, pieces));
  }
  return d.dtype == Q1_F16 ? launch_n<true>(a, pieces, s) : launch_n<false>(a, pieces, s);
}

}  // namespace q1
