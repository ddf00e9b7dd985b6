// Selective state space scan (q1_memory.h), single tokens and prompts.
//
// Single tokens: four lanes have a channel, a quarter of its states each, so that a
// state is read and written in whole lines and one sequence fills some hundred waves.
//
// Prompts: a lane has a channel and all of its states in registers; B and C are the
// same for all channels and come through scalar loads, a token ahead.  A prompt is cut
// into pieces so that the waves fill the chip, in three launches:
//   q1_scan_state  the state at the end of each piece from a zero state, and the sum
//                  of its deltas (the decay over the piece is exp(A * sum));
//   q1_scan_join   each piece's first state, one after the other;
//   q1_scan_out    the outputs, and from a sequence's last piece its final state.
// A sequence's last piece needs no q1_scan_state, so short sequences have none.  (Both
// are q1_scan_kernel, without and with outputs.)
//
// Bound by the vector units (93 % busy): a state costs a product, an exponential (8 cycles
// a wave, the others 4), a product and two multiply-adds a token, and without outputs one
// less, so that one walk over 16384 tokens of 5120 channels of 16 states cannot take less
// than 235 us at 2.15 GHz, both 430; with deltas, skip and gate they take 356 and 267, the
// join 27 (100 MB).  Reading and writing rows would take 136.
// Walking once would leave 80 waves for one sequence (9 ms), or, with a state a lane, 1280
// whose outputs need a sum over 16 lanes a token: by count of instructions no less than
// these, on 1024 SIMDs.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "q1_internal.h"
#include "q1_memory.h"
#include "q1_memory_device.h"

namespace q1 {
namespace {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr int kThreads = 256;

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef const __attribute__((address_space(4))) uint32_t* scalar_words;  // read through scalar loads

template <bool F16>
__device__ __forceinline__ float elem(uint32_t b) {
  return elem16<F16>(b, 0);
}

// log(1 + exp(s)) = max(s, 0) + log1p(u), u = exp(-|s|) <= 1, and with w = u / (2 + u) <= 1/3
// log1p(u) = 2 artanh w = 2 w p(w^2), p of degree 4 from the Chebyshev interpolation of
// artanh(w) / w over w^2 <= 1/9 (off by less than 2^-27 of it).  The rounding of |s| log2(e),
// which would be |s| units of u, is made good to first order; what is left, of the
// constant's own rounding, is a quarter of that.
__device__ __forceinline__ float softplus(float s) {
  const float v = -fabsf(s), r = v * kLog2e;
  const float low = fminf(__builtin_fmaf(v, kLog2e, -r), 1.0f);  // (far out, where u is 0, it may be anything)
  float u = __builtin_amdgcn_exp2f(r);
  u = __builtin_fmaf(u * low, 0.693147181f, u);
  const float w = u * __builtin_amdgcn_rcpf(2.0f + u), q = w * w;
  float p = 0.140788892f;
  p = __builtin_fmaf(p, q, 0.139825789f);
  p = __builtin_fmaf(p, q, 0.200122976f);
  p = __builtin_fmaf(p, q, 0.333331608f);
  p = __builtin_fmaf(p, q, 1.000000004f);
  return __builtin_fmaf(w * p, 2.0f, fmaxf(s, 0.f));
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

// An element of a pair, times x (fp16: with the conversion in the multiply-add).
template <bool F16>
__device__ __forceinline__ float times(uint32_t w, int hi, float x) {
  if constexpr (F16) return __builtin_fmaf(elem16<F16>(w, hi), x, 0.f);
  else return elem16<F16>(w, hi) * x;
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
  Divider by;
  int64_t blocks;  // of 64 channels
  Divider per_seq, channels;  // by Di * N and Di
  float* h;        // [pieces, N, Di]: behind piece p, of which its sequence has a next one
  float* sum;      // [pieces, Di]
};

constexpr int kBlock = 8;  // tokens of a block

// A wave's part of the LDS: a block's deltas, deltas times x, and sums over the states.
struct BlockLds {
  float delta[kBlock][64], dx[kBlock][64], y[kBlock][64];
};

// B and C of a token, in scalar registers.
template <int N, bool OUT>
struct Shared {
  uint32_t b[N / 2], c[OUT ? N / 2 : 1];
};

// A wave's walk over the rows [t0, t1) of a piece, 64 channels from c0 on.  Rows come in
// and go out by blocks of 8 tokens in which a lane has 8 channels of one token (16 bytes):
// so it makes the deltas and applies skip and gate.  Between these, through LDS, a lane
// has one channel and its states, token by token.
template <bool F16, bool DT32, int N, bool OUT>
struct Walk {
  static constexpr bool kPrefetch = N <= 16;  // (two tokens of more states do not fit the scalar registers)
  const q1_scan& d;
  BlockLds& m;
  const int64_t t1;
  const int lane, row;         // this lane's token of a block
  const uint32_t ch, c8;       // this lane's channel; first of its 8 channels of a row
  float h[N], A[N], bias[8], skip[OUT ? 8 : 1], sum = 0.f;
  u32x4 x, z, dt[DT32 ? 2 : 1];

  __device__ __forceinline__ Walk(const q1_scan& d, BlockLds& m, int64_t t1, uint32_t c0)
      : d(d), m(m), t1(t1), lane(threadIdx.x & 63), row(lane >> 3), ch(least(c0 + lane, (uint32_t)d.Di - 1)),
        c8(least(c0 + 8 * (lane & 7), (uint32_t)d.Di - 8)) {
    take(d.A + (int64_t)ch * N, A);
#pragma unroll
    for (int n = 0; n < N; ++n) A[n] *= kLog2e;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      bias[e] = d.dt_bias ? d.dt_bias[c8 + e] : 0.f;
      if constexpr (OUT) skip[e] = d.D ? d.D[c8 + e] : 0.f;
    }
  }

  static __device__ __forceinline__ void take(const float* from, float* to) {
#pragma unroll
    for (int n = 0; n < N / 4; ++n) {
      const f32x4 v = reinterpret_cast<const f32x4*>(from)[n];
#pragma unroll
      for (int j = 0; j < 4; ++j) to[4 * n + j] = v[j];
    }
  }

  static __device__ __forceinline__ uint32_t least(uint32_t a, uint32_t b) { return a < b ? a : b; }

  // The block of rows from t on (the last row again past the end).
  __device__ __forceinline__ void load(int64_t t) {
    const int64_t at = t + row < t1 ? t + row : t1 - 1;
    x = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(d.x) + at * d.x_ld + c8);
    if constexpr (DT32) {
      const u32x4* p = reinterpret_cast<const u32x4*>(static_cast<const float*>(d.dt) + at * d.dt_ld + c8);
      dt[0] = p[0];
      dt[1] = p[1];
    } else {
      dt[0] = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(d.dt) + at * d.dt_ld + c8);
    }
    if constexpr (OUT) {
      z = u32x4{0u, 0u, 0u, 0u};
      if (d.z != nullptr) z = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(d.z) + at * d.z_ld + c8);
    }
  }

  __device__ __forceinline__ void put_deltas() {
    float delta[8], dx[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float s = (DT32 ? __uint_as_float(dt[DT32 ? e >> 2 : 0][e & 3]) : elem16<F16>(dt[0][e >> 1], e & 1)) + bias[e];
      const float soft = softplus(s);
      delta[e] = d.softplus ? soft : s;
      dx[e] = delta[e] * elem16<F16>(x[e >> 1], e & 1);
    }
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      *reinterpret_cast<f32x4*>(&m.delta[row][8 * (lane & 7) + 4 * q]) = f32x4{delta[4 * q], delta[4 * q + 1], delta[4 * q + 2], delta[4 * q + 3]};
      *reinterpret_cast<f32x4*>(&m.dx[row][8 * (lane & 7) + 4 * q]) = f32x4{dx[4 * q], dx[4 * q + 1], dx[4 * q + 2], dx[4 * q + 3]};
    }
  }

  // B and C of the row `u` behind those at bp and cp.
  __device__ __forceinline__ void load_shared(const char* bp, const char* cp, uint32_t u, Shared<N, OUT>& s) const {
    const scalar_words b = (scalar_words)(uintptr_t)(bp + u * (uint32_t)(d.b_ld * 2));
    const scalar_words c = (scalar_words)(uintptr_t)(cp + u * (uint32_t)(d.c_ld * 2));
#pragma unroll
    for (int n = 0; n < N / 2; ++n) s.b[n] = b[n];
    if constexpr (OUT) {
#pragma unroll
      for (int n = 0; n < N / 2; ++n) s.c[n] = c[n];
    }
  }

  // Scalar loads come back in any order: what waits for one waits for all of them.  So
  // these are waited for here, before the next ones are issued.
  __device__ __forceinline__ void arrived(Shared<N, OUT>& s) const {
#pragma unroll
    for (int n = 0; n < N / 2; ++n) {
      asm volatile("" : "+s"(s.b[n]));
      if constexpr (OUT) asm volatile("" : "+s"(s.c[n]));
    }
    __builtin_amdgcn_sched_barrier(0);
  }

  __device__ __forceinline__ void token(int u, const Shared<N, OUT>& w) {
    const float delta = m.delta[u][lane], dx = m.dx[u][lane];
    if constexpr (!OUT) sum += delta;
    float y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int n = 0; n < N; ++n) {
      h[n] = __builtin_fmaf(__builtin_amdgcn_exp2f(delta * A[n]), h[n], times<F16>(w.b[n / 2], n & 1, dx));
      if constexpr (OUT) y[n & 3] = __builtin_fmaf(elem16<F16>(w.c[n / 2], n & 1), h[n], y[n & 3]);
    }
    if constexpr (OUT) m.y[u][lane] = (y[0] + y[1]) + (y[2] + y[3]);
  }

  __device__ __forceinline__ void put_rows(int64_t t, uint32_t first, u32x4 x, u32x4 z) const {
    float o[8];
    const f32x4 lo = *reinterpret_cast<const f32x4*>(&m.y[row][8 * (lane & 7)]);
    const f32x4 hi = *reinterpret_cast<const f32x4*>(&m.y[row][8 * (lane & 7) + 4]);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      o[e] = __builtin_fmaf(skip[e], elem16<F16>(x[e >> 1], e & 1), e < 4 ? lo[e & 3] : hi[e & 3]);
      const float gate = silu_fast(elem16<F16>(z[e >> 1], e & 1));
      o[e] = d.z != nullptr ? o[e] * gate : o[e];
    }
    if (t + row >= t1 || first + 8 * (lane & 7) >= d.Di) return;
    const int64_t at = (t + row) * d.Di + c8;
    if (d.out_dtype == F32) {
      f32x4* p = reinterpret_cast<f32x4*>(static_cast<float*>(d.out) + at);
      p[0] = f32x4{o[0], o[1], o[2], o[3]};
      p[1] = f32x4{o[4], o[5], o[6], o[7]};
    } else {
      u32x4 w;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        w[e] = d.out_dtype == F16 ? pack16<true>(o[2 * e], o[2 * e + 1]) : pack16<false>(o[2 * e], o[2 * e + 1]);
      *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(d.out) + at) = w;
    }
  }

  __device__ __forceinline__ void run(int64_t t0, uint32_t first) {
    load(t0);
    Shared<N, OUT> s[2];
    const char* bp = reinterpret_cast<const char*>(d.B) + t0 * d.b_ld * 2;
    const char* cp = reinterpret_cast<const char*>(d.C) + t0 * d.c_ld * 2;
    if constexpr (kPrefetch) load_shared(bp, cp, 0, s[0]);
    for (int64_t t = t0; t < t1; t += kBlock) {
      put_deltas();
      __builtin_amdgcn_wave_barrier();
      const u32x4 xc = x, zc = z;
      load(t + kBlock);
      if (t + kBlock <= t1) {
#pragma unroll
        for (int u = 0; u < kBlock; ++u) {
          if constexpr (kPrefetch) {
            arrived(s[u & 1]);
            load_shared(bp, cp, u + 1 < kBlock || t + kBlock < t1 ? u + 1 : u, s[(u + 1) & 1]);
            __builtin_amdgcn_sched_barrier(0);
          } else {
            load_shared(bp, cp, u, s[u & 1]);
          }
          token(u, s[u & 1]);
        }
      } else {  // a sequence's last few
        const int left = (int)(t1 - t);
#pragma clang loop unroll(disable)
        for (int u = 0; u < left; ++u) {
          load_shared(bp, cp, u, s[0]);
          token(u, s[0]);
        }
      }
      bp += kBlock * d.b_ld * 2;
      cp += kBlock * d.c_ld * 2;
      __builtin_amdgcn_wave_barrier();
      if constexpr (OUT) put_rows(t, first, xc, zc);
    }
  }
};

__device__ __forceinline__ int64_t slot_of(const q1_scan& d, int64_t seq) {
  const int64_t slot = d.slot_ids ? d.slot_ids[seq] : seq;
  return slot >= 0 && slot < d.slots ? slot : -1;
}

template <bool F16, bool DT32, int N, bool OUT>
__global__ __launch_bounds__(64) void q1_scan_kernel(const PromptArgs a) {
  const q1_scan& d = a.d;
  const int64_t piece = blockIdx.x / a.blocks, c0 = (blockIdx.x - piece * a.blocks) * 64 + threadIdx.x;
  const Piece p = scalar(find_piece_wave(a.r, piece, a.by, a.per));
  if (p.t0 >= p.t1) return;
  if (!OUT && p.last()) return;
  const bool live = c0 < d.Di;
  const int64_t ch = live ? c0 : d.Di - 1, slot = scalar(slot_of(d, p.seq));
  if (slot < 0) {
    if (OUT && live)
      for (int64_t t = p.t0; t < p.t1; ++t) store_out(d.out, d.out_dtype, t * d.Di + ch, 0.f);
    return;
  }
  __shared__ BlockLds m;
  const uint32_t first = (uint32_t)(blockIdx.x - piece * a.blocks) * 64;
  Walk<F16, DT32, N, OUT> w(d, m, p.t1, first);
  if constexpr (!OUT) {
#pragma unroll
    for (int n = 0; n < N; ++n) w.h[n] = 0.f;
  } else if (p.first()) {
    w.take(d.state + (slot * d.Di + ch) * N, w.h);
  } else {
#pragma unroll
    for (int n = 0; n < N; ++n) w.h[n] = a.h[((piece - 1) * N + n) * d.Di + ch];
  }
  w.run(p.t0, first);
  if (!live) return;
  if constexpr (!OUT) {
#pragma unroll
    for (int n = 0; n < N; ++n) a.h[(piece * N + n) * d.Di + ch] = w.h[n];
    a.sum[piece * d.Di + ch] = w.sum;
  } else if (p.last()) {
#pragma unroll
    for (int n = 0; n < N / 4; ++n)
      reinterpret_cast<f32x4*>(d.state + (slot * d.Di + ch) * N)[n] = f32x4{w.h[4 * n], w.h[4 * n + 1], w.h[4 * n + 2], w.h[4 * n + 3]};
  }
}

// A lane has one state of one channel of a sequence: from the ends of its pieces to
// their first states, in place.
__global__ __launch_bounds__(kThreads) void q1_scan_join(const PromptArgs a) {
  constexpr int U = 16;  // pieces in flight
  const q1_scan& d = a.d;
  const uint32_t i = blockIdx.x * kThreads + threadIdx.x, per = (uint32_t)(d.Di * d.N);
  const int64_t seq = divide(i, a.per_seq);
  if (seq >= a.r.nseq) return;
  const uint32_t w = i - (uint32_t)seq * per, n = divide(w, a.channels), ch = w - n * (uint32_t)d.Di;
  const int64_t slot = slot_of(d, seq);
  const uint32_t begin = cu_at(a.r, seq), end = cu_at(a.r, seq + 1);
  if (slot < 0 || end <= begin) return;
  const int64_t more = divide(end - begin - 1, a.by), first = divide(begin, a.by) + seq;  // pieces but the last one
  if (more == 0) return;
  const float A = d.A[(int64_t)ch * d.N + n] * kLog2e;
  float h = d.state[(slot * d.Di + ch) * d.N + n];
  float* hp = a.h + (first * d.N + n) * d.Di + ch;
  const float* sp = a.sum + first * d.Di + ch;
  for (int64_t j = 0; j < more; j += U) {
    float e[U], s[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t at = j + u < more ? j + u : more - 1;
      e[u] = hp[at * d.N * d.Di];
      s[u] = sp[at * d.Di];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      h = __builtin_fmaf(__builtin_amdgcn_exp2f(A * s[u]), h, e[u]);
      if (j + u < more) hp[(j + u) * d.N * d.Di] = h;
    }
  }
}

template <bool F16, bool DT32, int N>
hipError_t launch_prompt(const PromptArgs& a, int64_t pieces, hipStream_t s) {
  const dim3 grid((unsigned)(pieces * a.blocks));
  if (a.h != nullptr) {
    hipLaunchKernelGGL((q1_scan_kernel<F16, DT32, N, false>), grid, dim3(64), 0, s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t n = a.r.nseq * a.d.Di * N;
    hipLaunchKernelGGL(q1_scan_join, dim3((unsigned)((n + kThreads - 1) / kThreads)), dim3(kThreads), 0, s, a);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((q1_scan_kernel<F16, DT32, N, true>), grid, dim3(64), 0, s, a);
  return hipGetLastError();
}

template <bool F16, bool DT32>
hipError_t launch_n(const PromptArgs& a, int64_t pieces, hipStream_t s) {
  return a.d.N == 8    ? launch_prompt<F16, DT32, 8>(a, pieces, s)
         : a.d.N == 16 ? launch_prompt<F16, DT32, 16>(a, pieces, s)
         : a.d.N == 32 ? launch_prompt<F16, DT32, 32>(a, pieces, s)
                       : launch_prompt<F16, DT32, 64>(a, pieces, s);
}

size_t sums_at(const q1_scan& d, int64_t pieces) { return ((size_t)pieces * d.N * d.Di * 4 + 255) / 256 * 256; }

}  // namespace

// About three pieces for each wave that the chip holds at a time (four a SIMD), as they
// differ in length and the first to end make room; at least 24 tokens, or 16 where those
// would not be a wave a SIMD.  5120 channels of 16 states, us: 16384 tokens in pieces
// of 112 570, of 328 (one for each wave) 630, of 32 621, whole 8985; 4099 tokens of 7 sequences
// by 32 190, by 96 214, by 16 232; 8000 of 32 by 48 305, whole 618; 600 of one by 24 48, by 64 66;
// 77 of one by 16 24, by 24 29, whole 37.
int64_t scan_chunk(const q1_scan& d, int64_t tokens, int64_t nseq) {
  const int64_t blocks = (d.Di + 63) / 64, simds = (int64_t)device_cus() * 4;
  int64_t per = (tokens * blocks / (12 * simds) + kBlock - 1) / kBlock * kBlock;
  if (per < 24) per = tokens * blocks < 24 * simds ? 16 : 24;
  return tokens <= per ? 0 : per;  // (no sequence has a second piece)
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
  a.by = divider((uint32_t)a.per);
  a.blocks = (d.Di + 63) / 64;
  a.per_seq = divider((uint32_t)(d.Di * d.N));
  a.channels = divider((uint32_t)d.Di);
  if (per != 0) {
    a.h = reinterpret_cast<float*>(ws);
    a.sum = reinterpret_cast<float*>(ws + sums_at(d, pieces));
  }
  if (d.dt_dtype == F32) return d.dtype == Q1_F16 ? launch_n<true, true>(a, pieces, s) : launch_n<false, true>(a, pieces, s);
  return d.dtype == Q1_F16 ? launch_n<true, false>(a, pieces, s) : launch_n<false, false>(a, pieces, s);
}

}  // namespace q1
