// Selective state space scan (q1_memory.h), single tokens and prompts.
//
// Single tokens: four lanes have a channel, a quarter of its states each, so that a
// state is read and written in whole lines and one sequence fills some hundred waves.  One
// token of 5120 channels of 16 states takes 3.4 us in a graph, a launch's length.
//
// Prompts: the same, four waves for 64 channels.  A prompt is cut into pieces so that the
// waves fill the chip, in three launches:
//   q1_scan_kernel<.., false>  a sequence's first piece with its outputs; for the others the
//                              state at the end from a zero state, and the sum of the deltas
//                              (the decay over the piece is exp(A * sum));
//   q1_scan_join               the state before each piece, one after the other;
//   q1_scan_kernel<.., true>   the other outputs, and from a last piece the final state.
// A sequence's last piece needs no first walk, so short sequences have none.  (First pieces
// in the second launch, walked twice: 8000 tokens of 32 sequences 271 | 248 us, 4099 of 7 189 | 178,
// one long sequence the same.)
//
// Bound by the vector units (busy throughout): a state costs a product, an exponential (8
// cycles a wave, the others 4), a product and two multiply-adds a token, and without outputs
// one less, so that one walk over 16384 tokens of 5120 channels of 16 states cannot take less
// than 235 us at 2.15 GHz, both 430; with deltas, skip and gate 544 to 593 are measured.  Reading and
// writing rows would take 136.  A lane with all states of a channel, B and C in scalar
// registers, needs a tenth fewer instructions but four times the pieces: 602 us, 4099 tokens of 7
// sequences 206 | 164, 16000 of 60 (whole) 572 | 408, 77 of one 24 | 16.
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

// The sum of four neighbouring lanes' values.
__device__ __forceinline__ float sum_quad(float v) {
  v += __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), 0xb1, 0xf, 0xf, true));
  v += __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), 0x4e, 0xf, 0xf, true));
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

// Eight outputs of a row.
__device__ __forceinline__ void store_row(const q1_scan& d, int64_t at, const float* o) {
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

__device__ __forceinline__ int64_t slot_of(const q1_scan& d, int64_t seq) {
  const int64_t slot = d.slot_ids ? d.slot_ids[seq] : seq;
  return slot >= 0 && slot < d.slots ? slot : -1;
}

// A workgroup's walk over the rows [t0, t1) of a piece, 64 channels from `first` on.  Rows come
// in and go out by blocks of 32 tokens in which a lane has 8 channels of one token (16
// bytes): so it makes the deltas and applies skip and gate.  Between these, through LDS, four
// lanes have a channel, a quarter of its states each, token by token; B and C come from LDS
// as fp32.  (Without the places of `pair` and `four` the LDS, busy for 81 % of the time with a third
// of that conflicts, was the bound: 16384 tokens 613 us, with them 544.)
constexpr int kBlock = 32;

template <int N>
struct BlockLds {
  alignas(16) float2 dd[kBlock][64];  // delta, and delta times x, of the channel at pair(c)
  alignas(16) float y[kBlock][64];    // of the channel at four(c)
  alignas(16) float bc[kBlock][2 * N];
  // Places of a row's channels: eight lanes that write or read 8 channels each, 16 bytes at a
  // time, meet all banks.
  static __device__ __forceinline__ int pair(int c) { return c ^ (c >> 3 & 6); }
  static __device__ __forceinline__ int four(int c) { return c ^ (c >> 3 & 4); }
};

template <bool F16, bool DT32, int N, bool OUT>
struct Walk {
  static constexpr int M = N / 4;  // states of a lane
  const q1_scan& d;
  BlockLds<N>& m;
  const int64_t t1;
  const int row, part;    // this thread's token of a block, and eighth of it
  const int c, quad;      // this lane's channel of the 64, and quarter of its states
  const uint32_t first, c8;
  float h[M], A[M], bias[8], skip[OUT ? 8 : 1], sum = 0.f;
  u32x4 x, z, dt[DT32 ? 2 : 1];
  uint16_t b[N / 8], cc[OUT ? N / 8 : 1];

  __device__ __forceinline__ Walk(const q1_scan& d, BlockLds<N>& m, int64_t t1, uint32_t first)
      : d(d), m(m), t1(t1), row(threadIdx.x >> 3), part(threadIdx.x & 7), c(threadIdx.x >> 2), quad(threadIdx.x & 3), first(first),
        c8(first + 8 * part < (uint32_t)d.Di ? first + 8 * part : (uint32_t)d.Di - 8) {
    const uint32_t ch = channel();
#pragma unroll
    for (int n = 0; n < M; ++n) A[n] = d.A[(int64_t)ch * N + quad * M + n] * kLog2e;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      bias[e] = d.dt_bias ? d.dt_bias[c8 + e] : 0.f;
      if constexpr (OUT) skip[e] = d.D ? d.D[c8 + e] : 0.f;
    }
  }
  __device__ __forceinline__ bool live() const { return first + c < (uint32_t)d.Di; }
  __device__ __forceinline__ uint32_t channel() const { return live() ? first + c : (uint32_t)d.Di - 1; }

  template <typename T, int K>
  static __device__ __forceinline__ void take(const void* from, T (&to)[K]) {
    __builtin_memcpy(to, __builtin_assume_aligned(from, sizeof(T) * K), sizeof(T) * K);
  }

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
    take(static_cast<const uint16_t*>(d.B) + at * d.b_ld + part * (N / 8), b);
    if constexpr (OUT) {
      take(static_cast<const uint16_t*>(d.C) + at * d.c_ld + part * (N / 8), cc);
      z = u32x4{0u, 0u, 0u, 0u};
      if (d.z != nullptr) z = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(d.z) + at * d.z_ld + c8);
    }
  }

  __device__ __forceinline__ void put_deltas() {
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      f32x4 w;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float s = (DT32 ? __uint_as_float(dt[DT32 ? e >> 2 : 0][(e + j) & 3]) : elem16<F16>(dt[0][e >> 1], j)) + bias[e + j];
        const float soft = softplus(s);
        w[2 * j] = d.softplus ? soft : s;
        w[2 * j + 1] = w[2 * j] * elem16<F16>(x[e >> 1], j);
      }
      *reinterpret_cast<f32x4*>(&m.dd[row][m.pair(8 * part + e)]) = w;
    }
#pragma unroll
    for (int n = 0; n < N / 8; ++n) {
      m.bc[row][part * (N / 8) + n] = elem<F16>(b[n]);
      if constexpr (OUT) m.bc[row][N + part * (N / 8) + n] = elem<F16>(cc[n]);
    }
  }

  // Token u of the block: its states, and this lane's part of the output.
  __device__ __forceinline__ float token(int u) {
    const float2 w = m.dd[u][m.pair(c)];
    if constexpr (!OUT) sum += w.x;
    float y = 0.f;
#pragma unroll
    for (int n = 0; n < M; ++n) {
      h[n] = __builtin_fmaf(__builtin_amdgcn_exp2f(w.x * A[n]), h[n], w.y * m.bc[u][quad * M + n]);
      if constexpr (OUT) y = __builtin_fmaf(m.bc[u][N + quad * M + n], h[n], y);
    }
    return y;
  }

  static __device__ __forceinline__ float from1(float v) {  // of the lane whose number differs in bit 0
    return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), 0xb1, 0xf, 0xf, true));
  }
  static __device__ __forceinline__ float from2(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), 0x4e, 0xf, 0xf, true));
  }

  __device__ __forceinline__ void put_rows(int64_t t, u32x4 x, u32x4 z) const {
    float o[8];
    const f32x4 lo = *reinterpret_cast<const f32x4*>(&m.y[row][m.four(8 * part)]);
    const f32x4 hi = *reinterpret_cast<const f32x4*>(&m.y[row][m.four(8 * part + 4)]);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      o[e] = __builtin_fmaf(skip[e], elem16<F16>(x[e >> 1], e & 1), e < 4 ? lo[e & 3] : hi[e & 3]);
      const float gate = silu_fast(elem16<F16>(z[e >> 1], e & 1));
      o[e] = d.z != nullptr ? o[e] * gate : o[e];
    }
    if (t + row < t1 && first + 8 * part < d.Di) store_row(d, (t + row) * d.Di + c8, o);
  }

  __device__ __forceinline__ void run(int64_t t0) {
    load(t0);
    for (int64_t t = t0; t < t1; t += kBlock) {
      put_deltas();
      __syncthreads();
      const u32x4 xc = x, zc = z;
      load(t + kBlock);
      const int left = (int)(t1 - t < kBlock ? t1 - t : kBlock);
      int u = 0;
#pragma clang loop unroll_count(2)
      for (; u + 4 <= left; u += 4) {  // the sums of four tokens, one to each of a channel's lanes
        float y[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = token(u + j);
        if constexpr (OUT) {
          const bool odd = quad & 1, high = quad & 2;
          const float r0 = (odd ? y[1] : y[0]) + from1(odd ? y[0] : y[1]), r1 = (odd ? y[3] : y[2]) + from1(odd ? y[2] : y[3]);
          m.y[u + quad][m.four(c)] = (high ? r1 : r0) + from2(high ? r0 : r1);
        }
      }
      for (; u < left; ++u) {
        const float y = token(u);
        if constexpr (OUT) m.y[u][m.four(c)] = sum_quad(y);  // (the four write one value)
      }
      __syncthreads();
      if constexpr (OUT) put_rows(t, xc, zc);
    }
  }
};

// A piece, from the state before it (or, without outputs, from zeros).
template <bool F16, bool DT32, int N, bool OUT>
__device__ __forceinline__ void walk_piece(const PromptArgs& a, const Piece& p, int64_t piece, int64_t slot, uint32_t first, BlockLds<N>& m) {
  constexpr int M = N / 4;
  const q1_scan& d = a.d;
  Walk<F16, DT32, N, OUT> w(d, m, p.t1, first);
  const int64_t ch = w.channel();
  float* const st = d.state + (slot * d.Di + ch) * N + w.quad * M;
  float* const at = a.h + (piece * N + w.quad * M) * d.Di + ch;
#pragma unroll
  for (int n = 0; n < M; ++n) w.h[n] = !OUT ? 0.f : p.first() ? st[n] : at[(n - N) * d.Di];
  w.run(p.t0);
  if (!w.live()) return;
  if (OUT && p.last()) {
#pragma unroll
    for (int n = 0; n < M; ++n) st[n] = w.h[n];
  } else if (!OUT || p.first()) {
#pragma unroll
    for (int n = 0; n < M; ++n) at[n * d.Di] = w.h[n];
    if (!OUT && w.quad == 0) a.sum[piece * d.Di + ch] = w.sum;
  }
}

// LAST: the second walk.  The first piece of a sequence of several needs no state of another: the
// first walk makes its outputs.
template <bool F16, bool DT32, int N, bool LAST>
__global__ __launch_bounds__(kThreads) void q1_scan_kernel(const PromptArgs a) {
  const q1_scan& d = a.d;
  const int64_t piece = blockIdx.x / a.blocks;
  const uint32_t first = (uint32_t)(blockIdx.x - piece * a.blocks) * 64;
  const Piece p = scalar(find_piece_wave(a.r, piece, a.by, a.per));
  if (p.t0 >= p.t1) return;
  if (LAST ? p.first() && !p.last() : p.last()) return;
  const int64_t slot = scalar(slot_of(d, p.seq));
  if (slot < 0) {
    const uint32_t ch = first + (threadIdx.x & 63);
    if ((LAST || p.first()) && ch < d.Di)
      for (int64_t t = p.t0 + (threadIdx.x >> 6); t < p.t1; t += kThreads / 64) store_out(d.out, d.out_dtype, t * d.Di + ch, 0.f);
    return;
  }
  __shared__ BlockLds<N> m;
  if (LAST || p.first()) walk_piece<F16, DT32, N, true>(a, p, piece, slot, first, m);
  else walk_piece<F16, DT32, N, false>(a, p, piece, slot, first, m);
}

// A lane has one state of one channel of a sequence: from the ends of its pieces (the first
// one's as it is, the others' from a zero state) to the states before the next ones, in place.
__global__ __launch_bounds__(kThreads) void q1_scan_join(const PromptArgs a) {
  constexpr int U = 16;  // pieces in flight
  const q1_scan& d = a.d;
  const uint32_t i = blockIdx.x * kThreads + threadIdx.x, per = (uint32_t)(d.Di * d.N);
  const int64_t seq = divide(i, a.per_seq);
  if (seq >= a.r.nseq) return;
  const uint32_t w = i - (uint32_t)seq * per, n = divide(w, a.channels), ch = w - n * (uint32_t)d.Di;
  const uint32_t begin = cu_at(a.r, seq), end = cu_at(a.r, seq + 1);
  if (end <= begin || slot_of(d, seq) < 0) return;
  const int64_t more = divide(end - begin - 1, a.by), first = divide(begin, a.by) + seq;  // pieces but the last one
  if (more < 2) return;
  const float A = d.A[(int64_t)ch * d.N + n] * kLog2e;
  float* hp = a.h + (first * d.N + n) * d.Di + ch;
  const float* sp = a.sum + first * d.Di + ch;
  float h = hp[0];
  for (int64_t j = 1; j < more; j += U) {
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
    hipLaunchKernelGGL((q1_scan_kernel<F16, DT32, N, false>), grid, dim3(kThreads), 0, s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t n = a.r.nseq * a.d.Di * N;
    hipLaunchKernelGGL(q1_scan_join, dim3((unsigned)((n + kThreads - 1) / kThreads)), dim3(kThreads), 0, s, a);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((q1_scan_kernel<F16, DT32, N, true>), grid, dim3(kThreads), 0, s, a);
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

// Tokens of a piece, so that there are about seven workgroups a compute unit, but 64 to 256, and 32
// for little work.  Where the sequences alone are 16 workgroups a unit, an eighth of all tokens, up to
// 512: few of them have a second piece, but one that has nearly all tokens is still cut.  5120 channels
// of 16 states, us: 16384 tokens by 128 566, by 256 558, by 512 570, whole 2374; 4099 of 7 sequences by 64
// 167, 128 156, 192 162, 256 160, 512 225; 8000 of 32 by 128 251, 256 239, 512 282, whole 260; 600 of one by
// 32 45, 64 44, 128 50; 300 by 32 30, 64 32; 77 by 32 20, whole 16.  Sequences that fill the chip: 16000 of 60
// by 256 426, 512 408, whole 408; 60 of 267 by 256 374, 512 351, whole 344; 60 of 8 and one of 8000 by 256
// 336, 512 376, 1060 478, whole 1229; of 512 channels 600 of 27 by 64 94, 256 89, 512 87, whole 71, and 511
// of one token and one of 16384 by 64 138, 256 144, 512 201, 2112 638, whole 2399.
int64_t scan_chunk(const q1_scan& d, int64_t tokens, int64_t nseq) {
  const int64_t blocks = (d.Di + 63) / 64, cus = device_cus(), work = tokens * blocks;
  int64_t per = (work / (7 * cus) + kBlock / 2) / kBlock * kBlock;
  if (per > 256) per = 256;
  if (per < 64) per = work < 96 * cus ? 32 : 64;
  if (nseq * blocks >= 16 * cus && per < tokens / 8) {
    per = (tokens / 8 + kBlock - 1) / kBlock * kBlock;
    if (per > 512) per = 512;
  }
  return tokens <= (per > 96 ? per : 96) ? 0 : per;  // (no sequence has a second piece)
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
