// Short causal convolution with the activation behind it (q1_memory.h): prompts and
// single tokens with one kernel, so that both give the same bits.
//
// A lane has 8 channels (16 bytes of a row) of a piece of a sequence and slides over
// its tokens with the last W-1 rows in registers: a row is read once, but for the W-1
// before a piece.  The piece that starts a sequence reads the state and, since inputs
// are only read, writes the new one too: no other piece touches it.
//
// Bound by bytes: 16384 tokens of 10240 channels (672 MB) take 127 us, 5.3 TB/s, as a copy
// does.  Pieces of 16 tokens: by 4 184 us, by 8 133, by 32 134, by 64 145; 200 tokens of one
// sequence by 8 7.6, by 16 7.6, by 32 11.4, by 64 19.6.  8 single tokens: 3.5 in a graph, a launch.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "q1_internal.h"
#include "q1_kv_device.h"
#include "q1_memory.h"
#include "q1_memory_device.h"

namespace q1 {
namespace {

typedef kv_u32x4 u32x4;

constexpr int kThreads = 256;

struct ConvArgs {
  q1_conv d;
  Ragged r;          // r.cu == nullptr: T rows a sequence
  int64_t per;       // tokens of a piece
  Divider by;
  uint32_t n;        // lanes in all: pieces * C / 8
  uint32_t lanes;    // C / 8
  Divider per_row;   // by C / 8
};

template <bool F16, int W>
__global__ __launch_bounds__(kThreads) void q1_conv_kernel(const ConvArgs a) {
  constexpr int U = 4;  // rows in flight
  const q1_conv& d = a.d;
  const uint32_t i = blockIdx.x * kThreads + threadIdx.x;
  if (i >= a.n) return;
  const uint32_t piece = divide(i, a.per_row), c0 = (i - piece * a.lanes) * 8;
  Piece p;
  if (a.r.cu != nullptr) {
    p = find_piece(a.r, piece, a.by, a.per);
    if (p.t0 >= p.t1) return;
  } else {
    p.seq = piece;
    p.begin = p.t0 = (int64_t)piece * a.per;
    p.end = p.t1 = p.begin + a.per;
  }
  const int64_t slot = d.slot_ids ? d.slot_ids[p.seq] : p.seq;
  uint16_t* out = static_cast<uint16_t*>(d.out) + c0;
  if (slot < 0 || slot >= d.slots) {
    for (int64_t t = p.t0; t < p.t1; ++t) *reinterpret_cast<u32x4*>(out + t * d.C) = u32x4{0u, 0u, 0u, 0u};
    return;
  }
  const uint16_t* x = static_cast<const uint16_t*>(d.x) + c0;
  uint16_t* state = static_cast<uint16_t*>(d.state) + slot * (W - 1) * d.C + c0;

  u32x4 win[W - 1];  // rows t0 - (W-1) .. t0 - 1
  if (p.first()) {
#pragma unroll
    for (int j = 0; j < W - 1; ++j) win[j] = *reinterpret_cast<const u32x4*>(state + j * d.C);
    const int64_t len = p.end - p.begin;
    u32x4 keep[W - 1];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      const int64_t pos = len - (W - 1) + j;
      if (pos >= 0) {
        keep[j] = *reinterpret_cast<const u32x4*>(x + (p.begin + pos) * d.x_ld);
      } else {
        keep[j] = win[W - 2];
#pragma unroll
        for (int o = 0; o < W - 1; ++o)
          if (pos + W - 1 == o) keep[j] = win[o];
      }
    }
#pragma unroll
    for (int j = 0; j < W - 1; ++j) *reinterpret_cast<u32x4*>(state + j * d.C) = keep[j];
  } else {
#pragma unroll
    for (int j = 0; j < W - 1; ++j) win[j] = *reinterpret_cast<const u32x4*>(x + (p.t0 - (W - 1) + j) * d.x_ld);
  }

  float w[W][8], bias[8];
  {
    u32x4 raw[W];
#pragma unroll
    for (int j = 0; j < W; ++j)
      raw[j] = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(d.weight) + (int64_t)c0 * W + 8 * j);
#pragma unroll
    for (int c = 0; c < 8; ++c)
#pragma unroll
      for (int j = 0; j < W; ++j) w[j][c] = elem16<F16>(raw[(c * W + j) >> 3][((c * W + j) >> 1) & 3], (c * W + j) & 1);
    u32x4 b = {0u, 0u, 0u, 0u};
    if (d.bias != nullptr) b = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(d.bias) + c0);
#pragma unroll
    for (int c = 0; c < 8; ++c) bias[c] = elem16<F16>(b[c >> 1], c & 1);
  }

  const int64_t last = p.t1 - 1;
  u32x4 row[U], next[U];
#pragma unroll
  for (int u = 0; u < U; ++u) row[u] = *reinterpret_cast<const u32x4*>(x + (p.t0 + u < last ? p.t0 + u : last) * d.x_ld);
  for (int64_t t = p.t0; t < p.t1; t += U) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t tn = t + U + u;
      next[u] = *reinterpret_cast<const u32x4*>(x + (tn < last ? tn : last) * d.x_ld);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      u32x4 o;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float s[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int c = 2 * e + h;
          float acc = bias[c];
#pragma unroll
          for (int j = 0; j < W - 1; ++j) acc = __builtin_fmaf(w[j][c], elem16<F16>(win[j][e], h), acc);
          acc = __builtin_fmaf(w[W - 1][c], elem16<F16>(row[u][e], h), acc);
          s[h] = d.silu ? silu_fast(acc) : acc;
        }
        o[e] = pack16<F16>(s[0], s[1]);
      }
      if (t + u < p.t1) *reinterpret_cast<u32x4*>(out + (t + u) * d.C) = o;
#pragma unroll
      for (int j = 0; j + 1 < W - 1; ++j) win[j] = win[j + 1];
      win[W - 2] = row[u];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) row[u] = next[u];
  }
}

hipError_t launch(ConvArgs a, int64_t pieces, hipStream_t s) {
  a.lanes = (uint32_t)(a.d.C / 8);
  a.per_row = divider(a.lanes);
  a.by = divider((uint32_t)a.per);
  a.n = (uint32_t)(pieces * a.lanes);
  const dim3 grid((a.n + kThreads - 1) / kThreads), block(kThreads);
#define Q1_CV(H, N) hipLaunchKernelGGL((q1_conv_kernel<H, N>), grid, block, 0, s, a)
  if (a.d.dtype == Q1_F16) {
    if (a.d.W == 4) Q1_CV(true, 4);
    else if (a.d.W == 3) Q1_CV(true, 3);
    else Q1_CV(true, 2);
  } else {
    if (a.d.W == 4) Q1_CV(false, 4);
    else if (a.d.W == 3) Q1_CV(false, 3);
    else Q1_CV(false, 2);
  }
#undef Q1_CV
  return hipGetLastError();
}

}  // namespace

int64_t conv_pieces(const q1_conv&, int64_t tokens, int64_t nseq) { return ragged_pieces(tokens, nseq, kConvTokens); }

hipError_t launch_conv_step(const q1_conv& d, int64_t B, int64_t T, hipStream_t s) {
  ConvArgs a = {};
  a.d = d;
  a.per = T;
  return launch(a, B, s);
}

hipError_t launch_conv_prefill(const q1_conv& d, const Ragged& r, hipStream_t s) {
  ConvArgs a = {};
  a.d = d;
  a.r = r;
  a.per = kConvTokens;
  return launch(a, conv_pieces(d, r.tokens, r.nseq), s);
}

}  // namespace q1
