// Device functions shared by the kernels of q1_memory.h: pieces of a ragged batch,
// division, elements of 16 bits, the activation.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "q1_device.h"
#include "q1_memory.h"

namespace q1 {

// x / d for x below 2^31.
__device__ __forceinline__ uint32_t divide(uint32_t x, Divider d) { return (uint32_t)(((uint64_t)x * d.mul) >> d.shift); }

// The low or high element of a pair.
template <bool F16>
__device__ __forceinline__ float elem16(uint32_t w, int hi) {
  if constexpr (F16) return f16_bits_to_f32(hi ? w >> 16 : w & 0xffffu);
  else return __uint_as_float(hi ? w & 0xffff0000u : w << 16);
}

// Piece number `piece` of at most `per` tokens: rows [t0, t1) of sequence `seq`, whose
// own rows are [begin, end); nothing (t0 >= t1) where the batch has no such piece.
struct Piece {
  int64_t seq, begin, end, t0, t1;
  __device__ __forceinline__ bool first() const { return t0 == begin; }
  __device__ __forceinline__ bool last() const { return t1 == end; }
};

__device__ __forceinline__ int64_t cu_at(const Ragged& r, int64_t s) {
  const int64_t v = r.cu[s];
  return v < 0 ? 0 : v > r.tokens ? r.tokens : v;
}

__device__ __forceinline__ Piece find_piece(const Ragged& r, int64_t piece, int64_t per) {
  int64_t lo = 0, hi = r.nseq - 1;  // the last sequence whose first piece is not behind this one
  while (lo < hi) {
    const int64_t mid = (lo + hi + 1) >> 1;
    if (cu_at(r, mid) / per + mid <= piece) lo = mid;
    else hi = mid - 1;
  }
  Piece p;
  p.seq = lo;
  p.begin = cu_at(r, lo);
  p.end = cu_at(r, lo + 1);
  const int64_t j = piece - (p.begin / per + lo);
  p.t0 = p.begin + j * per;
  p.t1 = p.t0 + per < p.end ? p.t0 + per : p.end;
  if (j < 0) p.t1 = p.t0;  // rows before the first sequence
  return p;
}

// s / (1 + exp(-s)), off by a few units in the last place (and |s| more of them in the
// exponential, where it is large the other term is not).
__device__ __forceinline__ float silu_fast(float s) {
  return s * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(s * -1.44269504088896340736f));
}

}  // namespace q1
