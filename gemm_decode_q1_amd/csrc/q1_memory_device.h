// Device functions shared by the kernels of q1_memory.h: pieces of a ragged batch,
// division, elements of 16 bits, the activation.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "q1_device.h"
#include "q1_memory.h"

namespace q1 {

// x / d for x below 2^31.
__device__ __forceinline__ uint32_t divide(uint32_t x, Divider d) { return __umulhi(x << 1, d.mul) >> d.shift; }

// The low or high element of a pair.
template <bool F16>
__device__ __forceinline__ float elem16(uint32_t w, int hi) {
  if constexpr (F16) return f16_bits_to_f32(hi ? w >> 16 : w & 0xffffu);
  else return __uint_as_float(hi ? w & 0xffff0000u : w << 16);
}

// Two values rounded to a pair.
template <bool F16>
__device__ __forceinline__ uint32_t pack16(float x, float y) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  if constexpr (F16) return f32_to_f16_bits(x) | f32_to_f16_bits(y) << 16;
  else return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{x, y}, bf16x2));
}

// Piece number `piece` of at most `per` tokens: rows [t0, t1) of sequence `seq`, whose
// own rows are [begin, end); nothing (t0 >= t1) where the batch has no such piece.
struct Piece {
  int64_t seq, begin, end, t0, t1;
  __device__ __forceinline__ bool first() const { return t0 == begin; }
  __device__ __forceinline__ bool last() const { return t1 == end; }
};

__device__ __forceinline__ uint32_t cu_at(const Ragged& r, int64_t s) {
  const int32_t v = r.cu[s];
  return v < 0 ? 0u : v > r.tokens ? (uint32_t)r.tokens : (uint32_t)v;
}

// Sequence `seq`'s piece of the given number.
__device__ __forceinline__ Piece piece_of(const Ragged& r, int64_t piece, Divider by, int64_t per, int64_t seq) {
  Piece p;
  p.seq = seq;
  p.begin = cu_at(r, seq);
  p.end = cu_at(r, seq + 1);
  const int64_t j = piece - (divide((uint32_t)p.begin, by) + seq);
  p.t0 = p.begin + j * per;
  p.t1 = p.t0 + per < p.end ? p.t0 + per : p.end;
  if (j < 0) p.t1 = p.t0;  // rows before the first sequence
  return p;
}

// The last sequence whose first piece is not behind this one, by halving (by = `per`).
__device__ __forceinline__ Piece find_piece(const Ragged& r, int64_t piece, Divider by, int64_t per) {
  int64_t lo = 0, hi = r.nseq - 1;
  while (lo < hi) {
    const int64_t mid = (lo + hi + 1) >> 1;
    if (divide(cu_at(r, mid), by) + mid <= piece) lo = mid;
    else hi = mid - 1;
  }
  return piece_of(r, piece, by, per, lo);
}

// The same for a whole wave, which looks at 64 places at a time.
__device__ __forceinline__ Piece find_piece_wave(const Ragged& r, int64_t piece, Divider by, int64_t per) {
  int64_t lo = 0, n = r.nseq;  // among [lo, lo + n)
  while (n > 1) {
    const int64_t step = (n + 63) / 64, at = (int64_t)(threadIdx.x & 63) * step;
    const uint64_t hit = __ballot(at < n && (at == 0 || divide(cu_at(r, lo + at), by) + (lo + at) <= piece));
    const int64_t k = (63 - __builtin_clzll(hit)) * step;  // (lane 0 always hits)
    lo += k;
    n = n - k < step ? n - k : step;
  }
  return piece_of(r, piece, by, per, lo);
}

// The same piece in scalar registers, for a wave that walks over it as a whole.
__device__ __forceinline__ int64_t scalar(int64_t v) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v), hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
  return (int64_t)((uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ Piece scalar(const Piece& p) {
  return {scalar(p.seq), scalar(p.begin), scalar(p.end), scalar(p.t0), scalar(p.t1)};
}

// s / (1 + exp(-s)), off by a few units in the last place (and |s| more of them in the
// exponential, where it is large the other term is not).
__device__ __forceinline__ float silu_fast(float s) {
  return s * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(s * -1.44269504088896340736f));
}

}  // namespace q1
