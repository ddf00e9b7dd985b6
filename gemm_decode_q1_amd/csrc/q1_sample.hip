// Sampler: temperature, top-k, top-p, min-p and one draw per row, from a given
// random number.  One workgroup per row.
//
// The kept set is a threshold (key, ties): every logit with a larger key, and
// the first `ties` logits, in index order, of those that equal it.  Both
// thresholds come from a radix select over order-preserving 32-bit keys, by
// count (top-k) and by weight (top-p).  Weights are whole multiples of 2^-40,
// so all sums are exact and do not depend on the order of the additions.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "q1_decode.h"
#include "q1_device.h"
#include "q1_internal.h"

namespace q1 {
namespace {

constexpr int kThreads = 1024;
typedef unsigned long long u64;

template <int DT>
__device__ __forceinline__ float logit(const void* p, int64_t i) {
  float x;
  if (DT == F32) x = static_cast<const float*>(p)[i];
  else if (DT == BF16) x = bf16_bits_to_f32(static_cast<const uint16_t*>(p)[i]);
  else x = f16_bits_to_f32(static_cast<const uint16_t*>(p)[i]);
  return x != x ? -INFINITY : x + 0.0f;  // -0 and +0 are equal logits
}

// Larger logits have larger keys.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t u = __float_as_uint(x);
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}

__device__ __forceinline__ float exp_of(float x, float top, float T) { return x == top ? 1.0f : expf((x - top) / T); }

__device__ __forceinline__ u64 weight_of(float e) { return (u64)(e * 1099511627776.0f); }

// Sum over the workgroup; every thread gets it.
__device__ u64 block_sum(u64 v, u64* s) {
  __syncthreads();
  s[threadIdx.x] = v;
  __syncthreads();
  for (int w = kThreads / 2; w > 0; w >>= 1) {
    if ((int)threadIdx.x < w) s[threadIdx.x] += s[threadIdx.x + w];
    __syncthreads();
  }
  const u64 r = s[0];
  __syncthreads();
  return r;
}

template <int DT>
__global__ __launch_bounds__(kThreads) void q1_sample_row_kernel(const SampleArgs a) {
  __shared__ u64 sw[kThreads], hist[256];
  __shared__ uint32_t pick;
  __shared__ u64 over;
  const int64_t b = blockIdx.x;
  const int tid = threadIdx.x;
  const void* row = static_cast<const unsigned char*>(a.logits) + b * a.ld * (DT == F32 ? 4 : 2);
  const int V = (int)a.V;
  float T = a.temperature ? a.temperature[b] : 1.0f;
  const bool greedy = !(T > 0.f);
  if (greedy) T = 1.f;
  const int64_t k = greedy ? 1 : a.top_k && a.top_k[b] > 0 ? a.top_k[b] : V;
  const float p = a.top_p ? a.top_p[b] : 1.f;
  float mp = a.min_p ? a.min_p[b] : 0.f;
  mp = mp > 0.f ? fminf(mp, 1.f) : 0.f;

  float top = -INFINITY;
  for (int i = tid; i < V; i += kThreads) top = fmaxf(top, logit<DT>(row, i));
  float* sf = reinterpret_cast<float*>(sw);
  sf[tid] = top;
  __syncthreads();
  for (int w = kThreads / 2; w > 0; w >>= 1) {
    if (tid < w) sf[tid] = fmaxf(sf[tid], sf[tid + w]);
    __syncthreads();
  }
  top = sf[0];
  __syncthreads();
  if (top == -INFINITY) {
    if (tid == 0) {
      if (a.tokens_int64) static_cast<int64_t*>(a.tokens)[b] = -1;
      else static_cast<int32_t*>(a.tokens)[b] = -1;
      if (a.logprob) a.logprob[b] = -INFINITY;
    }
    return;
  }

  // Radix select, largest key first: the key at which the running sum of
  // `amount` (1 or the weight, counting at most `kties` of the key kthr)
  // reaches `want`, and the sum over the larger keys.
  uint32_t kthr = 0u;
  u64 kties = ~0ull;
  auto select = [&](bool weighted, u64 want, uint32_t* key, u64* above) {
    uint32_t prefix = 0u;
    u64 before = 0;
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int i = tid; i < 256; i += kThreads) hist[i] = 0;
      __syncthreads();
      for (int i = tid; i < V; i += kThreads) {
        const float x = logit<DT>(row, i);
        const uint32_t key_i = key_of(x);
        if (shift < 24 && (key_i >> (shift + 8)) != (prefix >> (shift + 8))) continue;
        if (weighted && key_i <= kthr) continue;  // the threshold key is added once, below
        atomicAdd(&hist[(key_i >> shift) & 255], weighted ? weight_of(exp_of(x, top, T)) : 1ull);
      }
      if (weighted && tid == 0 && kties != ~0ull && (shift == 24 || (kthr >> (shift + 8)) == (prefix >> (shift + 8)))) {
        const uint32_t bits = kthr >> 31 ? kthr ^ 0x80000000u : ~kthr;
        atomicAdd(&hist[(kthr >> shift) & 255], kties * weight_of(exp_of(__uint_as_float(bits), top, T)));
      }
      __syncthreads();
      if (tid == 0) {
        u64 c = before;
        int d = 255;
        for (; d > 0; --d) {
          if (c + hist[d] >= want) break;
          c += hist[d];
        }
        pick = (uint32_t)d;
        over = c;
      }
      __syncthreads();
      prefix |= pick << shift;
      before = over;
      __syncthreads();
    }
    *key = prefix;
    *above = before;
  };

  uint32_t thr = 0u;
  u64 ties = ~0ull;
  if (k < V) {
    u64 above;
    select(false, (u64)k, &thr, &above);
    ties = (u64)k - above;
    kthr = thr;
    kties = ties;
  }
  if (p < 1.f) {
    u64 mine = 0;
    for (int i = tid; i < V; i += kThreads) {
      const float x = logit<DT>(row, i);
      if (kties == ~0ull || key_of(x) > kthr) mine += weight_of(exp_of(x, top, T));
    }
    u64 total = block_sum(mine, sw);
    if (kties != ~0ull) {
      const uint32_t bits = kthr >> 31 ? kthr ^ 0x80000000u : ~kthr;
      total += kties * weight_of(exp_of(__uint_as_float(bits), top, T));
    }
    const double want = (double)p * (double)total;
    const u64 bound = want >= 1.0 ? (u64)want : 1;
    uint32_t key;
    u64 above;
    select(true, bound, &key, &above);
    const uint32_t bits = key >> 31 ? key ^ 0x80000000u : ~key;
    const u64 w = weight_of(exp_of(__uint_as_float(bits), top, T));
    const u64 n = w > 0 ? (bound - above + w - 1) / w : 1;
    if (key > kthr || kties == ~0ull || n < kties) ties = n;
    thr = key;
  }

  // Each thread's contiguous piece of the row: ties in it, then kept weight.
  const int piece = (V + kThreads - 1) / kThreads;
  const int i0 = tid * piece < V ? tid * piece : V, i1 = i0 + piece < V ? i0 + piece : V;
  u64 same = 0;
  for (int i = i0; i < i1; ++i) same += key_of(logit<DT>(row, i)) == thr;
  sw[tid] = same;
  __syncthreads();
  u64 rank0 = 0;
  for (int j = 0; j < tid; ++j) rank0 += sw[j];
  __syncthreads();
  auto kept = [&](int i, u64* rank) -> u64 {
    const float x = logit<DT>(row, i);
    const uint32_t key_i = key_of(x);
    const float e = exp_of(x, top, T);
    if (key_i < thr || e < mp) return 0;
    if (key_i == thr && (*rank)++ >= ties) return 0;
    return weight_of(e);
  };
  u64 mine = 0, rank = rank0;
  for (int i = i0; i < i1; ++i) mine += kept(i, &rank);
  sw[tid] = mine;
  __syncthreads();
  u64 start = 0, total = 0;
  for (int j = 0; j < kThreads; ++j) {
    if (j < tid) start += sw[j];
    total += sw[j];
  }
  const float u = a.u[b];
  u64 r = u > 0.f ? (u64)((double)fminf(u, 1.f) * (double)total) : 0;
  if (r >= total) r = total - 1;
  if (r >= start && r < start + mine) {
    u64 c = start;
    rank = rank0;
    for (int i = i0; i < i1; ++i) {
      const u64 w = kept(i, &rank);
      if (r < c + w) {
        if (a.tokens_int64) static_cast<int64_t*>(a.tokens)[b] = i;
        else static_cast<int32_t*>(a.tokens)[b] = i;
        if (a.logprob) a.logprob[b] = logf((float)((double)w / (double)total));
        break;
      }
      c += w;
    }
  }
}

}  // namespace

hipError_t launch_sample(const SampleArgs& a, unsigned char* ws, hipStream_t s) {
  (void)ws;
  const dim3 grid((unsigned)a.B), block(kThreads);
  if (a.dtype == F32) hipLaunchKernelGGL((q1_sample_row_kernel<F32>), grid, block, 0, s, a);
  else if (a.dtype == BF16) hipLaunchKernelGGL((q1_sample_row_kernel<BF16>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((q1_sample_row_kernel<F16>), grid, block, 0, s, a);
  return hipGetLastError();
}

}  // namespace q1
