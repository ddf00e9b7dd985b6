// Attention of a decode batch over a shared prefix and paged suffixes: one
// workgroup per (sequence, query head), a pass over the tokens in blocks of 256
// with a running maximum and sum.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "q1_decode.h"
#include "q1_device.h"
#include "q1_internal.h"

namespace q1 {
namespace {

constexpr int kThreads = 256;

__global__ __launch_bounds__(kThreads) void q1_attn_plain_kernel(const q1_attn a) {
  __shared__ float sc[kThreads], qs[256], red[kThreads];
  const int tid = threadIdx.x;
  const int64_t b = blockIdx.x / a.Hq;
  const int h = (int)(blockIdx.x - b * a.Hq), hk = h / (a.Hq / a.Hkv), D = a.D;
  const bool f16 = a.dtype == Q1_F16;
  auto cvt = [f16](uint16_t x) { return f16 ? f16_bits_to_f32(x) : bf16_bits_to_f32(x); };
  const auto* q = static_cast<const uint16_t*>(a.q) + b * a.q_ld + (int64_t)h * D;
  if (tid < D) qs[tid] = cvt(q[tid]);
  __syncthreads();
  int64_t suffix = 0;
  if (a.max_pages > 0) {
    suffix = a.suffix_lens[b];
    const int64_t most = a.max_pages * a.page_size;
    suffix = suffix < 0 ? 0 : suffix > most ? most : suffix;
  }
  const int64_t n = a.P + suffix;
  auto row = [&](int64_t t, const void* pre, const void* pag) -> const uint16_t* {
    if (t < a.P) return static_cast<const uint16_t*>(pre) + t * a.prefix_ld + (int64_t)hk * D;
    const int64_t s = t - a.P, pg = a.page_table[b * a.max_pages + s / a.page_size];
    if (pg < 0 || pg >= a.pages) return nullptr;
    return static_cast<const uint16_t*>(pag) + ((pg * a.page_size + s % a.page_size) * a.Hkv + hk) * D;
  };
  float m = -INFINITY, l = 0.f, o = 0.f;
  for (int64_t t0 = 0; t0 < n; t0 += kThreads) {
    const int64_t t = t0 + tid;
    float s = -INFINITY;
    if (t < n) {
      const uint16_t* k = row(t, a.k_prefix, a.k_pages);
      if (k != nullptr) {
        s = 0.f;
        for (int i = 0; i < D; ++i) s = __builtin_fmaf(qs[i], cvt(k[i]), s);
        s *= a.scale;
      }
    }
    red[tid] = s;
    __syncthreads();
    for (int w = kThreads / 2; w > 0; w >>= 1) {
      if (tid < w) red[tid] = fmaxf(red[tid], red[tid + w]);
      __syncthreads();
    }
    const float mn = fmaxf(m, red[0]);
    __syncthreads();
    const float p = s == -INFINITY ? 0.f : expf(s - mn);
    sc[tid] = p;
    red[tid] = p;
    __syncthreads();
    for (int w = kThreads / 2; w > 0; w >>= 1) {
      if (tid < w) red[tid] += red[tid + w];
      __syncthreads();
    }
    const float keep = m == -INFINITY ? 0.f : expf(m - mn);
    l = l * keep + red[0];
    if (tid < D) {
      o *= keep;
      for (int j = 0; j < kThreads && t0 + j < n; ++j) {
        if (sc[j] == 0.f) continue;
        const uint16_t* v = row(t0 + j, a.v_prefix, a.v_pages);
        if (v != nullptr) o = __builtin_fmaf(sc[j], cvt(v[tid]), o);
      }
    }
    m = mn;
    __syncthreads();
  }
  if (tid < D) store_out(a.out, a.out_dtype, (b * a.Hq + h) * D + tid, l > 0.f ? o / l : 0.f);
  if (tid == 0 && a.lse != nullptr) a.lse[b * a.Hq + h] = l > 0.f ? m + logf(l) : -INFINITY;
}

}  // namespace

hipError_t launch_prefix_attn(const q1_attn& a, unsigned char* ws, hipStream_t s) {
  (void)ws;
  hipLaunchKernelGGL(q1_attn_plain_kernel, dim3((unsigned)(a.B * a.Hq)), dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace q1
