// Sampler: temperature, top-k, top-p, min-p and one draw per row, from a given
// random number.
//
// A row is cut into contiguous chunks, one per wave; four launches:
//   q1_sample_top     largest logit of each workgroup's chunks, and of each small group
//                     of threads; a cleared histogram
//   q1_sample_hist    e = exp((x - top)/T), weight w = floor(e 2^40).  Rows with a top-k
//                     that is small beside the row (Row::few): all that it may keep, as
//                     candidates, from a bound that the groups' largest logits give.
//                     Others with top-k: counts in 2048 bins of (top - x)/T, with top-p:
//                     weights in them.  Rows with neither: each chunk's kept weight
//   q1_sample_cut     the bins in which the top-k and the top-p cut fall, from the
//                     histogram; each chunk's sum of the weights above them, and the
//                     elements in them as candidates
//   q1_sample_draw    one workgroup per row: the exact cut among the candidates and the
//                     draw; where it falls into a chunk, the token in that chunk
// so a row is read two or three times (once from HBM, then from the caches), never
// sorted, and any number of workgroups share it.  Weights are whole multiples of
// 2^-40, so sums are exact: no result depends on the order of the additions.
//
// Order of logits: composite = 32-bit key (larger logit, larger key) over the
// complement of the index, so equal logits go lowest index first and all
// composites differ; a cut is one composite, and kept are those not below it.
//
// Where a cut's bins hold more than kMost candidates (rows that are flat, or full
// of equal logits), or a top-k bound leaves more (the logits above -infinity lie in
// fewer groups than k), the draw falls back to a radix select over the row itself by
// one workgroup: 0.8 ms for 1 or 8 flat rows of 152064, 0.43 for 8000 logits in a run
// beside -infinity with top-k 200 (with top-k 100, 26 us).
//
// What bounds it: for many rows the first launch reads the logits at the rate of a
// plain read (192 rows of 152064 in fp32, 117 MB: 19 us, 6.1 TB/s); the second and
// third are bound by arithmetic, some 40 vector instructions an element for the
// exponential, the exact quotient, the weight and its bin (31 and 24 us), which is why
// elements that cannot matter are left out by one comparison before it; the draw is
// one workgroup's chain of selects (16 us).  For one row all four are latency: 3 + 6 +
// 2 + 9 us, near what four launches cost the caller (17 us); in a replayed graph a row
// takes 9 us greedy, 12 without a filter, 16 to 21 with top-k 50, 28 with top-p.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "q1_decode.h"
#include "q1_device.h"
#include "q1_internal.h"

namespace q1 {
namespace {

constexpr int kThreads = 1024, kWaves = kThreads / 64;
constexpr int kBins = 2048;            // of (top - x) / T in [0, 27.75): beyond, weights are zero
constexpr float kBinsPerUnit = 73.8f;
constexpr int kMost = 4096;            // candidates of one cut
typedef unsigned long long u64;
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

struct Hist {
  u64 weight[kBins];
  uint32_t count[kBins];
};

// Where a row's cuts fall (written by q1_sample_cut for q1_sample_draw).
struct Cut {
  u64 total;               // weight of the row
  u64 above_k, above_p;    // weight above the bins of the cut
  u64 want_k;              // elements to keep of the top-k bin
  uint32_t n_k, n_p;       // candidates, at most (from the histogram)
  int32_t bin_k, lo_p, hi_p;  // -1: not in use
  uint32_t first;          // greedy: the lowest index of the largest logit
  uint32_t got_k, got_p;   // candidates written
};

struct Ws {
  float* top;      // [B][S]
  float* most;     // [B][groups(S)]: largest logit of each group of threads
  Hist* hist;      // [B]
  Cut* cut;        // [B]
  u64* sums;       // [B][S * kWaves]
  ulonglong2* cand;  // [B][2][kMost]: composite, weight (top bit: below min_p)
};

template <int DT>
constexpr int kSize = DT == F32 ? 4 : 2;

template <int DT>
__device__ __forceinline__ float value_of(uint32_t bits) {
  return DT == F32 ? __uint_as_float(bits) : DT == BF16 ? bf16_bits_to_f32(bits) : f16_bits_to_f32(bits);
}

// NaN counts as -infinity, -0 and +0 are equal logits.
__device__ __forceinline__ float clean(float x) { return x != x ? -INFINITY : x + 0.0f; }

template <int DT>
__device__ __forceinline__ float logit(const void* p, int64_t i) {
  return clean(value_of<DT>(DT == F32 ? static_cast<const uint32_t*>(p)[i] : static_cast<const uint16_t*>(p)[i]));
}

// Larger logits have larger keys.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t u = __float_as_uint(x);
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}

__device__ __forceinline__ u64 composite(float x, int i) { return (u64)key_of(x) << 32 | (uint32_t)~i; }

__device__ __forceinline__ float exp_of(float x, float top, float T) { return x == top ? 1.0f : expf((x - top) / T); }

// floor(e 2^40) for 0 <= e <= 1, as the 17 bits down to 2^-16 and the 24 below: the
// scalings and the fraction are exact, the conversions cut off.
__device__ __forceinline__ u64 weight_of(float e) {
  const float f = e * 65536.0f;
  const uint32_t hi = (uint32_t)f, lo = (uint32_t)(__builtin_amdgcn_fractf(f) * 16777216.0f);
  return (u64)(hi >> 8) << 32 | (hi << 24 | lo);
}

__device__ __forceinline__ u64 bound_of(float p, u64 total) {
  const double want = (double)p * (double)total;
  return want >= 1.0 ? (u64)want : 1;
}

struct Row {
  float T, p, mp;
  int64_t k;
  bool greedy, use_k, use_p, few;
};

// Threads of a row's workgroups that have one largest logit together (1, 4 or 16), so that
// there are at most 4096 of these: every workgroup of the row goes through them.
__device__ __host__ __forceinline__ int group_lanes(int S) { return S <= 4 ? 1 : S <= 16 ? 4 : 16; }
__device__ __host__ __forceinline__ int groups(int S) { return S * kThreads / group_lanes(S); }

// few: all that top-k may keep are candidates (see q1_sample_hist).  The k-th largest of
// the groups' largest logits is near the k-th of all as long as k is a small part of the
// groups (at a quarter, about 1.15 k elements are above it, at all of them no bound is
// left).  Rows of up to kMost elements fit as they are.  It saves a pass over the row and
// wins while one wave's select takes the candidates: k = 50, 152064 logits, 1 / 64 / 192
// rows 15.6 / 33 / 60 us, with the histogram 18.2 / 39 / 80; k = 200, 20.6 / 35 / 61 and
// 19.3 / 40 / 79.  Past that the select by all waves costs 11 us, k = 400, 33 / 47 / 72 and
// 19.4 / 40 / 80, so only a batch whose pass takes longer does it (equal at 96 to 128 rows).
constexpr int kFew = 256;  // candidates that one wave works on (see cut_candidates)
__device__ __forceinline__ Row row_of(const SampleArgs& a, int64_t b, int S) {
  Row r;
  r.T = a.temperature ? a.temperature[b] : 1.0f;
  r.greedy = !(r.T > 0.f);
  if (r.greedy) r.T = 1.f;
  r.k = a.top_k ? a.top_k[b] : 0;
  r.p = a.top_p ? a.top_p[b] : 1.f;
  r.mp = a.min_p ? a.min_p[b] : 0.f;
  r.mp = r.mp > 0.f ? fminf(r.mp, 1.f) : 0.f;
  r.use_k = !r.greedy && r.k > 0 && r.k < a.V;
  r.use_p = !r.greedy && r.p < 1.f;
  const bool near = r.k <= groups(S) / 4 && (r.k <= kFew * 4 / 5 || a.B * a.V >= 1 << 24);
  r.few = r.use_k && (near || a.V <= kMost);
  return r;
}

// (x - top) / T of one logit, not below -64 (where weights are zero long since).
// The quotient has to be the correctly rounded one.  inv, the correctly rounded
// reciprocal, and what it lacks (rest) give it within a unit in the last place, and
// then one correction by the exact remainder rounds it correctly (Markstein); outside
// 2^+-40 for T the division itself is used.  NaN comes out as -64.
struct Scale {
  float top, T, inv, rest, least, bins;
  bool plain;
  __device__ Scale(float top_, float T_)
      : top(top_), T(T_), inv(1.0f / T_), rest(__builtin_fmaf(-inv, T_, 1.0f) * inv), least(-64.0f * T_),
        bins(kBinsPerUnit * inv), plain(!(T_ > 9e-13f && T_ < 1e12f) || top_ == INFINITY) {}
  __device__ __forceinline__ float exponent(float x) const {
    const float d = fmaxf(x - top, least);
    if (plain) return x == top ? 0.f : fmaxf(d / T, -64.f);
    const float q = __builtin_fmaf(d, inv, d * rest);
    return __builtin_fmaf(__builtin_fmaf(-q, T, d), inv, q);
  }
  // A bin that falls with the logit, where no weight is wanted: kBins for those past all bins and NaN.
  __device__ __forceinline__ int rank_bin(float x) const {
    const float f = plain ? -exponent(x) * kBinsPerUnit : (top - x) * bins;
    return (int)fminf(f, (float)kBins);
  }
  // Below it, every logit's bin is past `bin`.
  __device__ __forceinline__ float past(int bin) const {
    return plain ? -INFINITY : top - T * ((float)(bin + 1) / kBinsPerUnit) * 1.0001f - fabsf(top) * 1e-6f;
  }
};

__device__ __forceinline__ int bin_of(float t) { return (int)(-t * kBinsPerUnit); }

// Chunk c of a row: [c len, (c + 1) len), len = V over all chunks, rounded up.
__device__ __forceinline__ int chunk_len(int64_t V, int chunks) { return (int)((V + chunks - 1) / chunks); }

// f(index, logit as it is, whether there is one) for every element of [lo, hi), by one
// wave whose lanes call f together: 16-byte loads, four in flight, between the first and
// the last aligned element.
template <int DT, class F>
__device__ __forceinline__ void each(const void* row, int lo, int hi, F f) {
  constexpr int E = 16 / kSize<DT>;
  const int lane = threadIdx.x & 63;
  if (lo >= hi) return;
  const uintptr_t at = reinterpret_cast<uintptr_t>(row) + (int64_t)lo * kSize<DT>;
  int head = (int)((16 - at % 16) % 16) / kSize<DT>;
  if (head > hi - lo) head = hi - lo;
  const int a0 = lo + head, nv = (hi - a0) / E;
  const u32x4* v = reinterpret_cast<const u32x4*>(static_cast<const unsigned char*>(row) + (int64_t)a0 * kSize<DT>);
  auto all = [&](const u32x4& x, int i, bool ok) {
#pragma unroll
    for (int e = 0; e < E; ++e)
      f(a0 + i * E + e, value_of<DT>(DT == F32 ? x[e] : (x[e >> 1] >> (16 * (e & 1))) & 0xffffu), ok);
  };
  int i = lane;
  for (; i - lane + 256 <= nv; i += 256) {
    u32x4 x[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) x[u] = v[i + 64 * u];
#pragma unroll
    for (int u = 0; u < 4; ++u) all(x[u], i + 64 * u, true);
  }
  for (; i - lane < nv; i += 64) all(v[i < nv ? i : nv - 1], i, i < nv);
  // before and past the aligned part: at most 2 (E - 1) elements
  const int past = a0 + nv * E, n = head + hi - past;
  const int j = lane < head ? lo + lane : past + lane - head;
  const int c = lane < n ? j : lo;
  f(j, value_of<DT>(DT == F32 ? static_cast<const uint32_t*>(row)[c] : static_cast<const uint16_t*>(row)[c]), lane < n);
}

// One step of a scan over a wave's lanes: v plus (or the larger of v and) the value
// that the DPP control brings from another lane, where the row mask has this one.
template <int CTRL, int ROWS>
__device__ __forceinline__ u64 step_add(u64 v) {
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)v, CTRL, ROWS, 0xf, false);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(v >> 32), CTRL, ROWS, 0xf, false);
  return v + ((u64)hi << 32 | lo);
}

template <int CTRL, int ROWS>
__device__ __forceinline__ float step_max(float v) {
  const int none = (int)0xff800000u;  // -infinity
  return fmaxf(v, __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(none, __builtin_bit_cast(int, v), CTRL, ROWS, 0xf, false)));
}

// The value of another lane of the four (or of the row of 16) by a DPP control.
template <int CTRL>
__device__ __forceinline__ float with_lane(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xf, 0xf, false));
}

// Inclusive sum over the lanes of a wave: rows of 16 by shifts of 1, 2, 4, 8, then
// the last lane of a row to the next one, and of the lower half to the upper.
__device__ __forceinline__ u64 wave_scan(u64 v) {
  v = step_add<0x111, 0xf>(v);
  v = step_add<0x112, 0xf>(v);
  v = step_add<0x114, 0xf>(v);
  v = step_add<0x118, 0xf>(v);
  v = step_add<0x142, 0xa>(v);
  return step_add<0x143, 0xc>(v);
}

__device__ __forceinline__ u64 last_lane(u64 v) {
  return (u64)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(v >> 32), 63) << 32 |
         (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, 63);
}

__device__ __forceinline__ u64 wave_sum(u64 v) { return last_lane(wave_scan(v)); }

__device__ __forceinline__ float wave_max(float v) {
  v = step_max<0x111, 0xf>(v);
  v = step_max<0x112, 0xf>(v);
  v = step_max<0x114, 0xf>(v);
  v = step_max<0x118, 0xf>(v);
  v = step_max<0x142, 0xa>(v);
  v = step_max<0x143, 0xc>(v);
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
}

// Exclusive sum over the workgroup's threads in order; *total: of all of them.
// s: kWaves words that no thread reads or writes meanwhile.
__device__ __forceinline__ u64 block_scan(u64 v, u64* s, u64* total) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const u64 x = wave_scan(v);
  if (lane == 63) s[w] = x;
  __syncthreads();
  const u64 waves = wave_scan(lane < kWaves ? s[lane] : 0);
  *total = last_lane(waves);
  const u64 upto = (u64)__shfl((int64_t)waves, w);  // through wave w
  const u64 own = last_lane(x);
  return upto - own + x - v;
}

__device__ __forceinline__ void put_token(const SampleArgs& a, int64_t b, int64_t token, float logprob) {
  if (a.tokens_int64) static_cast<int64_t*>(a.tokens)[b] = token;
  else static_cast<int32_t*>(a.tokens)[b] = (int32_t)token;
  if (a.logprob) a.logprob[b] = logprob;
}

template <int DT>
__device__ __forceinline__ const void* row_ptr(const SampleArgs& a, int64_t b) {
  return static_cast<const unsigned char*>(a.logits) + b * a.ld * kSize<DT>;
}

// S is at most a wave's lanes.
__device__ __forceinline__ float row_top(const Ws& ws, int64_t b, int S) {
  const int lane = threadIdx.x & 63;
  return wave_max(lane < S ? ws.top[b * S + lane] : -INFINITY);
}

template <int DT>
__global__ __launch_bounds__(kThreads) void q1_sample_top(const SampleArgs a, const Ws ws, int S) {
  __shared__ float part[kWaves];
  const int64_t b = blockIdx.x / S;
  const int s = (int)(blockIdx.x - b * S), wave = threadIdx.x >> 6;
  const int len = chunk_len(a.V, S * kWaves), lo = (s * kWaves + wave) * len, end = lo + len;
  float top = -INFINITY;
  each<DT>(row_ptr<DT>(a, b), lo, end < a.V ? end : (int)a.V, [&](int, float x, bool ok) { top = fmaxf(top, ok ? x : -INFINITY); });
  if (a.top_k != nullptr) {
    const int L = group_lanes(S);
    float m = top;
    if (L > 1) m = fmaxf(with_lane<0xb1>(m), fmaxf(m, fmaxf(with_lane<0x4e>(m), with_lane<0x1b>(m))));
    if (L > 4) m = fmaxf(fmaxf(m, with_lane<0x124>(m)), fmaxf(with_lane<0x128>(m), with_lane<0x12c>(m)));
    if ((threadIdx.x & (L - 1)) == 0) ws.most[b * groups(S) + (s * kThreads + threadIdx.x) / L] = m;
  }
  top = wave_max(top);
  if ((threadIdx.x & 63) == 0) part[wave] = top;
  for (int i = s * kThreads + threadIdx.x; i < kBins; i += S * kThreads) {
    ws.hist[b].weight[i] = 0;
    ws.hist[b].count[i] = 0;
  }
  if (s == 0 && threadIdx.x == 0) {
    ws.cut[b].first = ~0u;
    ws.cut[b].got_k = ws.cut[b].got_p = 0;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < kWaves; ++i) top = fmaxf(top, part[i]);
    ws.top[b * S + s] = top;
  }
}

// take(index, logit) for the elements of [lo, hi) not below `past`, by one wave: they are
// collected in `queue`, so that the wave works on 64 of them at a time.
template <int DT, class F>
__device__ __forceinline__ void each_from(const void* row, int lo, int hi, float past, uint2 (&queue)[128], F take) {
  const int lane = threadIdx.x & 63;
  uint32_t in = 0, done = 0;
  each<DT>(row, lo, hi, [&](int i, float x, bool ok) {
    const u64 some = __ballot(ok && x >= past);
    if (some == 0) return;
    const uint32_t at = in + __builtin_amdgcn_mbcnt_hi((uint32_t)(some >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)some, 0));
    if (ok && x >= past) queue[at & 127] = uint2{(uint32_t)i, __float_as_uint(x)};
    in += (uint32_t)__builtin_popcountll(some);
    if (in - done >= 64) {
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      const uint2 m = queue[(done + lane) & 127];
      take((int)m.x, __uint_as_float(m.y));
      done += 64;
    }
  });
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  if (done + lane < in) {
    const uint2 m = queue[(done + lane) & 127];
    take((int)m.x, __uint_as_float(m.y));
  }
}

template <int DT>
__global__ __launch_bounds__(kThreads, 8) void q1_sample_hist(const SampleArgs a, const Ws ws, int S) {
  __shared__ Hist h;
  __shared__ uint2 queue[kWaves][128];
  __shared__ u64 scan[kWaves];
  __shared__ int last;
  const int64_t b = blockIdx.x / S;
  const int s = (int)(blockIdx.x - b * S), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = groups(S);
  float most[4];  // at most 4096 groups: four a thread, loaded before anything is waited for
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int at = i * kThreads + threadIdx.x;
    most[i] = a.top_k != nullptr && at < n ? ws.most[b * n + at] : -INFINITY;
  }
  const float top = row_top(ws, b, S);
  const Row r = row_of(a, b, S);
  if (top == -INFINITY) return;
  const int len = chunk_len(a.V, S * kWaves), c = s * kWaves + wave, lo = c * len;
  const int hi = lo + len < a.V ? lo + len : (int)a.V;
  const void* row = row_ptr<DT>(a, b);
  if (r.greedy) {
    int first = 0x7fffffff;
    each<DT>(row, lo, hi, [&](int i, float x, bool ok) {
      if (ok && x == top && i < first) first = i;
    });
    if (first != 0x7fffffff) atomicMin(&ws.cut[b].first, (uint32_t)first);
    return;
  }
  const Scale sc(top, r.T);
  if (!r.use_k && !r.use_p) {
    u64 sum = 0;
    each<DT>(row, lo, hi, [&](int, float x, bool ok) {
      const float e = expf(sc.exponent(x));
      if (ok && !(e < r.mp)) sum += weight_of(e);
    });
    sum = wave_sum(sum);
    if ((threadIdx.x & 63) == 0) ws.sums[b * S * kWaves + c] = sum;
    return;
  }
  if (r.few) {
    // the bin of the k-th largest of the groups' largest logits: k elements at least are
    // in it and those before it, and all of these are candidates
    h.count[threadIdx.x] = h.count[threadIdx.x + kThreads] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int bin = sc.rank_bin(most[i]);
      if (i * kThreads < n && bin < kBins) atomicAdd(&h.count[bin], 1u);
    }
    if (threadIdx.x == 0) last = kBins - 1;  // if there are fewer: every element with a weight
    __syncthreads();
    const uint32_t n0 = h.count[2 * threadIdx.x], n1 = h.count[2 * threadIdx.x + 1];
    u64 all;
    const u64 before = block_scan((u64)n0 + n1, scan, &all), k = (u64)r.k;
    if (before < k && k <= before + n0 + n1) last = 2 * threadIdx.x + (before + n0 < k);
    __syncthreads();
    const int bins = last;
    each_from<DT>(row, lo, hi, sc.past(bins), queue[wave], [&](int i, float x) {
      if (sc.rank_bin(x) > bins) return;
      const float e = expf(sc.exponent(x));
      const uint32_t at = atomicAdd(&ws.cut[b].got_k, 1u);
      if (at < kMost) ws.cand[(b * 2) * kMost + at] = ulonglong2{composite(clean(x), i), weight_of(e) | (e < r.mp ? 1ull << 63 : 0)};
    });
    return;
  }
  for (int i = threadIdx.x; i < kBins; i += kThreads) {
    h.weight[i] = 0;
    h.count[i] = 0;
  }
  __syncthreads();
  if (!r.use_p) {
    each<DT>(row, lo, hi, [&](int, float x, bool ok) {
      const int bin = sc.rank_bin(x);
      if (ok && bin < kBins) atomicAdd(&h.count[bin], 1u);
    });
  } else {
    each<DT>(row, lo, hi, [&](int, float x, bool ok) {
      const float t = sc.exponent(x);
      const u64 w = weight_of(expf(t));
      if (!ok || w == 0) return;
      const int bin = bin_of(t);
      atomicAdd(&h.weight[bin], w);
      if (r.use_k) atomicAdd(&h.count[bin], 1u);
    });
  }
  __syncthreads();
  for (int i = threadIdx.x; i < kBins; i += kThreads) {
    if (h.weight[i] != 0) atomicAdd(&ws.hist[b].weight[i], h.weight[i]);
    if (h.count[i] != 0) atomicAdd(&ws.hist[b].count[i], h.count[i]);
  }
}

// The bins of the cuts, from the histogram; every thread of the workgroup gets them.
// With both filters the top-p cut is known only once the top-k one is: its bins
// are those it can fall in, whatever of its bin top-k keeps.
struct Bins {  // a thread's two
  ulonglong2 w;
  uint2 n;
};

__device__ __forceinline__ Cut find_cut(const Bins& h, const Row& r, u64* s, Cut* out) {
  const int t = threadIdx.x;
  static_assert(kBins == 2 * kThreads, "two bins a thread");
  u64 wb = 0, nb = 0, all = 0, total = 0;
  const u64 w0 = h.w.x, w1 = h.w.y;
  const uint32_t n0 = h.n.x, n1 = h.n.y;
  if (t == 0) {
    out->bin_k = out->lo_p = out->hi_p = -1;
    out->n_k = out->n_p = 0;
    out->above_k = out->above_p = out->want_k = 0;
  }
  if (r.use_p) wb = block_scan(w0 + w1, s, &total);
  if (r.use_k) nb = block_scan((u64)n0 + n1, s + kWaves, &all);
  const u64 k = (u64)r.k;
  const bool use_k = r.use_k && k < all;  // else every element with a weight is kept
  u64 least = total, most = total;        // of the weight that top-k keeps
  if (use_k) {
    if (nb < k && k <= nb + n0 + n1) {
      const bool second = nb + n0 < k;
      out->bin_k = 2 * t + second;
      out->n_k = second ? n1 : n0;
      out->above_k = wb + (second ? w0 : 0);
      out->want_k = k - nb - (second ? n0 : 0);
      s[2 * kWaves] = second ? w1 : w0;
    }
    __syncthreads();
    least = out->above_k;
    most = least + s[2 * kWaves];
  }
  if (r.use_p) {
    const u64 p0 = bound_of(r.p, least), p1 = bound_of(r.p, most);
    if (wb < p0 && p0 <= wb + w0 + w1) {
      const bool second = wb + w0 < p0;
      out->lo_p = 2 * t + second;
      out->above_p = wb + (second ? w0 : 0);
    }
    if (wb < p1 && p1 <= wb + w0 + w1) out->hi_p = 2 * t + (wb + w0 < p1);
    __syncthreads();
    // at most: the bins' weights over the least weight in each
    const int lo = out->lo_p, hi = out->hi_p;
    if (2 * t + 1 >= lo && 2 * t <= hi) {
      u64 n = 0;
#pragma unroll
      for (int j = 0; j < 2; ++j)
        if (2 * t + j >= lo && 2 * t + j <= hi) {
          const u64 least_w = weight_of(0.999f * expf(-(float)(2 * t + j + 1) / kBinsPerUnit));
          n += (j ? w1 : w0) / (least_w > 0 ? least_w : 1);
        }
      atomicAdd(&out->n_p, (uint32_t)(n < (1u << 24) ? n : 1u << 24));
    }
  }
  __syncthreads();
  Cut c;
  c.total = total;
  c.bin_k = out->bin_k;
  c.lo_p = out->lo_p;
  c.hi_p = out->hi_p;
  c.n_k = out->n_k;
  c.n_p = out->n_p;
  c.above_k = out->above_k;
  c.above_p = out->above_p;
  c.want_k = out->want_k;
  return c;
}

template <int DT>
__global__ __launch_bounds__(kThreads, 8) void q1_sample_cut(const SampleArgs a, const Ws ws, int S) {
  __shared__ u64 s[2 * kWaves + 1];
  __shared__ Cut found;
  __shared__ uint2 queue[kWaves][128];
  const int64_t b = blockIdx.x / S;
  const int sl = (int)(blockIdx.x - b * S);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const float top = row_top(ws, b, S);
  const Bins bins = {reinterpret_cast<const ulonglong2*>(ws.hist[b].weight)[threadIdx.x],
                     reinterpret_cast<const uint2*>(ws.hist[b].count)[threadIdx.x]};
  const Row r = row_of(a, b, S);
  if ((!r.use_k && !r.use_p) || r.few || top == -INFINITY) return;
  const Cut c = find_cut(bins, r, s, &found);
  if (sl == 0 && threadIdx.x == 0) {
    Cut* o = &ws.cut[b];
    o->total = c.total;
    o->above_k = c.above_k;
    o->above_p = c.above_p;
    o->want_k = c.want_k;
    o->n_k = c.n_k;
    o->n_p = c.n_p;
    o->bin_k = c.bin_k;
    o->lo_p = c.lo_p;
    o->hi_p = c.hi_p;
  }
  if (c.n_k > kMost || c.n_p > kMost) return;
  // below the first bin of the deciding cut, everything is kept
  const int sure = r.use_p ? c.lo_p : c.bin_k >= 0 ? c.bin_k : kBins;
  const int last = c.bin_k > c.hi_p ? c.bin_k : c.hi_p;  // past it nothing is (none in use: -1, and sure has all)
  const Scale sc(top, r.T);
  const int len = chunk_len(a.V, S * kWaves), ch = sl * kWaves + wave, lo = ch * len;
  const int hi = lo + len < a.V ? lo + len : (int)a.V;
  u64 sum = 0;
  auto take = [&](int i, float x) {
    const float t = sc.exponent(x), e = expf(t);
    const int bin = r.use_p ? bin_of(t) : sc.rank_bin(x);
    const u64 w = weight_of(e);
    const bool low = e < r.mp;
    if (bin < sure && !low) sum += w;
    const ulonglong2 entry = {composite(clean(x), i), w | (low ? 1ull << 63 : 0)};
    // (with top-p, elements without a weight are in no bin's count, and there may be any number of them)
    if (bin == c.bin_k && (w != 0 || !r.use_p)) {
      const uint32_t at = atomicAdd(&ws.cut[b].got_k, 1u);
      if (at < kMost) ws.cand[(b * 2) * kMost + at] = entry;
    }
    if (w != 0 && bin >= c.lo_p && bin <= c.hi_p) {
      const uint32_t at = atomicAdd(&ws.cut[b].got_p, 1u);
      if (at < kMost) ws.cand[(b * 2 + 1) * kMost + at] = entry;
    }
  };
  each_from<DT>(row_ptr<DT>(a, b), lo, hi, sc.past(sure > last ? sure : last), queue[wave], take);
  sum = wave_sum(sum);
  if ((threadIdx.x & 63) == 0) ws.sums[b * S * kWaves + ch] = sum;
}

struct DrawShared {
  u64 bins[kThreads];
  u64 chunk[kThreads];  // weight in each chunk
  u64 s[3][kWaves];  // one for each sum or scan between barriers
  u64 over, cut;
  uint32_t pick, left;
};

template <int CTRL, int ROWS>
__device__ __forceinline__ u64 step_most(u64 v) {
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)v, CTRL, ROWS, 0xf, false);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(v >> 32), CTRL, ROWS, 0xf, false);
  const u64 o = (u64)hi << 32 | lo;
  return o > v ? o : v;
}

__device__ __forceinline__ u64 wave_most(u64 v) {
  v = step_most<0x111, 0xf>(v);
  v = step_most<0x112, 0xf>(v);
  v = step_most<0x114, 0xf>(v);
  v = step_most<0x118, 0xf>(v);
  v = step_most<0x142, 0xa>(v);
  return last_lane(step_most<0x143, 0xc>(v));
}

// The candidates of a cut are worked on by W waves, four a thread, in registers: by one
// wave up to kFew (every instruction costs the workgroup's 16 waves 16 cycles, and they
// would wait for each other: a row with all filters took 12 us so, and 7 with one
// wave), by all of them beyond.
constexpr int kEach = 4;
static_assert(kEach * 64 == kFew && kEach * kThreads == kMost, "four a thread");

template <int W>
__device__ __forceinline__ void group_sync() {
  if (W == 1) __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  else __syncthreads();
}

template <int W>
__device__ __forceinline__ u64 group_most(u64 v, u64* s) {
  v = wave_most(v);
  if (W == 1) return v;
  const int lane = threadIdx.x & 63;
  if (lane == 0) s[threadIdx.x >> 6] = v;
  __syncthreads();
  return wave_most(lane < W ? s[lane] : 0);
}

template <int W>
__device__ __forceinline__ u64 group_scan(u64 v, u64* s, u64* total) {
  if (W != 1) return block_scan(v, s, total);
  const u64 x = wave_scan(v);
  *total = last_lane(x);
  return x - v;
}

// Of the group's candidates (0: none), largest first, the one at which the running sum
// of their amounts reaches `want`; 0 if the sum stays below.  The interval of those left
// is cut into pieces of equal width (256 for one wave, 1024), the piece that the cut
// falls in is the next interval.
template <int W>
__device__ __forceinline__ u64 select_candidate(DrawShared& d, const u64 (&c)[kEach], const u64 (&amount)[kEach], u64 want) {
  constexpr int kPieces = W == 1 ? 256 : kThreads, kOwn = kPieces / (64 * W), kBits = W == 1 ? 8 : 10;
  const int t = threadIdx.x & (64 * W - 1);
  u64 lo = 1, hi = ~0ull, before = 0;
  for (;;) {
    u64 most = 0, least = 0;  // least: of the complements
#pragma unroll
    for (int k = 0; k < kEach; ++k)
      if (c[k] - lo <= hi - lo) {
        if (c[k] > most) most = c[k];
        if (~c[k] > least) least = ~c[k];
      }
#pragma unroll
    for (int k = 0; k < kOwn; ++k) d.bins[kOwn * t + k] = 0;
    hi = group_most<W>(most, d.s[0]);
    lo = ~group_most<W>(least, d.s[1]);
    group_sync<W>();
    if (hi == lo || hi == 0) return hi;  // one left, or none
    const int bits = 64 - __builtin_clzll(hi - lo), shift = bits > kBits ? bits - kBits : 0;
#pragma unroll
    for (int k = 0; k < kEach; ++k)
      if (c[k] - lo <= hi - lo) atomicAdd(&d.bins[(hi - c[k]) >> shift], amount[k]);
    group_sync<W>();
    u64 own[kOwn], sum = 0, all;
#pragma unroll
    for (int k = 0; k < kOwn; ++k) {
      own[k] = d.bins[kOwn * t + k];
      sum += own[k];
    }
    u64 at = before + group_scan<W>(sum, d.s[2], &all);
    if (before + all < want) return 0;
#pragma unroll
    for (int k = 0; k < kOwn; ++k) {
      if (at < want && want <= at + own[k]) {
        d.pick = (uint32_t)(kOwn * t + k);
        d.over = at;
      }
      at += own[k];
    }
    group_sync<W>();
    const u64 width = (1ull << shift) - 1;
    hi -= (u64)d.pick << shift;
    if (hi - lo > width) lo = hi - width;
    before = d.over;
  }
}

// floor(u total), below total.
__device__ __forceinline__ u64 drawn(float u, u64 total) {
  const u64 at = u > 0.f ? (u64)((double)fminf(u, 1.f) * (double)total) : 0;
  return at >= total ? total - 1 : at;
}

// A row's token by radix selects over the row itself (see the top of the file).
template <int DT>
__device__ void draw_from_row(const SampleArgs& a, int64_t b, const void* row, const Row& r, float top, u64* sw) {
  __shared__ u64 hist[256];
  __shared__ uint32_t pick;
  __shared__ u64 over;
  const int tid = threadIdx.x;
  const int V = (int)a.V;
  const float T = r.T, p = r.p, mp = r.mp;
  const int64_t k = r.use_k ? r.k : V;

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
    u64 total;
    __syncthreads();
    block_scan(mine, sw, &total);
    __syncthreads();
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
  const u64 at = drawn(u, total);
  if (at >= start && at < start + mine) {
    u64 c = start;
    rank = rank0;
    for (int i = i0; i < i1; ++i) {
      const u64 w = kept(i, &rank);
      if (at < c + w) {
        put_token(a, b, i, logf((float)((double)w / (double)total)));
        break;
      }
      c += w;
    }
  }
}

// The row's cuts among its candidates (own_k, own_p: the first of each list, for W = 1).
// Where they are all that may be kept (few), the draw among them too, in index order;
// else the lowest kept composite goes to d.cut, and the kept candidates' weights are
// added to their chunks'.
template <int W>
__device__ __forceinline__ void cut_candidates(DrawShared& d, const SampleArgs& a, int64_t b, const Row& r, const Cut& c,
                                               const ulonglong2* list, const ulonglong2 (&own_k)[kEach],
                                               const ulonglong2 (&own_p)[kEach], float u, int len) {
  const int t = threadIdx.x & (64 * W - 1);
  u64 comp[kEach] = {}, weight[kEach] = {}, amount[kEach];  // weight: 0 if below min-p
  u64 cut = 0, total = c.total;                   // total: of what top-k keeps
  for (int step = 0; step < (r.few ? 3 : 2); ++step) {
    u64 want;
    if (step == 0) {
      if (!r.few && c.bin_k < 0) continue;
      const uint32_t n = c.got_k;
#pragma unroll
      for (int k = 0; k < kEach; ++k) {
        const uint32_t i = (uint32_t)(t + 64 * W * k);
        const ulonglong2 e = i >= n ? ulonglong2{0, 0} : W == 1 ? own_k[k] : list[i];
        comp[k] = e.x;
        weight[k] = e.y;
        amount[k] = 1;
      }
      want = r.few ? (u64)r.k : c.want_k;
      if (r.few && want >= n) continue;  // all of them
    } else if (step == 1) {
      if (!r.use_p) continue;
      if (r.few || c.bin_k >= 0) {
        u64 mine = 0;
#pragma unroll
        for (int k = 0; k < kEach; ++k)
          if (comp[k] >= cut) mine += weight[k] & ~(1ull << 63);
        group_sync<W>();
        group_scan<W>(mine, d.s[2], &total);
        if (!r.few) total += c.above_k;
      }
#pragma unroll
      for (int k = 0; k < kEach; ++k) {
        if (!r.few) {
          const uint32_t i = (uint32_t)(t + 64 * W * k);
          const ulonglong2 e = i >= c.got_p ? ulonglong2{0, 0} : W == 1 ? own_p[k] : list[kMost + i];
          comp[k] = e.x;
          weight[k] = e.y;
        }
        amount[k] = weight[k] & ~(1ull << 63);
      }
      want = bound_of(r.p, total) - (r.few ? 0 : c.above_p);
    } else {
      u64 mine = 0;
#pragma unroll
      for (int k = 0; k < kEach; ++k) {
        amount[k] = comp[k] >= cut && !(weight[k] >> 63) ? weight[k] : 0;
        comp[k] &= 0xffffffffull;  // the complement of the index
        mine += amount[k];
      }
      group_sync<W>();
      group_scan<W>(mine, d.s[2], &total);
      want = drawn(u, total) + 1;
    }
    group_sync<W>();
    const u64 found = select_candidate<W>(d, comp, amount, want);
    if (step < 2) {
      cut = found;
      continue;
    }
#pragma unroll
    for (int k = 0; k < kEach; ++k)
      if (comp[k] == found)
        put_token(a, b, (int64_t)~(uint32_t)found, logf((float)((double)amount[k] / (double)total)));
  }
  if (r.few) return;
#pragma unroll
  for (int k = 0; k < kEach; ++k)
    if (comp[k] != 0 && comp[k] >= cut && !(weight[k] >> 63))
      atomicAdd(&d.chunk[~(uint32_t)comp[k] / (uint32_t)len], weight[k]);
  if (t == 0) d.cut = cut;
}

template <int DT>
__global__ __launch_bounds__(kThreads) void q1_sample_draw(const SampleArgs a, const Ws ws, int S) {
  __shared__ DrawShared d;
  const int64_t b = blockIdx.x;
  const int t = threadIdx.x, chunks = S * kWaves;
  // what does not depend on the row's filters, all loaded at once
  const ulonglong2* const list = ws.cand + b * 2 * kMost;
  const Cut c = ws.cut[b];
  ulonglong2 own_k[kEach] = {}, own_p[kEach] = {};
  if (t < 64 && (a.top_k != nullptr || a.top_p != nullptr)) {
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      own_k[k] = list[t + 64 * k];
      own_p[k] = list[kMost + t + 64 * k];
    }
  }
  const u64 chunk_sum = t < chunks ? ws.sums[b * chunks + t] : 0;
  const float u = a.u[b];
  const Row r = row_of(a, b, S);
  const float top = row_top(ws, b, S);
  if (top == -INFINITY) {
    if (t == 0) put_token(a, b, -1, -INFINITY);
    return;
  }
  if (r.greedy) {
    if (t == 0) put_token(a, b, c.first, 0.f);
    return;
  }
  const void* row = row_ptr<DT>(a, b);
  const int len = chunk_len(a.V, chunks);
  u64 cut = 0;  // the lowest kept composite
  d.chunk[t] = chunk_sum;
  __syncthreads();
  if (r.use_k || r.use_p) {
    if (r.few ? c.got_k > kMost : c.n_k > kMost || c.n_p > kMost) {
      draw_from_row<DT>(a, b, row, r, top, d.bins);
      return;
    }
    const uint32_t n_k = r.few || c.bin_k >= 0 ? c.got_k : 0, n_p = r.use_p && !r.few ? c.got_p : 0;
    if (n_k <= kFew && n_p <= kFew) {
      if (t < 64) cut_candidates<1>(d, a, b, r, c, list, own_k, own_p, u, len);
    } else {
      cut_candidates<kWaves>(d, a, b, r, c, list, own_k, own_p, u, len);
    }
    if (r.few) return;
    __syncthreads();
    cut = d.cut;
  }
  const u64 weight_here = d.chunk[t];
  u64 total;
  const u64 start = block_scan(weight_here, d.s[0], &total), at = drawn(u, total);
  if (at >= start && at < start + weight_here) {
    d.left = (uint32_t)t;
    d.over = at - start;
  }
  __syncthreads();
  // the token: consecutive elements of the chunk, a few per thread
  const int lo = (int)d.left * len, hi = lo + len < a.V ? lo + len : (int)a.V;
  const u64 want = d.over;
  const int per = (hi - lo + kThreads - 1) / kThreads;
  const int i0 = lo + t * per < hi ? lo + t * per : hi, i1 = i0 + per < hi ? i0 + per : hi;
  const Scale sc(top, r.T);
  auto weight = [&](int i) -> u64 {
    const float x = logit<DT>(row, i);
    const float e = expf(sc.exponent(x));
    return composite(x, i) >= cut && !(e < r.mp) ? weight_of(e) : 0;
  };
  u64 sum = 0;
  for (int i = i0; i < i1; ++i) sum += weight(i);
  u64 all;
  u64 run = block_scan(sum, d.s[1], &all);
  if (want >= run && want < run + sum)
    for (int i = i0; i < i1; ++i) {
      const u64 w = weight(i);
      if (want < run + w) {
        put_token(a, b, i, logf((float)((double)w / (double)total)));
        break;
      }
      run += w;
    }
}

template <int DT>
hipError_t launch_t(const SampleArgs& a, const Ws& w, int S, hipStream_t s) {
  const dim3 grid((unsigned)(a.B * S)), block(kThreads);
  hipLaunchKernelGGL((q1_sample_top<DT>), grid, block, 0, s, a, w, S);
  hipLaunchKernelGGL((q1_sample_hist<DT>), grid, block, 0, s, a, w, S);
  if (a.top_k != nullptr || a.top_p != nullptr) hipLaunchKernelGGL((q1_sample_cut<DT>), grid, block, 0, s, a, w, S);
  hipLaunchKernelGGL((q1_sample_draw<DT>), dim3((unsigned)a.B), block, 0, s, a, w, S);
  return hipGetLastError();
}

size_t up(size_t v) { return (v + 255) / 256 * 256; }

}  // namespace

// Workgroups per row: about two per compute unit in all, at least 4096 elements
// each, and no more chunks than the draw has threads.
int sample_split(int64_t B, int64_t V) {
  int64_t S = (512 + B - 1) / B, most = (V + 4095) / 4096;
  if (S > most) S = most;
  if (S > kThreads / kWaves) S = kThreads / kWaves;
  return S < 1 ? 1 : (int)S;
}

size_t sample_ws_bytes(int64_t B, int64_t V) {
  const size_t S = (size_t)sample_split(B, V), b = (size_t)B;
  return up(b * sizeof(Hist)) + up(b * 2 * kMost * sizeof(ulonglong2)) + up(b * sizeof(Cut)) +
         up(b * S * kWaves * sizeof(u64)) + up(b * S * sizeof(float)) + up(b * (size_t)groups((int)S) * sizeof(float));
}

hipError_t launch_sample(const SampleArgs& a, unsigned char* ws, hipStream_t s) {
  const int S = sample_split(a.B, a.V);
  const size_t b = (size_t)a.B;
  Ws w;
  w.hist = reinterpret_cast<Hist*>(ws);
  ws += up(b * sizeof(Hist));
  w.cand = reinterpret_cast<ulonglong2*>(ws);
  ws += up(b * 2 * kMost * sizeof(ulonglong2));
  w.cut = reinterpret_cast<Cut*>(ws);
  ws += up(b * sizeof(Cut));
  w.sums = reinterpret_cast<u64*>(ws);
  ws += up(b * (size_t)S * kWaves * sizeof(u64));
  w.top = reinterpret_cast<float*>(ws);
  ws += up(b * (size_t)S * sizeof(float));
  w.most = reinterpret_cast<float*>(ws);
  if (a.dtype == F32) return launch_t<F32>(a, w, S, s);
  if (a.dtype == BF16) return launch_t<BF16>(a, w, S, s);
  return launch_t<F16>(a, w, S, s);
}

}  // namespace q1
