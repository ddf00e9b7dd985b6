// Attention of a decode batch over a shared prefix and paged suffixes.
//
// Two launches: q1_attn_main computes, per work item, the running maximum m,
// sum l and unnormalised output o of some query rows over some tokens;
// q1_attn_join adds the items of a row.  A prefix item holds the rows of all
// sequences that share a key/value head (B * Hq/Hkv of them, in blocks), so a
// prefix token is read once per block and not once per sequence; a suffix item
// holds the Hq/Hkv rows of one sequence.  Tokens are split over items so that the
// launch fills the compute units (see plan_prefix_attn).
//
// An item has one of two forms.  By tokens (few rows: the bound is reading): each
// of the 4 waves takes every fourth tile of 32 tokens, by itself, with all the
// rows, and the waves are joined in LDS.  By rows (many): the waves share a tile
// in LDS, two tiles in turn, and each has rows of its own.  Either way, per tile:
//   S^T = K Q^T   keys are the A operand (lane: token l%16, 8 consecutive
//                 elements), queries the B operand.
//   softmax       a lane has one query (l%16) and 8 tokens: maximum and sum are
//                 in-lane, then over 4 lanes.
//   O^T = V^T P^T the weights come out of S^T as the B operand's layout (tokens
//                 4(l/16)..+3 of both 16-token halves); values lie in LDS as rows
//                 and come back transposed (ds_read_tr16).
// Weights enter the second product as two 16-bit parts (high and remainder), so
// that their rounding (2^-17) stays below a 16-bit output's; their sum, the maximum
// and the output are fp32.  A token that does not count (past the length, no such
// page) has the score -infinity, whatever its key, and zeros for its values.
//
// What bounds it: few rows over a long prefix, the reading of keys and values (8
// sequences of 32 heads, 8 of keys, over 65537 fp16 tokens: 311 MB in 60 us, 5.2 TB/s
// of a plain read's 6.2, and 5 us for the join); 192 rows to a head of 256 (32
// sequences over 8201 tokens, 77 MB), the products and softmax of a tile, one after the
// other in each of two workgroups a CU (34 us, of which reading would be 12, and 7 us
// for the join); a short prefix, the two launches (8 and 4 us).  Pages alone: 32
// sequences of 2000 tokens (24 heads, 4 of keys, D = 128, bf16) 131 MB in 29 us, 8 of
// 32000 524 MB in 106, one of 2000 4 MB in 9.4 (in a replayed graph).
//
// Loops have no branch around loads or products (a branch makes the compiler wait
// for every load in flight where the paths join): loads past the end are dropped
// by a buffer's range or go to a row that does count.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "q1_attn_tile.h"
#include "q1_decode.h"
#include "q1_device.h"
#include "q1_internal.h"

namespace q1 {
namespace {

constexpr int kOnce = 2;                // cache hint of a buffer load: not read again

__device__ __forceinline__ int64_t suffix_len(const q1_attn& a, int64_t b) {
  if (a.max_pages == 0 || a.pages == 0) return 0;
  const int64_t n = a.suffix_lens[b], most = a.max_pages * a.page_size;
  return n < 0 ? 0 : n > most ? most : n;
}

// Rows of an item: row r of its R belongs to (sequence, query head).
struct Rows {
  int64_t b0;
  int hk, group, R, row0;
  bool prefix;
  __device__ __forceinline__ int64_t seq(int r) const { return prefix ? r / group : b0; }
  __device__ __forceinline__ int head(int r) const { return hk * group + (prefix ? r % group : r); }
};

template <int D>
__device__ __forceinline__ u32x4 load_q(const q1_attn& a, const Rows& w, int r, int s, int grp) {
  if (r >= w.R) return u32x4{0u, 0u, 0u, 0u};
  return *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(a.q) + w.seq(r) * a.q_ld + (int64_t)w.head(r) * D +
                                         32 * s + 8 * grp);
}

// Queries stay in registers where they fit beside the output (D = 256: in LDS).
template <int D>
constexpr bool kQueriesInLds = D == 256;

template <int D, int NM>
constexpr int kTokenLds() {
  constexpr int q = kQueriesInLds<D> ? 16 * NM * (2 * D + 16) : 0;
  constexpr int vt = kWaves * kTile * (2 * D + 32) + q, jo = kWaves * 16 * NM * ((D + 4) * 4 + 8);
  return vt > jo ? vt : jo;
}

template <int D>
constexpr int kRowLds() {
  return 2 * kTile * ((2 * D + 16) + (2 * D + 32));
}

// Rows [0, n) of a strided operand: loads past them give zeros.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_of(const void* base, int64_t n, int64_t ld_bytes, int width_bytes) {
  const int bytes = n > 0 ? (int)((n < kTile ? n : kTile) - 1) * (int)ld_bytes + width_bytes : 0;
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, bytes, 0x00020000);
}

// An item by tokens.
template <bool F16, int D, int NM, bool PREFIX>
__device__ __forceinline__ void item_by_tokens(const q1_attn& a, const Rows& w, int64_t t0, int64_t t1, int64_t base,
                                               float* part_o, float2* part_ml, unsigned char* lds) {
  constexpr int KS = D / 32, DT = D / 16, VROW = 2 * D + 32;  // LDS bytes of a value row: rows start 8 banks apart
  constexpr int VCH = D / 8, VPI = 64 / VCH, VN = kTile / VPI;  // 16-byte pieces a row, rows and loads of a value tile
  constexpr bool QL = kQueriesInLds<D>;
  constexpr int QROW = 2 * D + 16;
  const int lane = threadIdx.x & 63, col = lane & 15, grp = lane >> 4;
  // in a scalar register: matrix-core products ignore the lane mask, so the loop they are in must be a scalar one
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  unsigned char* const ql = lds + kWaves * kTile * VROW;
  u32x4 Q[QL ? 1 : NM][QL ? 1 : KS];
  if constexpr (QL) {
    for (int i = threadIdx.x; i < 16 * NM * VCH; i += 64 * kWaves) {
      const int r = i / VCH, c = i % VCH;
      *reinterpret_cast<u32x4*>(ql + r * QROW + 16 * c) = load_q<D>(a, w, w.row0 + r, c >> 2, c & 3);
    }
    __syncthreads();
  } else {
#pragma unroll
    for (int n = 0; n < NM; ++n)
#pragma unroll
      for (int s = 0; s < KS; ++s) Q[n][s] = load_q<D>(a, w, w.row0 + 16 * n + col, s, grp);
  }

  const auto* kb = static_cast<const uint16_t*>(PREFIX ? a.k_prefix : a.k_pages) + (int64_t)w.hk * D;
  const auto* vb = static_cast<const uint16_t*>(PREFIX ? a.v_prefix : a.v_pages) + (int64_t)w.hk * D;
  const int64_t ld = PREFIX ? a.prefix_ld : (int64_t)a.Hkv * D;
  // Suffix: the page row of token t + (lane % 32), -1 if it does not count.
  auto row_of = [&](int64_t t) -> int {
    const int64_t tok = t + (lane & 31), last = t1 - 1;
    const uint32_t ps = (uint32_t)a.page_size, at = (uint32_t)(tok < last ? tok : last), pg = at / ps;
    const int id = a.page_table[w.b0 * a.max_pages + pg];
    return tok > last || id < 0 || id >= a.pages ? -1 : (int)((int64_t)id * ps + (at - pg * ps));
  };

  u32x4 K[2][KS], V[VN];
  int rows = 0;
  auto load_k = [&](int64_t t) {
    if constexpr (PREFIX) {
      const auto r = rows_of(kb + t * ld, t1 - t, ld * 2, 2 * D);
      const int at = col * (int)ld * 2 + 16 * grp;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int s = 0; s < KS; ++s)
          K[h][s] = __builtin_amdgcn_raw_buffer_load_b128(r, at + 16 * h * (int)ld * 2 + 64 * s, 0, kOnce);
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = __shfl(rows, 16 * h + col);
        const u32x4* k = reinterpret_cast<const u32x4*>(kb + (r < 0 ? 0 : r) * ld) + grp;
#pragma unroll
        for (int s = 0; s < KS; ++s) K[h][s] = k[4 * s];
      }
    }
  };
  auto load_v = [&](int64_t t) {
    if constexpr (PREFIX) {
      const auto r = rows_of(vb + t * ld, t1 - t, ld * 2, 2 * D);
      const int at = (lane / VCH) * (int)ld * 2 + 16 * (lane % VCH);
#pragma unroll
      for (int i = 0; i < VN; ++i) V[i] = __builtin_amdgcn_raw_buffer_load_b128(r, at + i * VPI * (int)ld * 2, 0, kOnce);
    } else {
#pragma unroll
      for (int i = 0; i < VN; ++i) {
        const int r = __shfl(rows, i * VPI + lane / VCH);
        V[i] = reinterpret_cast<const u32x4*>(vb + (r < 0 ? 0 : r) * ld)[lane % VCH];
      }
    }
  };

  f32x4 O[DT][NM];
  float m[NM], l[NM];
#pragma unroll
  for (int n = 0; n < NM; ++n) {
    m[n] = -INFINITY;
    l[n] = 0.f;
#pragma unroll
    for (int d = 0; d < DT; ++d) O[d][n] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  unsigned char* vt = lds + wave * (kTile * VROW);
  unsigned char* vw = vt + (lane / VCH) * VROW + 16 * (lane % VCH);
  const unsigned char* vr = vt + (4 * grp + col / 4) * VROW + 8 * (col & 3);
  const float sc = a.scale * kLog2e;

  int64_t t = t0 + wave * kTile;
  if (t < t1) {
    if constexpr (!PREFIX) rows = row_of(t);
    load_k(t);
    load_v(t);
  }
  for (; t < t1; t += kStep) {
    // which tokens of the tile count
    uint32_t in;
    if constexpr (PREFIX) in = t1 - t >= kTile ? ~0u : (1u << (int)(t1 - t)) - 1u;
    else in = (uint32_t)__ballot(rows >= 0);
    const int have = rows;
    const int64_t tn = t + kStep;
    if constexpr (!PREFIX) rows = row_of(tn);
    // scores, then the next tile's keys
    f32x4 S[NM][2];
#pragma unroll
    for (int n = 0; n < NM; ++n)
#pragma unroll
      for (int h = 0; h < 2; ++h) S[n][h] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
      for (int n = 0; n < NM; ++n) {
        u32x4 q;
        if constexpr (QL) q = *reinterpret_cast<const u32x4*>(ql + (16 * n + col) * QROW + 64 * s + 16 * grp);
        else q = Q[n][s];
#pragma unroll
        for (int h = 0; h < 2; ++h) S[n][h] = mma<F16>(K[h][s], q, S[n][h]);
      }
    load_k(tn);
#pragma unroll
    for (int i = 0; i < VN; ++i) {
      if constexpr (!PREFIX) {  // values of tokens that do not count (anything) are zeros
        const int r = __shfl(have, i * VPI + lane / VCH);
#pragma unroll
        for (int e = 0; e < 4; ++e) V[i][e] = r < 0 ? 0u : V[i][e];
      }
      *reinterpret_cast<u32x4*>(vw + i * VPI * VROW) = V[i];
    }
    load_v(tn);
    const uint32_t mine = (in >> (4 * grp) & 15u) | (in >> (16 + 4 * grp) & 15u) << 4;
    u32x4 hi[NM], lo[NM];
#pragma unroll
    for (int n = 0; n < NM; ++n)
      weigh<F16, DT>(S[n], mine, sc, m[n], l[n], &O[0][n], NM, hi[n], lo[n]);
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int d = 0; d < DT; ++d) {
      const u32x4 v = transposed(vr + 32 * d, 16 * VROW);
#pragma unroll
      for (int n = 0; n < NM; ++n)
        O[d][n] = mma<F16>(v, hi[n], O[d][n]);
#pragma unroll
      for (int n = 0; n < NM; ++n)
        O[d][n] = mma<F16>(v, lo[n], O[d][n]);
    }
    __builtin_amdgcn_wave_barrier();
  }

  // Join the waves in LDS (over the value tiles) and store the item's part.
  constexpr int OROW = D + 4;
  float* so = reinterpret_cast<float*>(lds);
  float2* sml = reinterpret_cast<float2*>(so + kWaves * 16 * NM * OROW);
  __syncthreads();
#pragma unroll
  for (int n = 0; n < NM; ++n) {
    const int r = wave * 16 * NM + 16 * n + col;
    const float sum = sum_groups(l[n]);
    if (grp == 0) sml[r] = float2{m[n], sum};
#pragma unroll
    for (int d = 0; d < DT; ++d) *reinterpret_cast<f32x4*>(so + r * OROW + 16 * d + 4 * grp) = O[d][n];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 16 * NM * (D / 4); i += 64 * kWaves) {
    const int r = i / (D / 4), c = 4 * (i % (D / 4));
    if (w.row0 + r >= w.R) continue;
    float top = -INFINITY;
#pragma unroll
    for (int v = 0; v < kWaves; ++v) top = fmaxf(top, sml[v * 16 * NM + r].x);
    f32x4 o = {0.f, 0.f, 0.f, 0.f};
    float sum = 0.f;
#pragma unroll
    for (int v = 0; v < kWaves; ++v) {
      const float2 ml = sml[v * 16 * NM + r];
      const float f = top == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(ml.x - top);
      o += f * *reinterpret_cast<const f32x4*>(so + (v * 16 * NM + r) * OROW + c);
      sum += f * ml.y;
    }
    const int64_t at = base + w.seq(w.row0 + r) * a.Hq + w.head(w.row0 + r);
    *reinterpret_cast<f32x4*>(part_o + at * D + c) = o;
    if (c == 0) part_ml[at] = float2{top, sum};
  }
}

// A prefix item by rows: wave w has rows row0 + 16 w .. +15.
template <bool F16, int D>
__device__ __forceinline__ void item_by_rows(const q1_attn& a, const Rows& w, int64_t t0, int64_t t1, int64_t base,
                                             float* part_o, float2* part_ml, unsigned char* lds) {
  constexpr int KS = D / 32, DT = D / 16, KROW = 2 * D + 16, VROW = 2 * D + 32, BUF = kTile * (KROW + VROW);
  constexpr int CH = D / 8, N = kTile * CH / (64 * kWaves);  // 16-byte pieces a row, loads of a tile per thread
  const int tid = threadIdx.x, lane = tid & 63, col = lane & 15, grp = lane >> 4;
  const int r = w.row0 + 16 * __builtin_amdgcn_readfirstlane(tid >> 6) + col;
  u32x4 Q[KS];
#pragma unroll
  for (int s = 0; s < KS; ++s) Q[s] = load_q<D>(a, w, r, s, grp);
  const auto* kb = static_cast<const uint16_t*>(a.k_prefix) + (int64_t)w.hk * D;
  const auto* vb = static_cast<const uint16_t*>(a.v_prefix) + (int64_t)w.hk * D;
  u32x4 K[N], V[N];
  const int ld = (int)a.prefix_ld * 2, at0 = (tid / CH) * ld + 16 * (tid % CH);
  auto load = [&](int64_t t) {
    const auto rk = rows_of(kb + t * a.prefix_ld, t1 - t, ld, 2 * D), rv = rows_of(vb + t * a.prefix_ld, t1 - t, ld, 2 * D);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      K[i] = __builtin_amdgcn_raw_buffer_load_b128(rk, at0 + i * (64 * kWaves / CH) * ld, 0, 0);
      V[i] = __builtin_amdgcn_raw_buffer_load_b128(rv, at0 + i * (64 * kWaves / CH) * ld, 0, 0);
    }
  };
  auto put = [&](unsigned char* buf) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int row = (i * 64 * kWaves + tid) / CH, c = tid % CH;
      *reinterpret_cast<u32x4*>(buf + row * KROW + 16 * c) = K[i];
      *reinterpret_cast<u32x4*>(buf + kTile * KROW + row * VROW + 16 * c) = V[i];
    }
  };
  f32x4 O[DT];
  float m = -INFINITY, l = 0.f;
#pragma unroll
  for (int d = 0; d < DT; ++d) O[d] = f32x4{0.f, 0.f, 0.f, 0.f};
  const float sc = a.scale * kLog2e;
  load(t0);
  put(lds);
  load(t0 + kTile);
  __syncthreads();
  int at = 0;
  for (int64_t t = t0; t < t1; t += kTile, at ^= BUF) {
    // the next tile to the other buffer, the one after it into registers
    put(lds + (at ^ BUF));
    load(t + 2 * kTile);
    const unsigned char* buf = lds + at;
    f32x4 S[2] = {f32x4{0.f, 0.f, 0.f, 0.f}, f32x4{0.f, 0.f, 0.f, 0.f}};
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        S[h] = mma<F16>(*reinterpret_cast<const u32x4*>(buf + (16 * h + col) * KROW + 64 * s + 16 * grp), Q[s], S[h]);
    const uint32_t in = t1 - t >= kTile ? ~0u : (1u << (int)(t1 - t)) - 1u;
    const uint32_t mine = (in >> (4 * grp) & 15u) | (in >> (16 + 4 * grp) & 15u) << 4;
    u32x4 hi, lo;
    weigh<F16, DT>(S, mine, sc, m, l, O, 1, hi, lo);
    const unsigned char* vr = buf + kTile * KROW + (4 * grp + col / 4) * VROW + 8 * (col & 3);
#pragma unroll
    for (int d = 0; d < DT; ++d) {
      const u32x4 v = transposed(vr + 32 * d, 16 * VROW);
      O[d] = mma<F16>(v, hi, O[d]);
      O[d] = mma<F16>(v, lo, O[d]);
    }
    __syncthreads();
  }
  const float sum = sum_groups(l);
  if (r >= w.R) return;
  const int64_t out = base + w.seq(r) * a.Hq + w.head(r);
  if (grp == 0) part_ml[out] = float2{m, sum};
#pragma unroll
  for (int d = 0; d < DT; ++d) *reinterpret_cast<f32x4*>(part_o + out * D + 16 * d + 4 * grp) = O[d];
}

// NM: blocks of 16 rows of an item by tokens.
template <bool F16, int D, int NM, bool BYROWS>
__global__ __launch_bounds__(64 * kWaves, NM * D > 256 ? 1 : 2) void q1_attn_main(const q1_attn a, const AttnPlan p, float* part_o, float2* part_ml) {
  extern __shared__ __align__(16) unsigned char lds[];
  Rows w;
  w.group = a.Hq / a.Hkv;
  w.prefix = blockIdx.x < (unsigned)p.prefix_wgs;
  w.b0 = 0;
  int64_t t0, t1;
  int split;
  if (w.prefix) {
    // blocks of rows over the same tokens are 8 workgroups apart: the same XCD's L2
    const int x = blockIdx.x & 7, y = blockIdx.x >> 3;
    const int pair = (y / p.prefix_rb) * 8 + x;
    if (pair >= a.Hkv * p.prefix_splits) return;
    w.hk = pair / p.prefix_splits;  // (an XCD reads a range of tokens for all heads: whole rows)
    split = pair % p.prefix_splits;
    w.R = (int)a.B * w.group;
    w.row0 = (y % p.prefix_rb) * (BYROWS ? 16 * kWaves : 16 * NM);
    t0 = (int64_t)split * p.prefix_tokens;
    t1 = t0 + p.prefix_tokens < a.P ? t0 + p.prefix_tokens : a.P;
  } else {
    int64_t i = blockIdx.x - p.prefix_wgs;
    w.hk = (int)(i % a.Hkv);
    i /= a.Hkv;
    w.row0 = (int)(i % p.suffix_rb) * 16 * NM;
    i /= p.suffix_rb;
    split = (int)(i % p.suffix_splits);
    w.b0 = i / p.suffix_splits;
    w.R = w.group;
    const int64_t n = suffix_len(a, w.b0);
    t0 = (int64_t)split * p.suffix_tokens;
    t1 = t0 + p.suffix_tokens < n ? t0 + p.suffix_tokens : n;
    split += p.prefix_splits;
    if (t0 >= t1) return;
  }
  const int64_t base = (int64_t)split * a.B * a.Hq;
  if constexpr (BYROWS) {
    if (w.prefix) item_by_rows<F16, D>(a, w, t0, t1, base, part_o, part_ml, lds);
    else item_by_tokens<F16, D, NM, false>(a, w, t0, t1, base, part_o, part_ml, lds);
  } else if (w.prefix) {
    item_by_tokens<F16, D, NM, true>(a, w, t0, t1, base, part_o, part_ml, lds);
  } else {
    item_by_tokens<F16, D, NM, false>(a, w, t0, t1, base, part_o, part_ml, lds);
  }
}

// One workgroup per (sequence, query head) adds its parts (at most 128): every wave
// finds the parts' factors, two per lane, and sums every fourth part.
template <int D>
__global__ __launch_bounds__(64 * kWaves) void q1_attn_join(const q1_attn a, const AttnPlan p, const float* part_o,
                                                            const float2* part_ml, float lift) {
  constexpr int E = D / 64;
  __shared__ float so[kWaves][D];
  const int64_t row = blockIdx.x, rows = a.B * a.Hq;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t n = suffix_len(a, row / a.Hq);
  const int parts = p.prefix_splits + (int)((n + p.suffix_tokens - 1) / p.suffix_tokens);
  const float2 none = {-INFINITY, 0.f};
  const float2 ml0 = lane < parts ? part_ml[lane * rows + row] : none;
  const float2 ml1 = lane + 64 < parts ? part_ml[(lane + 64) * rows + row] : none;
  float top = fmaxf(ml0.x, ml1.x);
  for (int off = 32; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor(top, off));
  const float base = top == -INFINITY ? 0.f : top;
  const float f0 = __builtin_amdgcn_exp2f(ml0.x - base), f1 = __builtin_amdgcn_exp2f(ml1.x - base);
  float sum = f0 * ml0.y + f1 * ml1.y;
  for (int off = 32; off > 0; off >>= 1) sum += __shfl_xor(sum, off);
  float o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
  for (int s0 = wave; s0 < parts; s0 += 4 * kWaves) {  // four parts' loads at a time
    float x[4][E];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int s = s0 + u * kWaves < parts ? s0 + u * kWaves : parts - 1;
      const float* po = part_o + (s * rows + row) * D + lane;
#pragma unroll
      for (int e = 0; e < E; ++e) x[u][e] = po[64 * e];
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int s = s0 + u * kWaves;
      const float f = s < parts ? __shfl(s < 64 ? f0 : f1, s & 63) : 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = __builtin_fmaf(f, x[u][e], o[e]);
    }
  }
#pragma unroll
  for (int e = 0; e < E; ++e) so[wave][64 * e + lane] = o[e];
  __syncthreads();
  const bool nothing = sum == 0.f;  // no token, or none above -infinity (a NaN stays one)
  const float inv = nothing ? 0.f : 1.0f / sum;
  if (threadIdx.x < D) {
    float t = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) t += so[w][threadIdx.x];
    store_out(a.out, a.out_dtype, row * D + threadIdx.x, t * inv);
  }
  if (threadIdx.x == 0 && a.lse != nullptr)
    a.lse[row] = nothing ? -INFINITY : (top - lift) * 0.69314718055994530942f + logf(sum);
}

template <bool F16, int D, int NM, bool BYROWS>
hipError_t launch(const q1_attn& a, const AttnPlan& p, float* po, float2* pml, hipStream_t s) {
  constexpr int tokens = kTokenLds<D, NM>(), rows = BYROWS ? kRowLds<D>() : 0;
  constexpr int bytes = tokens > rows ? tokens : rows;
  static const hipError_t attr = hipFuncSetAttribute(reinterpret_cast<const void*>(&q1_attn_main<F16, D, NM, BYROWS>),
                                                     hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (attr != hipSuccess) return attr;
  if (p.wgs > 0)
    hipLaunchKernelGGL((q1_attn_main<F16, D, NM, BYROWS>), dim3((unsigned)p.wgs), dim3(64 * kWaves), bytes, s, a, p, po, pml);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((q1_attn_join<D>), dim3((unsigned)(a.B * a.Hq)), dim3(64 * kWaves), 0, s, a, p, po, pml, kLift<F16>);
  return hipGetLastError();
}

template <bool F16, int D>
hipError_t launch_d(const q1_attn& a, const AttnPlan& p, float* po, float2* pml, hipStream_t s) {
  if (p.by_rows) return launch<F16, D, 1, true>(a, p, po, pml, s);
  return p.nm == 1 ? launch<F16, D, 1, false>(a, p, po, pml, s) : launch<F16, D, 2, false>(a, p, po, pml, s);
}

template <bool F16>
hipError_t launch_t(const q1_attn& a, const AttnPlan& p, float* po, float2* pml, hipStream_t s) {
  return a.D == 64 ? launch_d<F16, 64>(a, p, po, pml, s) : a.D == 128 ? launch_d<F16, 128>(a, p, po, pml, s) : launch_d<F16, 256>(a, p, po, pml, s);
}

int64_t up_div(int64_t x, int64_t y) { return (x + y - 1) / y; }

}  // namespace

// Few rows (up to 32 of them share a key/value head): items by tokens, all rows in
// an item; more: prefix items by rows, 64 a block, suffix items by tokens.  Measured at
// 32 rows, D = 128: over 65537 tokens by tokens 65 us, by rows 70 (8 heads, fp16, from
// HBM), 25 and 35 (1 head); but over 8000 tokens that caches hold 20 and 16, and with
// D = 256 and 30 rows 21 and 17.  Past 32, two blocks by tokens read the prefix twice:
// 36 rows over 8000 tokens 21 us, by rows 17 (D = 256: 23 and 18); over 1000 tokens equal
// (10.5), and at 64 rows 11 and 13.  (128 rows a block, two blocks a wave: 62 against
// 45 us at 192 rows of D = 256 over 8201 tokens, where it leaves one workgroup a CU,
// 41 against 38 us at 384 rows of D = 128 over 4000.)
AttnPlan plan_prefix_attn(const q1_attn& a) {
  AttnPlan p = {};
  const int64_t group = a.Hq / a.Hkv, R = a.P > 0 ? a.B * group : group;
  p.by_rows = a.P > 0 && R > 32;
  p.nm = !p.by_rows && R > 16 ? 2 : 1;
  p.prefix_rb = (int)up_div(a.B * group, 16 * p.nm * (p.by_rows ? kWaves : 1));
  p.suffix_rb = (int)up_div(group, 16 * p.nm);
  // units of work: kStep tokens by tokens, kTile by rows (about as long)
  const int64_t most = a.max_pages * a.page_size, punit = p.by_rows ? kTile : kStep;
  const int64_t pit = up_div(a.P, punit), sit = up_div(most, kStep);
  const int64_t total = pit * a.Hkv * p.prefix_rb + sit * a.B * a.Hkv * p.suffix_rb;
  const int64_t slots = (int64_t)device_cus() * (p.nm * a.D > 256 ? 1 : 2);  // workgroups at a time
  // units per item: the fewest with which all items run at a time (a second round of
  // workgroups would start when the first ends), at most 64 parts of a kind per row
  for (int64_t per = up_div(total, slots) > 1 ? up_div(total, slots) : 1;; per += up_div(per, 16)) {
    const int64_t pper = up_div(pit, 64) > per ? up_div(pit, 64) : per, sper = up_div(sit, 64) > per ? up_div(sit, 64) : per;
    p.prefix_splits = (int)up_div(pit, pper);
    p.prefix_tokens = pper * punit;
    p.suffix_splits = (int)up_div(sit, sper);
    p.suffix_tokens = sper * kStep;
    p.prefix_wgs = up_div(a.Hkv * (int64_t)p.prefix_splits, 8) * 8 * p.prefix_rb;
    p.wgs = p.prefix_wgs + (int64_t)p.suffix_splits * a.B * a.Hkv * p.suffix_rb;
    if (p.wgs <= slots || per >= 2 * up_div(total, slots)) break;
  }
  const size_t rows = (size_t)(p.prefix_splits + p.suffix_splits) * a.B * a.Hq;
  p.ml_off = (rows * a.D * 4 + 255) / 256 * 256;
  p.ws_bytes = p.ml_off + (rows * 8 + 255) / 256 * 256;
  return p;
}

hipError_t launch_prefix_attn(const q1_attn& a, const AttnPlan& p, unsigned char* ws, hipStream_t s) {
  float* po = reinterpret_cast<float*>(ws);
  float2* pml = reinterpret_cast<float2*>(ws + p.ml_off);
  return a.dtype == Q1_F16 ? launch_t<true>(a, p, po, pml, s) : launch_t<false>(a, p, po, pml, s);
}

}  // namespace q1
