// Attention over keys and values held in 4 or 8 bits (q1_memory.h).
//
// Two launches: q1_kv_main computes, per work item, the running maximum m, sum l and
// unnormalised output o of a block of query rows (the T * Hq/Hkv rows that share a
// key/value head of a sequence) over some tokens; q1_kv_join adds the items of a
// row.  Where the tokens are not split, the item writes the row itself.
//
// In an item each of the 4 waves takes every fourth tile of 32 tokens, by itself, and
// the waves are joined in LDS.  Codes go to bf16 in registers, which is exact, so the
// products are the ones of 16-bit attention (see q1_attn.hip for their layouts):
//   S^T = K Q^T   a lane has a quarter of the elements of one token in a row of bytes
//                 (for D = 128 one block with its scale), 8 of them a product: the
//                 order of the elements is free as long as the queries have it too.
//   O^T = V^T P^T values are loaded as keys are, go to LDS as bf16 rows and come back
//                 transposed.
// fp16 queries enter as two bf16 parts (11 bits of significand are 8 and 3), weights
// as two (2^-17).
//
// A token that a query does not see has the score -infinity, whatever its key.  Its
// weight 0 would still make a NaN of a NaN value, so a tile with a NaN block of values
// (a branch that hardly ever is taken) has zeros there, and the block's columns are
// made NaN for the queries that see the token.
//
// Bound by the bytes of the pages where rows are few.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "q1_attn_tile.h"
#include "q1_device.h"
#include "q1_internal.h"
#include "q1_kv_device.h"
#include "q1_memory.h"

namespace q1 {
namespace {

struct KvArgs {
  q1_kv c;
  q1_kv_query a;
  KvPlan p;
  float* part_o;
  float2* part_ml;
};

__device__ __forceinline__ int64_t length_of(const KvArgs& g, int64_t b) {
  if (g.c.pages == 0) return 0;
  const int64_t n = g.a.lens[b], most = g.a.max_pages * g.c.page_size;
  return n < 0 ? 0 : n > most ? most : n;
}

// Tokens that row r (of the T * group of a sequence and key/value head) sees.
__device__ __forceinline__ int64_t seen_by(const KvArgs& g, int64_t n, int64_t r, int group) {
  const int64_t s = n - (g.a.T - 1 - r / group);
  return s < 0 ? 0 : s;
}

// Queries stay in registers where they fit beside the output (D = 256: in LDS).
template <int D>
constexpr bool kQueriesInLds = D == 256;

template <int D, int NM, int QP>
constexpr int kMainLds() {
  constexpr int q = kQueriesInLds<D> ? 16 * NM * (2 * D * QP + 16) : 0;
  constexpr int vt = kWaves * kTile * (2 * D + 32) + q, jo = kWaves * 16 * NM * ((D + 4) * 4 + 8);
  return vt > jo ? vt : jo;
}

// 8 elements of a query row from element d on, as bf16 parts.
template <bool F16, int QP>
__device__ __forceinline__ void load_q(const KvArgs& g, int64_t b, int hk, int group, int64_t R, int64_t r, int d, u32x4* q) {
  u32x4 w = {0u, 0u, 0u, 0u};
  if (r < R) {
    const int64_t t = r / group;
    const int h = hk * group + (int)(r - t * group);
    w = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(g.a.q) + (b * g.a.T + t) * g.a.q_ld + (int64_t)h * g.c.D + d);
  }
  if constexpr (!F16) {
    q[0] = w;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float rx, ry, x0, x1;
      q[0][j] = round2<false>(f16_bits_to_f32(w[j] & 0xffffu), f16_bits_to_f32(w[j] >> 16), &rx, &ry);
      q[QP - 1][j] = round2<false>(rx, ry, &x0, &x1);
    }
  }
}

// What one lane holds of a tile: a quarter of the tokens col and 16 + col.
template <int BITS, int D>
struct Tile {
  static constexpr int KS = D / 32, W = D * BITS / 128, NB = D / 128 > 1 ? D / 128 : 1;  // products, dwords, scales a token
  uint32_t k[2][W], v[2][W];
  uint32_t ks[2], vs[2];  // NB scale bytes
  bool ok[2];             // the token counts
};

template <int BITS, int D>
__device__ __forceinline__ void load_tile(const q1_kv& c, const int64_t* page, const uint32_t* off, int grp, Tile<BITS, D>& x) {
  constexpr int W = Tile<BITS, D>::W, NB = Tile<BITS, D>::NB;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t row = page[h] + off[h];
    const unsigned char* kp = static_cast<const unsigned char*>(c.k) + row * (D * BITS / 8) + grp * (4 * W);
    const unsigned char* vp = static_cast<const unsigned char*>(c.v) + row * (D * BITS / 8) + grp * (4 * W);
    if constexpr (W == 2) {
      const uint2 kw = *reinterpret_cast<const uint2*>(kp), vw = *reinterpret_cast<const uint2*>(vp);
      x.k[h][0] = kw.x, x.k[h][1] = kw.y, x.v[h][0] = vw.x, x.v[h][1] = vw.y;
    } else {
#pragma unroll
      for (int i = 0; i < W / 4; ++i) {
        const u32x4 kw = reinterpret_cast<const u32x4*>(kp)[i], vw = reinterpret_cast<const u32x4*>(vp)[i];
#pragma unroll
        for (int j = 0; j < 4; ++j) x.k[h][4 * i + j] = kw[j], x.v[h][4 * i + j] = vw[j];
      }
    }
    const int64_t at = row * (D / kKvBlock) + (D == 64 ? grp >> 1 : grp * NB);
    const unsigned char* ksp = static_cast<const unsigned char*>(c.k_scales) + at;
    const unsigned char* vsp = static_cast<const unsigned char*>(c.v_scales) + at;
    if constexpr (NB == 2) {
      x.ks[h] = *reinterpret_cast<const uint16_t*>(ksp);
      x.vs[h] = *reinterpret_cast<const uint16_t*>(vsp);
    } else {
      x.ks[h] = *ksp;
      x.vs[h] = *vsp;
    }
  }
}

template <bool F16, int BITS, int D, int NM>
__global__ __launch_bounds__(64 * kWaves) void q1_kv_main(const KvArgs g) {
  constexpr int QP = F16 ? 2 : 1;
  using T = Tile<BITS, D>;
  constexpr int KS = T::KS, W = T::W, NB = T::NB, DT = D / 16, VROW = 2 * D + 32, QROW = 2 * D * QP + 16;
  constexpr bool QL = kQueriesInLds<D>;
  extern __shared__ unsigned char lds[];
  const q1_kv& c = g.c;
  const q1_kv_query& a = g.a;
  const int lane = threadIdx.x & 63, col = lane & 15, grp = lane >> 4;
  // in a scalar register: matrix-core products ignore the lane mask, so the loop they are in must be a scalar one
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

  int64_t i = blockIdx.x;
  const int hk = (int)(i % c.Hkv);
  i /= c.Hkv;
  const int rb = (int)(i % g.p.row_blocks);
  i /= g.p.row_blocks;
  const int split = (int)(i % g.p.splits);
  const int64_t b = i / g.p.splits;
  const int group = a.Hq / c.Hkv;
  const int64_t R = a.T * group, row0 = (int64_t)rb * 16 * NM;
  const int64_t n = length_of(g, b);
  // tokens that the block's last row sees: no row of it needs more
  const int64_t most = seen_by(g, n, row0 + 16 * NM < R ? row0 + 16 * NM - 1 : R - 1, group);
  const int64_t t0 = (int64_t)split * g.p.tokens;
  const int64_t t1 = t0 + g.p.tokens < most ? t0 + g.p.tokens : most;
  const bool direct = g.p.splits == 1;
  if (t0 >= t1 && !direct) return;

  unsigned char* const ql = lds + kWaves * kTile * VROW;
  u32x4 Q[QL ? 1 : NM][QL ? 1 : KS][QP];
  if constexpr (QL) {
    for (int x = threadIdx.x; x < 16 * NM * (D / 8); x += 64 * kWaves) {
      const int r = x / (D / 8), e = x % (D / 8);
      u32x4 q[QP];
      load_q<F16, QP>(g, b, hk, group, R, row0 + r, 8 * e, q);
#pragma unroll
      for (int s = 0; s < QP; ++s) *reinterpret_cast<u32x4*>(ql + r * QROW + s * 2 * D + 16 * e) = q[s];
    }
    __syncthreads();
  } else {
#pragma unroll
    for (int m = 0; m < NM; ++m)
#pragma unroll
      for (int s = 0; s < KS; ++s) load_q<F16, QP>(g, b, hk, group, R, row0 + 16 * m + col, grp * (D / 4) + 8 * s, Q[m][s]);
  }

  // The pages of this lane's two tokens of a tile, and their place in the page.
  const uint32_t last = (uint32_t)(t1 - 1);
  auto ids_of = [&](int64_t t, int32_t* id, uint32_t* off) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t tok = t + 16 * h + col;
      const uint32_t at = tok < t1 ? (uint32_t)tok : last, pg = divide(at, g.p.page);
      id[h] = a.page_table[b * a.max_pages + pg];
      off[h] = at - pg * (uint32_t)c.page_size;
    }
  };
  auto fetch = [&](int64_t t, const int32_t* id, const uint32_t* off, T& x) {
    int64_t page[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const bool in = id[h] >= 0 && id[h] < c.pages;
      x.ok[h] = in && t + 16 * h + col < t1;
      page[h] = ((int64_t)(in ? id[h] : 0) * c.Hkv + hk) * c.page_size;
    }
    load_tile<BITS, D>(c, page, off, grp, x);
  };

  f32x4 O[DT][NM];
  float m[NM], l[NM];
  int64_t lim[NM];  // tokens that this lane's query sees
#pragma unroll
  for (int x = 0; x < NM; ++x) {
    m[x] = -INFINITY;
    l[x] = 0.f;
    const int64_t r = row0 + 16 * x + col;
    lim[x] = seen_by(g, n, r < R ? r : R - 1, group);
#pragma unroll
    for (int d = 0; d < DT; ++d) O[d][x] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  unsigned char* const vt = lds + wave * (kTile * VROW);
  unsigned char* const vw = vt + col * VROW + grp * (D / 2);
  const unsigned char* const vr = vt + (4 * grp + col / 4) * VROW + 8 * (col & 3);
  const float sc = a.scale * kLog2e;

  auto work = [&](int64_t t, T& x) {
    // which tokens of the tile count
    const uint32_t in = (uint32_t)(__ballot(x.ok[0]) & 0xffffu) | (uint32_t)(__ballot(x.ok[1]) & 0xffffu) << 16;
    f32x4 S[NM][2];
#pragma unroll
    for (int q = 0; q < NM; ++q)
#pragma unroll
      for (int h = 0; h < 2; ++h) S[q][h] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      u32x4 K[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t e = NB == 2 ? (x.ks[h] >> (8 * (s / (KS / NB)))) & 255u : x.ks[h];
        K[h] = kv_bf16<BITS>(&x.k[h][s * (BITS / 4)], kv_scale(e));
      }
#pragma unroll
      for (int q = 0; q < NM; ++q)
#pragma unroll
        for (int y = 0; y < QP; ++y) {
          u32x4 w;
          if constexpr (QL) w = *reinterpret_cast<const u32x4*>(ql + (16 * q + col) * QROW + y * 2 * D + grp * (D / 2) + 16 * s);
          else w = Q[q][s][y];
#pragma unroll
          for (int h = 0; h < 2; ++h) S[q][h] = mma<false>(K[h], w, S[q][h]);
        }
    }
    // values to LDS; those of tokens that do not count (anything), and NaN blocks, as zeros
    uint64_t nan[2][NB];
    bool some = false;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        const uint32_t e = (x.vs[h] >> (8 * j)) & 255u;
        nan[h][j] = __ballot(x.ok[h] && e == 255u);
        some = some || nan[h][j] != 0;
        const bool use = x.ok[h] && e != 255u;
        const float scale = use ? __uint_as_float(e << 23) : 0.f;
#pragma unroll
        for (int s = 0; s < KS / NB; ++s) {
          uint32_t w[2] = {x.v[h][(j * (KS / NB) + s) * (BITS / 4)], 0u};
          if constexpr (BITS == 8) {
            w[1] = x.v[h][(j * (KS / NB) + s) * 2 + 1];
            w[0] = use ? w[0] : 0u;  // (an E4M3 code may be a NaN by itself)
            w[1] = use ? w[1] : 0u;
          }
          *reinterpret_cast<u32x4*>(vw + h * 16 * VROW + (j * (KS / NB) + s) * 16) = kv_bf16<BITS>(w, scale);
        }
      }
    u32x4 hi[NM], lo[NM];
    uint32_t vis[NM];
#pragma unroll
    for (int q = 0; q < NM; ++q) {
      const int64_t d = lim[q] - t;
      vis[q] = in & (d >= 32 ? ~0u : d <= 0 ? 0u : ~0u >> (32 - (int)d));
      const uint32_t mine = (vis[q] >> (4 * grp) & 15u) | (vis[q] >> (16 + 4 * grp) & 15u) << 4;
      weigh<false, DT>(S[q], mine, sc, m[q], l[q], &O[0][q], NM, hi[q], lo[q]);
    }
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int d = 0; d < DT; ++d) {
      const u32x4 v = transposed(vr + 32 * d, 16 * VROW);
#pragma unroll
      for (int q = 0; q < NM; ++q) O[d][q] = mma<false>(v, hi[q], O[d][q]);
#pragma unroll
      for (int q = 0; q < NM; ++q) O[d][q] = mma<false>(v, lo[q], O[d][q]);
    }
    if (some) {
#pragma unroll
      for (int d = 0; d < DT; ++d) {
        const int blk = d / 2, sh = 16 * (D == 64 ? 2 * blk : blk / NB), j = blk % NB;
        const uint32_t bad = (uint32_t)(nan[0][j] >> sh & 0xffffu) | (uint32_t)(nan[1][j] >> sh & 0xffffu) << 16;
#pragma unroll
        for (int q = 0; q < NM; ++q)
          if (vis[q] & bad) O[d][q] = f32x4{NAN, NAN, NAN, NAN};
      }
    }
    __builtin_amdgcn_wave_barrier();
  };

  int64_t t = t0 + wave * kTile;
  if (t < t1) {
    T x, y;
    int32_t id[2];
    uint32_t off[2];
    ids_of(t, id, off);
    fetch(t, id, off, x);
    ids_of(t + kStep, id, off);
    for (; t < t1; t += 2 * kStep) {
      fetch(t + kStep, id, off, y);
      ids_of(t + 2 * kStep, id, off);
      work(t, x);
      if (t + kStep >= t1) break;
      fetch(t + 2 * kStep, id, off, x);
      ids_of(t + 3 * kStep, id, off);
      work(t + kStep, y);
    }
  }

  // Join the waves in LDS (over the value tiles) and store the item's part, or the row.
  constexpr int OROW = D + 4;
  float* so = reinterpret_cast<float*>(lds);
  float2* sml = reinterpret_cast<float2*>(so + kWaves * 16 * NM * OROW);
  __syncthreads();
#pragma unroll
  for (int q = 0; q < NM; ++q) {
    const int r = wave * 16 * NM + 16 * q + col;
    const float sum = sum_groups(l[q]);
    if (grp == 0) sml[r] = float2{m[q], sum};
#pragma unroll
    for (int d = 0; d < DT; ++d) *reinterpret_cast<f32x4*>(so + r * OROW + 16 * d + 4 * grp) = O[d][q];
  }
  __syncthreads();
  for (int x = threadIdx.x; x < 16 * NM * (D / 4); x += 64 * kWaves) {
    const int r = x / (D / 4), e = 4 * (x % (D / 4));
    if (row0 + r >= R) continue;
    float top = -INFINITY;
#pragma unroll
    for (int v = 0; v < kWaves; ++v) top = fmaxf(top, sml[v * 16 * NM + r].x);
    f32x4 o = {0.f, 0.f, 0.f, 0.f};
    float sum = 0.f;
#pragma unroll
    for (int v = 0; v < kWaves; ++v) {
      const float2 ml = sml[v * 16 * NM + r];
      const float f = top == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(ml.x - top);
      o += f * *reinterpret_cast<const f32x4*>(so + (v * 16 * NM + r) * OROW + e);
      sum += f * ml.y;
    }
    const int64_t tq = (row0 + r) / group;
    const int64_t row = (b * a.T + tq) * a.Hq + hk * group + (int)(row0 + r - tq * group);
    if (direct) {
      const bool nothing = sum == 0.f;
      const float inv = nothing ? 0.f : 1.0f / sum;
#pragma unroll
      for (int j = 0; j < 4; ++j) store_out(a.out, a.out_dtype, row * D + e + j, nothing ? 0.f : o[j] * inv);
      if (e == 0 && a.lse != nullptr) a.lse[row] = nothing ? -INFINITY : top * 0.69314718055994530942f + logf(sum);
    } else {
      const int64_t at = (int64_t)split * a.B * a.T * a.Hq + row;
      *reinterpret_cast<f32x4*>(g.part_o + at * D + e) = o;
      if (e == 0) g.part_ml[at] = float2{top, sum};
    }
  }
}

// One workgroup per (query, head) adds its parts: every wave finds the parts'
// factors, a part a lane, and sums every fourth part.
template <int D>
__global__ __launch_bounds__(64 * kWaves) void q1_kv_join(const KvArgs g, int rows_of_block) {
  constexpr int E = D / 64;
  __shared__ float so[kWaves][D];
  const q1_kv_query& a = g.a;
  const int64_t row = blockIdx.x, rows = a.B * a.T * a.Hq;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t bt = row / a.Hq, b = bt / a.T;
  const int group = a.Hq / g.c.Hkv, h = (int)(row - bt * a.Hq);
  const int64_t R = a.T * group, r = (bt - b * a.T) * group + h % group;
  const int64_t end = r / rows_of_block * rows_of_block + rows_of_block;  // of its block of rows
  const int64_t most = seen_by(g, length_of(g, b), (end < R ? end : R) - 1, group);
  const int parts = (int)((most + g.p.tokens - 1) / g.p.tokens);
  const float2 ml = lane < parts ? g.part_ml[lane * rows + row] : float2{-INFINITY, 0.f};
  float top = ml.x;
  for (int off = 32; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor(top, off));
  const float f0 = __builtin_amdgcn_exp2f(ml.x - (top == -INFINITY ? 0.f : top));
  float sum = f0 * ml.y;
  for (int off = 32; off > 0; off >>= 1) sum += __shfl_xor(sum, off);
  float o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
  for (int s0 = wave; s0 < parts; s0 += 4 * kWaves) {  // four parts' loads at a time
    float x[4][E];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int s = s0 + u * kWaves < parts ? s0 + u * kWaves : parts - 1;
      const float* po = g.part_o + (s * rows + row) * D + lane;
#pragma unroll
      for (int e = 0; e < E; ++e) x[u][e] = po[64 * e];
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int s = s0 + u * kWaves;
      const float f = __shfl(f0, s & 63);
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = s < parts ? __builtin_fmaf(f, x[u][e], o[e]) : o[e];
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
    store_out(a.out, a.out_dtype, row * D + threadIdx.x, nothing ? 0.f : t * inv);
  }
  if (threadIdx.x == 0 && a.lse != nullptr)
    a.lse[row] = nothing ? -INFINITY : top * 0.69314718055994530942f + logf(sum);
}

template <bool F16, int BITS, int D, int NM>
hipError_t launch(const KvArgs& g, hipStream_t s) {
  constexpr int bytes = kMainLds<D, NM, F16 ? 2 : 1>();
  static const hipError_t attr = hipFuncSetAttribute(reinterpret_cast<const void*>(&q1_kv_main<F16, BITS, D, NM>),
                                                     hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (attr != hipSuccess) return attr;
  hipLaunchKernelGGL((q1_kv_main<F16, BITS, D, NM>), dim3((unsigned)g.p.wgs), dim3(64 * kWaves), bytes, s, g);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || g.p.splits == 1) return e;
  hipLaunchKernelGGL((q1_kv_join<D>), dim3((unsigned)(g.a.B * g.a.T * g.a.Hq)), dim3(64 * kWaves), 0, s, g, 16 * NM);
  return hipGetLastError();
}

template <bool F16, int BITS, int D>
hipError_t launch_n(const KvArgs& g, hipStream_t s) {
  return g.p.nm == 1 ? launch<F16, BITS, D, 1>(g, s) : launch<F16, BITS, D, 2>(g, s);
}

template <bool F16, int BITS>
hipError_t launch_d(const KvArgs& g, hipStream_t s) {
  return g.c.D == 64 ? launch_n<F16, BITS, 64>(g, s) : g.c.D == 128 ? launch_n<F16, BITS, 128>(g, s) : launch_n<F16, BITS, 256>(g, s);
}

int64_t up_div(int64_t x, int64_t y) { return (x + y - 1) / y; }

}  // namespace

KvPlan plan_kv_attn(const q1_kv& c, const q1_kv_query& a) {
  KvPlan p = {};
  const int64_t R = a.T * (a.Hq / c.Hkv), units = up_div(a.max_pages * c.page_size, kStep);
  p.nm = R > 16 ? 2 : 1;
  p.row_blocks = (int)up_div(R, 16 * p.nm);
  const int64_t others = a.B * c.Hkv * p.row_blocks;
  // the fewest units of kStep tokens an item with which all items run at a time, at most 64 items a row
  const int64_t slots = (int64_t)device_cus() * (p.nm * c.D > 256 ? 1 : 2);
  int64_t per = up_div(units * others, slots);
  if (per < up_div(units, 64)) per = up_div(units, 64);
  if (per < 1) per = 1;
  p.splits = units > 0 ? (int)up_div(units, per) : 1;
  p.tokens = per * kStep;
  p.wgs = others * p.splits;
  p.page = divider((uint32_t)c.page_size);
  if (p.splits > 1) {
    const size_t rows = (size_t)p.splits * a.B * a.T * a.Hq;
    p.ml_off = (rows * c.D * 4 + 255) / 256 * 256;
    p.ws_bytes = p.ml_off + (rows * 8 + 255) / 256 * 256;
  }
  return p;
}

hipError_t launch_kv_attn(const q1_kv& c, const q1_kv_query& a, const KvPlan& p, unsigned char* ws, hipStream_t s) {
  const KvArgs g = {c, a, p, reinterpret_cast<float*>(ws), reinterpret_cast<float2*>(ws + p.ml_off)};
  if (a.dtype == Q1_F16) return c.bits == 4 ? launch_d<true, 4>(g, s) : launch_d<true, 8>(g, s);
  return c.bits == 4 ? launch_d<false, 4>(g, s) : launch_d<false, 8>(g, s);
}

}  // namespace q1
