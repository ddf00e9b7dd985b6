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
  uint32_t* before;  // units before each entry, and of all
  float* part_o;     // [2 workgroups, rows of an item, D]
  float2* part_ml;
};

__device__ __forceinline__ uint32_t length_of(const KvArgs& g, uint32_t b) {
  if (g.c.pages == 0) return 0;
  const int64_t n = g.a.lens[b], most = g.a.max_pages * g.c.page_size;
  return n < 0 ? 0 : (uint32_t)(n > most ? most : n);
}

// Tokens that row r (of the T * group of a sequence and key/value head) sees, of n.
__device__ __forceinline__ uint32_t seen_by(const KvArgs& g, uint32_t n, uint32_t r) {
  const uint32_t behind = (uint32_t)g.a.T - 1 - divide(r, g.p.group);
  return n > behind ? n - behind : 0;
}

// An entry is a block of rows of a sequence; each of its key/value heads has this many
// units of kStep tokens: those that the block's last row sees.
__device__ __forceinline__ uint32_t units_of(const KvArgs& g, uint32_t entry) {
  const uint32_t b = divide(entry, g.p.blocks), end = (entry - b * g.p.row_blocks + 1) * g.p.rows;
  return (seen_by(g, length_of(g, b), (end < g.p.R ? end : g.p.R) - 1) + kStep - 1) / kStep;
}

// A workgroup's share of all units, in the order entry, head, tokens: an even cut.
struct Share {
  uint32_t each, longer;  // units of a workgroup, and how many first ones have one more
  __device__ __forceinline__ Share(uint32_t total, uint32_t wgs) : each(total / wgs), longer(total - each * wgs) {}
  __device__ __forceinline__ uint32_t first(uint32_t wg) const { return wg * each + (wg < longer ? wg : longer); }
  __device__ __forceinline__ uint32_t owner(uint32_t unit) const {
    const uint32_t head = longer * (each + 1);
    return unit < head ? unit / (each + 1) : longer + (unit - head) / each;
  }
};

// What a workgroup does next: tokens [t0, t1) of one entry and head.
struct Item {
  uint32_t entry, hk, t0, t1;
  uint32_t b, n, row0;   // sequence, its length, first row
  bool whole;            // all units of the entry and head
  uint32_t part;         // else: where its sums go
};

// The units before every entry, by the whole workgroup: returns all, and in *entry and
// *inside the place of unit `start` (inside: units of that entry before it).
__device__ __forceinline__ uint32_t scan_units(const KvArgs& g, uint32_t wgs, uint32_t* lds, Share* share, uint32_t* entry,
                                               uint32_t* inside) {
  if (g.p.entries <= 64) {  // (each wave for itself)
    const uint32_t lane = threadIdx.x & 63, u = lane < g.p.entries ? units_of(g, lane) * (uint32_t)g.c.Hkv : 0;
    uint32_t upto = u;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const uint32_t v = __shfl_up(upto, off);
      upto += (int)lane >= off ? v : 0;
    }
    const uint32_t total = __builtin_amdgcn_readlane(upto, 63);
    *share = Share(total, wgs);
    const uint32_t start = share->first(blockIdx.x);
    const uint64_t after = __ballot(upto > start);
    *entry = after ? __builtin_ctzll(after) : 0;
    *inside = start - __builtin_amdgcn_readlane(upto - u, *entry);
    if (blockIdx.x == 0 && threadIdx.x < 64) {
      if (lane < g.p.entries) g.before[lane] = upto - u;
      if (lane == 63) g.before[g.p.entries] = total;
    }
    return total;
  }
  const uint32_t tid = threadIdx.x, each = (g.p.entries + 64 * kWaves - 1) / (64 * kWaves), heads = (uint32_t)g.c.Hkv;
  const uint32_t e0 = tid * each, e1 = e0 + each < g.p.entries ? e0 + each : g.p.entries;
  uint32_t sum = 0;
  for (uint32_t e = e0; e < e1; ++e) sum += units_of(g, e) * heads;
  uint32_t upto = sum;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const uint32_t v = __shfl_up(upto, off);
    upto += (int)(tid & 63) >= off ? v : 0;
  }
  if ((tid & 63) == 63) lds[tid >> 6] = upto;
  __syncthreads();
  uint32_t total = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    upto += w < (int)(tid >> 6) ? lds[w] : 0;
    total += lds[w];
  }
  *share = Share(total, wgs);
  const uint32_t start = share->first(blockIdx.x);
  uint32_t at = upto - sum;
  const bool mine = start >= at && start < upto;
  if (mine || blockIdx.x == 0) {
    for (uint32_t e = e0; e < e1; ++e) {
      const uint32_t u = units_of(g, e) * heads;
      if (blockIdx.x == 0) g.before[e] = at;
      if (mine && start >= at && start < at + u) {
        lds[kWaves] = e;
        lds[kWaves + 1] = start - at;
      }
      at += u;
    }
    if (blockIdx.x == 0 && tid == 64 * kWaves - 1) g.before[g.p.entries] = total;
  }
  __syncthreads();
  *entry = __builtin_amdgcn_readfirstlane(lds[kWaves]);
  *inside = __builtin_amdgcn_readfirstlane(lds[kWaves + 1]);
  __syncthreads();
  return __builtin_amdgcn_readfirstlane(total);
}

// The item of all tokens of an entry and head, the longest (last rows) first.
__device__ __forceinline__ Item whole_item(const KvArgs& g, uint32_t i) {
  Item it;
  const uint32_t x = divide(i, g.p.kv_heads), y = divide(x, g.p.sequences);
  it.hk = i - x * (uint32_t)g.c.Hkv;
  it.b = x - y * (uint32_t)g.a.B;
  const uint32_t rb = g.p.row_blocks - 1 - y, past = (rb + 1) * g.p.rows;
  it.n = __builtin_amdgcn_readfirstlane(length_of(g, it.b));
  it.row0 = rb * g.p.rows;
  it.t0 = 0;
  it.t1 = __builtin_amdgcn_readfirstlane(seen_by(g, it.n, (past < g.p.R ? past : g.p.R) - 1));
  it.whole = true;
  it.entry = it.part = 0;
  return it;
}

// Calls f(item) for each of this workgroup's items.
template <typename F>
__device__ __forceinline__ void each_item(const KvArgs& g, uint32_t* lds, F f) {
  if (!g.p.cut) {
    f(whole_item(g, blockIdx.x));
    return;
  }
  Share share(0, 1);
  uint32_t entry, inside;
  const uint32_t total = scan_units(g, gridDim.x, lds, &share, &entry, &inside);
  const uint32_t first = share.first(blockIdx.x), end = __builtin_amdgcn_readfirstlane(share.first(blockIdx.x + 1));
  if (first >= total) return;
  uint32_t unit = __builtin_amdgcn_readfirstlane(first);
  Item it;
  it.entry = entry;
  uint32_t units = __builtin_amdgcn_readfirstlane(units_of(g, entry)), u = inside;
  it.hk = u / units;
  u -= it.hk * units;
  while (unit < end) {
    const uint32_t take = units - u < end - unit ? units - u : end - unit;
    it.b = divide(it.entry, g.p.blocks);
    it.n = __builtin_amdgcn_readfirstlane(length_of(g, it.b));
    it.row0 = (it.entry - it.b * g.p.row_blocks) * g.p.rows;
    const uint32_t past = it.row0 + g.p.rows, seen = seen_by(g, it.n, (past < g.p.R ? past : g.p.R) - 1);
    it.t0 = u * kStep;
    it.t1 = __builtin_amdgcn_readfirstlane((u + take) * kStep < seen ? (u + take) * kStep : seen);
    it.whole = take == units;
    it.part = 2 * blockIdx.x + (unit == first ? 0 : 1);
    f(it);
    unit += take;
    u = 0;
    if (++it.hk == (uint32_t)g.c.Hkv && unit < end) {
      it.hk = 0;
      do ++it.entry;
      while ((units = __builtin_amdgcn_readfirstlane(units_of(g, it.entry))) == 0);
    }
  }
}

// Queries stay in registers where they fit beside the output, and else go to LDS.
template <int D, int NM, int QP>
constexpr bool kQueriesInLds = D == 256 || (NM == 2 && D == 128);

template <int D, int NM, int QP>
constexpr int kTokenLds() {
  constexpr int q = kQueriesInLds<D, NM, QP> ? 16 * NM * (2 * D * QP + 16) : 0;
  constexpr int vt = kWaves * kTile * (2 * D + 32) + q, jo = kWaves * 16 * NM * ((D + 4) * 4 + 8);
  return vt > jo ? vt : jo;
}

// 8 elements of a query row from element d on, as bf16 parts.  They have the scale's sign
// (and are zeros for a scale of 0), so that the largest product is the largest score.
template <bool F16, int QP>
__device__ __forceinline__ void load_q(const KvArgs& g, const Item& it, uint32_t r, int d, u32x4* q) {
  u32x4 w = {0u, 0u, 0u, 0u};
  if (r < g.p.R) {
    const uint32_t t = divide(r, g.p.group), h = it.hk * g.p.heads_each + (r - t * g.p.heads_each);
    w = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(g.a.q) + ((int64_t)it.b * g.a.T + t) * g.a.q_ld +
                                        (int64_t)h * g.c.D + d);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) w[j] = g.a.scale == 0.f ? 0u : g.a.scale < 0.f ? w[j] ^ 0x80008000u : w[j];
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

  // Codes are read once; where a load has all of a line of two tokens (rows of 64 bytes; of
  // longer ones the next load has the rest) they need not be kept: 329 MB in 68 us, else 73,
  // but with rows of 128 bytes 320 MB in 76, else 70.
  static __device__ __forceinline__ u32x4 once(const u32x4* p) {
    if constexpr (W == 4) return __builtin_nontemporal_load(p);
    else return *p;
  }

  // From this lane's bytes of the tokens' rows on.
  __device__ __forceinline__ void load(const q1_kv& c, const uint64_t* at) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const unsigned char* kp = static_cast<const unsigned char*>(c.k) + at[h];
      const unsigned char* vp = static_cast<const unsigned char*>(c.v) + at[h];
      if constexpr (W == 2) {
        const uint2 kw = *reinterpret_cast<const uint2*>(kp), vw = *reinterpret_cast<const uint2*>(vp);
        k[h][0] = kw.x, k[h][1] = kw.y, v[h][0] = vw.x, v[h][1] = vw.y;
      } else {
#pragma unroll
        for (int i = 0; i < W / 4; ++i) {
          const u32x4 kw = once(reinterpret_cast<const u32x4*>(kp) + i), vw = once(reinterpret_cast<const u32x4*>(vp) + i);
#pragma unroll
          for (int j = 0; j < 4; ++j) k[h][4 * i + j] = kw[j], v[h][4 * i + j] = vw[j];
        }
      }
      // a scale is 4 * BITS bytes of codes: its place follows from theirs
      const uint64_t sat = at[h] / (4 * BITS);
      const unsigned char* ksp = static_cast<const unsigned char*>(c.k_scales) + sat;
      const unsigned char* vsp = static_cast<const unsigned char*>(c.v_scales) + sat;
      if constexpr (NB == 2) {
        ks[h] = *reinterpret_cast<const uint16_t*>(ksp);
        vs[h] = *reinterpret_cast<const uint16_t*>(vsp);
      } else {
        ks[h] = *ksp;
        vs[h] = *vsp;
      }
    }
  }

  static __device__ __forceinline__ uint32_t byte(uint32_t s, int j) { return NB == 2 ? s >> (8 * j) & 255u : s; }
};

// The softmax of one tile for a block of 16 queries: products of this lane's 8 tokens in,
// weights out as two operands; m, l and the output so far are brought to a new maximum
// where a product is so far above the old one that a weight could pass 2^8.  With ALL,
// every token counts, else those of `mine`.
template <bool ALL, int DT>
__device__ __forceinline__ void soften(const f32x4* S, uint32_t mine, float sc, float& m, float& l, f32x4* O, int stride,
                                       u32x4& hi, u32x4& lo) {
  float s[8], top = -INFINITY;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    s[j] = S[j >> 2][j & 3];
    if constexpr (!ALL) s[j] = (mine >> j) & 1u ? s[j] : -INFINITY;
    top = fmaxf(top, s[j]);
  }
  if (__any((top - m) * sc > 8.0f)) {  // (the first tile: m is -infinity)
    const float mn = fmaxf(m, max_groups(top));
    const float keep = m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f((m - mn) * sc);
    l *= keep;
#pragma unroll
    for (int d = 0; d < DT; ++d) O[d * stride] *= keep;
    m = mn;
  }
  const float base = m == -INFINITY ? 0.f : -m * sc;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    s[j] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[j], sc, base));
    l += s[j];
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float rx, ry, r0, r1;
    hi[j] = round2<false>(s[2 * j], s[2 * j + 1], &rx, &ry);
    lo[j] = round2<false>(rx, ry, &r0, &r1);
  }
}

// Four elements of a row: the row itself, or its part of it.
__device__ __forceinline__ void put_row(const KvArgs& g, const Item& it, uint32_t r, int e, f32x4 o, float top, float sum) {
  if (it.whole) {
    const uint32_t t = divide(r, g.p.group), h = it.hk * g.p.heads_each + (r - t * g.p.heads_each);
    const int64_t row = ((int64_t)it.b * g.a.T + t) * g.a.Hq + h, at = row * g.c.D + e;
    const bool nothing = sum == 0.f;  // no token, or none above -infinity (a NaN stays one)
    const float inv = nothing ? 0.f : 1.0f / sum;
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = nothing ? 0.f : o[j] * inv;
    if (g.a.out_dtype == F32) *reinterpret_cast<f32x4*>(static_cast<float*>(g.a.out) + at) = o;
    else if (g.a.out_dtype == F16) *reinterpret_cast<uint2*>(static_cast<uint16_t*>(g.a.out) + at) = uint2{pack16<true>(o[0], o[1]), pack16<true>(o[2], o[3])};
    else *reinterpret_cast<uint2*>(static_cast<uint16_t*>(g.a.out) + at) = uint2{pack16<false>(o[0], o[1]), pack16<false>(o[2], o[3])};
    if (e == 0 && g.a.lse != nullptr) g.a.lse[row] = nothing ? -INFINITY : top * 0.69314718055994530942f + logf(sum);
  } else {
    const int64_t at = (int64_t)it.part * g.p.rows + (r - it.row0);
    *reinterpret_cast<f32x4*>(g.part_o + at * g.c.D + e) = o;
    if (e == 0) g.part_ml[at] = float2{top, sum};
  }
}

// An item by tokens.
template <bool F16, int BITS, int D, int NM>
__device__ __forceinline__ void item_by_tokens(const KvArgs& g, const Item& it, unsigned char* lds) {
  constexpr int QP = F16 ? 2 : 1;
  using T = Tile<BITS, D>;
  constexpr int KS = T::KS, NB = T::NB, DT = D / 16, VROW = 2 * D + 32, QROW = 2 * D * QP + 16;
  constexpr bool QL = kQueriesInLds<D, NM, QP>;
  const q1_kv& c = g.c;
  const q1_kv_query& a = g.a;
  const int lane = threadIdx.x & 63, col = lane & 15, grp = lane >> 4;
  // in a scalar register: matrix-core products ignore the lane mask, so the loop they are in must be a scalar one
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int32_t end = (int32_t)it.t1;

  unsigned char* const ql = lds + kWaves * kTile * VROW;
  u32x4 Q[QL ? 1 : NM][QL ? 1 : KS][QP];
  if constexpr (QL) {
    for (int x = threadIdx.x; x < 16 * NM * (D / 8); x += 64 * kWaves) {
      const int r = x / (D / 8), e = x % (D / 8);
      u32x4 q[QP];
      load_q<F16, QP>(g, it, it.row0 + r, 8 * e, q);
#pragma unroll
      for (int s = 0; s < QP; ++s) *reinterpret_cast<u32x4*>(ql + r * QROW + s * 2 * D + 16 * e) = q[s];
    }
    __syncthreads();
  } else {
#pragma unroll
    for (int m = 0; m < NM; ++m)
#pragma unroll
      for (int s = 0; s < KS; ++s) load_q<F16, QP>(g, it, it.row0 + 16 * m + col, grp * (D / 4) + 8 * s, Q[m][s]);
  }

  // This lane's two tokens of the tile whose page ids are fetched next: page of the
  // sequence and place in it, which go on by kStep tokens (past the end: the last page).
  const uint32_t ps = (uint32_t)c.page_size, more_pg = kStep / ps, more_off = kStep - more_pg * ps;
  const uint32_t last_pg = it.t1 > 0 ? divide(it.t1 - 1, g.p.page) : 0;
  uint32_t pg[2], off[2];
  auto ids_of = [&](int32_t* id, uint32_t* place) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      id[h] = (a.page_table + it.b * a.max_pages)[pg[h] < last_pg ? pg[h] : last_pg];
      place[h] = off[h];
      pg[h] += more_pg;
      off[h] += more_off;
      const bool over = off[h] >= ps;
      pg[h] += over ? 1 : 0;
      off[h] -= over ? ps : 0;
    }
  };
  // bytes of a page of one tensor, and before this lane's in a page (both below 2^32)
  const uint32_t page_bytes = (uint32_t)(c.Hkv * c.page_size * (D * BITS / 8));
  const uint32_t lane_bytes = it.hk * (uint32_t)(c.page_size * (D * BITS / 8)) + grp * (D * BITS / 32);
  auto fetch = [&](int32_t t, const int32_t* id, const uint32_t* place, T& x) {
    uint64_t at[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const bool in = (uint32_t)id[h] < (uint32_t)c.pages;
      x.ok[h] = in && t + 16 * h + col < end;
      at[h] = (uint64_t)(in ? (uint32_t)id[h] : 0u) * page_bytes + (place[h] * (uint32_t)(D * BITS / 8) + lane_bytes);
    }
    x.load(c, at);
  };

  f32x4 O[DT][NM];
  float m[NM], l[NM];
  int32_t lim[NM];  // tokens that this lane's query sees
#pragma unroll
  for (int x = 0; x < NM; ++x) {
    m[x] = -INFINITY;
    l[x] = 0.f;
    const uint32_t r = it.row0 + 16 * x + col;
    lim[x] = (int32_t)seen_by(g, it.n, r < g.p.R ? r : g.p.R - 1);
#pragma unroll
    for (int d = 0; d < DT; ++d) O[d][x] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  const int32_t least = (int32_t)seen_by(g, it.n, it.row0);  // all queries see these
  unsigned char* const vt = lds + wave * (kTile * VROW);
  // (rows start 8 of 32 banks apart; in every other four rows the two 16-byte pieces of each 32
  // bytes change places, so that eight rows' writes of 16 bytes meet all banks, and reads still do)
  const int swap = 16 * (col >> 2 & 1);
  unsigned char* const vw = vt + col * VROW + grp * (D / 2);
  const unsigned char* const vr = vt + (4 * grp + col / 4) * VROW + ((16 * (col >> 1 & 1)) ^ (16 * (grp & 1))) + 8 * (col & 1);
  const float sc = a.scale == 0.f ? 1.0f : fabsf(a.scale) * kLog2e;

  // One tile; the next one's loads start as soon as this one's registers are free.
  auto work = [&](int32_t t, T& x, int32_t* id, uint32_t* place) {
    float ks[2][NB], vs[2][NB];
    uint32_t most = 0;  // of the scale bytes
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        const uint32_t ke = T::byte(x.ks[h], j), ve = T::byte(x.vs[h], j);
        ks[h][j] = __uint_as_float(ke << 23);
        vs[h][j] = __uint_as_float(ve << 23);
        most = most > ke ? most : ke;
        most = most > ve ? most : ve;
      }
    // Every token counts, and no block is a NaN: else which do, and which blocks of values are, by token
    const bool plain = __ballot(x.ok[0] && x.ok[1] && most != 255u) == ~0ull;
    uint32_t in = ~0u;
    uint64_t nan[2][NB];
    if (!plain) {
      in = (uint32_t)(__ballot(x.ok[0]) & 0xffffu) | (uint32_t)(__ballot(x.ok[1]) & 0xffffu) << 16;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int j = 0; j < NB; ++j) {
          const bool bad = T::byte(x.vs[h], j) == 255u;
          nan[h][j] = __ballot(x.ok[h] && bad);
          ks[h][j] = T::byte(x.ks[h], j) == 255u ? NAN : ks[h][j];
          vs[h][j] = x.ok[h] && !bad ? vs[h][j] : 1.0f;
#pragma unroll
          for (int w = 0; w < T::W / NB; ++w)  // values of tokens that do not count (anything), and NaN blocks, as zeros
            x.v[h][j * (T::W / NB) + w] = x.ok[h] && !bad ? x.v[h][j * (T::W / NB) + w] : 0u;
        }
      }
    }
    f32x4 S[NM][2];
#pragma unroll
    for (int q = 0; q < NM; ++q)
#pragma unroll
      for (int h = 0; h < 2; ++h) S[q][h] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      u32x4 K[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) K[h] = kv_bf16<BITS>(&x.k[h][s * (BITS / 4)], ks[h][s / (KS / NB)]);
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
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int s = 0; s < KS; ++s)
        *reinterpret_cast<u32x4*>(vw + (s & 1 ? -swap : swap) + h * 16 * VROW + 16 * s) =
            kv_bf16<BITS>(&x.v[h][s * (BITS / 4)], vs[h][s / (KS / NB)]);
    fetch(t + kStep, id, place, x);
    ids_of(id, place);
    u32x4 hi[NM], lo[NM];
    uint32_t vis[NM];
    if (plain && t + kTile <= least) {
#pragma unroll
      for (int q = 0; q < NM; ++q) soften<true, DT>(S[q], 0, sc, m[q], l[q], &O[0][q], NM, hi[q], lo[q]);
    } else {
#pragma unroll
      for (int q = 0; q < NM; ++q) {
        const int32_t d = lim[q] - t;
        vis[q] = in & (d >= 32 ? ~0u : d <= 0 ? 0u : ~0u >> (32 - d));
        const uint32_t mine = (vis[q] >> (4 * grp) & 15u) | (vis[q] >> (16 + 4 * grp) & 15u) << 4;
        soften<false, DT>(S[q], mine, sc, m[q], l[q], &O[0][q], NM, hi[q], lo[q]);
      }
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
    if (!plain) {
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

  int32_t t = (int32_t)it.t0 + wave * kTile;
  if (t < end) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      pg[h] = divide((uint32_t)(t + 16 * h + col), g.p.page);
      off[h] = (uint32_t)(t + 16 * h + col) - pg[h] * ps;
    }
    T x;
    int32_t id[2];
    uint32_t place[2];
    ids_of(id, place);
    fetch(t, id, place, x);
    ids_of(id, place);
    for (; t < end; t += kStep) work(t, x, id, place);
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
    if (grp == 0) sml[r] = float2{m[q] == -INFINITY ? m[q] : m[q] * sc, sum};
#pragma unroll
    for (int d = 0; d < DT; ++d) *reinterpret_cast<f32x4*>(so + r * OROW + 16 * d + 4 * grp) = O[d][q];
  }
  __syncthreads();
  for (int x = threadIdx.x; x < 16 * NM * (D / 4); x += 64 * kWaves) {
    const int r = x / (D / 4), e = 4 * (x % (D / 4));
    if (it.row0 + r >= g.p.R) continue;
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
    put_row(g, it, it.row0 + r, e, o, top, sum);
  }
  __syncthreads();
}

template <bool F16, int BITS, int D, int NM>
__global__ __launch_bounds__(64 * kWaves, 2) void q1_kv_tokens(const KvArgs g) {
  extern __shared__ unsigned char lds[];
  each_item(g, reinterpret_cast<uint32_t*>(lds), [&](const Item& it) { item_by_tokens<F16, BITS, D, NM>(g, it, lds); });
}

// The rows whose tokens several workgroups had, and those that see none: a row has R of a
// workgroup's 4 waves, of which each sums every R-th part.
template <int D, int R>
__global__ __launch_bounds__(64 * kWaves) void q1_kv_join(const KvArgs g) {
  constexpr int E = D / 64, U = 8;  // elements a lane, parts in flight
  typedef float vec __attribute__((ext_vector_type(E)));
  __shared__ vec so[kWaves][64];
  const q1_kv_query& a = g.a;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t rows = (uint32_t)(a.B * a.T * a.Hq), row = blockIdx.x * (kWaves / R) + wave / R;
  if (row >= rows) return;
  const uint32_t bt = divide(row, g.p.heads), h = row - bt * (uint32_t)a.Hq, b = divide(bt, g.p.queries);
  const uint32_t t = bt - b * (uint32_t)a.T, hk = divide(h, g.p.group);
  const uint32_t r = t * g.p.heads_each + (h - hk * g.p.heads_each), rb = r / g.p.rows, entry = b * g.p.row_blocks + rb;
  const uint32_t units = __builtin_amdgcn_readfirstlane(units_of(g, entry));
  uint32_t w0 = 0, parts = 0, second = 0;
  if (units > 0) {
    const Share share(__builtin_amdgcn_readfirstlane(g.before[g.p.entries]), g.p.wgs);
    const uint32_t first = __builtin_amdgcn_readfirstlane(g.before[entry]) + hk * units;
    w0 = share.owner(first);
    parts = share.owner(first + units - 1) - w0 + 1;
    if (parts == 1) return;  // whole: its workgroup wrote the row
    second = share.first(w0) != first ? 1 : 0;
  }
  // part s, of workgroup w0 + s: its first item, but for one that began with another entry or head
  auto at = [&](uint32_t s) { return (int64_t)(2 * (w0 + s) + (s == 0 ? second : 0)) * g.p.rows + (r - rb * g.p.rows); };
  vec o = 0.f;
  float top = -INFINITY, sum = 0.f;
  for (uint32_t c0 = 0; c0 < parts; c0 += 64) {  // 64 parts: their factors, one a lane, then every R-th of them
    const float2 ml = c0 + lane < parts ? g.part_ml[at(c0 + lane)] : float2{-INFINITY, 0.f};
    float now = fmaxf(top, ml.x);
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) now = fmaxf(now, __shfl_xor(now, off));
    const float base = now == -INFINITY ? 0.f : now, keep = __builtin_amdgcn_exp2f(top - base);
    const float f = __builtin_amdgcn_exp2f(ml.x - base);
    const uint32_t left = parts - c0 < 64 ? parts - c0 : 64;
    o = keep * o;
    sum = keep * sum + f * ml.y;  // (of this lane's parts)
    for (uint32_t s0 = wave % R; s0 < left; s0 += U * R) {
      vec x[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint32_t s = s0 + u * R < left ? s0 + u * R : left - 1;
        x[u] = reinterpret_cast<const vec*>(g.part_o + at(c0 + s) * D)[lane];
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint32_t s = s0 + u * R;
        const float fs = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(f), s & 63));
        o = s < left ? o + fs * x[u] : o;
      }
    }
    top = now;
  }
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) sum += __shfl_xor(sum, off);
  if constexpr (R > 1) {  // (every wave has the same top and sum)
    so[wave][lane] = o;
    __syncthreads();
    if (wave % R != 0) return;
#pragma unroll
    for (int w = 1; w < R; ++w) o = o + so[wave + w][lane];
  }
  const bool nothing = sum == 0.f;  // no token, or none above -infinity (a NaN stays one)
  const float inv = nothing ? 0.f : 1.0f / sum;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    float v;
    if constexpr (E == 1) v = o[0];
    else v = o[e];
    store_out(a.out, a.out_dtype, (int64_t)row * D + lane * E + e, nothing ? 0.f : v * inv);
  }
  if (lane == 0 && a.lse != nullptr) a.lse[row] = nothing ? -INFINITY : top * 0.69314718055994530942f + logf(sum);
}

template <int D>
hipError_t launch_join(const KvArgs& g, hipStream_t s) {
  // a wave a row where that fills the chip, else four
  const int64_t rows = g.a.B * g.a.T * g.a.Hq;
  if (rows < (int64_t)device_cus() * 4)
    hipLaunchKernelGGL((q1_kv_join<D, kWaves>), dim3((unsigned)rows), dim3(64 * kWaves), 0, s, g);
  else
    hipLaunchKernelGGL((q1_kv_join<D, 1>), dim3((unsigned)((rows + kWaves - 1) / kWaves)), dim3(64 * kWaves), 0, s, g);
  return hipGetLastError();
}

template <bool F16, int BITS, int D, int NM>
hipError_t launch(const KvArgs& g, hipStream_t s) {
  constexpr int bytes = kTokenLds<D, NM, F16 ? 2 : 1>();
  static const hipError_t attr = hipFuncSetAttribute(reinterpret_cast<const void*>(&q1_kv_tokens<F16, BITS, D, NM>),
                                                     hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (attr != hipSuccess) return attr;
  hipLaunchKernelGGL((q1_kv_tokens<F16, BITS, D, NM>), dim3((unsigned)g.p.wgs), dim3(64 * kWaves), bytes, s, g);
  const hipError_t e = hipGetLastError();
  return e != hipSuccess || !g.p.cut ? e : launch_join<D>(g, s);
}

template <bool F16, int BITS, int D>
hipError_t launch_n(const KvArgs& g, hipStream_t s) {
  if constexpr (D < 256) {
    if (g.p.nm == 2) return launch<F16, BITS, D, 2>(g, s);
  }
  return launch<F16, BITS, D, 1>(g, s);
}

template <bool F16, int BITS>
hipError_t launch_d(const KvArgs& g, hipStream_t s) {
  return g.c.D == 64 ? launch_n<F16, BITS, 64>(g, s) : g.c.D == 128 ? launch_n<F16, BITS, 128>(g, s) : launch_n<F16, BITS, 256>(g, s);
}

int64_t up_div(int64_t x, int64_t y) { return (x + y - 1) / y; }
size_t up256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

KvPlan plan_kv_attn(const q1_kv& c, const q1_kv_query& a) {
  KvPlan p = {};
  p.heads_each = (uint32_t)(a.Hq / c.Hkv);
  p.R = (uint32_t)(a.T * p.heads_each);
  p.nm = p.R > 16 && c.D < 256 ? 2 : 1;
  p.rows = 16 * p.nm;
  p.row_blocks = (uint32_t)up_div(p.R, p.rows);
  const int64_t items = a.B * p.row_blocks * c.Hkv, units = up_div(a.max_pages * c.page_size, kStep);
  p.too_large = items >= (int64_t)1 << 31 || (units > 0 && items >= ((int64_t)1 << 31) / units);
  p.entries = p.too_large ? 0 : (uint32_t)(a.B * p.row_blocks);
  const int64_t slots = (int64_t)device_cus() * 2;
  p.cut = units > 8 + items / 8 && items < slots * 4;
  if (!p.cut) {
    p.too_large |= items > (1 << 24) - 1;
    p.wgs = (uint32_t)items;
  } else {  // as many as run at a time, at most 64 for an item's rows on average, and one a unit
    int64_t wgs = slots;
    if (wgs > 64 * items) wgs = 64 * items;
    if (wgs > units * items) wgs = units * items;
    p.wgs = (uint32_t)wgs;
    const size_t rows = (size_t)2 * p.wgs * p.rows;
    p.o_off = up256(((size_t)p.entries + 1) * 4);
    p.ml_off = p.o_off + up256(rows * c.D * 4);
    p.ws_bytes = p.ml_off + up256(rows * 8);
  }
  p.page = divider((uint32_t)c.page_size);
  p.heads = divider((uint32_t)a.Hq);
  p.queries = divider((uint32_t)a.T);
  p.group = divider(p.heads_each);
  p.blocks = divider(p.row_blocks);
  p.kv_heads = divider((uint32_t)c.Hkv);
  p.sequences = divider((uint32_t)a.B);
  return p;
}

hipError_t launch_kv_attn(const q1_kv& c, const q1_kv_query& a, const KvPlan& p, unsigned char* ws, hipStream_t s) {
  const KvArgs g = {c, a, p, reinterpret_cast<uint32_t*>(ws), reinterpret_cast<float*>(ws + p.o_off), reinterpret_cast<float2*>(ws + p.ml_off)};
  if (a.dtype == Q1_F16) return c.bits == 4 ? launch_d<true, 4>(g, s) : launch_d<true, 8>(g, s);
  return c.bits == 4 ? launch_d<false, 4>(g, s) : launch_d<false, 8>(g, s);
}

}  // namespace q1
