// Attention over keys and values held in 4 or 8 bits (q1_memory.h).
//
// An item is a block of the T * Hq/Hkv query rows that share a key/value head of a
// sequence, and some of its tokens: running maximum m, sum l and unnormalised output o of
// each row.  The work, in units of 128 tokens, is cut evenly over as many workgroups as run
// at a time, and q1_kv_join adds the parts of a row; or each workgroup has a whole item and
// writes its rows itself (plan_kv_attn has the rule).  Codes go to bf16, which is exact, so
// the products are the ones of 16-bit attention (see q1_attn.hip for their layouts):
//   S^T = K Q^T     O^T = V^T P^T, values transposed on their way out of LDS.
// fp16 queries enter as two bf16 parts (11 bits of significand are 8 and 3), weights as
// two (2^-17: one would add an error of the size of the output's rounding).  The running
// maximum stays where it is until a token is 2^8 above it, so o is rescaled rarely, and for n
// tokens weights are relative to 2^8 2^bits(n) times the kept maximum: their sum is below 1, so o
// is finite wherever the values are (a power of two in a weight costs no bits; weights below
// n 2^-117 of the largest may become 0).
//
// By tokens (few rows): 4 waves, each with a quarter of the tokens and 16 or 32 rows,
// joined in LDS; keys go from memory to the matrix core through registers alone.  Bound by
// the bytes of the pages and by the vector instructions (98 a wave for 16 rows x 32 tokens).
// By rows (prompts): 8 waves, each with 32 rows (16 of D 256); a tile of 64 tokens is
// converted once for all of them.  Bound by the products, where there is much to do: 8000
// queries of 8000 tokens of 8 bits take 540 to 557 us for 590 Gflop (both parts of the weights),
// nine tenths of the rate of a large library product (1.11 to 1.22 PFLOP/s), fp16 ones 647 for 786.
//
// Measured (us): 32 sequences of up to 8201 tokens, D 256, 4 bits 51, 45 in a graph (the pages at
// the rate of a copy: 35); 8 of up to 65537, 3 queries each, D 128, 76 (66); 4 of up to 519 9.1;
// 2 x 1000 queries of 4525 and 5003 tokens, 24 heads of D 128, 8 bits 170 to 180 (129 at the rate
// above; the join and the parts it reads 20), of 3531 and 5003 176, of 4 bits 160, fp16 186 and 179.
//
// A token that a query does not see has the score -infinity, whatever its key.  Its weight 0
// would still make a NaN of a value that is not finite, so NaN blocks of values enter as zeros,
// and their columns are made NaN at the end for the queries that see the token.  In tiles that
// some query of the item does not see to their end, blocks with a NaN code, or a code that its
// scale carries out of bf16's range, are treated alike; elsewhere each such value makes its
// own column what it is.
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
template <int WAVES>
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
  const uint32_t tid = threadIdx.x, each = (g.p.entries + 64 * WAVES - 1) / (64 * WAVES), heads = (uint32_t)g.c.Hkv;
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
  for (int w = 0; w < WAVES; ++w) {
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
        lds[WAVES] = e;
        lds[WAVES + 1] = start - at;
      }
      at += u;
    }
    if (blockIdx.x == 0 && tid == 64 * WAVES - 1) g.before[g.p.entries] = total;
  }
  __syncthreads();
  *entry = __builtin_amdgcn_readfirstlane(lds[WAVES]);
  *inside = __builtin_amdgcn_readfirstlane(lds[WAVES + 1]);
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

// Weights of a sequence of n tokens are smaller than those relative to the kept maximum by 2^this.
__device__ __forceinline__ int down_of(uint32_t n) { return 8 + 32 - __builtin_clz(n | 1u); }

// What products are multiplied by (of queries with the scale's sign, see load_q): finite, so
// that a product of 0 is a score of 0 at any scale.
__device__ __forceinline__ float factor_of(float scale) {
  return scale == 0.f ? 1.0f : fminf(fabsf(scale) * kLog2e, 0x1.fffffep127f);
}

// Calls f(item) for each of this workgroup's items.
template <int WAVES, typename F>
__device__ __forceinline__ void each_item(const KvArgs& g, uint32_t* lds, F f) {
  if (!g.p.cut) {
    f(whole_item(g, blockIdx.x));
    return;
  }
  Share share(0, 1);
  uint32_t entry, inside;
  const uint32_t total = scan_units<WAVES>(g, gridDim.x, lds, &share, &entry, &inside);
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

// Whether one of 8 bf16 values is infinite or NaN.
__device__ __forceinline__ bool not_finite(u32x4 w) {
  uint32_t t = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) t |= (w[j] & 0x7f807f80u) + 0x00800080u;
  return (t & 0x80008000u) != 0;
}

// Products of this lane's 8 tokens: those of `vis` (by token of the tile) count.
__device__ __forceinline__ void hide(f32x4* S, uint32_t vis, int grp) {
  const uint32_t mine = (vis >> (4 * grp) & 15u) | (vis >> (16 + 4 * grp) & 15u) << 4;
#pragma unroll
  for (int j = 0; j < 8; ++j) S[j >> 2][j & 3] = (mine >> j) & 1u ? S[j >> 2][j & 3] : -INFINITY;
}

// The softmax of one tile for a block of 16 queries: products of this lane's 8 tokens in,
// weights out as two operands; m, l and the output so far are brought to a new maximum
// where a product is over 2^8 above the old one.  (One call for all tiles: where it was one of
// two, the output was copied at each, a quarter of the time.)
template <int DT>
__device__ __forceinline__ void soften(const f32x4* S, float sc, float down, float& m, float& l, f32x4* O, int stride, u32x4& hi, u32x4& lo) {
  float s[8], top = -INFINITY;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    s[j] = S[j >> 2][j & 3];
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
  const float base = m == -INFINITY ? 0.f : __builtin_fmaf(-m, sc, -down);
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

// log(sum 2^top), of weights smaller by 2^down.
__device__ __forceinline__ float lse_of(float top, float sum, int down) {
  return (top - (float)down) * 0.69314718055994530942f + logf(__builtin_ldexpf(sum, down));
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
    if (e == 0 && g.a.lse != nullptr) g.a.lse[row] = nothing ? -INFINITY : lse_of(top, sum, down_of(it.n));
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
  int32_t lim[NM];    // tokens that this lane's query sees
  uint32_t lost[NM];  // blocks of 32 columns of it that are NaN
#pragma unroll
  for (int x = 0; x < NM; ++x) {
    lost[x] = 0;
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
  const float sc = factor_of(a.scale), down = (float)down_of(it.n);

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
    // Every token counts, no block is a NaN and all queries see all tokens: else which tokens
    // count, and which blocks of values are not finite, by token
    const bool edge = __ballot(x.ok[0] && x.ok[1] && most != 255u) != ~0ull || t + kTile > least;
    uint32_t in = ~0u;
    uint64_t nan[2][NB];
    if (edge) {
      in = (uint32_t)(__ballot(x.ok[0]) & 0xffffu) | (uint32_t)(__ballot(x.ok[1]) & 0xffffu) << 16;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int j = 0; j < NB; ++j) {
          bool bad = T::byte(x.vs[h], j) == 255u;
#pragma unroll
          for (int s = 0; s < KS / NB; ++s)
            bad |= not_finite(kv_bf16<BITS>(&x.v[h][(j * (KS / NB) + s) * (BITS / 4)], vs[h][j]));
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
    if (edge) {
#pragma unroll
      for (int q = 0; q < NM; ++q) {
        const int32_t d = lim[q] - t;
        vis[q] = in & (d >= 32 ? ~0u : d <= 0 ? 0u : ~0u >> (32 - d));
        hide(S[q], vis[q], grp);
      }
    }
#pragma unroll
    for (int q = 0; q < NM; ++q) soften<DT>(S[q], sc, down, m[q], l[q], &O[0][q], NM, hi[q], lo[q]);
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int d = 0; d < DT; ++d) {
      const u32x4 v = transposed(vr + 32 * d, 16 * VROW);
#pragma unroll
      for (int q = 0; q < NM; ++q) O[d][q] = mma<false>(v, hi[q], O[d][q]);
#pragma unroll
      for (int q = 0; q < NM; ++q) O[d][q] = mma<false>(v, lo[q], O[d][q]);
    }
    if (edge) {
#pragma unroll
      for (int blk = 0; blk < D / kKvBlock; ++blk) {
        const int sh = 16 * (D == 64 ? 2 * blk : blk / NB), j = blk % NB;
        uint64_t n0 = nan[0][j], n1 = nan[1][j];
        if constexpr (D == 64) n0 |= n0 >> 16, n1 |= n1 >> 16;  // (two lanes have a block)
        const uint32_t bad = (uint32_t)(n0 >> sh & 0xffffu) | (uint32_t)(n1 >> sh & 0xffffu) << 16;
#pragma unroll
        for (int q = 0; q < NM; ++q) lost[q] |= vis[q] & bad ? 1u << blk : 0u;
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
    if (grp == 0) sml[r] = float2{m[q] == -INFINITY ? m[q] : __builtin_fmaf(m[q], sc, down), sum};
#pragma unroll
    for (int d = 0; d < DT; ++d)
      *reinterpret_cast<f32x4*>(so + r * OROW + 16 * d + 4 * grp) = lost[q] >> (d / 2) & 1u ? f32x4{NAN, NAN, NAN, NAN} : O[d][q];
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

// What one thread stages of a tile for the whole workgroup: an eighth of one token.
constexpr int kRowWaves = 8, kRowTile = 64, kParts = 64 * kRowWaves / kRowTile;

template <int BITS, int D>
struct Staged {
  static constexpr int EP = D / kParts, W = EP * BITS / 32;  // elements and dwords of a part
  static constexpr int KROW = 2 * D + 16, VROW = 2 * D + 32, kFlags = kRowTile * (KROW + VROW);
  static constexpr int kBytes = kFlags + kRowTile * kParts;
  uint32_t k[W], v[W], ks, vs;
  bool ok;  // the token counts

  static __device__ __forceinline__ void take(const unsigned char* p, uint32_t* to) {
    if constexpr (W == 1) {
      to[0] = *reinterpret_cast<const uint32_t*>(p);
    } else if constexpr (W == 2) {
      const uint2 w = *reinterpret_cast<const uint2*>(p);
      to[0] = w.x, to[1] = w.y;
    } else {
#pragma unroll
      for (int i = 0; i < W / 4; ++i) {
        const u32x4 w = reinterpret_cast<const u32x4*>(p)[i];
#pragma unroll
        for (int j = 0; j < 4; ++j) to[4 * i + j] = w[j];
      }
    }
  }

  __device__ __forceinline__ void load(const q1_kv& c, uint64_t at) {
    take(static_cast<const unsigned char*>(c.k) + at, k);
    take(static_cast<const unsigned char*>(c.v) + at, v);
    ks = static_cast<const unsigned char*>(c.k_scales)[at / (4 * BITS)];
    vs = static_cast<const unsigned char*>(c.v_scales)[at / (4 * BITS)];
  }

  // Pieces of 16 bytes that lie x apart, in each other's places.
  static __device__ __forceinline__ void swap(uint32_t* w, int x, bool yes) {
    constexpr int N = BITS / 4;  // dwords of codes a piece
#pragma unroll
    for (int i = 0; i < W; ++i)
      if (!(i / N & x)) {
        const uint32_t one = w[i], two = w[i + x * N];
        w[i] = yes ? two : one;
        w[i + x * N] = yes ? one : two;
      }
  }

  // A part with a value that is not finite is taken for one of a NaN block.
  __device__ __forceinline__ void mark_not_finite() {
    bool no = false;
#pragma unroll
    for (int s = 0; s < EP / 8; ++s) no |= not_finite(kv_bf16<BITS>(&v[s * (BITS / 4)], kv_scale(vs)));
    vs = no ? 255u : vs;
  }

  // To a buffer: keys, values (those of tokens that do not count, and NaN blocks, as zeros; in
  // every other four rows with neighbouring 16 bytes in each other's places, see item_by_tokens)
  // and a byte for each part: 1 where the token counts, and 2 where its values are a NaN block.
  // The parts of a row write their pieces in an order in which eight of them meet all banks.
  __device__ __forceinline__ void put(unsigned char* buf, int token, int part) {
    constexpr int NP = EP / 8;  // pieces of a part
    const bool bad = vs == 255u, use = ok && !bad;
    const float kscale = kv_scale(ks), vscale = use ? __uint_as_float(vs << 23) : 1.0f;
    unsigned char* const kr = buf + token * KROW;
    unsigned char* const vr = buf + kRowTile * KROW + token * VROW;
    const int turn = part * NP / 8;
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] = use ? v[i] : 0u;
#pragma unroll
    for (int x = 1; x < NP; x *= 2) {
      swap(k, x, turn & x);
      swap(v, x, turn & x);
    }
#pragma unroll
    for (int s = 0; s < NP; ++s) {
      const int piece = part * NP + (s ^ turn);
      *reinterpret_cast<u32x4*>(kr + 16 * piece) = kv_bf16<BITS>(&k[s * (BITS / 4)], kscale);
      *reinterpret_cast<u32x4*>(vr + 16 * (piece ^ (token >> 2 & 1))) = kv_bf16<BITS>(&v[s * (BITS / 4)], vscale);
    }
    buf[kFlags + token * kParts + part] = (ok ? 1 : 0) | (ok && bad ? 2 : 0);
  }
};

// An item by rows: each of 8 waves has 16 NM rows, the tiles of 64 tokens are converted once for
// all waves and lie in LDS, two in turn.  Against 16 rows a wave and two workgroups a compute
// unit, 32 rows and one workgroup halve what is converted, and what is read from LDS
// for each product.  2 x 1000 queries of 3531 and 5003 tokens, D 128, 8 bits: 181 | 176 us, fp16 213
// | 186, of 4 bits 165 | 160 and 194 | 179; 8000 of 8000 558 | 541, of 4 bits 532 | 552.  Loads a
// step ahead of their products and the priority, without and with: 186 | 176, 8000 566 | 541.
template <bool F16, int BITS, int D, int NM>
__device__ __forceinline__ void item_by_rows(const KvArgs& g, const Item& it, unsigned char* lds) {
  constexpr int QP = F16 ? 2 : 1, KS = D / 32, DT = D / 16;
  using T = Staged<BITS, D>;
  constexpr int KROW = T::KROW, VROW = T::VROW;
  const q1_kv& c = g.c;
  const q1_kv_query& a = g.a;
  const int tid = threadIdx.x, lane = tid & 63, col = lane & 15, grp = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int token = tid / kParts, part = tid % kParts;
  const uint32_t first = it.row0 + 16 * NM * wave, last = first + 16 * NM < g.p.R ? first + 16 * NM : g.p.R;  // of the wave
  const int32_t end = (int32_t)it.t1;

  u32x4 Q[NM][KS][QP];
  f32x4 O[NM][DT];
  float m[NM], l[NM];
  int32_t lim[NM];    // tokens that this lane's query sees
  uint32_t lost[NM];  // blocks of 32 columns of this lane's query that are NaN
#pragma unroll
  for (int y = 0; y < NM; ++y) {
    const uint32_t r = first + 16 * y + col;
#pragma unroll
    for (int s = 0; s < KS; ++s) load_q<F16, QP>(g, it, r, 32 * s + 8 * grp, Q[y][s]);
#pragma unroll
    for (int d = 0; d < DT; ++d) O[y][d] = f32x4{0.f, 0.f, 0.f, 0.f};
    m[y] = -INFINITY;
    l[y] = 0.f;
    lim[y] = (int32_t)seen_by(g, it.n, r < g.p.R ? r : g.p.R - 1);
    lost[y] = 0;
  }
  // all of the wave's queries see `least` tokens, none more than `most`
  const int32_t least = (int32_t)seen_by(g, it.n, first < g.p.R ? first : g.p.R - 1);
  const int32_t most = first < g.p.R ? (int32_t)seen_by(g, it.n, last - 1) : 0;
  const int32_t all = (int32_t)seen_by(g, it.n, it.row0);  // all queries of the item see these
  const float sc = factor_of(a.scale), down = (float)down_of(it.n);

  // This thread's token of the tile whose page id is fetched next, as in item_by_tokens.
  const uint32_t ps = (uint32_t)c.page_size, more_pg = kRowTile / ps, more_off = kRowTile - more_pg * ps;
  const uint32_t last_pg = it.t1 > 0 ? divide(it.t1 - 1, g.p.page) : 0;
  uint32_t pg = divide(it.t0 + token, g.p.page), off = it.t0 + token - pg * ps;
  int32_t id = 0;
  uint32_t place = 0;
  auto id_of = [&] {
    id = (a.page_table + it.b * a.max_pages)[pg < last_pg ? pg : last_pg];
    place = off;
    pg += more_pg;
    off += more_off;
    const bool over = off >= ps;
    pg += over ? 1 : 0;
    off -= over ? ps : 0;
  };
  const uint32_t page_bytes = (uint32_t)(c.Hkv * c.page_size * (D * BITS / 8));
  const uint32_t lane_bytes = it.hk * (uint32_t)(c.page_size * (D * BITS / 8)) + part * (T::EP * BITS / 8);
  T x;
  auto fetch = [&](int32_t t) {
    const bool in = (uint32_t)id < (uint32_t)c.pages;
    x.ok = in && t + token < end;
    x.load(c, (uint64_t)(in ? (uint32_t)id : 0u) * page_bytes + (place * (uint32_t)(D * BITS / 8) + lane_bytes));
  };

  const int32_t t0 = (int32_t)it.t0;
  if (t0 < end) {
    id_of();
    fetch(t0);
    id_of();
  }
  int turn = 0;
  for (int32_t t = t0; t < end; t += kRowTile, turn ^= 1) {
    unsigned char* const buf = lds + turn * T::kBytes;
    if (t + kRowTile > all) x.mark_not_finite();
    x.put(buf, token, part);
    __syncthreads();
    fetch(t + kRowTile);
    id_of();
    const uint2 flags = reinterpret_cast<const uint2*>(buf + T::kFlags)[lane];  // of token t + lane
    const bool plain = __ballot(flags.x == 0x01010101u && flags.y == 0x01010101u) == ~0ull;
#pragma unroll
    for (int sub = 0; sub < kRowTile / kTile; ++sub) {
      const int32_t ts = t + kTile * sub;
      if (ts >= most) break;
      const unsigned char* const kb = buf + (kTile * sub + col) * KROW + 16 * grp;
      const unsigned char* const vb = buf + kRowTile * KROW + (kTile * sub + 4 * grp + col / 4) * VROW +
                                      ((16 * (col >> 1 & 1)) ^ (16 * (grp & 1))) + 8 * (col & 1);
      f32x4 S[NM][2];
#pragma unroll
      for (int y = 0; y < NM; ++y) S[y][0] = S[y][1] = f32x4{0.f, 0.f, 0.f, 0.f};
      // what the next products take is loaded before these: the compiler would load it after them
      u32x4 K[2][2];
      auto load_k = [&](int s) {
#pragma unroll
        for (int h = 0; h < 2; ++h) K[s & 1][h] = *reinterpret_cast<const u32x4*>(kb + 16 * h * KROW + 64 * s);
      };
      load_k(0);
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        if (s + 1 < KS) load_k(s + 1);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int y = 0; y < NM; ++y)
#pragma unroll
            for (int q = 0; q < QP; ++q) S[y][h] = mma<false>(K[s & 1][h], Q[y][s][q], S[y][h]);
        __builtin_amdgcn_sched_barrier(0);
      }
      u32x4 hi[NM], lo[NM];
      uint32_t vis[NM];
#pragma unroll
      for (int y = 0; y < NM; ++y) vis[y] = ~0u;
      if (!plain || ts + kTile > least) {
        const uint32_t count = (uint32_t)(__ballot(flags.x & 1u) >> (kTile * sub));
#pragma unroll
        for (int y = 0; y < NM; ++y) {
          const int32_t d = lim[y] - ts;
          vis[y] = count & (d >= 32 ? ~0u : d <= 0 ? 0u : ~0u >> (32 - d));
          hide(S[y], vis[y], grp);
        }
      }
      __builtin_amdgcn_s_setprio(1);  // the other wave's products need few instructions
#pragma unroll
      for (int y = 0; y < NM; ++y) soften<DT>(S[y], sc, down, m[y], l[y], O[y], 1, hi[y], lo[y]);
      __builtin_amdgcn_s_setprio(0);
      u32x4 v[2];
      v[0] = transposed(vb, 16 * VROW);
#pragma unroll
      for (int d = 0; d < DT; ++d) {
        if (d + 1 < DT) v[(d + 1) & 1] = transposed(vb + 32 * (d + 1), 16 * VROW);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int y = 0; y < NM; ++y) {
          O[y][d] = mma<false>(v[d & 1], hi[y], O[y][d]);
          O[y][d] = mma<false>(v[d & 1], lo[y], O[y][d]);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      if (!plain) {
#pragma unroll
        for (int blk = 0; blk < D / kKvBlock; ++blk) {
          constexpr int PB = kKvBlock / T::EP;  // its parts, p the first of them
          constexpr uint32_t two = PB == 4 ? 0x02020202u : PB == 2 ? 0x0202u : 0x02u;
          const int p = blk * PB;
          const uint32_t bad = (uint32_t)(__ballot(((p < 4 ? flags.x : flags.y) >> (8 * (p % 4)) & two) != 0) >> (kTile * sub));
#pragma unroll
          for (int y = 0; y < NM; ++y) lost[y] |= vis[y] & bad ? 1u << blk : 0u;
        }
      }
    }
  }
#pragma unroll
  for (int y = 0; y < NM; ++y) {
    const uint32_t r = first + 16 * y + col;
    const float sum = sum_groups(l[y]), top = m[y] == -INFINITY ? m[y] : __builtin_fmaf(m[y], sc, down);
#pragma unroll
    for (int d = 0; d < DT; ++d)
      if (r < g.p.R) put_row(g, it, r, 16 * d + 4 * grp, lost[y] >> (d / 2) & 1u ? f32x4{NAN, NAN, NAN, NAN} : O[y][d], top, sum);
  }
  __syncthreads();
}

template <bool F16, int BITS, int D, int NM>
__global__ __launch_bounds__(64 * kRowWaves, 2) void q1_kv_rows(const KvArgs g) {
  extern __shared__ unsigned char lds[];
  each_item<kRowWaves>(g, reinterpret_cast<uint32_t*>(lds), [&](const Item& it) { item_by_rows<F16, BITS, D, NM>(g, it, lds); });
}

template <bool F16, int BITS, int D, int NM>
__global__ __launch_bounds__(64 * kWaves, 2) void q1_kv_tokens(const KvArgs g) {
  extern __shared__ unsigned char lds[];
  each_item<kWaves>(g, reinterpret_cast<uint32_t*>(lds), [&](const Item& it) { item_by_tokens<F16, BITS, D, NM>(g, it, lds); });
}

// Where the parts of an item's rows are: of workgroups w0 .. w0 + count - 1, each of which had it
// as its first item, but for one that began with another.  One alone has written the rows.
struct Parts {
  uint32_t w0, count, second, units;
  __device__ __forceinline__ Parts(const KvArgs& g, uint32_t entry, uint32_t hk) : w0(0), count(0), second(0) {
    units = __builtin_amdgcn_readfirstlane(units_of(g, entry));
    if (units == 0) return;
    const Share share(__builtin_amdgcn_readfirstlane(g.before[g.p.entries]), g.p.wgs);
    const uint32_t first = __builtin_amdgcn_readfirstlane(g.before[entry]) + hk * units;
    w0 = share.owner(first);
    count = share.owner(first + units - 1) - w0 + 1;
    second = share.first(w0) != first ? 1 : 0;
  }
  // Row `row` of the item in part s.
  __device__ __forceinline__ int64_t at(const KvArgs& g, uint32_t s, uint32_t row) const {
    return (int64_t)(2 * (w0 + s) + (s == 0 ? second : 0)) * g.p.rows + row;
  }
};

// The rows whose tokens several workgroups had, and those that see none.  A wave has J rows of
// an item, and R waves of a workgroup the same ones, of which each sums every R-th part.
template <int D, int R, int J>
__global__ __launch_bounds__(64 * kWaves) void q1_kv_join(const KvArgs g) {
  constexpr int E = D / 64, U = 8 / J;  // elements a lane, parts in flight
  typedef float vec __attribute__((ext_vector_type(E)));
  __shared__ vec so[kWaves][J][64];
  const q1_kv_query& a = g.a;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t i = blockIdx.x * (kWaves / R) + wave / R;  // of groups of J rows: of an item, then head, entry
  const uint32_t item = divide(i, g.p.groups), row0 = (i - item * g.p.groups_each) * J;
  const uint32_t entry = divide(item, g.p.kv_heads), hk = item - entry * (uint32_t)g.c.Hkv;
  if (entry >= g.p.entries) return;
  const uint32_t b = divide(entry, g.p.blocks), first = (entry - b * g.p.row_blocks) * g.p.rows + row0;
  if (first >= g.p.R) return;
  const Parts parts(g, entry, hk);
  if (parts.count == 1) return;
  vec o[J];
  float top[J], sum[J];
#pragma unroll
  for (int j = 0; j < J; ++j) {
    o[j] = 0.f;
    top[j] = -INFINITY;
    sum[j] = 0.f;
  }
  for (uint32_t c0 = 0; c0 < parts.count; c0 += 64) {  // 64 parts: their factors, one a lane, then every R-th of them
    const uint32_t left = parts.count - c0 < 64 ? parts.count - c0 : 64;
    float f[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const float2 ml = c0 + lane < parts.count ? g.part_ml[parts.at(g, c0 + lane, row0 + j)] : float2{-INFINITY, 0.f};
      float now = fmaxf(top[j], ml.x);
#pragma unroll
      for (int off = 32; off > 0; off >>= 1) now = fmaxf(now, __shfl_xor(now, off));
      const float base = now == -INFINITY ? 0.f : now, keep = __builtin_amdgcn_exp2f(top[j] - base);
      f[j] = __builtin_amdgcn_exp2f(ml.x - base);
      o[j] = keep * o[j];
      sum[j] = keep * sum[j] + f[j] * ml.y;  // (of this lane's parts)
      top[j] = now;
    }
    for (uint32_t s0 = wave % R; s0 < left; s0 += U * R) {
      vec x[U][J];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint32_t s = s0 + u * R < left ? s0 + u * R : left - 1;
#pragma unroll
        for (int j = 0; j < J; ++j) x[u][j] = reinterpret_cast<const vec*>(g.part_o + parts.at(g, c0 + s, row0 + j) * D)[lane];
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint32_t s = s0 + u * R;
#pragma unroll
        for (int j = 0; j < J; ++j) {
          const float fs = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(f[j]), s & 63));
          o[j] = s < left ? o[j] + fs * x[u][j] : o[j];
        }
      }
    }
  }
  if constexpr (R > 1) {  // (every wave has the same top and sum)
#pragma unroll
    for (int j = 0; j < J; ++j) so[wave][j][lane] = o[j];
    __syncthreads();
    if (wave % R != 0) return;
#pragma unroll
    for (int w = 1; w < R; ++w)
#pragma unroll
      for (int j = 0; j < J; ++j) o[j] = o[j] + so[wave + w][j][lane];
  }
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const uint32_t r = first + j;
    if (r >= g.p.R) break;
    const uint32_t t = divide(r, g.p.group), h = hk * g.p.heads_each + (r - t * g.p.heads_each);
    const int64_t row = ((int64_t)b * a.T + t) * a.Hq + h;
    float all = sum[j];
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) all += __shfl_xor(all, off);
    const bool nothing = all == 0.f;  // no token, or none above -infinity (a NaN stays one)
    const float inv = nothing ? 0.f : 1.0f / all;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      float v;
      if constexpr (E == 1) v = o[j][0];
      else v = o[j][e];
      store_out(a.out, a.out_dtype, row * D + lane * E + e, nothing ? 0.f : v * inv);
    }
    if (lane == 0 && a.lse != nullptr) a.lse[row] = nothing ? -INFINITY : lse_of(top[j], all, down_of(length_of(g, b)));
  }
}

template <int D>
hipError_t launch_join(const KvArgs& g, hipStream_t s) {
  const int64_t groups = (int64_t)g.p.entries * g.c.Hkv * g.p.groups_each;
  if (g.p.join_rows == 1)
    hipLaunchKernelGGL((q1_kv_join<D, kWaves, 1>), dim3((unsigned)groups), dim3(64 * kWaves), 0, s, g);
  else
    hipLaunchKernelGGL((q1_kv_join<D, 1, 4>), dim3((unsigned)((groups + kWaves - 1) / kWaves)), dim3(64 * kWaves), 0, s, g);
  return hipGetLastError();
}

template <int D, typename K>
hipError_t launch(K kernel, int waves, int bytes, hipError_t attr, const KvArgs& g, hipStream_t s) {
  if (attr != hipSuccess) return attr;
  hipLaunchKernelGGL(kernel, dim3((unsigned)g.p.wgs), dim3(64 * waves), bytes, s, g);
  const hipError_t e = hipGetLastError();
  return e != hipSuccess || !g.p.cut ? e : launch_join<D>(g, s);
}

template <bool F16, int BITS, int D, int NM>
hipError_t launch_tokens(const KvArgs& g, hipStream_t s) {
  constexpr int bytes = kTokenLds<D, NM, F16 ? 2 : 1>();
  static const hipError_t attr = hipFuncSetAttribute(reinterpret_cast<const void*>(&q1_kv_tokens<F16, BITS, D, NM>),
                                                     hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  return launch<D>(q1_kv_tokens<F16, BITS, D, NM>, kWaves, bytes, attr, g, s);
}

template <bool F16, int BITS, int D>
hipError_t launch_rows(const KvArgs& g, hipStream_t s) {
  constexpr int bytes = 2 * Staged<BITS, D>::kBytes, NM = D < 256 ? 2 : 1;
  static const hipError_t attr = hipFuncSetAttribute(reinterpret_cast<const void*>(&q1_kv_rows<F16, BITS, D, NM>),
                                                     hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  return launch<D>(q1_kv_rows<F16, BITS, D, NM>, kRowWaves, bytes, attr, g, s);
}

template <bool F16, int BITS, int D>
hipError_t launch_n(const KvArgs& g, hipStream_t s) {
  if (g.p.by_rows) return launch_rows<F16, BITS, D>(g, s);
  if constexpr (D < 256) {
    if (g.p.nm == 2) return launch_tokens<F16, BITS, D, 2>(g, s);
  }
  return launch_tokens<F16, BITS, D, 1>(g, s);
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
  p.nm = p.R > 16 && c.D < 256 ? 2 : 1;  // groups of 16 rows a wave: 256 registers hold two of D 128
  const int64_t cus = device_cus(), units = up_div(a.max_pages * c.page_size, kStep);
  // By rows where that form has a full item for half of the compute units, and many tokens.  D 128,
  // group 6, 4 heads of keys, 4 bits, tokens | rows: 8000 queries of 8000 tokens 729 | 552 us, 2 x 1000
  // of 3531 and 5003 199 | 163; few tokens or few items: 2048 of 2048 64 | 91, 512 of 512 14 | 30.
  // Lengths are on the device, so `units` is what the table has room for: a wide table of short
  // sequences is taken for long ones (4 x 512 queries of 512 in a table for 4096 or more 35 | 46,
  // 2048 of 2048 64 | 97; single tokens are cut then, 4 x 519 9.8 | 11, 32 x 2000 21 | 18).
  const int64_t row_items = a.B * (p.R / (16 * p.nm * kRowWaves)) * c.Hkv;
  p.by_rows = 2 * row_items >= cus && units >= 32;
  p.rows = 16 * p.nm * (p.by_rows ? kRowWaves : 1);
  p.row_blocks = (uint32_t)up_div(p.R, p.rows);
  const int64_t items = a.B * p.row_blocks * c.Hkv;
  p.too_large = items >= (int64_t)1 << 31 || (units > 0 && items >= ((int64_t)1 << 31) / units);
  p.entries = p.too_large ? 0 : (uint32_t)(a.B * p.row_blocks);
  // Whole items, or an even cut of all of their units over the workgroups that run at a time:
  // where the last round of whole items would leave more units of time unused than joining costs
  // (a unit of an item by rows takes 4.7 us, one by tokens 1 to 2).  Whole | cut by tokens, 4 bits:
  // 304 items of 40 units 64 | 54 us, 752 of 40 90 | 106, 600 of 16 38 | 51, 512 of 16 33 | 35, 16 of 5
  // 10.2 | 11.5, and at the border 128 of 16 21.8 | 18.8; by rows: 192 of 40 213 | 174, 188 of 40
  // (D 256) 224 | 195, 752 of 63 543 | 748.  Two workgroups by tokens are counted for a compute unit;
  // of D 64 and 128 with 16 rows three or four would fit, of fp16 and D 256 only one does (86 KB of
  // LDS): 32 sequences of 6000 to 8201 tokens 73 us, of bf16 49.
  const int64_t slots = cus * (p.by_rows ? 1 : 2), room = up_div(items, slots) * slots;
  p.cut = !p.too_large && units * (room - items) > (p.by_rows ? 4 : 10 + items / 64) * room;
  if (!p.cut) {
    p.too_large |= items >= ((int64_t)1 << 32) / (64 * (p.by_rows ? kRowWaves : kWaves));  // lanes of a launch
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
  p.group = divider(p.heads_each);
  p.blocks = divider(p.row_blocks);
  // joining: four waves a row where rows are few, else a wave four rows
  p.join_rows = items * p.rows < (int64_t)device_cus() * 16 ? 1 : 4;
  const uint32_t used = p.rows < p.R ? p.rows : p.R;  // rows of an item
  p.groups_each = (uint32_t)up_div(used, p.join_rows);
  p.groups = divider(p.groups_each);
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
