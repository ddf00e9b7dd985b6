// Gated delta rule over whole prompts: chunks of 64 tokens on the matrix cores.
//
// With G_i the running sum of g in a chunk, D_ij = exp(G_i - G_j) (j <= i), S0 the
// state before it and r_i, s_i the norms' reciprocals of k_i and q_i:
//   A_ij = beta_i r_i r_j (k_i.k_j) D_ij (j < i),   T = (I + A)^-1 diag(beta)
//   R = V - diag(r e^G) K S0,   V' = T R
//   O = scale (diag(s e^G) Q S0 + P V'),   P_ij = s_i r_j (q_i.k_j) D_ij (j <= i)
//   S1 = e^{G_63} S0 + K^T diag(r e^{G_63 - G}) V'
// T, P and the factors need no state: q1_chunk_prep makes them for all chunks at
// once.  q1_chunk_run then goes through a sequence's chunks with the state of 32
// columns in registers (columns are independent).
//
// The state is held and returned in fp32 and nothing that reaches it may lose
// that: an fp32 operand of a matrix-core product is taken as three bf16 parts
// (8 significant bits each, cut off, all 24 together), k, q and v as they are
// (bf16, or two parts of an fp16 value: exact).  A product of two fp32 operands
// (T R) sums the products of parts down to 2^-21: what it leaves out is below that
// of the summed magnitudes.  Outputs in fp32 are made the same way.  Those in 16 bits
// take P and V' in two parts, and what these leave out is, of the summed magnitudes,
// below 2^-13 with bf16 operands (P V' without the product of its low parts) and below
// 2^-15 with fp16 ones (low parts to the nearest, all four products; S0 in two parts).
// That is small beside their rounding (2^-9, 2^-12); the rest would be 2 % of the time
// of a long bf16 prompt (688 against 675 us), or 3 % of a ragged fp16 batch's.
// G is summed in 64 bits, so that a difference of two sums is as exact as the
// decays between them whatever came before; the inverse is made by substitution
// and fp32 products.
//
// Operand layouts (16x16x32): lane l has row (or column) l % 16 and eight k
// indices; a result lane has column l % 16, rows 4 (l / 16) .. +3.  Which k
// indices a lane has is free as long as both operands agree, so two result
// tiles (16 rows each) are the operand of the next product as they are: lane l
// has k = 4 (l / 16) .. +3 of both.  The state, R and V' go from product to
// product this way, through LDS only to reach the other waves.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "q1_decode.h"
#include "q1_device.h"
#include "q1_internal.h"

namespace q1 {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef double f64x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

constexpr int C = kDeltaChunk;

// Workspace of one (value head, chunk), a head's chunks one after another (the run
// walks through them; a chunk's heads together cost it a new page every chunk): T
// and P in 10 tiles (it, jt <= it) of 64 lanes x 16 bytes -- T: row 16 it + l%16,
// columns 16 jt + 4(l/16) .. +3 in fp32; P: the same elements as four high and four
// low parts, or in fp32 for outputs in fp32 -- then the factors.  T as the three bf16 parts that the run takes it in,
// and pairs of tiles with zeros, were 31 KB instead of 21.
struct ChunkWs {
  f32x4 T[10][64];
  u32x4 P[10][64];
  float in[C], out[C], read[C];  // r e^G, r e^{G63-G}, scale s e^G
  float keep, pad[63];           // e^{G63}
};
static_assert(sizeof(ChunkWs) == kDeltaChunkBytes, "workspace of a chunk");

// As operands, two tiles side by side: 16 rows it and 32 columns k.
constexpr int pair_of(int it, int k) { return it < 2 ? it : 2 * it - 2 + k; }

__device__ __forceinline__ f32x4 mma(u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

template <bool F16>
__device__ __forceinline__ f32x4 mma_in(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (F16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  else
    return mma(a, b, c);
}

__device__ __forceinline__ f32x4 mma4(f32x4 a, f32x4 b, f32x4 c) {
#pragma unroll
  for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[i], b[i], c, 0, 0, 0);
  return c;
}

// The upper halves of two words.
__device__ __forceinline__ uint32_t tops(uint32_t lo, uint32_t hi) { return __builtin_amdgcn_perm(hi, lo, 0x07060302u); }

__device__ __forceinline__ float rest(float x) { return x - __uint_as_float(__float_as_uint(x) & 0xffff0000u); }

// The leading 8 significant bits of four floats as bf16; x becomes what is left.
__device__ __forceinline__ u32x2 part(f32x4& x) {
  const u32x2 r = {tops(__float_as_uint(x[0]), __float_as_uint(x[1])), tops(__float_as_uint(x[2]), __float_as_uint(x[3]))};
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = rest(x[i]);
  return r;
}

// Four floats rounded to the nearest bf16.
__device__ __forceinline__ u32x2 nearest(f32x4 x) { return __builtin_bit_cast(u32x2, __builtin_convertvector(x, bf16x4)); }

__device__ __forceinline__ void clamp_range(const DeltaArgs& a, int64_t s, int64_t* lo, int64_t* hi) {
  const int64_t l = a.cu[s], h = a.cu[s + 1];
  *lo = l < 0 ? 0 : l > a.tokens ? a.tokens : l;
  *hi = h < 0 ? 0 : h > a.tokens ? a.tokens : h;
}

// Chunk c of sequence s is slot start/64 + s + c: one slot per chunk, no two the
// same (sequences do not overlap), below tokens/64 + nseq + 1.
__device__ __forceinline__ int64_t slot_base(int64_t start, int64_t s) { return start / C + s; }

// Rows [0, n) of a strided operand: loads and stores past them are dropped (loads
// give zeros), so that a chunk that ends early needs no branch.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_of(const void* base, int n, int64_t ld_bytes, int width_bytes) {
  const int bytes = n > 0 ? (int)((n - 1) * ld_bytes) + width_bytes : 0;
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, bytes, 0x00020000);
}

// Workgroups go to the XCDs in turn; each XCD gets a contiguous run of units.
__device__ __forceinline__ int64_t xcd_unit(int64_t units) {
  const int64_t per = (units + 7) / 8;
  return (int64_t)(blockIdx.x & 7) * per + (blockIdx.x >> 3);
}

// v plus the value that the DPP control brings from another lane, where the row mask has this one.
template <int CTRL, int ROWS>
__device__ __forceinline__ double scan_step(double v) {
  const u32x2 b = __builtin_bit_cast(u32x2, v);
  const u32x2 o = {(uint32_t)__builtin_amdgcn_update_dpp(0, (int)b[0], CTRL, ROWS, 0xf, false),
                   (uint32_t)__builtin_amdgcn_update_dpp(0, (int)b[1], CTRL, ROWS, 0xf, false)};
  return v + __builtin_bit_cast(double, o);
}

constexpr int AS = 68;  // LDS row of A in floats

// One workgroup of 4 waves per (chunk, value head); wave `it` has rows 16 it .. +15
// of A, P and T.  Bound by a chunk's chain of steps (some 20000 cycles) with 16 waves
// on a CU to hide it; 16384 tokens of 48 heads, 264 MB of workspace, take 120 us, a
// prompt of two chunks 7.5.
template <bool F16, int DK>
__global__ __launch_bounds__(256, 4) void q1_chunk_prep(const DeltaArgs a, ChunkWs* ws, int64_t slots, int64_t units) {
  constexpr int KS = DK / 32;
  __shared__ __align__(16) float A[C * AS], Kt[C * AS];  // (A's rows first hold the queries)
  __shared__ __align__(16) double Gs[C];
  __shared__ __align__(16) float rks[C], bs[C];
  const int64_t unit = xcd_unit(units);
  if (unit >= units) return;
  const uint32_t slot = (uint32_t)unit / (uint32_t)a.Hv;  // (there are fewer units than 2^31)
  const uint32_t h = (uint32_t)unit - slot * (uint32_t)a.Hv, hk = h / ((uint32_t)a.Hv / (uint32_t)a.Hk);
  int64_t s0 = 0, s1 = a.nseq;  // the last sequence whose first slot is not past this one
  while (s1 - s0 > 1) {
    const int64_t m = (s0 + s1) / 2;
    int64_t lo, hi;
    clamp_range(a, m, &lo, &hi);
    if (slot_base(lo, m) <= slot) s0 = m;
    else s1 = m;
  }
  int64_t lo, hi;
  clamp_range(a, s0, &lo, &hi);
  const int64_t c = slot - slot_base(lo, s0);
  const int64_t t0 = lo + c * C;
  if (c < 0 || t0 >= hi) return;
  const int n = hi - t0 < C ? (int)(hi - t0) : C;
  const int lane = threadIdx.x & 63, col = lane & 15, grp = lane >> 4;
  // in a scalar register: matrix-core products ignore the lane mask, so what they are in must be a scalar branch
  const int it = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  ChunkWs* w = ws + h * slots + slot;

  // lane = token: log decay, write strength; rows past the end are zeros
  const bool in = lane < n;
  float gv = in ? a.g[(t0 + lane) * a.Hv + h] : 0.f;
  const float beta = in ? a.beta[(t0 + lane) * a.Hv + h] : 0.f;
  const auto kr = rows_of(a.k + t0 * a.k_ld + hk * DK, n, a.k_ld * 2, 2 * DK);
  const auto qr = rows_of(a.q + t0 * a.q_ld + hk * DK, n, a.q_ld * 2, 2 * DK);
  // The wave's 16 rows of k and q, through LDS: as operands (rows side by side in a load's
  // lanes) each load took four times as long, and the four waves' took most of the launch.
  constexpr int CH = DK / 8, RL = 64 / CH;  // 16-byte pieces of a row, rows of a load
  u32x4 K[KS], Q[KS];
  {
    u32x4 kv[KS], qv[KS];
    const int r0 = 16 * it + lane / CH, c0 = 16 * (lane % CH);
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      kv[s] = __builtin_amdgcn_raw_buffer_load_b128(kr, (r0 + RL * s) * (int)a.k_ld * 2 + c0, 0, 0);
      qv[s] = __builtin_amdgcn_raw_buffer_load_b128(qr, (r0 + RL * s) * (int)a.q_ld * 2 + c0, 0, 0);
    }
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      *reinterpret_cast<u32x4*>(&Kt[(r0 + RL * s) * AS + c0 / 4]) = kv[s];
      *reinterpret_cast<u32x4*>(&A[(r0 + RL * s) * AS + c0 / 4]) = qv[s];
    }
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
  for (int s = 0; s < KS; ++s) {
    K[s] = *reinterpret_cast<const u32x4*>(&Kt[(16 * it + col) * AS + 4 * grp + 16 * s]);
    Q[s] = *reinterpret_cast<const u32x4*>(&A[(16 * it + col) * AS + 4 * grp + 16 * s]);
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");

  gv = gv < -1000.f ? -1000.f : gv;  // exp is 0 there and below; a sum with -infinity in it would not be a number
  double G = (double)gv * 1.4426950408889634074;  // decay sums in units of log2
  G = scan_step<0x111, 0xf>(G);  // inclusive over the lanes: within rows of 16, then row to row
  G = scan_step<0x112, 0xf>(G);
  G = scan_step<0x114, 0xf>(G);
  G = scan_step<0x118, 0xf>(G);
  G = scan_step<0x142, 0xa>(G);
  G = scan_step<0x143, 0xc>(G);
  const u32x2 last = __builtin_bit_cast(u32x2, G);
  const double G63 = __builtin_bit_cast(
      double, u32x2{(uint32_t)__builtin_amdgcn_readlane((int)last[0], 63), (uint32_t)__builtin_amdgcn_readlane((int)last[1], 63)});
  float rq = 1.f;  // of row 16 it + col
  if (it == 0) {
    Gs[lane] = G;
    bs[lane] = beta;
  }
  if (a.l2norm) {
    f32x4 kk = {0.f, 0.f, 0.f, 0.f}, qq = kk;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      kk = mma_in<F16>(K[s], K[s], kk);
      qq = mma_in<F16>(Q[s], Q[s], qq);
    }
    // the diagonal: lane (col, grp) with col / 4 == grp has it, in place col % 4
    const int e = col & 3;
    const float dk = e == 0 ? kk[0] : e == 1 ? kk[1] : e == 2 ? kk[2] : kk[3];
    const float dq = e == 0 ? qq[0] : e == 1 ? qq[1] : e == 2 ? qq[2] : qq[3];
    const int from = col + 16 * (col >> 2);
    if (grp == col >> 2) rks[16 * it + col] = 1.0f / sqrtf(dk + 1e-6f);
    rq = 1.0f / sqrtf(__shfl(dq, from) + 1e-6f);
  } else if (grp == 0) {
    rks[16 * it + col] = 1.f;
  }
  __syncthreads();
  const int i = 16 * it + col;
  const double Gi = Gs[i];
  if (grp == 0) {
    const float eG = __builtin_amdgcn_exp2f((float)Gi);
    w->in[i] = rks[i] * eG;
    w->out[i] = rks[i] * __builtin_amdgcn_exp2f((float)(G63 - Gi));
    w->read[i] = a.scale * rq * eG;
    if (i == 0) w->keep = __builtin_amdgcn_exp2f((float)G63);
  }

  // A (rows i = l % 16, columns j = 4 (l / 16) .. +3 of a tile) to LDS, P to the workspace
  {
    const float bi = bs[i] * rks[i], qi = a.scale * rq;
    auto tile = [&](int jt) {
      f32x4 kk = {0.f, 0.f, 0.f, 0.f}, qk = kk;
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        const u32x4 kj = *reinterpret_cast<const u32x4*>(&Kt[(16 * jt + col) * AS + 4 * grp + 16 * s]);
        kk = mma_in<F16>(kj, K[s], kk);
        qk = mma_in<F16>(kj, Q[s], qk);
      }
      const int j0 = 16 * jt + 4 * grp;
      const f32x4 rj = *reinterpret_cast<const f32x4*>(&rks[j0]);
      const f64x2 Ga = *reinterpret_cast<const f64x2*>(&Gs[j0]), Gb = *reinterpret_cast<const f64x2*>(&Gs[j0 + 2]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const double Gj = e < 2 ? Ga[e & 1] : Gb[e & 1];
        const float d = rj[e] * __builtin_amdgcn_exp2f((float)(Gi - Gj));
        kk[e] = i > j0 + e ? bi * kk[e] * d : 0.f;
        qk[e] = i >= j0 + e ? qi * qk[e] * d : 0.f;
      }
      *reinterpret_cast<f32x4*>(&A[i * AS + j0]) = kk;
      u32x4 pw = __builtin_bit_cast(u32x4, qk);
      if (a.out_dtype != F32) {
        const u32x2 ph = part(qk), pl = nearest(qk);
        pw = u32x4{ph[0], ph[1], pl[0], pl[1]};
      }
      w->P[it * (it + 1) / 2 + jt][lane] = pw;
    };
    for (int jt = 0; jt <= it; ++jt) tile(jt);
  }
  __syncthreads();

  // Inverse of I + A in place.  The four diagonal blocks by substitution, all by one
  // wave (a block per 16 lanes, a column per lane) ...
  if (it == 0) {
    float x[16];
    float* Ab = &A[(16 * grp) * AS + 16 * grp];
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      float s0v = 0.f, s1v = 0.f;
#pragma unroll
      for (int k = 0; k < r; k += 4) {
        const f32x4 y = *reinterpret_cast<const f32x4*>(Ab + r * AS + k);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (k + e < r) {
            if (e & 1) s1v = __builtin_fmaf(y[e], x[k + e], s1v);
            else s0v = __builtin_fmaf(y[e], x[k + e], s0v);
          }
      }
      x[r] = (r == col ? 1.f : 0.f) - (s0v + s1v);
    }
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int r = 0; r < 16; ++r) Ab[r * AS + col] = x[r];
  }
  __syncthreads();
  // ... then, with I, J the blocks of the lower and upper half: T_IJ = -T_II' A_I'J' T_J'J,
  // first for halves of 16 rows (waves 1 and 3), then of 32 (a wave each block).
  auto row4 = [&](int I, int J) { return *reinterpret_cast<const f32x4*>(&A[(16 * I + col) * AS + 16 * J + 4 * grp]); };
  auto col4 = [&](int I, int J) {
    f32x4 r;
#pragma unroll
    for (int e = 0; e < 4; ++e) r[e] = A[(16 * I + 4 * grp + e) * AS + 16 * J + col];
    return r;
  };
  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
  if (it & 1) {
    const f32x4 y = mma4(row4(it, it - 1), col4(it - 1, it - 1), zero);
    const f32x4 x = mma4(y, row4(it, it), zero);
    *reinterpret_cast<f32x4*>(&A[(16 * it + col) * AS + 16 * (it - 1) + 4 * grp]) = -x;
  }
  __syncthreads();
  {
    const int I = it >> 1, J = it & 1;
    auto half = [&](int r) {  // rows 2 + r of A times the upper half's inverse, columns J
      f32x4 y = mma4(row4(2 + r, 1), col4(1, J), zero);
      if (J == 0) y = mma4(row4(2 + r, 0), col4(0, 0), y);
      return y;
    };
    const f32x4 y0 = half(0);
    f32x4 x;
    if (I == 0) x = mma4(y0, row4(2, 2), zero);
    else x = mma4(half(1), row4(3, 3), mma4(y0, row4(3, 2), zero));
    __syncthreads();
    *reinterpret_cast<f32x4*>(&A[(32 + 16 * I + col) * AS + 16 * J + 4 * grp]) = -x;
  }
  __syncthreads();
#pragma unroll
  for (int jt = 0; jt < 4; ++jt)
    if (jt <= it) w->T[it * (it + 1) / 2 + jt][lane] = row4(it, jt) * *reinterpret_cast<const f32x4*>(&bs[16 * jt + 4 * grp]);
}

// One workgroup of 8 waves per (sequence, value head, 32 columns of the state).
// Waves 0..3 carry the state, waves 4..7 make the output; of each, wave (sl, hf) has
// the 16 columns sl, the tokens 32 hf .. +31 of a chunk and (state) the rows
// hf DK/2 .. of the state.  What a wave makes itself it uses from its registers;
// LDS only carries the other half.  Loads are those of the next chunk, into the
// registers that a product has just read.
//
// A chunk has three parts between barriers: K S0 and R with the half of V' that needs
// no other wave; the other half, W and half of the new state; the rest of it and its
// parts.  Bound by this chain: 2.4 us a chunk (bf16, 128x128), of which the matrix
// cores are busy 0.6 and the vector units 0.75; the output waves' work is dealt so
// that the first two do not wait for it, and the third hardly (with the output made in
// the first part and Q S0 in the second, 8192 tokens of 48 heads took 378 us instead of
// 362; a product more in the third costs 2 %, in the first nothing).  Three bf16
// parts keep the state in fp32.  Four waves with 16 columns and no division of labour
// took 932 us for 16384 tokens when eight with 32 took 863.
constexpr int kRunThreads = 512;

// The sequence in `place` by length, the longest first, among its block of 64: the longest
// ones have to start first, or the launch waits for them at its end (7 sequences of 39 to
// 1969 tokens with 32 heads: 302 us in the order given, an XCD after the other, 127 so).
__device__ __forceinline__ int64_t by_length(const DeltaArgs& a, int64_t place) {
  const int lane = threadIdx.x & 63;
  const int64_t base = place & ~(int64_t)63;
  const int n = a.nseq - base < 64 ? (int)(a.nseq - base) : 64;
  int64_t lo = 0, hi = 0;
  if (lane < n) clamp_range(a, base + lane, &lo, &hi);
  const int mine = (int)(hi - lo);
  int before = 0;
  for (int i = 0; i < n; ++i) {
    const int other = __builtin_amdgcn_readlane(mine, i);
    before += other > mine || (other == mine && i < lane);
  }
  const uint64_t found = __ballot(lane < n && before == (int)(place - base));
  return base + __builtin_ctzll(found);
}

constexpr int kVRow = 64 + 16;  // LDS bytes of a row of 32 values

template <bool F16, int DK, bool OUT32>
__global__ __launch_bounds__(kRunThreads) void q1_chunk_run(const DeltaArgs a, const ChunkWs* ws, int64_t slots) {
  constexpr int KS = DK / 32, HS = KS / 2, KP = F16 ? 2 : 1, ST = DK / 32;  // k steps (a half), parts of k and q, state tiles
  constexpr int KROW = 2 * DK + (F16 && DK == 128 ? 16 : 32), CH = DK / 8, NL = C * CH / 256;  // LDS bytes of a key row, 16-byte pieces, loads
  __shared__ __align__(16) unsigned char kt[2][KP][C * KROW], qt[C * KROW], vt[C * kVRow];
  __shared__ __align__(16) u32x4 Ss[2][KS][3][64], Rs[2][3][64], Ws[2][2][3][64];
  __shared__ __align__(16) u32x4 Ts[6][3][64];
  __shared__ __align__(16) f32x4 Vs[2][4][64];
  // (sequence, head) pairs go to the XCDs in turn, a pair's column slices to the same one,
  // and where the heads divide evenly an XCD has neighbours, which share keys.  (There are
  // fewer workgroups than 2^31.)
  const uint32_t slices = (uint32_t)(a.Dv + 31) / 32, Hv = (uint32_t)a.Hv, at = blockIdx.x >> 3;
  const uint32_t pair = at / slices * 8 + (blockIdx.x & 7), place = pair / Hv, j = pair - place * Hv;
  if (place >= (uint64_t)a.nseq) return;
  const uint32_t h = Hv % 8 == 0 ? (j & 7) * (Hv / 8) + (j >> 3) : j, hk = h / (Hv / (uint32_t)a.Hk);
  const int64_t seq = a.nseq == 1 ? 0 : by_length(a, place);
  const int lane = threadIdx.x & 63, col = lane & 15, grp = lane >> 4;
  // in a scalar register: matrix-core products ignore the lane mask, so what they are in must be a scalar branch
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int sl = (wave >> 1) & 1, hf = wave & 1;
  const int c0 = (int)(at % slices) * 32 + 16 * sl;
  const bool live = c0 < a.Dv;  // Dv may end with the first 16 columns
  int64_t lo, hi;
  clamp_range(a, seq, &lo, &hi);
  if (lo >= hi) return;
  const int64_t slot = a.slot_ids ? a.slot_ids[seq] : seq;
  constexpr int esz = OUT32 ? 4 : 2;
  unsigned char* ob = static_cast<unsigned char*>(a.out) + (int64_t)h * a.Dv * esz;
  const int64_t o_ld = (int64_t)a.Hv * a.Dv * esz;
  constexpr int kNone = 1 << 30;  // an offset past every range
  if (slot < 0 || slot >= a.slots) {  // no state: zeros
    for (int64_t t = lo + (threadIdx.x >> 2); t < hi; t += kRunThreads / 4) {
      const int c = (c0 & ~31) + 8 * (threadIdx.x & 3);
      if (c < a.Dv)
#pragma unroll
        for (int e = 0; e < 8 * esz / 16; ++e)
          *reinterpret_cast<u32x4*>(ob + t * o_ld + c * esz + 16 * e) = u32x4{0u, 0u, 0u, 0u};
    }
    return;
  }
  const ChunkWs* w = ws + h * slots + slot_base(lo, seq);
  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
  auto left = [&](int64_t t0) { return hi - t0 < C ? (int)(hi - t0) : C; };
  // k's fp16 pairs as two bf16 parts (11 bits: exact)
  auto halves = [](uint32_t w2, uint32_t* hi_, uint32_t* lo_) {
    const float x = f16_bits_to_f32(w2 & 0xffffu), y = f16_bits_to_f32(w2 >> 16);
    *hi_ = tops(__float_as_uint(x), __float_as_uint(y));
    *lo_ = tops(__float_as_uint(rest(x)), __float_as_uint(rest(y)));
  };

  if (wave < 4) {
    // ---- state ----
    // tile t is rows hf DK/2 + 32 (t/2) + 4 (t%2) + 8 grp .. +3, column col
    f32x4 S[ST];
    u32x4 Sp[HS][3];
    float* sp = a.state + ((slot * a.Hv + h) * DK + hf * (DK / 2) + 8 * grp) * (int64_t)a.Dv + c0 + col;
    auto row = [](int t, int e) { return 32 * (t >> 1) + 4 * (t & 1) + e; };
#pragma unroll
    for (int t = 0; t < ST; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) S[t][e] = live ? sp[(int64_t)row(t, e) * a.Dv] : 0.f;
    auto put_state = [&]() {
#pragma unroll
      for (int s = 0; s < HS; ++s) {
        f32x4 x = S[2 * s], y = S[2 * s + 1];
#pragma unroll
        for (int p = 0; p < 3; ++p) {
          const u32x2 xp = part(x), yp = part(y);
          Sp[s][p] = u32x4{xp[0], xp[1], yp[0], yp[1]};
          Ss[sl][hf * HS + s][p][lane] = Sp[s][p];
        }
      }
    };
    f32x4 in[2], outf[2];
    float keep;
    auto load_in = [&](const ChunkWs* cw) {
#pragma unroll
      for (int i = 0; i < 2; ++i) in[i] = *reinterpret_cast<const f32x4*>(&cw->in[32 * hf + 16 * i + 4 * grp]);
    };
    // pairs of T with the own columns: (0,0) (1,0) or (2,1) (3,1); with the others: none or (2,0) (3,0)
    const int t_own = hf ? 3 : 0, t_oth = 2, t_step = hf ? 2 : 1;
    auto load_out = [&](const ChunkWs* cw) {
#pragma unroll
      for (int i = 0; i < 2; ++i) outf[i] = *reinterpret_cast<const f32x4*>(&cw->out[32 * hf + 16 * i + 4 * grp]);
      keep = cw->keep;
    };
    // K S0 of this wave's tokens: with its own half of the state (from registers), with the other (from LDS)
    f32x4 ks[2];
    auto scores = [&](int o, int b) {
#pragma unroll
      for (int s = 0; s < HS; ++s) {
        const int kk = (o ? 1 - hf : hf) * HS + s;
        u32x4 sv[3];
#pragma unroll
        for (int p = 0; p < 3; ++p) sv[p] = o ? Ss[sl][kk][p][lane] : Sp[s][p];
        u32x4 kop[2][KP];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int p = 0; p < KP; ++p)
            kop[i][p] = *reinterpret_cast<const u32x4*>(&kt[b][p][(32 * hf + 16 * i + col) * KROW + 64 * kk + 16 * grp]);
#pragma unroll
        for (int p = 2; p >= 0; --p)
#pragma unroll
          for (int i = 0; i < 2; ++i) ks[i] = mma(kop[i][0], sv[p], ks[i]);
        if constexpr (F16) {
#pragma unroll
          for (int p = 1; p >= 0; --p)
#pragma unroll
            for (int i = 0; i < 2; ++i) ks[i] = mma(kop[i][KP - 1], sv[p], ks[i]);
        }
      }
    };
    load_in(w);
    load_out(w);
    put_state();
    __syncthreads();
    int buf = 0;
    ks[0] = ks[1] = zero;
    scores(0, 0);
    for (int64_t t0 = lo; t0 < hi; t0 += C, buf ^= 1) {
      const ChunkWs* wn = t0 + C < hi ? w + 1 : w;
      // K S0: the rest, with the other half's state from LDS
      scores(1, buf);
      f32x4 rr[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const s16x4 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (lds_s16x4*)&vt[(32 * hf + 16 * i + 4 * grp + col / 4) * kVRow + 32 * sl + 8 * (col & 3)]);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          rr[i][e] = (F16 ? f16_bits_to_f32((uint16_t)v[e]) : bf16_bits_to_f32((uint16_t)v[e])) - in[i][e] * ks[i][e];
      }
      load_in(wn);
      u32x4 R[3];
#pragma unroll
      for (int p = 0; p < 3; ++p) {
        const u32x2 x = part(rr[0]), y = part(rr[1]);
        R[p] = u32x4{x[0], x[1], y[0], y[1]};
        if (hf == 0) Rs[sl][p][lane] = R[p];
      }
      // V' = T R: the six products of parts down to 2^-24
      f32x4 vn[2] = {zero, zero};
      auto times = [&](int o, const u32x4* r) {
        u32x4 T[2][3];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int p = 0; p < 3; ++p) T[i][p] = Ts[(o ? t_oth : t_own) + i * t_step][p][lane];
#pragma unroll
        for (int x = 2; x >= 0; --x)
#pragma unroll
          for (int p = 0; p <= x; ++p)
#pragma unroll
            for (int i = 0; i < 2; ++i) vn[i] = mma(T[i][p], r[x - p], vn[i]);
      };
      times(0, R);
      __syncthreads();
      if (hf == 1) {
        u32x4 r0[3];
#pragma unroll
        for (int p = 0; p < 3; ++p) r0[p] = Rs[sl][p][lane];
        times(1, r0);
      }
      u32x4 W[3];
      {
        f32x4 x = outf[0] * vn[0], y = outf[1] * vn[1];
#pragma unroll
        for (int p = 0; p < 3; ++p) {
          const u32x2 xp = part(x), yp = part(y);
          W[p] = u32x4{xp[0], xp[1], yp[0], yp[1]};
          Ws[sl][hf][p][lane] = W[p];
        }
        Vs[sl][2 * hf][lane] = vn[0];
        Vs[sl][2 * hf + 1][lane] = vn[1];
      }
#pragma unroll
      for (int t = 0; t < ST; ++t) S[t] *= keep;
      load_out(wn);
      // S1 = e^{G63} S0 + K^T W
      auto update = [&](int k, const u32x4* wv) {
        u32x4 kop[ST][KP];
#pragma unroll
        for (int t = 0; t < ST; ++t)
#pragma unroll
          for (int p = 0; p < KP; ++p) {
            const unsigned char* kr = &kt[buf][p][(32 * k + 4 * grp + col / 4) * KROW + DK * hf + 64 * (t >> 1) + 8 * (t & 1) + 16 * (col & 3)];
            const s16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)kr);
            const s16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(kr + 16 * KROW));
            const u32x2 xw = __builtin_bit_cast(u32x2, x), yw = __builtin_bit_cast(u32x2, y);
            kop[t][p] = u32x4{xw[0], xw[1], yw[0], yw[1]};
          }
#pragma unroll
        for (int p = 2; p >= 0; --p)
#pragma unroll
          for (int t = 0; t < ST; ++t) S[t] = mma(kop[t][0], wv[p], S[t]);
        if constexpr (F16) {
#pragma unroll
          for (int p = 1; p >= 0; --p)
#pragma unroll
            for (int t = 0; t < ST; ++t) S[t] = mma(kop[t][KP - 1], wv[p], S[t]);
        }
      };
      update(hf, W);
      __syncthreads();
#pragma unroll
      for (int p = 0; p < 3; ++p) W[p] = Ws[sl][1 - hf][p][lane];
      update(1 - hf, W);
      put_state();
      ks[0] = ks[1] = zero;
      scores(0, buf ^ 1);  // (the next keys are there since the barrier before)
      __syncthreads();
      w = wn;
    }
    if (live)
#pragma unroll
      for (int t = 0; t < ST; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) sp[(int64_t)row(t, e) * a.Dv] = S[t][e];
  } else {
    // ---- output, and the next chunk's keys ----
    const int tid = threadIdx.x & 255;
    u32x4 Kn[NL], Qn[NL], Vn, P[2][4];  // (n: the next chunk's)
    f32x4 Tn[3];
    float read[2];
    const int k_off = (tid / CH) * (int)a.k_ld * 2 + 16 * (tid % CH), k_step = (256 / CH) * (int)a.k_ld * 2;
    const int q_off = (tid / CH) * (int)a.q_ld * 2 + 16 * (tid % CH), q_step = (256 / CH) * (int)a.q_ld * 2;
    const int vc = (c0 & ~31) + 8 * (tid & 3);
    const int v_off = vc < a.Dv ? (tid >> 2) * (int)a.v_ld * 2 + 2 * vc : kNone;
    auto load_k = [&](int64_t t0) {
      const auto r = rows_of(a.k + t0 * a.k_ld + hk * DK, left(t0), a.k_ld * 2, 2 * DK);
#pragma unroll
      for (int i = 0; i < NL; ++i) Kn[i] = __builtin_amdgcn_raw_buffer_load_b128(r, k_off + i * k_step, 0, 0);
      const auto rv = rows_of(a.v + t0 * a.v_ld + (int64_t)h * a.Dv, left(t0), a.v_ld * 2, 2 * a.Dv);
      Vn = __builtin_amdgcn_raw_buffer_load_b128(rv, v_off, 0, 0);
    };
    auto load_q = [&](int64_t t0) {
      const auto r = rows_of(a.q + t0 * a.q_ld + hk * DK, left(t0), a.q_ld * 2, 2 * DK);
#pragma unroll
      for (int i = 0; i < NL; ++i) Qn[i] = __builtin_amdgcn_raw_buffer_load_b128(r, q_off + i * q_step, 0, 0);
    };
    auto put_q = [&]() {
#pragma unroll
      for (int i = 0; i < NL; ++i)
        *reinterpret_cast<u32x4*>(&qt[((i * 256 + tid) / CH) * KROW + 16 * (tid % CH)]) = Qn[i];
    };
    auto put_kv = [&](int b) {
      *reinterpret_cast<u32x4*>(&vt[(tid >> 2) * kVRow + 16 * (tid & 3)]) = Vn;
#pragma unroll
      for (int i = 0; i < NL; ++i) {
        const int at = ((i * 256 + tid) / CH) * KROW + 16 * (tid % CH);
        if constexpr (F16) {
          u32x4 p0, p1;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t x0, x1;
            halves(Kn[i][e], &x0, &x1);
            p0[e] = x0;
            p1[e] = x1;
          }
          *reinterpret_cast<u32x4*>(&kt[b][0][at]) = p0;
          *reinterpret_cast<u32x4*>(&kt[b][KP - 1][at]) = p1;
        } else {
          *reinterpret_cast<u32x4*>(&kt[b][0][at]) = Kn[i];
        }
      }
    };
    // tiles (2 hf + i, j) of P; those above the diagonal are past the range: zeros
    int p_off[2][4];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int it = 2 * hf + i;
        p_off[i][j] = j <= it ? (it * (it + 1) / 2 + j) * 1024 + 16 * lane : kNone;
      }
    auto load_p = [&](const ChunkWs* cw) {
      const auto r = __builtin_amdgcn_make_buffer_rsrc(const_cast<u32x4*>(&cw->P[0][0]), (short)0, (int)sizeof(cw->P), 0x00020000);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int j = 0; j < 4; ++j) P[i][j] = __builtin_amdgcn_raw_buffer_load_b128(r, p_off[i][j], 0, 0);
        read[i] = cw->read[32 * hf + 16 * i + col];
      }
    };
    // T: wave x of the four takes tiles x, x + 4, x + 8 (of 10) from the workspace to LDS, in three parts
    const int tw = wave & 3;
    auto load_t = [&](const ChunkWs* cw) {
      const auto r = __builtin_amdgcn_make_buffer_rsrc(const_cast<f32x4*>(&cw->T[0][0]), (short)0, (int)sizeof(cw->T), 0x00020000);
#pragma unroll
      for (int i = 0; i < 3; ++i)
        Tn[i] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(r, (tw + 4 * i) * 1024 + 16 * lane, 0, 0));
    };
    u32x2 Tp[3][3];
    auto split_t = [&]() {
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        f32x4 x = Tn[i];
#pragma unroll
        for (int p = 0; p < 3; ++p) Tp[i][p] = part(x);
      }
    };
    auto put_t = [&]() {
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        const int t = tw + 4 * i, it = t < 1 ? 0 : t < 3 ? 1 : t < 6 ? 2 : 3, jt = t - it * (it + 1) / 2;
        if (t < 10) {
#pragma unroll
          for (int p = 0; p < 3; ++p)
            reinterpret_cast<u32x2*>(&Ts[it < 2 ? it : 2 * it - 2 + (jt >> 1)][p][lane])[jt & 1] = Tp[i][p];
        }
      }
    };
    u32x4 Pp[2][2][OUT32 ? 3 : 1];  // P's parts, for outputs in fp32: made before the output needs them, where
                                    // these waves wait (16384 tokens of 48 heads 774 us, with the output 821)
    auto split_p = [&]() {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          f32x4 x = __builtin_bit_cast(f32x4, P[i][2 * k]), y = __builtin_bit_cast(f32x4, P[i][2 * k + 1]);
#pragma unroll
          for (int p = 0; p < (OUT32 ? 3 : 1); ++p) {
            const u32x2 xp = part(x), yp = part(y);
            Pp[i][k][p] = u32x4{xp[0], xp[1], yp[0], yp[1]};
          }
        }
    };
    const int o_off = live ? (32 * hf + col) * (int)o_ld + (c0 + 4 * grp) * esz : kNone;
    f32x4 qs[2] = {zero, zero};
    // O^T = scale s e^G (Q S0)^T + V'^T P^T; a lane has token 32 hf + 16 i + col
    f32x4 o[2] = {zero, zero};
    auto finish = [&]() {
      o[0] = read[0] * qs[0];
      o[1] = read[1] * qs[1];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        f32x4 x = Vs[sl][2 * k][lane], y = Vs[sl][2 * k + 1][lane];
        if constexpr (OUT32) {  // three parts of both, as in the state
          u32x4 vp[3];
#pragma unroll
          for (int p = 0; p < 3; ++p) {
            const u32x2 xp = part(x), yp = part(y);
            vp[p] = u32x4{xp[0], xp[1], yp[0], yp[1]};
          }
#pragma unroll
          for (int n = 2; n >= 0; --n)
#pragma unroll
            for (int p = 0; p <= n; ++p)
#pragma unroll
              for (int i = 0; i < 2; ++i) o[i] = mma(vp[p], Pp[i][k][n - p], o[i]);
          continue;
        }
        const u32x2 x0 = part(x), x1 = F16 ? nearest(x) : part(x), y0 = part(y), y1 = F16 ? nearest(y) : part(y);
        const u32x4 v0 = {x0[0], x0[1], y0[0], y0[1]}, v1 = {x1[0], x1[1], y1[0], y1[1]};
        u32x4 ph[2], pl[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          ph[i] = u32x4{P[i][2 * k][0], P[i][2 * k][1], P[i][2 * k + 1][0], P[i][2 * k + 1][1]};
          pl[i] = u32x4{P[i][2 * k][2], P[i][2 * k][3], P[i][2 * k + 1][2], P[i][2 * k + 1][3]};
        }
        if constexpr (F16) {
#pragma unroll
          for (int i = 0; i < 2; ++i) o[i] = mma(v1, pl[i], o[i]);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) o[i] = mma(v1, ph[i], o[i]);
#pragma unroll
        for (int i = 0; i < 2; ++i) o[i] = mma(v0, pl[i], o[i]);
#pragma unroll
        for (int i = 0; i < 2; ++i) o[i] = mma(v0, ph[i], o[i]);
      }
    };
    auto store = [&](int64_t t, int n) {
      const auto ores = rows_of(ob + t * o_ld, n, o_ld, a.Dv * esz);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if constexpr (OUT32) {
          __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, o[i]), ores, o_off + 16 * i * (int)o_ld, 0, 0);
        } else {
          const u32x2 b16 = __builtin_bit_cast(u32x2, __builtin_convertvector(o[i], bf16x4));
          const u32x2 h16 = __builtin_bit_cast(u32x2, __builtin_convertvector(o[i], f16x4));
          __builtin_amdgcn_raw_buffer_store_b64(a.out_dtype == BF16 ? b16 : h16, ores, o_off + 16 * i * (int)o_ld, 0, 0);
        }
      }
    };
    load_k(lo);
    load_q(lo);
    load_p(w);
    load_t(w);
    put_kv(0);
    put_q();
    // the upper halves of pairs (0,0) and (2,1) stay zero
    if (tw == 0)
#pragma unroll
      for (int p = 0; p < 3; ++p)
        reinterpret_cast<u32x2*>(&Ts[pair_of(0, 0)][p][lane])[1] = reinterpret_cast<u32x2*>(&Ts[pair_of(2, 1)][p][lane])[1] = u32x2{0u, 0u};
    split_t();
    put_t();
    load_t(lo + C < hi ? w + 1 : w);
    load_k(lo + C);
    load_q(lo + C);
    __syncthreads();
    int buf = 0, done = 0;  // rows of the chunk before that wait for store(): none at first
    for (int64_t t0 = lo; t0 < hi; t0 += C, buf ^= 1) {
      // while the state waves make R: the chunk before goes out, (Q S0)^T
      store(t0 - done, done);
      done = C;
      qs[0] = qs[1] = zero;
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        const u32x4 s0 = Ss[sl][s][0][lane], s1 = Ss[sl][s][1][lane], s2 = Ss[sl][s][2][lane];
        u32x4 Q[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) Q[i] = *reinterpret_cast<const u32x4*>(&qt[(32 * hf + 16 * i + col) * KROW + 64 * s + 16 * grp]);
        if constexpr (F16) {
          u32x4 q0[2], q1[2];
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t h0, h1;
              halves(Q[i][e], &h0, &h1);
              q0[i][e] = h0;
              q1[i][e] = h1;
            }
          if constexpr (OUT32) {
#pragma unroll
            for (int i = 0; i < 2; ++i) qs[i] = mma(s2, q0[i], qs[i]);
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) qs[i] = mma(s1, q1[i], qs[i]);
#pragma unroll
          for (int i = 0; i < 2; ++i) qs[i] = mma(s0, q1[i], qs[i]);
#pragma unroll
          for (int i = 0; i < 2; ++i) qs[i] = mma(s1, q0[i], qs[i]);
#pragma unroll
          for (int i = 0; i < 2; ++i) qs[i] = mma(s0, q0[i], qs[i]);
        } else {
#pragma unroll
          for (int i = 0; i < 2; ++i) qs[i] = mma(s2, Q[i], qs[i]);
#pragma unroll
          for (int i = 0; i < 2; ++i) qs[i] = mma(s1, Q[i], qs[i]);
#pragma unroll
          for (int i = 0; i < 2; ++i) qs[i] = mma(s0, Q[i], qs[i]);
        }
      }
      if constexpr (OUT32) split_p();
      __syncthreads();
      // while they make V' and half of the new state: the next keys, values and queries
      split_t();
      put_kv(buf ^ 1);
      load_k(t0 + 2 * C);
      put_q();
      load_q(t0 + 2 * C);
      __syncthreads();
      // while they make the rest of it: the output, and the next T
      const ChunkWs* wn = t0 + C < hi ? w + 1 : w;
      finish();
      load_p(wn);
      put_t();
      load_t(t0 + 2 * C < hi ? wn + 1 : wn);
      w = wn;
      __syncthreads();
    }
    const int64_t last = lo + (hi - lo - 1) / C * C;
    store(last, (int)(hi - last));
  }
}

template <bool F16, int DK>
hipError_t launch_t(const DeltaArgs& a, ChunkWs* ws, hipStream_t s) {
  const int64_t slots = delta_chunk_slots(a.tokens, a.nseq), prep = slots * a.Hv;
  hipLaunchKernelGGL((q1_chunk_prep<F16, DK>), dim3((unsigned)((prep + 7) / 8 * 8)), dim3(256), 0, s, a, ws, slots, prep);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const dim3 grid((unsigned)((a.nseq * a.Hv + 7) / 8 * 8 * ((a.Dv + 31) / 32)));
  if (a.out_dtype == F32)
    hipLaunchKernelGGL((q1_chunk_run<F16, DK, true>), grid, dim3(kRunThreads), 0, s, a, ws, slots);
  else
    hipLaunchKernelGGL((q1_chunk_run<F16, DK, false>), grid, dim3(kRunThreads), 0, s, a, ws, slots);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_delta_chunk(const DeltaArgs& a, bool f16, int Dk, unsigned char* ws, hipStream_t s) {
  ChunkWs* w = reinterpret_cast<ChunkWs*>(ws);
  if (f16) return Dk == 128 ? launch_t<true, 128>(a, w, s) : launch_t<true, 64>(a, w, s);
  return Dk == 128 ? launch_t<false, 128>(a, w, s) : launch_t<false, 64>(a, w, s);
}

}  // namespace q1
