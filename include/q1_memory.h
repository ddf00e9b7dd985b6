/*
 * q1_memory.h -- what a decoder remembers between tokens, beside the gated delta
 * rule's states (q1_decode.h): keys and values in pages of 4 or 8 bits with the
 * attention that reads them, the window of a short causal convolution, and the
 * states of a selective state space scan.
 *
 * The conventions of q1.h and q1_decode.h hold: caller-owned device memory,
 * argument checks before any HIP call, then the workspace check, then the device
 * check; calls only enqueue work on `stream`, allocate nothing, keep nothing
 * between calls, and can be captured in a HIP graph.  Workspaces need no initial
 * contents; calls that may run at the same time need separate ones.  A workspace
 * query returns 0 for a call that needs none, and with an error text for one that is
 * refused.  Outputs must not overlap inputs, but for states, which are updated in place.
 *
 * Numbers the kernels read from device memory (lengths, offsets, page and slot
 * ids) cannot be checked by the call; each one below says what an id outside
 * its range does.  No such value makes a kernel read or write out of bounds.
 */
#ifndef Q1_MEMORY_H
#define Q1_MEMORY_H

#include "q1.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Pages of keys and values.  32 consecutive elements of a (token, head) are a
 * block with one scale 2^e, held as the byte e + 127; an element is a code c of
 * bits = 4: sign and one of 0, 0.5, 1, 1.5, 2, 3, 4, 6 (E2M1), two to a byte, the even
 *           element in the low half;
 * bits = 8: E4M3, largest 448;
 * and stands for c * 2^e, exact in bf16.  q1_kv_write takes the smallest e with
 * max |x| <= 1.75 * 2^(e + p), p = 2 or 8 (so the largest element is off by at most
 * half of its own step), and the nearest code, ties to even.  The byte is kept within
 * 2..252 (bits = 4) or 10..246 (bits = 8), and up to 140 or 134 for fp16 operands: the
 * values are normal numbers and finite in the operands' type; what is larger takes
 * the largest code.  A block with a NaN or an infinity has the byte 255 and zero
 * codes, and is NaN as a whole.
 */
typedef struct q1_kv {
  void* k;            /* [pages, Hkv, page_size, D * bits / 8]; 16-byte aligned */
  void* v;            /* as k */
  void* k_scales;     /* [pages, Hkv, page_size, D / 32] bytes; 8-byte aligned */
  void* v_scales;     /* as k_scales */
  int64_t pages;      /* pages * page_size below 2^31 */
  int64_t page_size;  /* Hkv * page_size * D below 2^31 */
  int32_t Hkv;
  int32_t D;          /* 64, 128 or 256 */
  int32_t bits;       /* 4 or 8 */
  int32_t reserved;   /* 0 */
} q1_kv;

/*
 * q1_kv_write -- quantises `tokens` rows of keys and values into the pages: row t
 * goes to token slots[t] % page_size of page slots[t] / page_size.  Slots are
 * distinct (of one that comes twice, the row is a mixture of both); a row whose
 * slot is outside [0, pages * page_size) is not written.
 *   k, v   token t, head j, element i: k[t*k_ld + j*D + i], in dtype (Q1_BF16 or
 *          Q1_F16); 16-byte aligned, k_ld and v_ld multiples of 8, below 2^23
 *   slots  device int32 [tokens]
 */
q1_status q1_kv_write(const q1_kv* c, const void* k, const void* v, int32_t dtype, int64_t k_ld, int64_t v_ld,
                      int64_t tokens, const int32_t* slots, void* stream);

/*
 * q1_kv_read -- the values of `rows` rows, rounded to out_dtype (exact for Q1_F32
 * and Q1_BF16, and for Q1_F16 where they are in its range): row i is slot slots[i],
 * zeros where that is outside [0, pages * page_size).  Slots may repeat.
 *   k, v   [rows, Hkv, D] in out_dtype; 16-byte aligned
 */
q1_status q1_kv_read(const q1_kv* c, const int32_t* slots, int64_t rows, void* k, void* v, int32_t out_dtype,
                     void* stream);

/*
 * q1_kv_attn -- T queries of each of B sequences over the pages; the queries are
 * the last T of the lens[b] tokens, so query t sees the first
 * n(b, t) = lens[b] - (T - 1 - t):
 *   out[b, t, h] = softmax(scale * q[b, t, h] . K^T) V,  lse[b, t, h] = log sum exp
 * over tokens j < n(b, t) of key/value head h / (Hq/Hkv).  Token j of sequence b is
 * row j % page_size of page page_table[b, j / page_size]; several sequences may share
 * pages.  Lengths are clamped to [0, max_pages * page_size]; a token whose page id
 * is outside [0, pages) is left out.  A query that sees no token gives zeros and
 * lse = -infinity.  Rows that a query does not see are never used, whatever they
 * hold.  Scores, softmax and sums are fp32; keys, values and queries enter the
 * products as they are, a weight as two bf16 parts (2^-17); of n tokens, those whose
 * weight is below n 2^-117 of the largest may be left out.  A NaN block of a key that
 * a query sees makes its row and its lse NaN, one of a value its 32 columns.  Bytes that
 * q1_kv_write does not make (the codes 0x7f and 0xff of 8 bits, larger scales) may stand
 * for a NaN or for more than bf16 holds: of a value, that makes at least its own column
 * NaN or infinite for the queries that see it, and at most the block's 32.
 */
typedef struct q1_kv_query {
  const void* q;              /* [B, T, Hq, D], q_ld elements between tokens (b*T + t); 16-byte aligned */
  const int32_t* page_table;  /* device [B, max_pages] */
  const int32_t* lens;        /* device [B] */
  void* out;                  /* [B, T, Hq, D] in out_dtype; 16-byte aligned */
  float* lse;                 /* [B, T, Hq], or NULL */
  int64_t q_ld;               /* a multiple of 8 */
  int64_t B, T, max_pages;    /* max_pages * page_size up to 2^31 - 2^16 */
  int32_t Hq;                 /* Hq % Hkv == 0 */
  int32_t dtype;              /* of q: Q1_BF16 or Q1_F16 */
  int32_t out_dtype;          /* Q1_F32, Q1_F16 or Q1_BF16 */
  float scale;                /* finite */
} q1_kv_query;

q1_status q1_kv_attn(const q1_kv* c, const q1_kv_query* a, void* workspace, size_t workspace_bytes, void* stream);

size_t q1_kv_attn_workspace_bytes(const q1_kv* c, const q1_kv_query* a);

/*
 * Short causal convolution, per channel c and token t of a sequence:
 *   y[t, c] = act(bias[c] + sum_{w < W} weight[c, w] * x[t - (W-1) + w, c])
 * with act(s) = s / (1 + exp(-s)) for silu = 1 and s for silu = 0.  Rows before the
 * sequence's first are the state, oldest first, which then holds the last W-1 rows.
 * Sums are fp32.
 */
typedef struct q1_conv {
  const void* x;           /* token t, channel i: x[t*x_ld + i]; 16-byte aligned, x_ld % 8 == 0, below 2^23 */
  const void* weight;      /* [C, W] in dtype; 16-byte aligned */
  const void* bias;        /* [C] in dtype, 16-byte aligned, or NULL */
  void* state;             /* [slots, W-1, C] in dtype, read and written; 16-byte aligned */
  const int32_t* slot_ids; /* device [sequences], distinct; NULL: sequence b uses slot b.  A sequence whose
                              id is outside [0, slots) touches no state and its outputs are zeros */
  void* out;               /* [tokens, C] in dtype; 16-byte aligned */
  int64_t x_ld, slots;
  int64_t C;               /* a multiple of 8, up to 2^20 */
  int32_t W;               /* 2, 3 or 4 */
  int32_t dtype;           /* Q1_BF16 or Q1_F16 */
  int32_t silu;            /* 0 or 1 */
  int32_t reserved;        /* 0 */
} q1_conv;

/* q1_conv_step -- T tokens of each of B sequences; token t of sequence b is row b*T + t. */
q1_status q1_conv_step(const q1_conv* d, int64_t B, int64_t T, void* stream);

/*
 * q1_conv_prefill -- whole prompts: `tokens` rows, sequence s = rows cu_seqlens[s] ..
 * cu_seqlens[s+1]-1 (device int32 [nseq + 1], not decreasing, from 0 to `tokens`;
 * offsets outside [0, tokens] are clamped, an empty sequence keeps its state, rows of
 * no sequence are not written).  The same bits as q1_conv_step over the same tokens.
 */
q1_status q1_conv_prefill(const q1_conv* d, int64_t tokens, int64_t nseq, const int32_t* cu_seqlens, void* stream);

/*
 * Selective state space scan, per channel d and token t of a sequence, with a
 * state h [N] per channel:
 *   s_t = dt_t + dt_bias,  delta_t = log(1 + exp(s_t)) for softplus = 1, else s_t
 *   h_t[n] = exp(delta_t A[n]) h_{t-1}[n] + delta_t x_t B_t[n]
 *   y_t = (sum_n C_t[n] h_t[n] + D x_t) * z_t / (1 + exp(-z_t))
 * (without D: D = 0; without z: no gate).  States, sums and exponentials are fp32;
 * outputs are rounded once.
 */
typedef struct q1_scan {
  const void* x;           /* token t, channel i: x[t*x_ld + i] in dtype; 16-byte aligned */
  const void* dt;          /* as x, with dt_ld, in dt_dtype */
  const void* B;           /* token t: B[t*b_ld + n] in dtype; 16-byte aligned */
  const void* C;           /* as B, with c_ld */
  const void* z;           /* as x, with z_ld; or NULL */
  const float* A;          /* [Di, N]; 16-byte aligned */
  const float* D;          /* [Di], or NULL */
  const float* dt_bias;    /* [Di], or NULL */
  float* state;            /* [slots, Di, N], read and written; 16-byte aligned */
  const int32_t* slot_ids; /* as for q1_conv */
  void* out;               /* [tokens, Di] in out_dtype; 16-byte aligned */
  int64_t x_ld, dt_ld, b_ld, c_ld, z_ld; /* multiples of 8, below 2^23 */
  int64_t slots;
  int64_t Di;              /* a multiple of 8, up to 2^18 */
  int32_t N;               /* 8, 16, 32 or 64 */
  int32_t dtype;           /* of x, B, C and z: Q1_BF16 or Q1_F16 */
  int32_t dt_dtype;        /* dtype or Q1_F32 */
  int32_t out_dtype;       /* Q1_F32, Q1_F16 or Q1_BF16 */
  int32_t softplus;        /* 0 or 1 */
  int32_t reserved;        /* 0 */
} q1_scan;

/*
 * q1_scan_step -- T tokens of each of B sequences; token t of sequence b is row
 * b*T + t.  States end after all T tokens, none between is kept.
 */
q1_status q1_scan_step(const q1_scan* d, int64_t B, int64_t T, void* stream);

/*
 * q1_scan_prefill -- whole prompts, as for q1_conv_prefill.  The same result as
 * q1_scan_step over the same tokens, to fp32 rounding.
 *   workspace  q1_scan_prefill_workspace_bytes(...) bytes, 256-byte aligned.
 */
q1_status q1_scan_prefill(const q1_scan* d, int64_t tokens, int64_t nseq, const int32_t* cu_seqlens, void* workspace,
                          size_t workspace_bytes, void* stream);

size_t q1_scan_prefill_workspace_bytes(const q1_scan* d, int64_t tokens, int64_t nseq);

#ifdef __cplusplus
}
#endif

#endif /* Q1_MEMORY_H */
