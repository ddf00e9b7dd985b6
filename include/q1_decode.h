/*
 * q1_decode.h -- the calls between the packed Q1 projections of a decode step:
 * the gated delta rule (single tokens and whole prompts), attention of a decode
 * batch over a shared prefix, and the sampler of the tied head's logits.
 *
 * The conventions of q1.h hold: caller-owned device memory, argument checks
 * before any HIP call, then the workspace check, then the device check; calls
 * only enqueue work on `stream`, allocate nothing, keep nothing between calls,
 * and can be captured in a HIP graph.  Workspaces here need no initial
 * contents (the reserved block of q1.h is not used); calls that may run at the
 * same time, and calls of several threads on one stream, need separate ones (a
 * call is several launches that hand data on through its workspace).
 *
 * Numbers the kernels read from device memory (lengths, offsets, page and slot
 * ids) cannot be checked by the call; each one below says what an id outside
 * its range does.  No such value makes a kernel read or write out of bounds.
 */
#ifndef Q1_DECODE_H
#define Q1_DECODE_H

#include "q1.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Gated delta rule.  Per sequence and value head h (key head h / (Hv/Hk)), with
 * a state S [Dk, Dv] in fp32 and a_t = exp(g_t):
 *   S_t = a_t S_{t-1} + k_t (x) beta_t (v_t - a_t S_{t-1}^T k_t)
 *   o_t = scale * S_t^T q_t
 * With l2norm = 1, q and k are first divided by sqrt(sum of squares + 1e-6).
 * State, sums and exponentials are fp32; outputs are rounded once (of prompts
 * with a 16-bit out_dtype, see q1_delta_prefill).
 * g = -infinity (a = 0) forgets a finite state exactly.
 */
typedef struct q1_delta {
  const void* q;           /* token t, key head j, element i: q[t*q_ld + j*Dk + i]; 16-byte aligned */
  const void* k;           /* as q, with k_ld */
  const void* v;           /* v[t*v_ld + h*Dv + i]; 16-byte aligned */
  int64_t q_ld, k_ld, v_ld; /* elements between tokens; multiples of 8, below 2^23 */
  const float* g;          /* [tokens, Hv] log decay */
  const float* beta;       /* [tokens, Hv] write strength */
  float* state;            /* [slots, Hv, Dk, Dv], read and written; 16-byte aligned */
  const int32_t* slot_ids; /* device [sequences], distinct; NULL: sequence b uses slot b.  A sequence whose
                              id is outside [0, slots) touches no state and its outputs are zeros */
  void* out;               /* [tokens, Hv, Dv] in out_dtype; 16-byte aligned */
  int64_t slots;           /* states in the pool */
  int32_t Hk, Hv;          /* Hv % Hk == 0 */
  int32_t Dk, Dv;          /* Dk 64 or 128; Dv a multiple of 16, at most 256 */
  int32_t dtype;           /* of q, k, v: Q1_BF16 or Q1_F16 */
  int32_t out_dtype;       /* Q1_F32, Q1_F16 or Q1_BF16 */
  int32_t l2norm;          /* 0 or 1 */
  float scale;             /* of the output, usually 1/sqrt(Dk) */
} q1_delta;

/*
 * q1_delta_step -- T tokens (one or a few) of each of B sequences; token t of
 * sequence b is row b*T + t.  States are read and written once: they end after all
 * T tokens, none between is kept.  A caller that may take drafted tokens back
 * starts them from a copy of the state, in another slot.
 */
q1_status q1_delta_step(const q1_delta* d, int64_t B, int64_t T, void* stream);

/*
 * q1_delta_prefill -- whole prompts: `tokens` rows, sequence s = rows
 * cu_seqlens[s] .. cu_seqlens[s+1]-1 (device int32 [nseq + 1], not decreasing,
 * from 0 to `tokens`; offsets outside [0, tokens] are clamped, an empty
 * sequence keeps its state, rows of no sequence are not written).  The same
 * result as q1_delta_step over the same tokens, to fp32 rounding; outputs in a
 * 16-bit type are rounded from sums that are up to 2^-13 of their terms' magnitudes
 * off with bf16 operands, 2^-15 with fp16 ones.  A NaN or
 * infinity in q, k, v or beta spreads to the whole chunk of up to 64 tokens it is in
 * (and, as in the recurrence, to what follows).
 *   workspace  q1_delta_prefill_workspace_bytes(...) bytes, 256-byte aligned.
 */
q1_status q1_delta_prefill(const q1_delta* d, int64_t tokens, int64_t nseq, const int32_t* cu_seqlens,
                           void* workspace, size_t workspace_bytes, void* stream);

size_t q1_delta_prefill_workspace_bytes(const q1_delta* d, int64_t tokens, int64_t nseq);

/*
 * q1_prefix_attn -- one query per sequence over a prefix that the whole batch
 * shares and a suffix of its own, read from pages:
 *   out[b, h] = softmax(scale * q[b, h] . K^T) V,  lse[b, h] = log sum exp
 * over the P prefix tokens and the suffix_lens[b] suffix tokens of key/value
 * head h / (Hq/Hkv).  Suffix token t of sequence b is row t % page_size of page
 * page_table[b, t / page_size].  Lengths are clamped to [0, max_pages *
 * page_size]; a token whose page id is outside [0, pages) is left out.  A row
 * with no token at all gives zeros and lse = -infinity.  Rows past a length
 * are never used, whatever they hold.  Scores, softmax and sums are fp32; the
 * weights' products with the values take a weight as two 16-bit parts (2^-17).
 * A NaN or +infinite score of a token that counts makes its row's out and lse
 * NaN.  A NaN or infinite value of such a token makes its column of the row
 * NaN, or infinite where it is (weights enter the product in two parts, of which
 * one may be 0 or negative: an infinite sum can become NaN).
 */
typedef struct q1_attn {
  const void* q;               /* [B, Hq, D] with q_ld elements between sequences; 16-byte aligned, q_ld % 8 == 0 */
  const void* k_prefix;        /* token t, head j: k_prefix[t*prefix_ld + j*D + i]; 16-byte aligned; NULL iff P == 0 */
  const void* v_prefix;        /* as k_prefix */
  const void* k_pages;         /* [pages, page_size, Hkv, D]; 16-byte aligned; NULL iff pages == 0 */
  const void* v_pages;         /* as k_pages */
  const int32_t* page_table;   /* device [B, max_pages]; NULL iff max_pages == 0 */
  const int32_t* suffix_lens;  /* device [B]; NULL iff max_pages == 0 */
  void* out;                   /* [B, Hq, D] in out_dtype; 16-byte aligned */
  float* lse;                  /* [B, Hq], or NULL */
  int64_t q_ld, prefix_ld;     /* prefix_ld % 8 == 0, below 2^23 */
  int64_t B, P, pages, max_pages, page_size; /* P, pages * page_size and max_pages * page_size below 2^31 */
  int32_t Hq, Hkv;             /* Hq % Hkv == 0 */
  int32_t D;                   /* 64, 128 or 256 */
  int32_t dtype;               /* of q, keys and values: Q1_BF16 or Q1_F16 */
  int32_t out_dtype;           /* Q1_F32, Q1_F16 or Q1_BF16 */
  float scale;
} q1_attn;

q1_status q1_prefix_attn(const q1_attn* a, void* workspace, size_t workspace_bytes, void* stream);

size_t q1_prefix_attn_workspace_bytes(const q1_attn* a);

/*
 * q1_sample -- one token per row of logits, from a given random number.
 * Row b, with T = temperature[b] and top = the largest logit:
 *   e_i = exp((logit_i - top) / T) in fp32,  w_i = floor(e_i * 2^40) as an integer;
 *   keep the top_k[b] largest logits (equal logits: lowest index first);
 *   of these, in that order, keep those before which less than
 *     max(1, floor(top_p[b] * sum of the kept w)) of weight lies;
 *   of these, keep e_i >= min_p[b];
 *   token = the first i, in index order, where the running sum of the kept w
 *   exceeds floor(u[b] * their sum);  logprob = log(w_token / their sum).
 * Sums of weights are exact integers, so the token depends on the row alone:
 * not on the batch, the split of the row or the order of the additions.
 *   temperature <= 0 (or NaN): the largest logit, lowest index first.
 *   top_k <= 0, top_p >= 1, min_p <= 0 (or NaN) are off; a NULL array is off for
 *   every row (NULL temperature: 1).  min_p above 1 acts as 1.
 *   u is taken as 0 when below 0 or NaN, and below 1 otherwise.
 *   A NaN logit counts as -infinity; logits of +infinity share the draw.
 *   A row with nothing above -infinity gives token -1 and logprob -infinity.
 *   logits   [B, V] in dtype, `ld` >= V elements between rows; 1 <= V <= 2^22
 *   tokens   [B] int32 (tokens_are_int64 = 0) or int64 (= 1)
 *   logprob  [B], or NULL
 *   workspace  q1_sample_workspace_bytes(...) bytes, 256-byte aligned.
 */
q1_status q1_sample(const void* logits, int32_t dtype, int64_t B, int64_t V, int64_t ld, const float* u,
                    const float* temperature, const int32_t* top_k, const float* top_p, const float* min_p,
                    void* tokens, int32_t tokens_are_int64, float* logprob, void* workspace, size_t workspace_bytes,
                    void* stream);

size_t q1_sample_workspace_bytes(int64_t B, int64_t V);

#ifdef __cplusplus
}
#endif

#endif /* Q1_DECODE_H */
