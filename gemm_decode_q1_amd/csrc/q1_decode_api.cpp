// C ABI of the decode-step operators: argument checks and dispatch.  Order of
// checks as everywhere in the library: arguments (no HIP call), the workspace,
// the current device.
#include <hip/hip_runtime.h>

#include <cmath>

#include "../../include/q1_decode.h"
#include "q1_decode.h"
#include "q1_internal.h"
#include "q1_status.h"

using namespace q1;

namespace {

constexpr int64_t kMaxGrid = (int64_t)1 << 30;  // workgroups of one launch

// Shapes and dtypes of a delta call (what the workspace query needs).
q1_status check_delta_shape(const q1_delta* d) {
  if (d == nullptr) return fail(Q1_ERR_INVALID_ARG, "delta descriptor is NULL");
  if (d->dtype != Q1_BF16 && d->dtype != Q1_F16) return fail(Q1_ERR_UNSUPPORTED, "q, k and v must be bf16 or fp16");
  if (!valid_out_dtype(d->out_dtype)) return fail(Q1_ERR_INVALID_ARG, "out dtype must be Q1_F32, Q1_F16 or Q1_BF16");
  if (d->Hk <= 0 || d->Hv <= 0 || d->Hv % d->Hk != 0)
    return fail(Q1_ERR_INVALID_ARG, "value heads (%d) must be a positive multiple of key heads (%d)", d->Hv, d->Hk);
  if (d->Dk != 64 && d->Dk != 128) return fail(Q1_ERR_UNSUPPORTED, "Dk must be 64 or 128 (got %d)", d->Dk);
  if (d->Dv <= 0 || d->Dv % 16 != 0 || d->Dv > 256)
    return fail(Q1_ERR_UNSUPPORTED, "Dv must be a multiple of 16 up to 256 (got %d)", d->Dv);
  if (d->Hv > 4096) return fail(Q1_ERR_UNSUPPORTED, "too many heads (%d)", d->Hv);
  if (d->l2norm != 0 && d->l2norm != 1) return fail(Q1_ERR_INVALID_ARG, "l2norm must be 0 or 1");
  return Q1_OK;
}

q1_status check_delta(const q1_delta* d, int64_t tokens, int64_t nseq) {
  if (d->q == nullptr || d->k == nullptr || d->v == nullptr || d->g == nullptr || d->beta == nullptr ||
      d->state == nullptr || d->out == nullptr)
    return fail(Q1_ERR_INVALID_ARG, "q, k, v, g, beta, state and out must not be NULL");
  if (!aligned(d->q, 16) || !aligned(d->k, 16) || !aligned(d->v, 16) || !aligned(d->state, 16) || !aligned(d->out, 16))
    return fail(Q1_ERR_INVALID_ARG, "q, k, v, state and out must be 16-byte aligned");
  if (!aligned(d->g, 4) || !aligned(d->beta, 4) || !aligned(d->slot_ids, 4))
    return fail(Q1_ERR_INVALID_ARG, "g, beta and slot_ids must be 4-byte aligned");
  const int64_t qk = (int64_t)d->Hk * d->Dk, vv = (int64_t)d->Hv * d->Dv;
  if (d->q_ld < qk || d->k_ld < qk || d->v_ld < vv)
    return fail(Q1_ERR_INVALID_ARG, "row strides must cover the heads (q %lld, k %lld, v %lld)", (long long)d->q_ld,
                (long long)d->k_ld, (long long)d->v_ld);
  if (d->q_ld % 8 != 0 || d->k_ld % 8 != 0 || d->v_ld % 8 != 0)
    return fail(Q1_ERR_INVALID_ARG, "row strides must be multiples of 8 elements");
  if (d->slots <= 0) return fail(Q1_ERR_INVALID_ARG, "slots must be positive");
  if (d->slot_ids == nullptr && nseq > d->slots)
    return fail(Q1_ERR_INVALID_ARG, "%lld sequences need as many state slots (got %lld)", (long long)nseq,
                (long long)d->slots);
  const int64_t ld = d->q_ld > d->k_ld ? (d->q_ld > d->v_ld ? d->q_ld : d->v_ld) : (d->k_ld > d->v_ld ? d->k_ld : d->v_ld);
  if (ld >= (int64_t)1 << 23) return fail(Q1_ERR_UNSUPPORTED, "row strides must be below 2^23 elements");
  if (tokens >= (int64_t)1 << 31 || tokens > ((int64_t)1 << 46) / ld || nseq > kMaxGrid / ((int64_t)d->Hv * 16) ||
      d->slots > ((int64_t)1 << 46) / ((int64_t)d->Hv * d->Dk * d->Dv))
    return fail(Q1_ERR_UNSUPPORTED, "call too large");
  return Q1_OK;
}

DeltaArgs delta_args(const q1_delta* d) {
  DeltaArgs a = {};
  a.q = static_cast<const uint16_t*>(d->q);
  a.k = static_cast<const uint16_t*>(d->k);
  a.v = static_cast<const uint16_t*>(d->v);
  a.q_ld = d->q_ld;
  a.k_ld = d->k_ld;
  a.v_ld = d->v_ld;
  a.g = d->g;
  a.beta = d->beta;
  a.state = d->state;
  a.slot_ids = d->slot_ids;
  a.out = d->out;
  a.slots = d->slots;
  a.Hk = d->Hk;
  a.Hv = d->Hv;
  a.Dv = d->Dv;
  a.out_dtype = d->out_dtype;
  a.l2norm = d->l2norm;
  a.scale = d->scale;
  return a;
}

q1_status check_attn(const q1_attn* a) {
  if (a == nullptr) return fail(Q1_ERR_INVALID_ARG, "attention descriptor is NULL");
  if (a->dtype != Q1_BF16 && a->dtype != Q1_F16) return fail(Q1_ERR_UNSUPPORTED, "q, keys and values must be bf16 or fp16");
  if (!valid_out_dtype(a->out_dtype)) return fail(Q1_ERR_INVALID_ARG, "out dtype must be Q1_F32, Q1_F16 or Q1_BF16");
  if (a->Hq <= 0 || a->Hkv <= 0 || a->Hq % a->Hkv != 0)
    return fail(Q1_ERR_INVALID_ARG, "query heads (%d) must be a positive multiple of key/value heads (%d)", a->Hq, a->Hkv);
  if (a->Hq > 4096) return fail(Q1_ERR_UNSUPPORTED, "too many heads (%d)", a->Hq);
  if (a->D != 64 && a->D != 128 && a->D != 256) return fail(Q1_ERR_UNSUPPORTED, "D must be 64, 128 or 256 (got %d)", a->D);
  if (a->B < 0 || a->P < 0 || a->pages < 0 || a->max_pages < 0)
    return fail(Q1_ERR_INVALID_ARG, "B, P, pages and max_pages must be >= 0");
  if (a->max_pages > 0 && a->page_size <= 0) return fail(Q1_ERR_INVALID_ARG, "page_size must be positive");
  const int64_t row = (int64_t)a->Hkv * a->D;
  if (a->P > 0 && a->prefix_ld < row) return fail(Q1_ERR_INVALID_ARG, "prefix_ld must cover the heads (got %lld)", (long long)a->prefix_ld);
  if (a->q_ld < (int64_t)a->Hq * a->D) return fail(Q1_ERR_INVALID_ARG, "q_ld must cover the heads (got %lld)", (long long)a->q_ld);
  if ((a->P > 0 && a->prefix_ld % 8 != 0) || a->q_ld % 8 != 0)
    return fail(Q1_ERR_INVALID_ARG, "q_ld and prefix_ld must be multiples of 8 elements");
  const int64_t lim = (int64_t)1 << 46;
  if (a->P > 0 && a->prefix_ld >= (int64_t)1 << 23) return fail(Q1_ERR_UNSUPPORTED, "prefix_ld must be below 2^23 elements");
  if (a->B > kMaxGrid / 4096 || a->q_ld > lim / (a->B + 1) || (a->P > 0 && a->P >= (int64_t)1 << 31) ||
      (a->P > 0 && a->prefix_ld > lim / a->P))
    return fail(Q1_ERR_UNSUPPORTED, "call too large");
  if (a->max_pages > 0 &&
      (a->page_size >= (int64_t)1 << 31 || a->max_pages >= (int64_t)1 << 31 || a->pages >= (int64_t)1 << 31 ||
       a->max_pages * a->page_size >= (int64_t)1 << 31 || a->pages * a->page_size >= (int64_t)1 << 31))
    return fail(Q1_ERR_UNSUPPORTED, "call too large");
  return Q1_OK;
}

}  // namespace

extern "C" {

q1_status q1_delta_step(const q1_delta* d, int64_t B, int64_t T, void* stream) {
  q1_status st = check_delta_shape(d);
  if (st != Q1_OK) return st;
  if (B < 0 || T < 0) return fail(Q1_ERR_INVALID_ARG, "B and T must be >= 0 (got %lld, %lld)", (long long)B, (long long)T);
  if (B == 0 || T == 0) return ok();
  if (B >= ((int64_t)1 << 31) / T) return fail(Q1_ERR_UNSUPPORTED, "call too large");
  st = check_delta(d, B * T, B);
  if (st == Q1_OK) st = check_current_device();
  if (st != Q1_OK) return st;
  DeltaArgs a = delta_args(d);
  a.T = T;
  a.nseq = B;
  return hip_status(launch_delta_recurrent(a, d->dtype == Q1_F16, d->Dk, static_cast<hipStream_t>(stream)),
                    "delta step launch");
}

size_t q1_delta_prefill_workspace_bytes(const q1_delta* d, int64_t tokens, int64_t nseq) {
  if (check_delta_shape(d) != Q1_OK) return 0;
  if (tokens < 0 || nseq < 0) {
    fail(Q1_ERR_INVALID_ARG, "tokens and nseq must be >= 0");
    return 0;
  }
  if (tokens >= (int64_t)1 << 31 || nseq >= (int64_t)1 << 31) {
    fail(Q1_ERR_UNSUPPORTED, "call too large");
    return 0;
  }
  ok();
  if (tokens == 0 || nseq == 0) return 0;
  return (size_t)delta_chunk_slots(tokens, nseq) * d->Hv * kDeltaChunkBytes;
}

q1_status q1_delta_prefill(const q1_delta* d, int64_t tokens, int64_t nseq, const int32_t* cu_seqlens, void* workspace,
                           size_t workspace_bytes, void* stream) {
  q1_status st = check_delta_shape(d);
  if (st != Q1_OK) return st;
  if (tokens < 0 || nseq < 0) return fail(Q1_ERR_INVALID_ARG, "tokens and nseq must be >= 0");
  if (tokens == 0 || nseq == 0) return ok();
  st = check_delta(d, tokens, nseq);
  if (st == Q1_OK && delta_chunk_slots(tokens, nseq) * d->Hv > kMaxGrid) st = fail(Q1_ERR_UNSUPPORTED, "call too large");
  if (st != Q1_OK) return st;
  if (cu_seqlens == nullptr || !aligned(cu_seqlens, 4))
    return fail(Q1_ERR_INVALID_ARG, "cu_seqlens must be a 4-byte aligned device pointer");
  const size_t need = q1_delta_prefill_workspace_bytes(d, tokens, nseq);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need))
    return fail(Q1_ERR_WORKSPACE, "workspace too small: need %zu bytes, got %zu", need, workspace ? workspace_bytes : 0);
  if (need > 0 && !aligned(workspace, 256)) return fail(Q1_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  st = check_current_device();
  if (st != Q1_OK) return st;
  DeltaArgs a = delta_args(d);
  a.cu = cu_seqlens;
  a.tokens = tokens;
  a.nseq = nseq;
  return hip_status(launch_delta_chunk(a, d->dtype == Q1_F16, d->Dk, static_cast<unsigned char*>(workspace),
                                       static_cast<hipStream_t>(stream)),
                    "delta prefill launch");
}

size_t q1_prefix_attn_workspace_bytes(const q1_attn* a) {
  if (check_attn(a) != Q1_OK) return 0;
  ok();
  return a->B == 0 ? 0 : plan_prefix_attn(*a).ws_bytes;
}

q1_status q1_prefix_attn(const q1_attn* a, void* workspace, size_t workspace_bytes, void* stream) {
  q1_status st = check_attn(a);
  if (st != Q1_OK) return st;
  if (a->B == 0) return ok();
  if (a->q == nullptr || a->out == nullptr) return fail(Q1_ERR_INVALID_ARG, "q and out must not be NULL");
  if (a->P > 0 && (a->k_prefix == nullptr || a->v_prefix == nullptr))
    return fail(Q1_ERR_INVALID_ARG, "k_prefix and v_prefix must not be NULL");
  if (a->pages > 0 && (a->k_pages == nullptr || a->v_pages == nullptr))
    return fail(Q1_ERR_INVALID_ARG, "k_pages and v_pages must not be NULL");
  if (a->max_pages > 0 && (a->page_table == nullptr || a->suffix_lens == nullptr))
    return fail(Q1_ERR_INVALID_ARG, "page_table and suffix_lens must not be NULL");
  if (!aligned(a->q, 16) || !aligned(a->out, 16) || !aligned(a->k_prefix, 16) || !aligned(a->v_prefix, 16) ||
      !aligned(a->k_pages, 16) || !aligned(a->v_pages, 16))
    return fail(Q1_ERR_INVALID_ARG, "q, out, keys and values must be 16-byte aligned");
  if (!aligned(a->page_table, 4) || !aligned(a->suffix_lens, 4) || !aligned(a->lse, 4))
    return fail(Q1_ERR_INVALID_ARG, "page_table, suffix_lens and lse must be 4-byte aligned");
  const AttnPlan plan = plan_prefix_attn(*a);
  if (plan.wgs > kMaxGrid) return fail(Q1_ERR_UNSUPPORTED, "call too large");
  const size_t need = plan.ws_bytes;
  if (need > 0 && (workspace == nullptr || workspace_bytes < need))
    return fail(Q1_ERR_WORKSPACE, "workspace too small: need %zu bytes, got %zu", need, workspace ? workspace_bytes : 0);
  if (need > 0 && !aligned(workspace, 256)) return fail(Q1_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  st = check_current_device();
  if (st != Q1_OK) return st;
  return hip_status(launch_prefix_attn(*a, plan, static_cast<unsigned char*>(workspace), static_cast<hipStream_t>(stream)),
                    "attention launch");
}

size_t q1_sample_workspace_bytes(int64_t B, int64_t V) {
  if (B < 0 || V < 1) {
    fail(Q1_ERR_INVALID_ARG, "B must be >= 0 and V >= 1");
    return 0;
  }
  if (B > (int64_t)1 << 20 || V > (int64_t)1 << 22) {
    fail(Q1_ERR_UNSUPPORTED, "call too large");
    return 0;
  }
  ok();
  return B == 0 ? 0 : sample_ws_bytes(B, V);
}

q1_status q1_sample(const void* logits, int32_t dtype, int64_t B, int64_t V, int64_t ld, const float* u,
                    const float* temperature, const int32_t* top_k, const float* top_p, const float* min_p,
                    void* tokens, int32_t tokens_are_int64, float* logprob, void* workspace, size_t workspace_bytes,
                    void* stream) {
  if (!valid_out_dtype(dtype)) return fail(Q1_ERR_INVALID_ARG, "logits must be Q1_F32, Q1_F16 or Q1_BF16");
  if (B < 0) return fail(Q1_ERR_INVALID_ARG, "B must be >= 0 (got %lld)", (long long)B);
  if (V < 1) return fail(Q1_ERR_INVALID_ARG, "V must be positive (got %lld)", (long long)V);
  if (V > (int64_t)1 << 22) return fail(Q1_ERR_UNSUPPORTED, "V must be at most 2^22 (got %lld)", (long long)V);
  if (ld < V) return fail(Q1_ERR_INVALID_ARG, "row stride %lld is below V = %lld", (long long)ld, (long long)V);
  if (tokens_are_int64 != 0 && tokens_are_int64 != 1) return fail(Q1_ERR_INVALID_ARG, "tokens_are_int64 must be 0 or 1");
  if (B > (int64_t)1 << 20 || ld > ((int64_t)1 << 46) / (B + 1)) return fail(Q1_ERR_UNSUPPORTED, "call too large");
  if (B == 0) return ok();
  if (logits == nullptr || u == nullptr || tokens == nullptr)
    return fail(Q1_ERR_INVALID_ARG, "logits, u and tokens must not be NULL");
  if (!aligned(logits, dtype_size(dtype))) return fail(Q1_ERR_INVALID_ARG, "logits are misaligned");
  if (!aligned(u, 4) || !aligned(temperature, 4) || !aligned(top_k, 4) || !aligned(top_p, 4) || !aligned(min_p, 4) ||
      !aligned(logprob, 4) || !aligned(tokens, tokens_are_int64 ? 8 : 4))
    return fail(Q1_ERR_INVALID_ARG, "u, the row parameters, tokens and logprob must be aligned to their elements");
  const size_t need = q1_sample_workspace_bytes(B, V);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need))
    return fail(Q1_ERR_WORKSPACE, "workspace too small: need %zu bytes, got %zu", need, workspace ? workspace_bytes : 0);
  if (need > 0 && !aligned(workspace, 256)) return fail(Q1_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  const q1_status st = check_current_device();
  if (st != Q1_OK) return st;
  SampleArgs a;
  a.logits = logits;
  a.dtype = dtype;
  a.B = B;
  a.V = V;
  a.ld = ld;
  a.u = u;
  a.temperature = temperature;
  a.top_k = top_k;
  a.top_p = top_p;
  a.min_p = min_p;
  a.tokens = tokens;
  a.tokens_int64 = tokens_are_int64;
  a.logprob = logprob;
  return hip_status(launch_sample(a, static_cast<unsigned char*>(workspace), static_cast<hipStream_t>(stream)),
                    "sampler launch");
}

}  // extern "C"
