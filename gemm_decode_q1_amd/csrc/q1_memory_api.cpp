// C ABI of q1_memory.h: argument checks and dispatch.  Order of checks as
// everywhere in the library: arguments (no HIP call), the workspace, the current
// device.
#include <hip/hip_runtime.h>

#include <cmath>

#include "../../include/q1_memory.h"
#include "q1_internal.h"
#include "q1_memory.h"
#include "q1_status.h"

using namespace q1;

namespace {

constexpr int64_t kMaxGrid = ((int64_t)1 << 24) - 1;  // workgroups of one launch (2^32 lanes)
constexpr int64_t kMost = (int64_t)1 << 46;     // elements of one operand
constexpr int64_t k31 = (int64_t)1 << 31;
constexpr int64_t kMostTokens = k31 - (1 << 16);  // of a sequence: the tile behind its last one is still counted in 31 bits

// Shapes of the pages (what the workspace query needs).
q1_status check_kv_shape(const q1_kv* c) {
  if (c == nullptr) return fail(Q1_ERR_INVALID_ARG, "descriptor of the pages is NULL");
  if (c->bits != 4 && c->bits != 8) return fail(Q1_ERR_UNSUPPORTED, "bits must be 4 or 8 (got %d)", c->bits);
  if (c->D != 64 && c->D != 128 && c->D != 256) return fail(Q1_ERR_UNSUPPORTED, "D must be 64, 128 or 256 (got %d)", c->D);
  if (c->Hkv <= 0) return fail(Q1_ERR_INVALID_ARG, "Hkv must be positive (got %d)", c->Hkv);
  if (c->Hkv > 4096) return fail(Q1_ERR_UNSUPPORTED, "too many heads (%d)", c->Hkv);
  if (c->pages < 0 || c->page_size <= 0) return fail(Q1_ERR_INVALID_ARG, "pages must be >= 0 and page_size positive");
  if (c->reserved != 0) return fail(Q1_ERR_INVALID_ARG, "reserved must be 0");
  if (c->pages >= k31 || c->page_size >= k31 || c->pages * c->page_size >= k31 ||
      c->page_size * c->Hkv >= k31 || c->page_size * c->Hkv * c->D >= k31)
    return fail(Q1_ERR_UNSUPPORTED, "pages too large");
  return Q1_OK;
}

q1_status check_kv(const q1_kv* c) {
  if (c->pages == 0) return Q1_OK;
  if (c->k == nullptr || c->v == nullptr || c->k_scales == nullptr || c->v_scales == nullptr)
    return fail(Q1_ERR_INVALID_ARG, "k, v and their scales must not be NULL");
  if (!aligned(c->k, 16) || !aligned(c->v, 16)) return fail(Q1_ERR_INVALID_ARG, "pages must be 16-byte aligned");
  if (!aligned(c->k_scales, 8) || !aligned(c->v_scales, 8)) return fail(Q1_ERR_INVALID_ARG, "scales must be 8-byte aligned");
  return Q1_OK;
}

q1_status check_kv_query(const q1_kv* c, const q1_kv_query* a) {
  q1_status st = check_kv_shape(c);
  if (st != Q1_OK) return st;
  if (a == nullptr) return fail(Q1_ERR_INVALID_ARG, "attention descriptor is NULL");
  if (a->dtype != Q1_BF16 && a->dtype != Q1_F16) return fail(Q1_ERR_UNSUPPORTED, "q must be bf16 or fp16");
  if (!valid_out_dtype(a->out_dtype)) return fail(Q1_ERR_INVALID_ARG, "out dtype must be Q1_F32, Q1_F16 or Q1_BF16");
  if (a->Hq <= 0 || a->Hq % c->Hkv != 0)
    return fail(Q1_ERR_INVALID_ARG, "query heads (%d) must be a positive multiple of key/value heads (%d)", a->Hq, c->Hkv);
  if (a->Hq > 4096) return fail(Q1_ERR_UNSUPPORTED, "too many heads (%d)", a->Hq);
  if (a->B < 0 || a->T < 0 || a->max_pages < 0) return fail(Q1_ERR_INVALID_ARG, "B, T and max_pages must be >= 0");
  if (a->q_ld < (int64_t)a->Hq * c->D) return fail(Q1_ERR_INVALID_ARG, "q_ld must cover the heads (got %lld)", (long long)a->q_ld);
  if (a->q_ld % 8 != 0) return fail(Q1_ERR_INVALID_ARG, "q_ld must be a multiple of 8 elements");
  if (!std::isfinite(a->scale)) return fail(Q1_ERR_INVALID_ARG, "scale must be finite");
  if (a->max_pages >= k31 || a->max_pages * c->page_size > kMostTokens || a->B >= k31 || a->T >= k31 / a->Hq ||
      (a->T > 0 && a->B >= k31 / (a->T * a->Hq)) || a->q_ld > kMost / (a->B * a->T + 1) ||
      (a->max_pages > 0 && a->B > kMost / a->max_pages))
    return fail(Q1_ERR_UNSUPPORTED, "call too large");
  return Q1_OK;
}

q1_status check_operands(int32_t dtype, int32_t reserved) {
  if (dtype != Q1_BF16 && dtype != Q1_F16) return fail(Q1_ERR_UNSUPPORTED, "operands must be bf16 or fp16");
  if (reserved != 0) return fail(Q1_ERR_INVALID_ARG, "reserved must be 0");
  return Q1_OK;
}

q1_status check_step(int64_t B, int64_t T) {
  if (B < 0 || T < 0) return fail(Q1_ERR_INVALID_ARG, "B and T must be >= 0 (got %lld, %lld)", (long long)B, (long long)T);
  if (B > 0 && T > 0 && B >= k31 / T) return fail(Q1_ERR_UNSUPPORTED, "call too large");
  return Q1_OK;
}

q1_status check_ragged(int64_t tokens, int64_t nseq, const int32_t* cu) {
  if (cu == nullptr || !aligned(cu, 4)) return fail(Q1_ERR_INVALID_ARG, "cu_seqlens must be a 4-byte aligned device pointer");
  if (tokens >= k31 || nseq >= k31) return fail(Q1_ERR_UNSUPPORTED, "call too large");
  return Q1_OK;
}

q1_status check_slots(const int32_t* ids, int64_t slots, int64_t nseq) {
  if (!aligned(ids, 4)) return fail(Q1_ERR_INVALID_ARG, "slot_ids must be 4-byte aligned");
  if (slots <= 0) return fail(Q1_ERR_INVALID_ARG, "slots must be positive");
  if (ids == nullptr && nseq > slots)
    return fail(Q1_ERR_INVALID_ARG, "%lld sequences need as many state slots (got %lld)", (long long)nseq, (long long)slots);
  return Q1_OK;
}

// Row strides of `n` operands of at least `width` elements.
q1_status check_lds(const int64_t* ld, const int64_t* width, int n, int64_t tokens) {
  for (int i = 0; i < n; ++i) {
    if (ld[i] < width[i]) return fail(Q1_ERR_INVALID_ARG, "row strides must cover the row (got %lld)", (long long)ld[i]);
    if (ld[i] % 8 != 0) return fail(Q1_ERR_INVALID_ARG, "row strides must be multiples of 8 elements");
    if (ld[i] >= (int64_t)1 << 23) return fail(Q1_ERR_UNSUPPORTED, "row strides must be below 2^23 elements");
    if (tokens > kMost / ld[i]) return fail(Q1_ERR_UNSUPPORTED, "call too large");
  }
  return Q1_OK;
}

q1_status check_conv(const q1_conv* d, int64_t tokens, int64_t nseq) {
  q1_status st = check_operands(d->dtype, d->reserved);
  if (st != Q1_OK) return st;
  if (d->W < 2 || d->W > 4) return fail(Q1_ERR_UNSUPPORTED, "W must be 2, 3 or 4 (got %d)", d->W);
  if (d->C <= 0 || d->C % 8 != 0) return fail(Q1_ERR_INVALID_ARG, "C must be a positive multiple of 8 (got %lld)", (long long)d->C);
  if (d->C > (int64_t)1 << 20) return fail(Q1_ERR_UNSUPPORTED, "C must be at most 2^20 (got %lld)", (long long)d->C);
  if (d->silu != 0 && d->silu != 1) return fail(Q1_ERR_INVALID_ARG, "silu must be 0 or 1");
  if (d->x == nullptr || d->weight == nullptr || d->state == nullptr || d->out == nullptr)
    return fail(Q1_ERR_INVALID_ARG, "x, weight, state and out must not be NULL");
  if (!aligned(d->x, 16) || !aligned(d->weight, 16) || !aligned(d->bias, 16) || !aligned(d->state, 16) || !aligned(d->out, 16))
    return fail(Q1_ERR_INVALID_ARG, "x, weight, bias, state and out must be 16-byte aligned");
  st = check_slots(d->slot_ids, d->slots, nseq);
  if (st == Q1_OK) st = check_lds(&d->x_ld, &d->C, 1, tokens);
  if (st != Q1_OK) return st;
  if (d->slots > kMost / (3 * d->C) || nseq >= k31 / (d->C / 8)) return fail(Q1_ERR_UNSUPPORTED, "call too large");
  return Q1_OK;
}

// Shapes of a scan (what the workspace query needs).
q1_status check_scan_shape(const q1_scan* d) {
  if (d == nullptr) return fail(Q1_ERR_INVALID_ARG, "scan descriptor is NULL");
  const q1_status st = check_operands(d->dtype, d->reserved);
  if (st != Q1_OK) return st;
  if (d->dt_dtype != d->dtype && d->dt_dtype != Q1_F32)
    return fail(Q1_ERR_UNSUPPORTED, "dt must have the operands' dtype or be fp32");
  if (!valid_out_dtype(d->out_dtype)) return fail(Q1_ERR_INVALID_ARG, "out dtype must be Q1_F32, Q1_F16 or Q1_BF16");
  if (d->N != 8 && d->N != 16 && d->N != 32 && d->N != 64)
    return fail(Q1_ERR_UNSUPPORTED, "N must be 8, 16, 32 or 64 (got %d)", d->N);
  if (d->Di <= 0 || d->Di % 8 != 0)
    return fail(Q1_ERR_INVALID_ARG, "Di must be a positive multiple of 8 (got %lld)", (long long)d->Di);
  if (d->Di > (int64_t)1 << 18) return fail(Q1_ERR_UNSUPPORTED, "Di must be at most 2^18 (got %lld)", (long long)d->Di);
  if (d->softplus != 0 && d->softplus != 1) return fail(Q1_ERR_INVALID_ARG, "softplus must be 0 or 1");
  return Q1_OK;
}

q1_status check_scan(const q1_scan* d, int64_t tokens, int64_t nseq) {
  if (d->x == nullptr || d->dt == nullptr || d->B == nullptr || d->C == nullptr || d->A == nullptr ||
      d->state == nullptr || d->out == nullptr)
    return fail(Q1_ERR_INVALID_ARG, "x, dt, B, C, A, state and out must not be NULL");
  if (!aligned(d->x, 16) || !aligned(d->dt, 16) || !aligned(d->B, 16) || !aligned(d->C, 16) || !aligned(d->z, 16) ||
      !aligned(d->A, 16) || !aligned(d->state, 16) || !aligned(d->out, 16))
    return fail(Q1_ERR_INVALID_ARG, "x, dt, B, C, z, A, state and out must be 16-byte aligned");
  if (!aligned(d->D, 4) || !aligned(d->dt_bias, 4)) return fail(Q1_ERR_INVALID_ARG, "D and dt_bias must be 4-byte aligned");
  q1_status st = check_slots(d->slot_ids, d->slots, nseq);
  if (st != Q1_OK) return st;
  const int64_t ld[5] = {d->x_ld, d->dt_ld, d->b_ld, d->c_ld, d->z_ld}, width[5] = {d->Di, d->Di, d->N, d->N, d->Di};
  st = check_lds(ld, width, d->z != nullptr ? 5 : 4, tokens);
  if (st != Q1_OK) return st;
  if (d->slots > kMost / (d->Di * d->N) || nseq >= k31 / (4 * d->Di)) return fail(Q1_ERR_UNSUPPORTED, "call too large");
  return Q1_OK;
}

// Whether a launch of the prompt's scan would have too many workgroups.
bool scan_too_large(const q1_scan& d, int64_t tokens, int64_t nseq) {
  return scan_pieces(d, tokens, nseq) > kMaxGrid / ((d.Di + 63) / 64) || nseq >= k31 / (d.Di * d.N);
}

}  // namespace

extern "C" {

q1_status q1_kv_write(const q1_kv* c, const void* k, const void* v, int32_t dtype, int64_t k_ld, int64_t v_ld,
                      int64_t tokens, const int32_t* slots, void* stream) {
  q1_status st = check_kv_shape(c);
  if (st == Q1_OK) st = check_operands(dtype, 0);
  if (st != Q1_OK) return st;
  if (tokens < 0) return fail(Q1_ERR_INVALID_ARG, "tokens must be >= 0 (got %lld)", (long long)tokens);
  const int64_t width = (int64_t)c->Hkv * c->D;
  if (tokens >= k31 / (width / 8)) return fail(Q1_ERR_UNSUPPORTED, "call too large");
  if (tokens == 0) return ok();
  st = check_kv(c);
  if (st != Q1_OK) return st;
  if (k == nullptr || v == nullptr || slots == nullptr) return fail(Q1_ERR_INVALID_ARG, "k, v and slots must not be NULL");
  if (!aligned(k, 16) || !aligned(v, 16)) return fail(Q1_ERR_INVALID_ARG, "k and v must be 16-byte aligned");
  if (!aligned(slots, 4)) return fail(Q1_ERR_INVALID_ARG, "slots must be 4-byte aligned");
  const int64_t ld[2] = {k_ld, v_ld}, widths[2] = {width, width};
  st = check_lds(ld, widths, 2, tokens);
  if (st == Q1_OK) st = check_current_device();
  if (st != Q1_OK) return st;
  if (c->pages == 0) return ok();  // no slot is inside
  return hip_status(launch_kv_write(*c, k, v, dtype == Q1_F16, k_ld, v_ld, tokens, slots, static_cast<hipStream_t>(stream)),
                    "cache write launch");
}

q1_status q1_kv_read(const q1_kv* c, const int32_t* slots, int64_t rows, void* k, void* v, int32_t out_dtype,
                     void* stream) {
  q1_status st = check_kv_shape(c);
  if (st != Q1_OK) return st;
  if (!valid_out_dtype(out_dtype)) return fail(Q1_ERR_INVALID_ARG, "out dtype must be Q1_F32, Q1_F16 or Q1_BF16");
  if (rows < 0) return fail(Q1_ERR_INVALID_ARG, "rows must be >= 0 (got %lld)", (long long)rows);
  if (rows >= k31 / ((int64_t)c->Hkv * c->D / 8)) return fail(Q1_ERR_UNSUPPORTED, "call too large");
  if (rows == 0) return ok();
  st = check_kv(c);
  if (st != Q1_OK) return st;
  if (k == nullptr || v == nullptr || slots == nullptr) return fail(Q1_ERR_INVALID_ARG, "k, v and slots must not be NULL");
  if (!aligned(k, 16) || !aligned(v, 16)) return fail(Q1_ERR_INVALID_ARG, "k and v must be 16-byte aligned");
  if (!aligned(slots, 4)) return fail(Q1_ERR_INVALID_ARG, "slots must be 4-byte aligned");
  st = check_current_device();
  if (st != Q1_OK) return st;
  return hip_status(launch_kv_read(*c, slots, rows, k, v, out_dtype, static_cast<hipStream_t>(stream)), "cache read launch");
}

size_t q1_kv_attn_workspace_bytes(const q1_kv* c, const q1_kv_query* a) {
  if (check_kv_query(c, a) != Q1_OK) return 0;
  ok();
  if (a->B == 0 || a->T == 0) return 0;
  const KvPlan plan = plan_kv_attn(*c, *a);
  if (plan.too_large) fail(Q1_ERR_UNSUPPORTED, "call too large");
  return plan.ws_bytes;
}

q1_status q1_kv_attn(const q1_kv* c, const q1_kv_query* a, void* workspace, size_t workspace_bytes, void* stream) {
  q1_status st = check_kv_query(c, a);
  if (st != Q1_OK) return st;
  if (a->B == 0 || a->T == 0) return ok();
  st = check_kv(c);
  if (st != Q1_OK) return st;
  if (a->q == nullptr || a->out == nullptr) return fail(Q1_ERR_INVALID_ARG, "q and out must not be NULL");
  if (a->lens == nullptr || (a->max_pages > 0 && a->page_table == nullptr))
    return fail(Q1_ERR_INVALID_ARG, "page_table and lens must not be NULL");
  if (!aligned(a->q, 16) || !aligned(a->out, 16)) return fail(Q1_ERR_INVALID_ARG, "q and out must be 16-byte aligned");
  if (!aligned(a->page_table, 4) || !aligned(a->lens, 4) || !aligned(a->lse, 4))
    return fail(Q1_ERR_INVALID_ARG, "page_table, lens and lse must be 4-byte aligned");
  const KvPlan plan = plan_kv_attn(*c, *a);
  if (plan.too_large) return fail(Q1_ERR_UNSUPPORTED, "call too large");
  const size_t need = plan.ws_bytes;
  if (need > 0 && (workspace == nullptr || workspace_bytes < need))
    return fail(Q1_ERR_WORKSPACE, "workspace too small: need %zu bytes, got %zu", need, workspace ? workspace_bytes : 0);
  if (need > 0 && !aligned(workspace, 256)) return fail(Q1_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  st = check_current_device();
  if (st != Q1_OK) return st;
  return hip_status(launch_kv_attn(*c, *a, plan, static_cast<unsigned char*>(workspace), static_cast<hipStream_t>(stream)),
                    "cache attention launch");
}

q1_status q1_conv_step(const q1_conv* d, int64_t B, int64_t T, void* stream) {
  if (d == nullptr) return fail(Q1_ERR_INVALID_ARG, "convolution descriptor is NULL");
  q1_status st = check_step(B, T);
  if (st != Q1_OK) return st;
  if (B == 0 || T == 0) return ok();
  st = check_conv(d, B * T, B);
  if (st == Q1_OK) st = check_current_device();
  if (st != Q1_OK) return st;
  return hip_status(launch_conv_step(*d, B, T, static_cast<hipStream_t>(stream)), "convolution step launch");
}

q1_status q1_conv_prefill(const q1_conv* d, int64_t tokens, int64_t nseq, const int32_t* cu_seqlens, void* stream) {
  if (d == nullptr) return fail(Q1_ERR_INVALID_ARG, "convolution descriptor is NULL");
  if (tokens < 0 || nseq < 0) return fail(Q1_ERR_INVALID_ARG, "tokens and nseq must be >= 0");
  if (tokens == 0 || nseq == 0) return ok();
  q1_status st = check_ragged(tokens, nseq, cu_seqlens);
  if (st == Q1_OK) st = check_conv(d, tokens, nseq);
  if (st == Q1_OK && conv_pieces(*d, tokens, nseq) >= k31 / (d->C / 8)) st = fail(Q1_ERR_UNSUPPORTED, "call too large");
  if (st == Q1_OK) st = check_current_device();
  if (st != Q1_OK) return st;
  return hip_status(launch_conv_prefill(*d, Ragged{cu_seqlens, tokens, nseq}, static_cast<hipStream_t>(stream)),
                    "convolution launch");
}

q1_status q1_scan_step(const q1_scan* d, int64_t B, int64_t T, void* stream) {
  q1_status st = check_scan_shape(d);
  if (st == Q1_OK) st = check_step(B, T);
  if (st != Q1_OK) return st;
  if (B == 0 || T == 0) return ok();
  st = check_scan(d, B * T, B);
  if (st == Q1_OK) st = check_current_device();
  if (st != Q1_OK) return st;
  return hip_status(launch_scan_step(*d, B, T, static_cast<hipStream_t>(stream)), "scan step launch");
}

size_t q1_scan_prefill_workspace_bytes(const q1_scan* d, int64_t tokens, int64_t nseq) {
  if (check_scan_shape(d) != Q1_OK) return 0;
  if (tokens < 0 || nseq < 0) {
    fail(Q1_ERR_INVALID_ARG, "tokens and nseq must be >= 0");
    return 0;
  }
  ok();
  if (tokens == 0 || nseq == 0) return 0;
  if (tokens >= k31 || nseq >= k31 / (4 * d->Di) || scan_too_large(*d, tokens, nseq)) {
    fail(Q1_ERR_UNSUPPORTED, "call too large");
    return 0;
  }
  return scan_ws_bytes(*d, tokens, nseq);
}

q1_status q1_scan_prefill(const q1_scan* d, int64_t tokens, int64_t nseq, const int32_t* cu_seqlens, void* workspace,
                          size_t workspace_bytes, void* stream) {
  q1_status st = check_scan_shape(d);
  if (st != Q1_OK) return st;
  if (tokens < 0 || nseq < 0) return fail(Q1_ERR_INVALID_ARG, "tokens and nseq must be >= 0");
  if (tokens == 0 || nseq == 0) return ok();
  st = check_ragged(tokens, nseq, cu_seqlens);
  if (st == Q1_OK) st = check_scan(d, tokens, nseq);
  if (st == Q1_OK && scan_too_large(*d, tokens, nseq)) st = fail(Q1_ERR_UNSUPPORTED, "call too large");
  if (st != Q1_OK) return st;
  const size_t need = scan_ws_bytes(*d, tokens, nseq);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need))
    return fail(Q1_ERR_WORKSPACE, "workspace too small: need %zu bytes, got %zu", need, workspace ? workspace_bytes : 0);
  if (need > 0 && !aligned(workspace, 256)) return fail(Q1_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  st = check_current_device();
  if (st != Q1_OK) return st;
  return hip_status(launch_scan_prefill(*d, Ragged{cu_seqlens, tokens, nseq}, static_cast<unsigned char*>(workspace),
                                        static_cast<hipStream_t>(stream)),
                    "scan launch");
}

}  // extern "C"
