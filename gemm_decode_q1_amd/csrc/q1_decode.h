// Internal interface between the C ABI of the decode-step operators
// (q1_decode_api.cpp) and their HIP kernels.  Not part of the public boundary.
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

#include "../../include/q1_decode.h"

namespace q1 {

// ---- gated delta rule -------------------------------------------------------

// Rows of a sequence: T each (single tokens), or from cu[s] to cu[s + 1] (prompts).
struct DeltaArgs {
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  int64_t q_ld, k_ld, v_ld;
  const float* g;
  const float* beta;
  float* state;
  const int32_t* slot_ids;
  void* out;
  int64_t slots;
  int32_t Hk, Hv, Dv;
  int32_t out_dtype, l2norm;
  float scale;
  int64_t T;        // single tokens: tokens per sequence
  const int32_t* cu;
  int64_t tokens;   // prompts: rows in all
  int64_t nseq;
};

hipError_t launch_delta_recurrent(const DeltaArgs& a, bool f16, int Dk, hipStream_t s);

// Prompts in chunks of kDeltaChunk tokens (q1_delta_chunk.hip).
constexpr int kDeltaChunk = 64;
constexpr size_t kDeltaChunkBytes = (10 + 10 + 1) * 1024;  // workspace per chunk and value head
// Chunks the workspace has room for, whatever the sequences' lengths.
inline int64_t delta_chunk_slots(int64_t tokens, int64_t nseq) { return tokens / kDeltaChunk + nseq + 1; }
hipError_t launch_delta_chunk(const DeltaArgs& a, bool f16, int Dk, unsigned char* ws, hipStream_t s);

// ---- attention over a shared prefix -----------------------------------------

// How a call is cut into work items (see q1_attn.hip).
struct AttnPlan {
  int32_t nm;                            // blocks of 16 query rows per item by tokens
  int32_t by_rows;                       // 1: waves of a prefix item share its tokens
  int32_t prefix_rb, suffix_rb;          // items along the rows
  int32_t prefix_splits, suffix_splits;  // items along the tokens
  int64_t prefix_tokens, suffix_tokens;  // tokens per item
  int64_t prefix_wgs, wgs;
  size_t ml_off, ws_bytes;
};

AttnPlan plan_prefix_attn(const q1_attn& a);
hipError_t launch_prefix_attn(const q1_attn& a, const AttnPlan& p, unsigned char* ws, hipStream_t s);

// ---- sampler ----------------------------------------------------------------

struct SampleArgs {
  const void* logits;
  int32_t dtype;
  int64_t B, V, ld;
  const float* u;
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  void* tokens;
  int32_t tokens_int64;
  float* logprob;
};

size_t sample_ws_bytes(int64_t B, int64_t V);
hipError_t launch_sample(const SampleArgs& a, unsigned char* ws, hipStream_t s);

}  // namespace q1
