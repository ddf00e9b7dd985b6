// Internal interface between the C ABI of q1_memory.h (q1_memory_api.cpp) and
// its HIP kernels.  Not part of the public boundary.
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

#include "../../include/q1_memory.h"

namespace q1 {

constexpr int kKvBlock = 32;  // elements that share a scale

// ---- keys and values in pages -------------------------------------------------

hipError_t launch_kv_write(const q1_kv& c, const void* k, const void* v, bool f16, int64_t k_ld, int64_t v_ld,
                           int64_t tokens, const int32_t* slots, hipStream_t s);
hipError_t launch_kv_read(const q1_kv& c, const int32_t* slots, int64_t rows, void* k, void* v, int32_t out_dtype,
                          hipStream_t s);

// Division of whole numbers below 2^31 by d >= 1: x / d = (2 x * mul) >> 32 >> shift.
struct Divider {
  uint32_t mul;
  int32_t shift;
};
inline Divider divider(uint32_t d) {
  // 2^(31 + l) / d rounded up, l = ceil(log2 d): off by less than 2^l / d of a unit per 2^31
  int l = 0;
  while (((uint64_t)1 << l) < d) ++l;
  return {(uint32_t)((((uint64_t)1 << (31 + l)) + d - 1) / d), l};
}

// How a call is cut into work items (see q1_kv_attn.hip).
struct KvPlan {
  int32_t nm;              // blocks of 16 query rows of a wave
  int32_t by_rows;         // 1: waves of an item share its tokens
  uint32_t heads_each, R;  // query heads and rows of a key/value head
  uint32_t rows;           // rows of an item
  uint32_t row_blocks;     // items along the rows
  uint32_t entries;        // sequences times row_blocks
  int32_t cut;             // 1: workgroups have equal shares of all tokens, else an item each
  uint32_t wgs;
  int32_t too_large;       // more units of work than are counted in 31 bits
  uint32_t join_rows, groups_each;  // rows of a wave that joins, and such groups of an item
  Divider page, group, blocks, kv_heads, sequences, groups;  // by page_size, heads_each, row_blocks, Hkv, B, groups_each
  size_t o_off, ml_off, ws_bytes;
};

KvPlan plan_kv_attn(const q1_kv& c, const q1_kv_query& a);
hipError_t launch_kv_attn(const q1_kv& c, const q1_kv_query& a, const KvPlan& p, unsigned char* ws, hipStream_t s);

// ---- short convolution and scan ------------------------------------------------

// A sequence's rows: T each (single tokens, cu == nullptr), or from cu[s] to cu[s + 1].
struct Ragged {
  const int32_t* cu;
  int64_t tokens, nseq;
};

// Tokens of a piece of a prompt's convolution, and its pieces.
constexpr int64_t kConvTokens = 16;
int64_t conv_pieces(const q1_conv& d, int64_t tokens, int64_t nseq);
hipError_t launch_conv_step(const q1_conv& d, int64_t B, int64_t T, hipStream_t s);
hipError_t launch_conv_prefill(const q1_conv& d, const Ragged& r, hipStream_t s);

hipError_t launch_scan_step(const q1_scan& d, int64_t B, int64_t T, hipStream_t s);

// Tokens of a chunk of a prompt's scan: 0 for whole sequences.
int64_t scan_chunk(const q1_scan& d, int64_t tokens, int64_t nseq);
int64_t scan_pieces(const q1_scan& d, int64_t tokens, int64_t nseq);
size_t scan_ws_bytes(const q1_scan& d, int64_t tokens, int64_t nseq);
hipError_t launch_scan_prefill(const q1_scan& d, const Ragged& r, unsigned char* ws, hipStream_t s);

// Pieces of at most `per` tokens of a ragged batch: sequence s has the pieces from
// cu[s] / per + s on, so a piece's sequence is found by its number alone; there are
// at most this many, some of them empty.
inline int64_t ragged_pieces(int64_t tokens, int64_t nseq, int64_t per) { return tokens / per + nseq; }

}  // namespace q1
