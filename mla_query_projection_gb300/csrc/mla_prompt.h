// mla_prompt.h - arguments of the prompt's operators (mla_prompt_rows.cu,
// mla_prompt_attn.cu).
#pragma once

#include <stdint.h>

#include "mla_internal.h"

namespace mla {

constexpr int kRopePairs = kRope / 2;

// A rotation: what pair p turns a position (a 64-bit fraction of a turn), the
// axis its positions come from, whether pairs are neighbours or halves.
struct RopeSpec {
  uint64_t turns[kRopePairs];
  uint8_t axis[kRopePairs];
  int axes;
  int interleaved;
  float scale;  // of cosine and sine
};

struct RopeArgs {
  RopeSpec spec;
  const int32_t* positions;  // [axes][pos_stride]
  int64_t pos_stride;
  int64_t offset;  // added to every position
};

struct CacheWriteArgs {
  int64_t tokens;
  const uint16_t* kv_c;
  const uint16_t* k_pe;
  int64_t kv_c_stride, k_pe_stride;
  const uint16_t* gamma;  // or null: rows are normalised
  float eps;
  RopeArgs rope;  // positions null: no rotation
  const int64_t* slots;
  uint8_t* cache;
  int64_t capacity;  // slots
  int page_size;
  const float* k_scale;
  uint16_t* rows;  // [tokens][rows_stride] or null
  int64_t rows_stride;
  unsigned* flags;  // or null
};

struct CacheReadArgs {
  const uint8_t* cache;
  int64_t num_pages;
  int page_size;
  const float* k_scale;
  const int32_t* table;
  int64_t bt_stride, bt_cols;
  int requests;
  const int32_t* cu;     // [requests + 1]
  const int32_t* first;  // [requests] or null
  int64_t max_rows;
  uint16_t* rows;
  int64_t rows_stride;
  unsigned* flags;  // or null
};

// Attention of packed documents (mla_prompt_attn.cu).
struct PromptInputs {
  const void *q_nope, *q_pe, *k_nope, *k_pe, *v;
  int64_t qn_ts, qn_hs, qp_ts, qp_hs, kn_ts, kn_hs, kp_ts, v_ts, v_hs;  // elements
};
struct PromptArgs {
  const int32_t* cu_q;    // [docs + 1]
  const int32_t* cu_k;    // [docs + 1]
  const int32_t* prefix;  // [docs] or null
  const float* slopes;    // [heads] or null
  int docs, heads;
  int q_tokens, k_tokens;
  int causal;
  float scale, cap;  // cap 0: none
  uint16_t* out;
  int64_t o_ts, o_hs;
  float* lse;  // [q_tokens][heads] or null
  float above, times;  // how much lower exponents are taken (base 2); 2 to that
  int splits;
  float* part_o;    // [splits][heads][q_tokens][128], each part's output
  float2* part_ml;  // [splits][heads][q_tokens] reference in base 2, sum
  const uint16_t* v;
  int64_t v_ts, v_hs;
  int tiles;       // the most tiles of 256 query rows that the documents can have together
  int group;       // heads that are handed out together
  uint32_t* next;  // items handed out beside each CTA's first, CTAs that are done; zero between calls
  uint32_t* err;
};
struct PromptMaps {
  CUtensorMap q_nope, q_pe, k_nope, k_pe, v;
};
cudaError_t prepare_prompt();
cudaError_t launch_prompt(const PromptArgs& a, const PromptInputs& in, int ctas, cudaStream_t stream);

}  // namespace mla
