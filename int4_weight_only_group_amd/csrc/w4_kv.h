// The paged key/value cache as the kernels see it, and the launchers of the operators on it.
#pragma once

#include "w4_internal.h"

namespace w4 {

// Element (page, head, token of the page, d) of K lies at
// k[page * stride_page + head * stride_head + token * stride_token + d]; V alike.
struct KvCache {
  void* k;
  void* v;
  const float* k_scale;  // e4m3: the value of a code is code * scale[head] (nullptr: 1)
  const float* v_scale;
  int64_t stride_page, stride_head, stride_token;  // elements
  int pages, page_size, heads, dim;
  bool e4m3;
};

// A norm of each query and key head before it turns: x w / sqrt(mean(x^2) + eps).
struct HeadNorm {
  const float *q, *k;  // weights of the dims; nullptr: 1
  float eps;
};

// norm == nullptr: none
void launch_rope(const void* x, bool f32, int64_t ldx, const int32_t* pos, const float* freq, uint16_t* y, int64_t ldy,
                 int T, int H, int D, int R, bool interleaved, bool inverse, float mscale, const HeadNorm* norm,
                 hipStream_t st);
// q == nullptr: nothing but the append
void launch_kv_append(const void* q, int64_t ldq, uint16_t* q_out, int64_t ldqo, int Hq, const void* k, int64_t ldk,
                      const void* v, int64_t ldv, bool f32, const KvCache& c, const int64_t* slots, const int32_t* pos,
                      const float* freq, int T, int R, bool interleaved, float mscale, const HeadNorm* norm,
                      hipStream_t st);

// Pages, row starts, positions and slots of a step; see kv_plan in w4.h.
struct PlanArgs {
  const int32_t *kv_len, *new_len, *depth;  // depth: nullptr: rows follow each other
  int32_t *table, *owned, *free, *free_count;
  int64_t ldt;
  int32_t *q_start, *kv_total, *pos, *status;
  int64_t* slot;
  int B, W, pages, page_size, T;
};
void launch_plan(const PlanArgs& a, hipStream_t st);

// Attention of T new tokens of B sequences over the cache; see attention_paged and attention_paged_tree in w4.h.
struct AttnArgs {
  const uint16_t* q;
  uint16_t* out;
  int64_t ldq, ldo;
  KvCache c;
  const int32_t* table;
  int64_t ldt;
  const int32_t* kv_len;
  const int32_t* q_start;  // nullptr: one token each
  int W, B, T, max_q, Hq, window;
  float scale;
  const uint64_t* mask = nullptr;  // [T][ldm]: which new tokens of its sequence a row sees; nullptr: those up to itself
  int64_t ldm = 0;
};
bool attention_ws_bytes(const AttnArgs& a, size_t& bytes);  // false: no launch holds so many workgroups
void launch_attention(const AttnArgs& a, void* ws, hipStream_t st);
void launch_attention_tree(const AttnArgs& a, void* ws, hipStream_t st);  // with a mask

}  // namespace w4
