// What the entry points and the kernels of the prompt's operators share.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace mla {

// Rows [token][head] of a tensor: strides in elements, columns contiguous.
struct HeadRows {
  const void* p;
  int64_t token_stride, head_stride;
};

// One call of the expanded attention.
struct PrefillCall {
  HeadRows q_nope, q_pe, k_nope, k_pe, v, out;
  float* lse;
  const int32_t* cu_q;
  const int32_t* cu_k;
  int batch, num_heads, num_tokens_q, num_tokens_k;
  bool causal;
  float scale;
  void* workspace;
};
int prefill_items(int num_tokens_q, int batch);

// How a call is cut up.
struct PrefillForm {
  int item_rows;  // query rows of an item: 512 on a pair of CTAs, 256 on one
  int parts;      // of a row block's keys, at most
  int group;      // heads whose items are mixed
  size_t workspace;
};
PrefillForm prefill_form(int num_tokens_q, int num_tokens_k, int batch, int num_heads, int sms);
size_t prefill_workspace(int num_tokens_q, int num_tokens_k, int batch, int num_heads, int sms);

}  // namespace mla
