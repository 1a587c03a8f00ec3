// What the 4-bit cache's kernels and the C ABI share.
#pragma once

#include "awq_internal.h"

namespace awq {

// A cache's arrays and sizes; `shift` is log2 of the tokens of a page.
struct Kv4 {
  uint32_t *k_codes, *v_codes;  // kv4_device.h has their order
  uint32_t *k_params, *v_params;
  int64_t pages;
  int heads, shift, dim, group;
};

struct Kv4Rows {  // keys and values of tokens, strides in values
  const void *k, *v;
  int64_t k_token, k_head, v_token, v_head;
};
hipError_t launch_kv4_append(const Kv4& c, const Kv4Rows& rows, int type, int64_t tokens,
                             const int32_t* slots, hipStream_t stream);
hipError_t launch_kv4_gather(const Kv4& c, int64_t tokens, const int32_t* slots, void* k, void* v,
                             int type, hipStream_t stream);

struct Kv4Attention {
  Kv4 cache;
  const void* q;
  void* out;
  int type, heads;  // heads: the queries'
  int64_t tokens, q_token, q_head;
  int64_t seqs, per_seq;  // per_seq: entries of a sequence in the table
  const int32_t *starts, *table, *lens;
  float scale;
  void* ws;
};
size_t kv4_attention_workspace(const Kv4Attention& a);
hipError_t launch_kv4_attention(const Kv4Attention& a, hipStream_t stream);

}  // namespace awq
