// mk_attn.cuh -- causal attention of packed query rows over keys and values
// that lie packed beside them or in a paged cache.
//
//   o_t = sum_j p_tj v_j / sum_j p_tj,  p_tj = exp(scale q_t . k_j - m_t)
//
// over the keys j <= len - T + t of the row's own sequence (T new tokens, len
// keys).
#pragma once
#include "mk_rows.cuh"

namespace mk {
namespace at {

struct AttnArgs {
  const unsigned char* q;
  unsigned char* out;
  float* lse;                          // [rows][q_heads], or null
  long long q_ts, q_hs, o_ts, o_hs;    // token and head strides, values
  const int* cu_q;                     // [batch + 1] first row of each sequence
  int rows, batch, q_heads, kv_heads, group;
  float scale_log2;                    // scale * log2(e)
  // packed keys and values
  const unsigned char *k, *v;
  long long k_ts, k_hs, v_ts, v_hs;
  // or a paged cache
  PagedView c;
  const int* table;                    // [batch][table_stride]
  int table_stride;
  const int* seq_lens;
};

}  // namespace at
}  // namespace mk
