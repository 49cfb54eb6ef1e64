// kv8_fwd.h - parameters of the kernels behind attn_paged_kv8_fwd.
#pragma once

#include "kv8.cuh"

namespace attn {
namespace kv8 {

struct FwdParams {
  Cache c;
  int Hq, num_queries, max_queries, causal, device;
  float scale_log2;            // scale * log2(e): scores are kept in the log2 domain
  const int32_t* q_offsets;    // [num_seqs + 1]
  const int32_t* positions;    // [num_queries] or nullptr (the newest tokens)
  const void* q;               // [num_queries, Hq, D]
  const uint8_t *k_codes, *v_codes;
  const float *k_scale, *v_scale;
  void* out;
  float* lse;  // [num_queries, Hq] or nullptr
  void* ws;
};

}  // namespace kv8
}  // namespace attn
