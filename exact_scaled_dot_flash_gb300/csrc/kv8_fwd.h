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

// Calls with at most this many rows (queries x heads) of a kv head share out
// the keys (attn_kv8_decode.cuh).
constexpr int DECODE_ROWS = 32;
inline bool decode_rows(int max_queries, int heads) {
  return static_cast<int64_t>(max_queries) * heads <= DECODE_ROWS;
}

// Ranges that the keys of a call are cut into, each for Hkv CTAs: two CTAs for
// each of the 152 SMs (the kernel for 8 rows fits twice); with many heads four
// waves of smaller ones, so that a last wave that is not full costs little;
// never more than there can be blocks of 128 keys.
inline int decode_ranges(int num_seqs, int Hkv, int max_pages, int page_size) {
  const int64_t keys = static_cast<int64_t>(max_pages) * page_size;
  const int64_t blocks = num_seqs * ((keys + 127) / 128 > 1 ? (keys + 127) / 128 : 1);
  int64_t r = (Hkv > 16 ? 4 : 1) * 304 / Hkv;
  if (r > blocks) r = blocks;
  return static_cast<int>(r > 1 ? r : 1);
}

// Partials: CTA c (range, head) owns slots 2c (its first sequence) and 2c + 1
// (its last), each rows x (D floats) and rows x (m, l).
struct DecodeLayout {
  int64_t slots, rows;
  int64_t ml_offset(int D) const { return (slots * rows * D * 4 + 255) / 256 * 256; }
  int64_t bytes(int D) const { return ml_offset(D) + slots * rows * 8; }
};

template <bool BF16>
cudaError_t launch_decode(const FwdParams& p, int fmt, cudaStream_t st);

}  // namespace kv8
}  // namespace attn
