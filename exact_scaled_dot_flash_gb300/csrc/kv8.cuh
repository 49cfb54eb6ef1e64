// kv8.cuh - the 8-bit paged cache: its layout and its codes.
//
// Codes K, V [pages, page_size, Hkv, D], one byte each, and a float scale for
// every `group` consecutive tokens of a head, [pages, Hkv, page_size / group]
// (the scales of one head lie side by side, as the attention that streams a
// head's keys reads them). A value is code * scale.
//   int8: a two's complement integer (the writer makes -127..127).
//   e4m3: 1 sign, 4 exponent (bias 7) and 3 mantissa bits, gradual underflow,
//         largest value 448. The writer never makes the codes 0x7f and 0xff;
//         read back they stand for +-480, so that a byte never is a NaN and a
//         masked token's byte cannot leak through 0 * NaN.
#pragma once

#include "params.h"
#include "ptx.cuh"

namespace attn {
namespace kv8 {

constexpr int FMT_INT8 = 0, FMT_E4M3 = 1;
// Scales below this would make 1/scale overflow; a group of zeros has it too.
constexpr float SCALE_FLOOR = 7.888609052210118e-31f;  // 2^-100

struct Cache {
  int num_pages, page_size, Hkv, D, group, per;  // per = page_size / group scales of a (page, head)
  int num_seqs, max_pages;
  const int32_t* block_table;  // [num_seqs, max_pages]
  const int32_t* seq_lens;     // [num_seqs]
  int* status;
};

// The fp32 values of the 4 codes of a 32-bit word (lowest byte first).
template <int FMT>
__device__ __forceinline__ float4 decode4(uint32_t w) {
  if constexpr (FMT == FMT_INT8) {
    return make_float4(static_cast<float>(static_cast<int8_t>(w)), static_cast<float>(static_cast<int8_t>(w >> 8)),
                       static_cast<float>(static_cast<int8_t>(w >> 16)), static_cast<float>(static_cast<int8_t>(w >> 24)));
  } else {
    // sign to bit 31 and the 7 other bits to the top of the fp32 exponent and
    // mantissa: the value times 2^(7 - 127), subnormals included; one exact
    // multiplication by 2^120 puts the exponent right
    constexpr float K = 1.329227995784916e36f;  // 2^120
    auto one = [](uint32_t b) { return __uint_as_float(((b & 0x80u) << 24) | ((b & 0x7fu) << 20)) * K; };
    return make_float4(one(w & 0xffu), one((w >> 8) & 0xffu), one((w >> 16) & 0xffu), one(w >> 24));
  }
}

__device__ __forceinline__ int seq_len(const Cache& c, int s) {
  return min(max(__ldg(c.seq_lens + s), 0), c.max_pages * c.page_size);
}

// Physical page of key block `b` of sequence s, or -1 (outside the table or the cache).
__device__ __forceinline__ int page_of(const Cache& c, int s, int b) {
  if (b < 0 || b >= c.max_pages) return -1;
  const int p = __ldg(c.block_table + static_cast<size_t>(s) * c.max_pages + b);
  return p >= 0 && p < c.num_pages ? p : -1;
}

__device__ __forceinline__ size_t scale_index(const Cache& c, int page, int row, int h) {
  return (static_cast<size_t>(page) * c.Hkv + h) * c.per + row / c.group;
}

// Packed rows: sequence s has rows off[s] .. off[s+1]-1, clamped to [0, n].
__device__ __forceinline__ void row_range(const int32_t* off, int s, int n, int& lo, int& hi) {
  lo = min(max(__ldg(off + s), 0), n);
  hi = min(max(__ldg(off + s + 1), lo), n);
}

}  // namespace kv8
}  // namespace attn
