// kv8_fwd.h - parameters of the kernels behind attn_paged_kv8_fwd.
#pragma once

#include <math.h>

#include <algorithm>
#include <atomic>

#include "host_checks.h"
#include "kv8.cuh"

namespace attn {
namespace kv8 {

struct FwdParams {
  Cache c;
  int Hq, num_queries, max_queries, causal, device;
  bool bf16;                   // type of q and out in the 16-bit kernels (else F16)
  uint32_t group_magic;        // row / group = umulhi(row, group_magic) for group > 1, row < 65536
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

// How a call with few rows is cut (attn_kv8_decode.cuh). A CTA takes up to 32
// rows of a kv head (8 nt); more rows go to `row_groups` CTAs that read the same
// codes (the second from L2).
struct DecodePlan {
  int rows = 0, row_groups = 0, nt = 0, ranges = 0, aligned = 0;  // aligned: a range is a sequence
  bool few_keys = false;  // fewer ranges than three quarters of what the SMs hold
  bool cuts() const { return !aligned && ranges > 1; }            // sequences may be cut: workspace
  int slot_rows() const { return row_groups * nt * 8; }
  // Partials: CTA c (range, head) owns slots 2c (its first sequence) and 2c + 1
  // (its last), each slot_rows x D floats; then slot_rows x (m, l) for each slot;
  // then a counter for each (range, head, row group).
  int64_t ml_offset(int Hkv, int D) const { return 2ll * ranges * Hkv * slot_rows() * D * 4; }
  int64_t counter_offset(int Hkv, int D) const { return ml_offset(Hkv, D) + 2ll * ranges * Hkv * slot_rows() * 8; }
  int64_t bytes(int Hkv, int D) const { return cuts() ? counter_offset(Hkv, D) + 4ll * ranges * Hkv * row_groups : 0; }
};

// Opts a kernel in to `smem` bytes of shared memory, once for each device.
template <typename K>
cudaError_t allow_smem(K kern, int smem, int device, std::atomic<unsigned long long>& configured) {
  const unsigned long long bit = device >= 0 && device < 64 ? 1ull << device : 0ull;
  if (bit && (configured.load(std::memory_order_acquire) & bit)) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess) configured.fetch_or(bit, std::memory_order_acq_rel);
  return e;
}

// Ranges that the keys of a call are cut into, each for Hkv CTAs (and row
// groups): as many CTAs as the 152 SMs hold at once, three each of the kernels
// for 8 and 16 rows, two of the others (twice as many, or a second set of small
// ones for the SMs that are done first, cost more in partials than the balance
// gave: 123 us instead of 114 us for 64 sequences of 1k-8k keys). A sequence of n
// blocks of 128 keys that is cut every m blocks is streamed in m times some 1 us
// and leaves n / m parts to one CTA, which combines 4 rows of 8 parts in some 1 us:
// a range has at least the m where the two are equal. Sequences of at most 512 keys (4 blocks)
// are a range each: cutting them would cost a second launch and a workspace.
inline DecodePlan decode_plan(int num_seqs, int Hkv, int heads, int max_queries, int max_pages, int page_size) {
  DecodePlan d;
  d.rows = static_cast<int>(static_cast<int64_t>(max_queries) * heads);
  d.row_groups = (d.rows + 31) / 32;
  const int group_rows = (d.rows + d.row_groups - 1) / d.row_groups;
  d.nt = (group_rows + 7) / 8;
  const int64_t keys = static_cast<int64_t>(max_pages) * page_size;
  const int64_t blocks = num_seqs * (keys > 128 ? (keys + 127) / 128 : 1);
  const int64_t side = static_cast<int64_t>(Hkv) * d.row_groups;
  d.aligned = keys <= 512;
  int64_t r = d.aligned ? num_seqs : SMS * (d.nt <= 2 ? 3 : 2) / side;
  if (!d.aligned) {
    const double n = static_cast<double>(blocks) / num_seqs;
    const double m = sqrt(n * ((group_rows + 3) / 4) / 8);
    const int64_t most = static_cast<int64_t>(blocks / (m > 1 ? m : 1));
    d.few_keys = 4 * most < 3 * r;
    r = std::min(r, most);
  }
  d.ranges = static_cast<int>(r > 1 ? r : 1);
  return d;
}

template <int FMT>
cudaError_t launch_decode(const FwdParams& p, const DecodePlan& plan, cudaStream_t st);

// Many rows, F16/BF16, D in {64, 128} (attn_kv8_tc.cuh): CTAs of 256 packed rows
// of a sequence and kv head. Where they fill at most half the 152 SMs, their keys
// are cut into runs of at least 4 tiles of 128, as many as fill the SMs (48 CTAs
// over up to 3.5k keys: 41 us, 67 whole); over 8k keys and more, 51 to 114 CTAs are
// cut to fill them twice (up to 16k keys, 100 rows of 20 sequences, 80 CTAs: 138 us,
// 228 whole; 104 CTAs: 174, 229; but 112 CTAs over up to 3.5k keys: 77, 68). From 115
// CTAs on it depends on how far the lengths lie apart, which the host does not know:
// 120 CTAs, 3k-16k keys: 170 us, 227 whole; all of 16k: 246, 234. Nor are these borders
// sharp: 80 CTAs over 2k-7.9k keys take 74 us cut, 113 whole, as they are run.
// The workspace then holds for each run and row D floats and (m, l).
inline int64_t key_tiles(int max_pages, int page_size) { return (static_cast<int64_t>(max_pages) * page_size + 127) / 128; }
inline int64_t tc_qblocks(int max_queries, int heads) { return (static_cast<int64_t>(max_queries) * heads + 255) / 256; }
inline int tc_splits(int num_seqs, int Hkv, int64_t qblocks, int max_pages, int page_size) {
  const int64_t ctas = num_seqs * qblocks * Hkv;
  const int64_t tiles = key_tiles(max_pages, page_size);
  int64_t s = ctas <= 0 ? 1 : ctas > 50 && ctas <= 114 && tiles >= 64 ? 2 * SMS / ctas : SMS / ctas;
  if (s > tiles / 4) s = tiles / 4;
  if (s > 32) s = 32;
  return static_cast<int>(s > 1 ? s : 1);
}

// Which of the two takes a call. More than 64 rows: the kernel for many. 17 to 64
// rows of so few keys that the other one's CTAs would not fill the SMs: it too (30
// rows, one sequence of some 6k keys, 4 kv heads: 28 against 50 us; 12 sequences: 87
// against 75). 49 to 64 rows: where its CTAs, cut or not, fill the SMs, or have few
// keys, since its time is that of its longest CTA and the other one's that of all
// keys. 4k-16k keys, CTAs whole, 50 to 64 rows: up to 120 CTAs the few-row kernel is
// the faster one (2k-7.9k keys, 80 CTAs: 88 against 113 us; 3k-16k keys, 120: 170, 227),
// from there on they cross (2k-7.9k, 148: 131 against 115; 3k-16k, 148: 203, 229). Fewer
// keys, any number of CTAs: the many-row one (4 to 960 CTAs, up to 500 keys: 1.0 to 1.35
// times as fast, up to 2k keys 1.3 to 1.7 times; 80 to 148 CTAs up to 3.5k keys: 59 to 61
// against 57 to 80 us).
inline bool decode_takes(int num_seqs, int Hkv, int heads, int max_queries, int max_pages, int page_size) {
  const int64_t rows = static_cast<int64_t>(max_queries) * heads;
  if (rows > 64) return false;
  if (rows <= 16) return true;
  if (decode_plan(num_seqs, Hkv, heads, max_queries, max_pages, page_size).few_keys) return false;
  return rows <= 48 || (tc_splits(num_seqs, Hkv, 1, max_pages, page_size) == 1 && key_tiles(max_pages, page_size) >= 32 &&
                        static_cast<int64_t>(num_seqs) * Hkv <= 120);
}
template <int FMT>
cudaError_t launch_tc(const FwdParams& p, cudaStream_t st);

}  // namespace kv8
}  // namespace attn
