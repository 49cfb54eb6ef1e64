// prefix.cuh - attention over a paged cache for groups of sequences that share a
// prefix (attn_paged_prefix_fwd): parameters, workspace and what the kernels read of
// the metadata.
//
// A row (query, head) sees the keys j < lim of its sequence. Group g's first `pre`
// keys are the same for all its members, so a call has two stages:
//   prefix: a unit is a group, its rows all the queries of its members (packed, so they
//           lie side by side), its keys [0, pre). A row leaves `parts` parts (m, l, O) in
//           the workspace, one for each run of keys that its unit was cut into:
//           O = sum_j 2^(x_j - m) v_j, l = sum_j 2^(x_j - m), x in log2 units.
//   suffix: a unit is a sequence, its keys [pre, L) (all of them outside a group). It
//           joins its own part with those of the prefix and writes out and lse.
#pragma once

#include <atomic>

#include "host_checks.h"
#include "params.h"
#include "ptx.cuh"

namespace attn {
namespace prefix {

constexpr float LN2 = 0.6931471805599453f;
constexpr int MAX_PARTS = 32;

struct Params {
  int num_seqs, num_queries, num_groups, Hq, Hkv, D, page_size, num_pages, max_pages;
  int max_queries, max_group_queries;
  int causal, device;
  float scale_log2;
  const int32_t *block_table, *seq_lens, *q_offsets, *positions, *group_offsets, *prefix_lens;
  const void *q, *k, *v;
  void* out;
  float* lse;
  int* status;
  // workspace
  int most_parts;   // slots of a row
  int32_t* parts;   // [num_groups] parts of each row of the group
  float2* ml;       // [most_parts, num_queries * Hq]
  float* o;         // [most_parts, num_queries * Hq, D]
};

__device__ __forceinline__ int capacity(const Params& p) { return p.max_pages * p.page_size; }

__device__ __forceinline__ int seq_len(const Params& p, int s) { return min(max(__ldg(p.seq_lens + s), 0), capacity(p)); }

__device__ __forceinline__ int query_at(const Params& p, int s) { return min(max(__ldg(p.q_offsets + s), 0), p.num_queries); }

__device__ __forceinline__ void group_range(const Params& p, int g, int& a, int& b) {
  a = min(max(__ldg(p.group_offsets + g), 0), p.num_seqs);
  b = min(max(__ldg(p.group_offsets + g + 1), a), p.num_seqs);
}

__device__ __forceinline__ int prefix_len(const Params& p, int g) { return min(max(__ldg(p.prefix_lens + g), 0), capacity(p)); }

// The last i in [lo, hi) with off[i] <= x, or lo.
__device__ __forceinline__ int last_at_most(const int32_t* off, int lo, int hi, int x) {
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(off + mid) <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Group of sequence s, or -1.
__device__ __forceinline__ int group_of(const Params& p, int s) {
  if (p.num_groups == 0) return -1;
  const int g = last_at_most(p.group_offsets, 0, p.num_groups, s);
  int a, b;
  group_range(p, g, a, b);
  return s >= a && s < b ? g : -1;
}

// Keys that query `i` of sequence s sees: j < the result.
__device__ __forceinline__ int limit_of(const Params& p, int s, int i) {
  const int L = seq_len(p, s);
  if (!p.causal) return L;
  int pos;
  if (p.positions) pos = in_bounds(p.status, i, p.num_queries) ? __ldg(p.positions + i) : -1;
  else pos = L - query_at(p, s + 1) + i;
  return pos < 0 ? 0 : min(L, pos < L ? pos + 1 : L);
}

// Physical page of key block b of sequence s, or -1.
__device__ __forceinline__ int page_of(const Params& p, int s, int b) {
  if (b < 0 || b >= p.max_pages) return -1;
  const int page = __ldg(p.block_table + static_cast<int64_t>(s) * p.max_pages + b);
  return page >= 0 && page < p.num_pages ? page : -1;
}

// The member of [a, b) whose row the prefix is read through: the first with the most
// tokens of it. Every thread of the CTA calls it.
__device__ __forceinline__ int reader_of(const Params& p, int a, int b, int pre) {
  __shared__ unsigned long long best;
  if (threadIdx.x == 0) best = 0;
  __syncthreads();
  unsigned long long mine = 0;
  for (int s = a + threadIdx.x; s < b; s += blockDim.x) {
    const unsigned long long x = (static_cast<unsigned long long>(min(seq_len(p, s), pre)) << 32) | static_cast<uint32_t>(~s);
    mine = x > mine ? x : mine;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const unsigned long long x = __shfl_xor_sync(0xffffffffu, mine, o);
    mine = x > mine ? x : mine;
  }
  if ((threadIdx.x & 31) == 0 && mine) atomicMax(&best, mine);
  __syncthreads();
  return static_cast<int>(~static_cast<uint32_t>(best));
}

// Opts a kernel in to `smem` bytes of shared memory, once for each device.
template <typename K>
cudaError_t allow_smem(K kern, int smem, int device, std::atomic<unsigned long long>& configured) {
  const unsigned long long bit = device >= 0 && device < 64 ? 1ull << device : 0ull;
  if (bit && (configured.load(std::memory_order_acquire) & bit)) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess) configured.fetch_or(bit, std::memory_order_acq_rel);
  return e;
}

// ------------------------------------------------------------------ few rows (prefix_rows.cuh)
namespace rows {

constexpr int WARPS = 4;
constexpr int THREADS = WARPS * 32;
constexpr int BLOCK = 16 * WARPS;  // keys of a block: 16 a warp
constexpr int LEAST_BLOCKS = 4;    // of a range

// CTAs of an SM: what the shared memory holds, and enough registers for the outputs.
__host__ __device__ constexpr int ctas_of_sm(int D, int nt) { return D == 128 ? 2 : nt <= 2 ? 4 : 3; }

// Groups of 8 rows that a CTA takes.
inline int nt_of(int64_t rows) { return rows <= 8 ? 1 : rows <= 16 ? 2 : rows <= 24 ? 3 : 4; }

// Workspace of the sequences that are cut: CTA c (range, head) owns slots 2c (its first unit) and
// 2c + 1 (its last), each 8 nt x D floats and 8 nt (m, l); a counter for each CTA.
struct Cuts {
  float* o;
  float2* ml;
  int* counters;
};

// counters: cleared by the prefix stage, which is always launched before the suffix stage.
template <bool BF16>
cudaError_t launch_prefix(const Params& p, int nt, int* counters, int num_counters, cudaStream_t st);
template <bool BF16>
cudaError_t launch_suffix(const Params& p, int nt, const Cuts& cuts, int ranges, cudaStream_t st);

}  // namespace rows

// ------------------------------------------------------------------ many rows (prefix_tc.cuh)
namespace tc {

// One stage; counters as above (prefix stage).
template <bool BF16, bool PREFIX>
cudaError_t launch(EncodeTiledFn enc, const Params& p, int* counters, int num_counters, cudaStream_t st);

}  // namespace tc

}  // namespace prefix
}  // namespace attn
