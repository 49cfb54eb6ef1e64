// prefix.cuh - attention over a paged cache for groups of sequences that share a
// prefix (attn_paged_prefix_fwd): parameters, workspace and what the kernels read of
// the metadata.
//
// A row (query, head) sees the keys j < lim of its sequence. Group g's first `pre`
// keys are the same for all its members, so a call has two stages:
//   prefix: a unit is a group, its rows all the queries of its members (packed, so they
//           lie side by side), its keys [0, pre). A row leaves parts (m, l, O) in the
//           workspace, one for each run of keys that its unit was cut into:
//           O = sum_j 2^(x_j - m) v_j, l = sum_j 2^(x_j - m), x in log2 units.
//           The 16-bit kernels share out the work in equal ranges: the blocks (a run of
//           keys for a block of rows and a head) of all groups, in one order, are cut into
//           as many ranges as there are CTAs, so a row's parts are the ranges that its
//           unit's blocks lie in (Head, Rec, parts_of).
//   suffix: a unit is a sequence, its keys [pre, L) (all of them outside a group). For many
//           rows it joins its own part with those of the prefix and writes out and lse;
//           for few rows it leaves parts too, and does not need the prefix's: the stages then run side
//           by side, the prefix on as many SMs as let it end with the suffix (share_out),
//           and a last kernel joins the parts of each row in their order.
#pragma once

#include <atomic>

#include "host_checks.h"
#include "launch.cuh"
#include "params.h"
#include "ptx.cuh"

namespace attn {
namespace prefix {

constexpr float LN2 = 0.6931471805599453f;
constexpr int MAX_PARTS = 32, MIN_PARTS = 2;  // room for the parts of a row

// How the prefix stage was shared out, in the workspace: block total and ranges of the call; of each
// group its first block, the blocks of one (row block, head), the row blocks, whether the last
// one has at most half the rows (its blocks then hold twice the keys, and a range leaves two
// parts), and the first query.
struct Head {
  int64_t total;
  int32_t ranges, row_block;
};
struct Rec {
  int64_t first;
  int32_t nb, rbs, half, q_lo;
};

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
  int most_parts;   // slots of a row; from 4 on, a last row block of half the rows or fewer splits its keys
  Head* head;
  Rec* rec;         // [num_groups]
  float2* ml;       // [most_parts, num_queries * Hq]
  float* o;         // [most_parts, num_queries * Hq, D]
  // of the few-row suffix stage: blocks and ranges as above; each sequence's first block; the
  // parts of units that lie in one range; those of units that are cut: CTA c (range, head) owns
  // slots 2c (its first unit) and 2c + 1 (its last), suffix_rows rows each
  int suffix_rows, suffix_ranges;
  Head* suffix_head;
  int64_t* suffix_first;  // [num_seqs]
  float2 *own_ml, *cut_ml;
  float *own_o, *cut_o;
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

__device__ __forceinline__ int64_t cut(int64_t total, int r, int ranges) { return total * r / ranges; }  // first block of range r

// The range that block x lies in (ranges <= total).
__device__ __forceinline__ int range_of(int64_t x, int64_t total, int ranges) {
  return static_cast<int>(((x + 1) * ranges + total - 1) / total) - 1;
}

// Queries of the sequences [a, b), from q_lo on, at most `most`.
__device__ __forceinline__ int queries_of(const Params& p, int a, int b, int most, int& q_lo) {
  q_lo = query_at(p, a);
  return a < b ? min(max(query_at(p, b) - q_lo, 0), most) : 0;
}

// Keys of sequence s that are its own: [start, L); `pre`: tokens its group shares.
struct Own {
  int group, pre, start, L;
};

__device__ __forceinline__ Own own_of(const Params& p, int s, int L) {
  Own o;
  o.L = L;
  if (p.num_groups == 1) {  // the common case, without a search
    int a, b;
    group_range(p, 0, a, b);
    const int pre = prefix_len(p, 0);
    o.group = s >= a && s < b ? 0 : -1;
    o.pre = o.group == 0 ? pre : 0;
  } else {
    o.group = group_of(p, s);
    o.pre = o.group >= 0 ? prefix_len(p, o.group) : 0;
  }
  o.start = min(o.pre, o.L);
  return o;
}

__device__ __forceinline__ Own own_of(const Params& p, int s) { return own_of(p, s, seq_len(p, s)); }

// What a group brings to the prefix stage: `first` is filled in by the caller.
__device__ __forceinline__ Rec rec_of(const Params& p, int g, int key_block, int row_block, bool halves) {
  int a, b;
  group_range(p, g, a, b);
  Rec r;
  r.first = 0;
  const int64_t rows = static_cast<int64_t>(queries_of(p, a, b, p.max_group_queries, r.q_lo)) * (p.Hq / p.Hkv);
  r.nb = (prefix_len(p, g) + key_block - 1) / key_block;
  r.rbs = r.nb > 0 ? static_cast<int>((rows + row_block - 1) / row_block) : 0;
  r.half = halves && r.rbs > 0 && rows - static_cast<int64_t>(r.rbs - 1) * row_block <= row_block / 2;
  return r;
}

__device__ __forceinline__ int64_t full_blocks(const Params& p, const Rec& r) { return static_cast<int64_t>(r.rbs - r.half) * p.Hkv * r.nb; }

__device__ __forceinline__ int64_t blocks_of(const Params& p, const Rec& r) {
  return full_blocks(p, r) + (r.half ? static_cast<int64_t>(p.Hkv) * ((r.nb + 1) / 2) : 0);
}

// Shares out the prefix stage: the ranges, this CTA's blocks [u0, u1), and the group that u0 lies in with its
// first block. Every thread of the CTA calls it; CTA 0 leaves Head and Rec in the workspace.
struct Share {
  int64_t total, u0, u1, first;
  int ranges, g;
};

// Microseconds, measured where the two stages run side by side: a block of 256 rows and 128 keys of 128
// elements on an SM, and what a piece costs besides; KB of keys and values that the few-row suffix stage streams in one of them, on one SM
// and on all.
constexpr float BLOCK_US = 2.4f, PIECE_US = 10.f, SM_KB_US = 40.f, ALL_KB_US = 5500.f;

template <int THREADS, bool BESIDE>
__device__ __forceinline__ Share share_out(const Params& p, int ctas, int key_block, int row_block, bool halves) {
  __shared__ int64_t warp_sum[THREADS / 32];
  __shared__ int most_full, most_half, found_g;
  __shared__ int64_t found_first;
  __shared__ unsigned long long own_keys;  // of all sequences
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (p.num_groups + THREADS - 1) / THREADS;
  const int g0 = min(tid * per, p.num_groups), g1 = min(g0 + per, p.num_groups);
  if (tid == 0) most_full = most_half = found_g = 0, found_first = 0, own_keys = 0;
  __syncthreads();
  int64_t mine = 0, keys = 0;
  int full = 0, half = 0;
  if constexpr (BESIDE) {
    for (int s = tid; s < p.num_seqs; s += THREADS) keys += seq_len(p, s);
  }
  Rec r0{};
  for (int g = g0; g < g1; ++g) {
    const Rec r = rec_of(p, g, key_block, row_block, halves);
    if (g == g0) r0 = r;
    mine += blocks_of(p, r);
    if (r.rbs > r.half) full = max(full, r.nb);
    if (r.half) half = max(half, (r.nb + 1) / 2);
    if constexpr (BESIDE) {
      int a, b;
      group_range(p, g, a, b);
      keys -= static_cast<int64_t>(b - a) * prefix_len(p, g);
    }
  }
  if constexpr (BESIDE) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) keys += __shfl_xor_sync(0xffffffffu, keys, o);
    if (lane == 0) atomicAdd(&own_keys, static_cast<unsigned long long>(keys));
  }
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  if (lane == 31) warp_sum[warp] = incl;
  full = __reduce_max_sync(0xffffffffu, full);
  half = __reduce_max_sync(0xffffffffu, half);
  if (lane == 0 && full) atomicMax(&most_full, full);
  if (lane == 0 && half) atomicMax(&most_half, half);
  __syncthreads();
  Share s;
  int64_t before = incl - mine;
  s.total = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < warp) before += warp_sum[w];
    s.total += warp_sum[w];
  }
  // as many ranges as CTAs, if they leave a row no more parts than its room: n blocks lie in
  // at most n ranges / total + 1 ranges
  int64_t ranges = min(static_cast<int64_t>(ctas), s.total);
  if constexpr (BESIDE) {
    // Of 8, 16 .. SMs for this stage the number with which both are done first: the other one
    // streams on the rest meanwhile, then on all.
    const float us = static_cast<float>(s.total) * BLOCK_US * (p.D == 128 ? 1.f : 0.7f);
    const float kb = fmaxf(static_cast<float>(static_cast<long long>(own_keys)), 0.f) * p.Hkv * p.D * (4.f / 1024.f);
    const int n = min(8 * (lane + 1), ctas);
    const float own = PIECE_US + us / n;
    const float rest = fmaxf(kb - own * fminf(SM_KB_US * (SMS - n), ALL_KB_US), 0.f);
    const uint32_t t = static_cast<uint32_t>(fminf((own + rest / ALL_KB_US) * 16.f, 1e8f)), best = __reduce_min_sync(0xffffffffu, t);
    ranges = min(ranges, static_cast<int64_t>(min(8 * (32 - __clz(__ballot_sync(0xffffffffu, t == best))), ctas)));
  }
  if (most_full) ranges = min(ranges, s.total * (p.most_parts - 1) / most_full);
  if (most_half) ranges = min(ranges, s.total * (p.most_parts / 2 - 1) / most_half);
  s.ranges = static_cast<int>(max(ranges, static_cast<int64_t>(1)));
  const bool mine_too = static_cast<int>(blockIdx.x) < s.ranges;
  s.u0 = mine_too ? cut(s.total, blockIdx.x, s.ranges) : s.total;
  s.u1 = mine_too ? cut(s.total, blockIdx.x + 1, s.ranges) : s.total;
  if (blockIdx.x == 0 || (s.u0 >= before && s.u0 < before + mine)) {
    int64_t at = before;
    for (int g = g0; g < g1; ++g) {
      Rec r = g == g0 ? r0 : rec_of(p, g, key_block, row_block, halves);
      const int64_t n = blocks_of(p, r);
      if (s.u0 >= at && s.u0 < at + n) {
        found_g = g;
        found_first = at;
      }
      r.first = at;
      if (blockIdx.x == 0) p.rec[g] = r;
      at += n;
    }
  }
  if (blockIdx.x == 0 && tid == 0) *p.head = Head{s.total, s.ranges, row_block};
  __syncthreads();
  s.g = found_g;
  s.first = found_first;
  return s;
}

// Parts of the prefix that row (query, head h * heads + hr) of group g has.
__device__ __forceinline__ int parts_of(const Params& p, int g, int query, int hr, int h) {
  const int64_t total = __ldcg(reinterpret_cast<const long long*>(&p.head->total));
  const int ranges = __ldcg(&p.head->ranges), row_block = __ldcg(&p.head->row_block);
  const Rec* const at = p.rec + g;
  const int64_t first = __ldcg(reinterpret_cast<const long long*>(&at->first));
  const int nb = __ldcg(&at->nb), rbs = __ldcg(&at->rbs), half = __ldcg(&at->half), q_lo = __ldcg(&at->q_lo);
  const int64_t row = static_cast<int64_t>(query - q_lo) * (p.Hq / p.Hkv) + hr;
  const int rb = static_cast<int>(row / row_block);
  if (row < 0 || rb >= rbs || total <= 0) return 0;
  const bool two = half && rb == rbs - 1;
  const int n = two ? (nb + 1) / 2 : nb;
  const int64_t start = first + static_cast<int64_t>(rb) * p.Hkv * nb + static_cast<int64_t>(h) * n;
  const int pieces = range_of(start + n - 1, total, ranges) - range_of(start, total, ranges) + 1;
  return min(two ? 2 * pieces : pieces, p.most_parts);
}

// 8 floats of the workspace: 32 bytes, one sector.
__device__ __forceinline__ void load8cg(float (&r)[8], const float* at) {
  asm volatile("ld.global.cg.v8.f32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7])
               : "l"(at)
               : "memory");
}
__device__ __forceinline__ void store8(float* at, const float (&r)[8]) {
  asm volatile("st.global.v8.f32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::"f"(r[0]), "f"(r[1]), "f"(r[2]), "f"(r[3]), "f"(r[4]),
               "f"(r[5]), "f"(r[6]), "f"(r[7]), "l"(at)
               : "memory");
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

constexpr int WARPS = 2;
constexpr int THREADS = WARPS * 32;
constexpr int BLOCK = 16 * WARPS;  // keys of a block: 16 a warp

constexpr int LEAST_BLOCKS = 4;    // of a range of the suffix stage, where units are cut

// CTAs of an SM: what the shared memory holds, and enough registers for the outputs.
__host__ __device__ constexpr int ctas_of_sm(int D, int nt) { return D == 128 ? (nt <= 2 ? 6 : 4) : nt <= 2 ? 8 : 6; }

// Groups of 8 rows that a CTA takes.
inline int nt_of(int64_t rows) { return rows <= 8 ? 1 : rows <= 16 ? 2 : rows <= 24 ? 3 : 4; }

template <bool BF16>
cudaError_t launch_prefix(const Params& p, int nt, cudaStream_t st);
template <bool BF16>
cudaError_t launch_suffix(const Params& p, int nt, bool after_prefix, cudaStream_t st);
template <bool BF16>
cudaError_t launch_join(const Params& p, cudaStream_t st);

}  // namespace rows

// ------------------------------------------------------------------ many rows (prefix_tc.cuh)
namespace tc {

// One stage; after_prefix: the launch before it is the prefix stage.
template <bool BF16, bool PREFIX>
cudaError_t launch(EncodeTiledFn enc, const Params& p, bool after_prefix, cudaStream_t st);

}  // namespace tc

}  // namespace prefix
}  // namespace attn
