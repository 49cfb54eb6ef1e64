// attn_pages.cu - the pages of a paged cache: copying, forking, freeing, reserving
// (copy on write) and compacting them.
//
// State: block_table [num_seqs, max_pages], seq_lens [num_seqs] and refs [num_pages], the
// number of entries of the table that name a page. A table entry changes hands by
// an atomic exchange wherever two rows of a call may name the same row of the
// table, so that refs counts entries whatever the caller passes.
//
// reserve and compact plan on one cluster of CTAs (reserve_kernel, compact_kernel), since what they
// hand out depends on the order of all sequences and of all pages: three prefix sums over
// the cluster in reserve, two in compact, a few thousand instructions in all, bound by the trips to L2
// between its barriers (reserve, 64 of 128 rows, 8700 pages: 19 us with cold caches, a
// beam step with it 23 us as a graph; compact, 6000 pages: 9 us). The copies that follow
// from the plan are a kernel of their own over the whole GPU, bound by the bytes of the
// moved pages, each read once and written once (1.27 GB: 194 us, 6.5 TB/s, 98% of the copy
// bandwidth).
#include <algorithm>

#include "attn.h"
#include "host_checks.h"
#include "launch.cuh"
#include "params.h"
#include "ptx.cuh"

namespace attn {
namespace pages {

constexpr int THREADS = 256;

struct Pool {
  int num_seqs, max_pages, page_size, num_pages;
  int32_t* table;
  int32_t* lens;
  int32_t* refs;
  int* status;
};

__device__ __forceinline__ bool in_pool(int page, int num_pages) { return page >= 0 && page < num_pages; }

__device__ __forceinline__ int tokens_of(const Pool& p, int s) {
  return min(max(p.lens[s], 0), p.max_pages * p.page_size);
}

// One (row of the list, run of its blocks) for a CTA: a thread takes one entry. The
// entry's old page and its new one change their counts by atomics, which commute.
template <bool FORK>
__global__ void __launch_bounds__(THREADS) rows_kernel(const __grid_constant__ Pool p, const int32_t* __restrict__ from,
                                                       const int32_t* __restrict__ rows) {
  wait_before();
  const int s = __ldg(rows + blockIdx.x);
  if (s < 0 || s >= p.num_seqs) return;
  int parent = -1, held = 0, tokens = 0;
  if constexpr (FORK) {
    parent = __ldg(from + blockIdx.x);
    if (parent < 0 || parent >= p.num_seqs || parent == s) return;
    tokens = tokens_of(p, parent);
    held = tokens > 0 ? (tokens - 1) / p.page_size + 1 : 0;  // tokens may be 2^31 - 1
  }
  if (blockIdx.y == 0 && threadIdx.x == 0) p.lens[s] = tokens;
  const int b = blockIdx.y * THREADS + threadIdx.x;
  if (b >= p.max_pages) return;
  int page = -1;
  if constexpr (FORK) {
    if (b < held) page = *static_cast<volatile int32_t*>(p.table + static_cast<int64_t>(parent) * p.max_pages + b);
    if (!in_pool(page, p.num_pages)) page = -1;
    if (page >= 0) atomicAdd(p.refs + page, 1);
  }
  const int old = atomicExch(p.table + static_cast<int64_t>(s) * p.max_pages + b, page);
  if (in_pool(old, p.num_pages)) atomicSub(p.refs + old, 1);
}

// ------------------------------------------------------------------ copies
constexpr int MAX_BUFS = 64;       // buffers of one launch
constexpr int PIECE = 16 * 1024;   // bytes that a CTA moves at a time

struct CopyParams {
  const int32_t *src, *dst;
  const int32_t* count;  // pairs, or nullptr: n
  int n, num_pages, num_bufs;
  int pieces;                // pieces of one page in all buffers
  int first_piece[MAX_BUFS]; // of each buffer
  void* buf[MAX_BUFS];
  int64_t bytes[MAX_BUFS];
  // compaction: the table's entries follow their pages
  int32_t* table;
  const int32_t* map;
  int64_t entries;
  int* status;
};

template <typename T>
__device__ __forceinline__ void move_as(uint8_t* to, const uint8_t* from, int n) {
  constexpr int BATCH = 4;
  const int units = n / static_cast<int>(sizeof(T));
  for (int i = threadIdx.x; i < units; i += THREADS * BATCH) {
    T x[BATCH];
#pragma unroll
    for (int u = 0; u < BATCH; ++u)
      if (i + u * THREADS < units) x[u] = reinterpret_cast<const T*>(from)[i + u * THREADS];
#pragma unroll
    for (int u = 0; u < BATCH; ++u)
      if (i + u * THREADS < units) reinterpret_cast<T*>(to)[i + u * THREADS] = x[u];
  }
}

__global__ void __launch_bounds__(THREADS) copy_kernel(const __grid_constant__ CopyParams p) {
  wait_before();  // the plan is complete
  const int64_t items = static_cast<int64_t>(p.count ? __ldcg(p.count) : p.n) * p.pieces;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int pair = static_cast<int>(it / p.pieces), r = static_cast<int>(it - static_cast<int64_t>(pair) * p.pieces);
    const int src = __ldcg(p.src + pair), dst = __ldcg(p.dst + pair);
    if (!in_pool(src, p.num_pages) || !in_pool(dst, p.num_pages) || src == dst) continue;
    int b = 0;
    for (int k = 1; k < p.num_bufs; ++k)
      if (r >= p.first_piece[k]) b = k;
    const int64_t bytes = p.bytes[b], at = static_cast<int64_t>(r - p.first_piece[b]) * PIECE;
    const int n = static_cast<int>(min(static_cast<int64_t>(PIECE), bytes - at));
    if (!range_in_bounds(p.status, dst * bytes + at, n, p.num_pages * bytes)) continue;
    const uint8_t* const from = static_cast<const uint8_t*>(p.buf[b]) + src * bytes + at;
    uint8_t* const to = static_cast<uint8_t*>(p.buf[b]) + dst * bytes + at;
    const uint32_t all = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p.buf[b])) | static_cast<uint32_t>(bytes);
    if (all % 16 == 0) move_as<uint4>(to, from, n);
    else if (all % 4 == 0) move_as<uint32_t>(to, from, n);
    else move_as<uint8_t>(to, from, n);
  }
  if (p.table) {
    for (int64_t e = static_cast<int64_t>(blockIdx.x) * THREADS + threadIdx.x; e < p.entries;
         e += static_cast<int64_t>(gridDim.x) * THREADS) {
      const int page = p.table[e];
      if (!in_pool(page, p.num_pages)) continue;
      const int to = __ldcg(p.map + page);
      if (to >= 0 && to != page) p.table[e] = to;
    }
  }
}

// ------------------------------------------------------------------ plans
constexpr int PLAN_THREADS = 1024;
constexpr int MAX_CLUSTER = 8;

// Places of the workspace's arrays, in ints.
struct Space {
  int64_t list, owner, left, src, dst, first, counts, total;
};

__host__ __device__ inline Space space_of(int64_t num_pages, int64_t num_seqs) {
  auto up = [](int64_t n) { return (n + 3) / 4 * 4; };
  Space w;
  w.list = 0;  // free pages, in order; compaction: destinations
  w.owner = w.list + up(num_pages);
  w.left = w.owner + up(num_pages);
  w.src = w.left + up(num_pages);  // compaction has more pairs than sequences: its sources are at `owner`
  w.dst = w.src + up(num_seqs);
  w.first = w.dst + up(num_seqs);  // first candidate of each sequence
  w.counts = w.first + up(num_seqs);
  w.total = w.counts + 8;
  return w;
}

// Run `me` of n things dealt to `threads` in equal runs: [lo, hi).
__device__ __forceinline__ void run_of(int n, int me, int threads, int& lo, int& hi) {
  const int64_t per = (static_cast<int64_t>(n) + threads - 1) / threads;
  lo = static_cast<int>(min(me * per, static_cast<int64_t>(n)));
  hi = static_cast<int>(min(lo + per, static_cast<int64_t>(n)));
}

__device__ __forceinline__ void cluster_sync() {
  cluster_arrive();
  cluster_wait();
}

__device__ __forceinline__ int ld_cluster(uint32_t addr) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// The sum of v over the threads of the cluster before this one, and over all of
// them. Every thread calls it; global writes before it are seen after it.
__device__ __forceinline__ int cluster_scan(int v, int ctas, int rank, int& total) {
  __shared__ int warp_sum[PLAN_THREADS / 32];
  __shared__ int cta_sum;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    int x = warp_sum[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    warp_sum[lane] = x;
    if (lane == 31) cta_sum = x;
  }
  cluster_sync();
  int before = incl - v + (warp > 0 ? warp_sum[warp - 1] : 0);
  total = 0;
  for (int r = 0; r < ctas; ++r) {
    const int x = ld_cluster(peer_addr(smem_u32(&cta_sum), r));
    if (r < rank) before += x;
    total += x;
  }
  cluster_sync();  // the sums are read before the next scan writes them
  return before;
}

// Blocks that sequence s is about to write: [b0, b1).
__device__ __forceinline__ void written(const Pool& p, const int32_t* new_tokens, int s, int& tokens, int& b0, int& b1) {
  tokens = tokens_of(p, s);
  const int room = p.max_pages * p.page_size - tokens;
  const int n = min(max(__ldg(new_tokens + s), 0), room);
  b0 = tokens / p.page_size;
  b1 = n > 0 ? (tokens + n - 1) / p.page_size + 1 : b0;
}

// The candidates (blocks about to be written, in the order of sequence and block) are dealt
// to the threads in runs; so are the pages. Of a page with R references that k
// candidates are about to write, the sequential rule lets each of them take a new
// page while other references remain: all k if k < R, all but the last if k = R. So
// `left` = R - k and `owner`, the last candidate, decide each one by itself.
__global__ void __launch_bounds__(PLAN_THREADS) reserve_kernel(const __grid_constant__ Pool p,
                                                               const int32_t* __restrict__ new_tokens, int32_t* ws,
                                                               int32_t* result, int ctas) {
  wait_before();
  let_next();  // the copies may come up; they wait
  const Space w = space_of(p.num_pages, p.num_seqs);
  int32_t *const list = ws + w.list, *const owner = ws + w.owner, *const left = ws + w.left, *const first = ws + w.first;
  const int rank = static_cast<int>(cluster_rank());
  const int threads = ctas * PLAN_THREADS, me = rank * PLAN_THREADS + threadIdx.x;
  if (me == 0) ws[w.counts] = 0;

  // first candidate of each sequence
  int s0, s1;
  run_of(p.num_seqs, me, threads, s0, s1);
  int mine = 0, cands, tokens, b0, b1;
  for (int s = s0; s < s1; ++s) {
    written(p, new_tokens, s, tokens, b0, b1);
    mine += b1 - b0;
  }
  int at = cluster_scan(mine, ctas, rank, cands);
  for (int s = s0; s < s1; ++s) {
    first[s] = at;
    written(p, new_tokens, s, tokens, b0, b1);
    at += b1 - b0;
  }
  if (cands == 0) {
    if (me == 0) result[0] = result[1] = 0;
    return;
  }
  cluster_sync();

  // This thread's run of candidates, and the sequence that it begins in: the last one whose first is
  // at most c0. Each CTA looks in a copy of its own, a search in L2 would take a trip for each step.
  constexpr int KEPT = 4096;
  __shared__ int kept[KEPT];
  const bool keep = p.num_seqs <= KEPT;
  if (keep)
    for (int s = threadIdx.x; s < p.num_seqs; s += PLAN_THREADS) kept[s] = __ldcg(first + s);
  __syncthreads();
  auto first_of = [&](int s) { return keep ? kept[s] : __ldcg(first + s); };
  int c0, c1;
  run_of(cands, me, threads, c0, c1);
  int begin = 0;
  if (c0 < c1) {
    int hi = p.num_seqs;
    while (hi - begin > 1) {
      const int mid = (begin + hi) >> 1;
      if (first_of(mid) <= c0) begin = mid;
      else hi = mid;
    }
  }
  // f(candidate, block, tokens of its sequence, table entry, page): a run of one candidate is read once
  int32_t* one = nullptr;
  int one_block = 0, one_tokens = 0, one_page = 0;
  if (c0 + 1 == c1) {
    written(p, new_tokens, begin, one_tokens, b0, b1);
    one_block = b0 + (c0 - first_of(begin));
    one = p.table + static_cast<int64_t>(begin) * p.max_pages + one_block;
    one_page = *one;
  }
  auto each = [&](auto&& f) {
    if (one) {
      f(c0, one_block, one_tokens, one, one_page);
      return;
    }
    int s = begin;
    for (int c = c0; c < c1; ++s) {
      written(p, new_tokens, s, tokens, b0, b1);
      for (int b = b0 + (c - first_of(s)); b < b1 && c < c1; ++b, ++c) {
        int32_t* const e = p.table + static_cast<int64_t>(s) * p.max_pages + b;
        f(c, b, tokens, e, *e);
      }
    }
  };
  each([&](int, int, int, int32_t*, int page) {
    if (!in_pool(page, p.num_pages)) return;
    owner[page] = -1;
    left[page] = max(p.refs[page], 1);
  });
  cluster_sync();
  each([&](int c, int, int, int32_t*, int page) {
    if (!in_pool(page, p.num_pages)) return;
    atomicMax(owner + page, c);
    atomicSub(left + page, 1);
  });
  cluster_sync();
  auto keeps = [&](int c, int page) { return in_pool(page, p.num_pages) && __ldcg(left + page) == 0 && __ldcg(owner + page) == c; };
  int wants = 0, need;
  each([&](int c, int, int, int32_t*, int page) { wants += keeps(c, page) ? 0 : 1; });
  int next = cluster_scan(wants, ctas, rank, need);
  if (need == 0) {
    if (me == 0) result[0] = result[1] = 0;
    return;
  }

  // the lowest free pages
  int p0, p1;
  run_of(p.num_pages, me, threads, p0, p1);
  int spare = 0, free_pages;
  for (int i = p0; i < p1; ++i) spare += p.refs[i] <= 0;
  int place = cluster_scan(spare, ctas, rank, free_pages);
  if (me == 0) {
    result[0] = need <= free_pages ? need : 0;
    result[1] = max(need - free_pages, 0);
  }
  if (need > free_pages) return;
  if (spare > 0)
    for (int i = p0; i < p1 && place < need; ++i)
      if (p.refs[i] <= 0) list[place++] = i;
  cluster_sync();

  each([&](int c, int b, int held, int32_t* e, int page) {
    if (keeps(c, page)) return;
    const int fresh = __ldcg(list + next++);
    *e = fresh;
    p.refs[fresh] = 1;
    if (!in_pool(page, p.num_pages)) return;
    atomicSub(p.refs + page, 1);
    if (static_cast<int64_t>(b) * p.page_size < held) {  // one block of a sequence at most
      const int i = atomicAdd(ws + w.counts, 1);
      if (!in_bounds(p.status, i, p.num_seqs)) return;
      ws[w.src + i] = page;
      ws[w.dst + i] = fresh;
    }
  });
}

// Pages in runs, one for each thread. With U pages in use, a free page below U is hole
// number (pages below it) - (pages in use below it), and a page in use from U on is
// mover number (pages in use below it) - (pages in use below U).
__global__ void __launch_bounds__(PLAN_THREADS) compact_kernel(const __grid_constant__ Pool p, int32_t* __restrict__ map,
                                                               int32_t* used_out, int32_t* ws, int ctas) {
  wait_before();
  let_next();
  const Space w = space_of(p.num_pages, p.num_seqs);
  int32_t *const holes = ws + w.list, *const movers = ws + w.owner;
  const int rank = static_cast<int>(cluster_rank());
  const int threads = ctas * PLAN_THREADS, me = rank * PLAN_THREADS + threadIdx.x;
  int p0, p1;
  run_of(p.num_pages, me, threads, p0, p1);
  int mine = 0, used, low = 0, below;
  for (int i = p0; i < p1; ++i) mine += p.refs[i] > 0;
  const int before = cluster_scan(mine, ctas, rank, used);
  for (int i = p0; i < min(p1, used); ++i) low += p.refs[i] > 0;
  cluster_scan(low, ctas, rank, below);  // below: pages in use below U
  int k = before;
  for (int i = p0; i < p1; ++i) {
    const bool in_use = p.refs[i] > 0;
    if (in_use) {
      if (i < used) map[i] = i;
      else movers[k - below] = i;
      ++k;
    } else {
      map[i] = -1;
      if (i < used) holes[i - k] = i;
    }
  }
  cluster_sync();
  k = p0 < used ? below : before;
  for (int i = max(p0, used); i < p1; ++i) {  // what lies below U is written here and not read
    if (p.refs[i] <= 0) continue;
    const int to = __ldcg(holes + k++ - below);
    map[i] = to;
    p.refs[to] = p.refs[i];
    p.refs[i] = 0;
  }
  if (me == 0) {
    *used_out = used;
    ws[w.counts] = used - below;
  }
}

// A cluster of one CTA up to 1024 pages or sequences, of eight from 4097 on: a thread
// looks at one of each up to 8192.
inline int plan_ctas(int64_t work) {
  int c = 1;
  while (c < MAX_CLUSTER && static_cast<int64_t>(c) * PLAN_THREADS < work) c *= 2;
  return c;
}

// Launches the copies of p.src -> p.dst in all buffers, 64 of them at a time. `most`:
// an upper bound on the pairs.
inline cudaError_t launch_copies(CopyParams p, void* const* bufs, const int64_t* page_bytes, int num_bufs, int64_t most,
                                 cudaStream_t st) {
  int32_t* const table = p.table;
  for (int b0 = 0; b0 < num_bufs || (b0 == 0 && table); b0 += MAX_BUFS) {
    p.num_bufs = std::min(MAX_BUFS, num_bufs - b0);
    int64_t pieces = 0;
    for (int b = 0; b < p.num_bufs; ++b) {
      p.buf[b] = bufs[b0 + b];
      p.bytes[b] = page_bytes[b0 + b];
      p.first_piece[b] = static_cast<int>(pieces);
      pieces += (p.bytes[b] + PIECE - 1) / PIECE;
    }
    p.pieces = static_cast<int>(pieces);
    p.table = b0 == 0 ? table : nullptr;
    const int64_t items = std::max(most * pieces, p.table ? (p.entries + THREADS - 1) / THREADS : 1);
    const cudaError_t e = launch_early(copy_kernel, dim3(static_cast<unsigned>(std::min<int64_t>(items, SMS * 8))), THREADS, 0, st, 0, p);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace pages
}  // namespace attn

namespace {

using attn::aligned;
using attn::Buf;
using attn::meet;
using attn::pages::CopyParams;
using attn::pages::Pool;
using attn::pages::Space;

int check_pool(const attn_pages_t& s) {
  if (s.num_seqs < 0 || s.max_pages < 0 || s.page_size <= 0 || s.num_pages < 0) return ATTN_ERR_SHAPE;
  if (static_cast<int64_t>(s.max_pages) * s.page_size > 0x7fffffffLL ||
      static_cast<int64_t>(s.num_seqs) * s.max_pages > 0x7fffffffLL ||
      s.max_pages > 65535 * attn::pages::THREADS)
    return ATTN_ERR_SHAPE;
  return ATTN_OK;
}

// Buffers: pointers, sizes inside 64 bits, none sharing a byte with another or with `others`.
int check_buffers(void* const* bufs, const int64_t* page_bytes, int num_bufs, int num_pages, const Buf* others, int n) {
  if (num_bufs < 0 || num_bufs > ATTN_PAGES_MAX_BUFFERS) return ATTN_ERR_SHAPE;
  if (num_bufs > 0 && (!bufs || !page_bytes)) return ATTN_ERR_NULL;
  int64_t pieces = 0;
  for (int i = 0; i < num_bufs; ++i) {
    if (page_bytes[i] <= 0 || page_bytes[i] > (1ll << 40) || static_cast<double>(page_bytes[i]) * num_pages > 1e17)
      return ATTN_ERR_SHAPE;
    if (!bufs[i] && num_pages > 0) return ATTN_ERR_NULL;
    pieces += (page_bytes[i] + attn::pages::PIECE - 1) / attn::pages::PIECE;
  }
  if (pieces > 0x7fffffffLL) return ATTN_ERR_SHAPE;
  auto span = [&](int i) { return Buf{bufs[i], page_bytes[i] * num_pages}; };
  bool rising = true;  // as one allocation's slices are: then neighbours are enough
  for (int i = 1; i < num_bufs && rising; ++i)
    rising = reinterpret_cast<uintptr_t>(bufs[i - 1]) + static_cast<uintptr_t>(page_bytes[i - 1] * num_pages) <=
             reinterpret_cast<uintptr_t>(bufs[i]);
  for (int i = 0; i < num_bufs; ++i) {
    if (!rising)
      for (int j = 0; j < i; ++j)
        if (meet(span(i), span(j))) return ATTN_ERR_OVERLAP;
    for (int j = 0; j < n; ++j)
      if (meet(span(i), others[j])) return ATTN_ERR_OVERLAP;
  }
  return ATTN_OK;
}

// The first `written` of n arrays share no byte with another one.
bool apart(const Buf* b, int written, int n) {
  for (int i = 0; i < written; ++i)
    for (int j = 0; j < n; ++j)
      if (j != i && meet(b[i], b[j])) return false;
  return true;
}

bool ints_aligned(const Buf* b, int n) {
  for (int i = 0; i < n; ++i)
    if (!aligned(b[i].p, 4)) return false;
  return true;
}

int pool_of(const attn_pages_t& s, int32_t* table, const int32_t* lens, int32_t* refs, Pool& p) {
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return attn::record_cuda_error(e);
  p = Pool{s.num_seqs, s.max_pages, s.page_size, s.num_pages, table, const_cast<int32_t*>(lens), refs,
           attn::status_word(dev)};
  return ATTN_OK;
}

int done(cudaError_t e) { return e == cudaSuccess ? ATTN_OK : attn::record_cuda_error(e); }

int64_t table_bytes(const attn_pages_t& s) { return static_cast<int64_t>(s.num_seqs) * s.max_pages * 4; }

}  // namespace

extern "C" int attn_pages_copy(int num_pages, void* const* bufs, const int64_t* page_bytes, int num_bufs,
                               const int32_t* src, const int32_t* dst, int n, void* stream) {
  if (num_pages < 0 || n < 0) return ATTN_ERR_SHAPE;
  const Buf lists[] = {{src, n * 4ll}, {dst, n * 4ll}};
  if (!ints_aligned(lists, 2)) return ATTN_ERR_ALIGN;
  if (const int rc = check_buffers(bufs, page_bytes, num_bufs, num_pages, lists, 2)) return rc;
  if (n == 0 || num_pages == 0 || num_bufs == 0) return ATTN_OK;
  if (!src || !dst) return ATTN_ERR_NULL;
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return attn::record_cuda_error(e);
  CopyParams p{};
  p.src = src;
  p.dst = dst;
  p.n = n;
  p.num_pages = num_pages;
  p.status = attn::status_word(dev);
  return done(attn::pages::launch_copies(p, bufs, page_bytes, num_bufs, n, static_cast<cudaStream_t>(stream)));
}

extern "C" int attn_pages_fork(const attn_pages_t* pool, int32_t* block_table, int32_t* seq_lens, int32_t* refs,
                               const int32_t* parents, const int32_t* children, int n, void* stream) {
  if (!pool) return ATTN_ERR_NULL;
  const attn_pages_t s = *pool;
  if (const int rc = check_pool(s)) return rc;
  if (n < 0) return ATTN_ERR_SHAPE;
  const Buf b[] = {{block_table, table_bytes(s)}, {seq_lens, s.num_seqs * 4ll}, {refs, s.num_pages * 4ll},
                   {parents, n * 4ll}, {children, n * 4ll}};
  if (!ints_aligned(b, 5)) return ATTN_ERR_ALIGN;
  if (n == 0 || s.num_seqs == 0) return ATTN_OK;
  if (!seq_lens || !parents || !children || (s.max_pages > 0 && !block_table) || (s.num_pages > 0 && !refs))
    return ATTN_ERR_NULL;
  if (!apart(b, 3, 5)) return ATTN_ERR_OVERLAP;
  Pool p;
  if (const int rc = pool_of(s, block_table, seq_lens, refs, p)) return rc;
  const dim3 grid(static_cast<unsigned>(n), static_cast<unsigned>(std::max(1, (s.max_pages + 255) / 256)));
  return done(attn::launch_early(attn::pages::rows_kernel<true>, grid, attn::pages::THREADS, 0, static_cast<cudaStream_t>(stream), 0, p,
                                 parents, children));
}

extern "C" int attn_pages_free(const attn_pages_t* pool, int32_t* block_table, int32_t* seq_lens, int32_t* refs,
                               const int32_t* seqs, int n, void* stream) {
  if (!pool) return ATTN_ERR_NULL;
  const attn_pages_t s = *pool;
  if (const int rc = check_pool(s)) return rc;
  if (n < 0) return ATTN_ERR_SHAPE;
  const Buf b[] = {{block_table, table_bytes(s)}, {seq_lens, s.num_seqs * 4ll}, {refs, s.num_pages * 4ll}, {seqs, n * 4ll}};
  if (!ints_aligned(b, 4)) return ATTN_ERR_ALIGN;
  if (n == 0 || s.num_seqs == 0) return ATTN_OK;
  if (!seq_lens || !seqs || (s.max_pages > 0 && !block_table) || (s.num_pages > 0 && !refs)) return ATTN_ERR_NULL;
  if (!apart(b, 3, 4)) return ATTN_ERR_OVERLAP;
  Pool p;
  if (const int rc = pool_of(s, block_table, seq_lens, refs, p)) return rc;
  const dim3 grid(static_cast<unsigned>(n), static_cast<unsigned>(std::max(1, (s.max_pages + 255) / 256)));
  return done(attn::launch_early(attn::pages::rows_kernel<false>, grid, attn::pages::THREADS, 0, static_cast<cudaStream_t>(stream), 0, p,
                                 static_cast<const int32_t*>(nullptr), seqs));
}

extern "C" int attn_pages_workspace_bytes(const attn_pages_t* pool, size_t* bytes) {
  if (!pool || !bytes) return ATTN_ERR_NULL;
  if (const int rc = check_pool(*pool)) return rc;
  *bytes = static_cast<size_t>(attn::pages::space_of(pool->num_pages, pool->num_seqs).total) * 4;
  return ATTN_OK;
}

extern "C" int attn_pages_reserve(const attn_pages_t* pool, int32_t* block_table, const int32_t* seq_lens, int32_t* refs,
                                  const int32_t* new_tokens, void* const* bufs, const int64_t* page_bytes, int num_bufs,
                                  int32_t* result, void* workspace, size_t workspace_bytes, void* stream) {
  size_t need = 0;
  if (const int rc = attn_pages_workspace_bytes(pool, &need)) return rc;
  const attn_pages_t s = *pool;
  if (!result) return ATTN_ERR_NULL;
  if (s.num_seqs > 0 && (!seq_lens || !new_tokens || (s.max_pages > 0 && !block_table))) return ATTN_ERR_NULL;
  if (s.num_pages > 0 && !refs) return ATTN_ERR_NULL;
  const Buf b[] = {{block_table, table_bytes(s)}, {refs, s.num_pages * 4ll}, {result, 8}, {workspace, static_cast<int64_t>(need)},
                   {seq_lens, s.num_seqs * 4ll}, {new_tokens, s.num_seqs * 4ll}};
  if (!workspace || workspace_bytes < need) return ATTN_ERR_WORKSPACE;
  if (!ints_aligned(b, 6) || !aligned(workspace, 16)) return ATTN_ERR_ALIGN;
  if (!apart(b, 4, 6)) return ATTN_ERR_OVERLAP;
  if (const int rc = check_buffers(bufs, page_bytes, num_bufs, s.num_pages, b, 6)) return rc;
  Pool p;
  if (const int rc = pool_of(s, block_table, seq_lens, refs, p)) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int32_t* const ws = static_cast<int32_t*>(workspace);
  const int ctas = attn::pages::plan_ctas(std::max(s.num_pages, s.num_seqs));
  cudaError_t e = attn::launch_early(attn::pages::reserve_kernel, dim3(ctas), attn::pages::PLAN_THREADS, 0, st, ctas, p, new_tokens, ws, result, ctas);
  if (e != cudaSuccess || num_bufs == 0 || s.num_pages == 0) return done(e);
  const Space w = attn::pages::space_of(s.num_pages, s.num_seqs);
  CopyParams c{};
  c.src = ws + w.src;
  c.dst = ws + w.dst;
  c.count = ws + w.counts;
  c.num_pages = s.num_pages;
  c.status = p.status;
  return done(attn::pages::launch_copies(c, bufs, page_bytes, num_bufs, s.num_seqs, st));
}

extern "C" int attn_pages_compact(const attn_pages_t* pool, int32_t* block_table, int32_t* refs, void* const* bufs,
                                  const int64_t* page_bytes, int num_bufs, int32_t* page_map, int32_t* used,
                                  void* workspace, size_t workspace_bytes, void* stream) {
  size_t need = 0;
  if (const int rc = attn_pages_workspace_bytes(pool, &need)) return rc;
  const attn_pages_t s = *pool;
  if (!used || (s.num_pages > 0 && (!refs || !page_map)) || (s.num_seqs > 0 && s.max_pages > 0 && !block_table))
    return ATTN_ERR_NULL;
  const Buf b[] = {{block_table, table_bytes(s)}, {refs, s.num_pages * 4ll}, {page_map, s.num_pages * 4ll}, {used, 4},
                   {workspace, static_cast<int64_t>(need)}};
  if (!workspace || workspace_bytes < need) return ATTN_ERR_WORKSPACE;
  if (!ints_aligned(b, 5) || !aligned(workspace, 16)) return ATTN_ERR_ALIGN;
  if (!apart(b, 5, 5)) return ATTN_ERR_OVERLAP;
  if (const int rc = check_buffers(bufs, page_bytes, num_bufs, s.num_pages, b, 5)) return rc;
  Pool p;
  if (const int rc = pool_of(s, block_table, nullptr, refs, p)) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int32_t* const ws = static_cast<int32_t*>(workspace);
  const int ctas = attn::pages::plan_ctas(s.num_pages);
  const cudaError_t e = attn::launch_early(attn::pages::compact_kernel, dim3(ctas), attn::pages::PLAN_THREADS, 0, st, ctas, p, page_map, used, ws, ctas);
  if (e != cudaSuccess || s.num_pages == 0) return done(e);
  const Space w = attn::pages::space_of(s.num_pages, s.num_seqs);
  CopyParams c{};
  c.src = ws + w.owner;
  c.dst = ws + w.list;
  c.count = ws + w.counts;
  c.num_pages = s.num_pages;
  c.status = p.status;
  c.table = block_table;
  c.map = page_map;
  c.entries = static_cast<int64_t>(s.num_seqs) * s.max_pages;
  if (c.entries == 0) c.table = nullptr;
  return done(attn::pages::launch_copies(c, bufs, page_bytes, num_bufs, s.num_pages / 2, st));
}
