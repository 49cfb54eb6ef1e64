// prefix_tc.cuh - both stages of attn_paged_prefix_fwd (prefix.cuh) for many rows, on the tcgen05
// tensor cores (F16/BF16, D in {64, 128}, page_size a multiple of 8 that divides 128 or a
// multiple of 128): the prefix of a group with more than 32 rows (queries x heads of a kv
// head), and the own keys of sequences with many new tokens.
//
// The pipeline is the dense forward's (attn_tc.cuh: two tiles of 128 rows, S and P in tensor
// memory, MMA order S_0 PV_1 S_1 PV_0, lazy rescale), with
//  - rows packed as row = query * heads + head, whatever the number of heads: each softmax
//    thread copies its own row of q into the swizzled tile (a TMA box would want heads
//    to divide 128);
//  - 128-key tiles gathered page by page, one TMA box each, from a 4-D view
//    [pages, page_size, Hkv, D] of the cache;
//  - values past the last key and before the first set to zero in shared memory before their
//    product: a page's unwritten rows may hold NaN, and the prefix's last values infinities, which a
//    probability of 0 does not remove;
//  - key tiles that some row of a row tile does not see in full looked through for values that are no
//    numbers (there are one or two of them in a causal sequence): where there are some, the softmax threads
//    add the tile's product to their rows themselves, each the keys that its row sees. That costs 4%
//    (24 prompts of 16-128 tokens behind 4096: 162 us, 156 without any care for such values);
//  - one CTA an SM that goes through several pieces of work without a break: a warp works out
//    the next piece from the metadata while the others compute, and the copies of its
//    first tiles fly during the epilogue of the piece before.
// Prefix stage: pieces of equal ranges of all groups' blocks (prefix.cuh), 128 keys for 256
// rows. Where a unit has 128 rows or fewer (the last rows of a group), the two row tiles take the
// same rows and half of the key tiles each, and leave a part each: a block is 256 keys. (Halves, not
// every other tile: the keys are then read at the time that the group's other rows read them.)
// Suffix stage: a piece is all own keys of a sequence for 256 rows, joined with the prefix's parts.
// Measured (32/8 heads, D 128, BF16): the prefix of 24 prompts of 16-128 tokens behind 4096 keys 117 us, 0.99
// PFLOP/s, their own keys 61 us; 96 rows over 60001 keys 117 us, 0.81 PFLOP/s. Bound by the softmax's latency between
// the products of two row tiles (tensor pipe 49% active); the second case also by the keys of a head
// being read for each of its two row blocks (475 MB instead of 246).
#pragma once

#include <algorithm>
#include <type_traits>

#include "prefix.cuh"

namespace attn {
namespace prefix {
namespace tc {

constexpr int BM = 128;
constexpr int BN = 128;
constexpr int NQ = 2;
constexpr int ROWS = BM * NQ;
constexpr int NUM_THREADS = 384;
constexpr int WARP_TMA = 8, WARP_MMA = 9, WARP_PLAN = 10;
constexpr int TMEM_COLS = 512;
constexpr int REG_SOFTMAX = 200;
constexpr int REG_OTHER = 96;
constexpr float RESCALE_LOG2 = 8.0f;

template <int D>
struct Cfg {
  static constexpr int NCHUNK = D / 64;
  static constexpr int CHUNK_BYTES = BN * 128;
  static constexpr int TILE_BYTES = NCHUNK * CHUNK_BYTES;
  static constexpr int STAGES = D == 128 ? 5 : 8;
  static constexpr uint32_t LAYOUT = 2u;  // 128-byte swizzle
  static constexpr int SBO = 1024;
  static constexpr int KSTEPS_QK = D / 16;
  static constexpr int KSTEPS_PV = BN / 16;
  static constexpr int COL_P = 64;
  static constexpr int OFF_KV = NQ * TILE_BYTES;
  static constexpr int OFF_BAR = OFF_KV + STAGES * TILE_BYTES;
  static constexpr int BAR_FULL = 0, BAR_EMPTY = STAGES, BAR_Q = 2 * STAGES, BAR_S = BAR_Q + NQ;
  static constexpr int BAR_P = BAR_S + NQ, BAR_O = BAR_P + NQ, BAR_DONE = BAR_O + NQ;
  static constexpr int BAR_WORK = BAR_DONE + 1, BAR_FREE = BAR_WORK + 2;  // the pieces' ring
  static constexpr int BAR_TEAM = BAR_FREE + 2;                           // the four softmax warps of a row tile
  static constexpr int OFF_MISC = OFF_BAR + (BAR_TEAM + NQ) * 8;
  static constexpr int OFF_TEAM = OFF_MISC + 16;
  static constexpr int OFF_WORK = (OFF_TEAM + NQ * 64 + 15) / 16 * 16;
  static constexpr int SMEM_BYTES = OFF_WORK + 2 * 64 + 1024;
};

// A piece of work: rows row0 .. of a unit (queries from q_lo on, nq of them, times heads), keys
// [lo, to), of which the key tiles j0 .. j0 + n - 1 of a row tile are this piece's.
struct Work {
  int s0, s1;          // the unit's sequences
  int table;           // row of the table that names the pages
  int q_lo, nq, h, row0;
  int lo, to, j0;
  int n[NQ];           // key tiles of each row tile; split: both have the same rows, and tiles from j0 and from j0 + n[0] on
  int split, part, group;
  int state;           // 0: no more work, 1: rows may see fewer keys than [lo, to), 2: every row sees all
};
static_assert(sizeof(Work) == 64);

// What the softmax warps of a row tile tell one another and the issuing warp. Meetings take the two slots by
// turns: who writes for meeting m + 2 has met the others at m + 1, and they had read those of m before.
struct Team {
  int least[2][4];  // fewest keys that a row of each warp sees
  int strange[2];   // m + 1: a warp has found a value that is no number at meeting m
  int alone;        // 1: the warps have added this tile's product themselves
  int unused[5];    // to 64 bytes
};
static_assert(sizeof(Team) == 64);

__device__ __forceinline__ bool halves(const Params& p) { return p.most_parts >= 4; }

// The most keys that one of the queries [q, q + n) of the sequences [a, b) sees. A warp calls it.
__device__ __forceinline__ int most_seen(const Params& p, int a, int b, int q, int n) {
  int most = 0;
  for (int i = q + static_cast<int>(threadIdx.x & 31); i < q + n; i += 32)
    most = max(most, limit_of(p, last_at_most(p.q_offsets, a, b, i), i));
  return __reduce_max_sync(0xffffffffu, most);
}

// The pieces of a CTA, one after another. A warp calls it, all lanes with the same results.
template <bool PREFIX>
struct Planner {
  int64_t u, u1, first;  // prefix: blocks, first one of group g
  int g;
  int64_t item, items;   // suffix
  int qblocks;
  Share sh;
  bool fresh;
  Rec rec;
  int a, b, pre, table, to, q_lo, nq;
  bool open;

  __device__ __forceinline__ void load_group(const Params& p) {
    rec = rec_of(p, g, BN, ROWS, halves(p));
    group_range(p, g, a, b);
    nq = queries_of(p, a, b, p.max_group_queries, q_lo);
    pre = prefix_len(p, g);
    // the member whose row covers the most of the prefix, and whether a row sees less of it
    unsigned long long best = 0;
    int least = 0x7fffffff;
    for (int s = a + static_cast<int>(threadIdx.x & 31); s < b; s += 32) {
      const int L = seq_len(p, s), n = query_at(p, s + 1) - query_at(p, s);
      const unsigned long long x = (static_cast<unsigned long long>(min(L, pre)) << 32) | static_cast<uint32_t>(~s);
      best = x > best ? x : best;
      if (n > 0) least = min(least, p.causal ? L - n + 1 : L);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const unsigned long long x = __shfl_xor_sync(0xffffffffu, best, o);
      best = x > best ? x : best;
    }
    least = __reduce_min_sync(0xffffffffu, least);
    table = static_cast<int>(~static_cast<uint32_t>(best));
    to = static_cast<int>(best >> 32);
    open = least >= to && !(p.causal && p.positions);
  }

  __device__ __forceinline__ bool next(const Params& p, Work& w) {
    const int heads = p.Hq / p.Hkv;
    if constexpr (PREFIX) {
      if (u >= u1) return false;
      while (fresh || u >= first + blocks_of(p, rec)) {
        if (!fresh) {
          first += blocks_of(p, rec);
          ++g;
        }
        fresh = false;
        rec = rec_of(p, g, BN, ROWS, halves(p));
        if (u < first + blocks_of(p, rec)) load_group(p);
      }
      const int64_t off = u - first, full = full_blocks(p, rec);
      w.split = off >= full;
      const int n = w.split ? (rec.nb + 1) / 2 : rec.nb;
      const int64_t in = w.split ? off - full : off;
      const int unit = static_cast<int>(in / n), k0 = static_cast<int>(in - static_cast<int64_t>(unit) * n);
      const int take = static_cast<int>(min(static_cast<int64_t>(n - k0), u1 - u));
      const int piece = static_cast<int>(blockIdx.x) - range_of(u - k0, sh.total, sh.ranges);
      u += take;
      w.s0 = a;
      w.s1 = b;
      w.table = table;
      w.q_lo = q_lo;
      w.nq = nq;
      w.h = unit % p.Hkv;
      w.row0 = (w.split ? rec.rbs - 1 : unit / p.Hkv) * ROWS;
      w.lo = 0;
      w.to = to;
      if (!open) {  // what no row of the piece sees is not there
        const int q0 = w.row0 / heads, q1 = min(nq - 1, (w.row0 + (w.split ? BM : ROWS) - 1) / heads);
        w.to = min(to, most_seen(p, a, b, q_lo + q0, q1 - q0 + 1));
      }
      w.group = g;
      const int tiles = (w.to + BN - 1) / BN;  // with keys; a reader shorter than the prefix has fewer than nb
      if (w.split) {
        w.part = 2 * piece;
        w.j0 = 2 * k0;
        const int k = max(min(2 * (k0 + take), tiles) - w.j0, 0);
        w.n[0] = (k + 1) / 2;
        w.n[1] = k / 2;
      } else {
        w.part = piece;
        w.j0 = k0;
        w.n[0] = max(min(k0 + take, tiles) - k0, 0);
        w.n[1] = w.row0 + BM < nq * heads ? w.n[0] : 0;
      }
      w.state = open ? 2 : 1;
      return true;
    } else {
      for (; item < items; item += gridDim.x) {
        int64_t r = item;
        w.h = static_cast<int>(r % p.Hkv);
        r /= p.Hkv;
        w.row0 = static_cast<int>(qblocks - 1 - r % qblocks) * ROWS;  // the last blocks see the most keys and go first
        w.s0 = w.table = static_cast<int>(r / qblocks);
        w.s1 = w.s0 + 1;
        w.nq = queries_of(p, w.s0, w.s1, p.max_queries, w.q_lo);
        if (w.row0 >= static_cast<int64_t>(w.nq) * heads) continue;
        const Own own = own_of(p, w.s0);
        w.group = own.pre > 0 ? own.group : -1;
        w.lo = own.start;
        w.to = own.L;
        w.j0 = own.start / BN;
        w.split = w.part = 0;
        const int all = query_at(p, w.s1) - w.q_lo;
        if (p.causal && p.positions) {  // what no row of the piece sees is not there
          const int q0 = w.row0 / heads, q1 = min(w.nq - 1, (w.row0 + ROWS - 1) / heads);
          w.to = min(w.to, most_seen(p, w.s0, w.s1, w.q_lo + q0, q1 - q0 + 1));
        }
#pragma unroll
        for (int t = 0; t < NQ; ++t) {
          const int r0 = w.row0 + t * BM;
          w.n[t] = 0;
          if (r0 >= static_cast<int64_t>(w.nq) * heads) continue;
          int end = w.to;  // keys that the tile's rows see
          if (p.causal && !p.positions) end = min(end, own.L - all + min(w.nq - 1, (r0 + BM - 1) / heads) + 1);
          w.n[t] = end > w.lo ? (end + BN - 1) / BN - w.j0 : 0;
        }
        w.state = 1;
        item += gridDim.x;
        return true;
      }
      return false;
    }
  }
};

// A value that is the same in all lanes of a warp, from a reduction, whose result is uniform.
__device__ __forceinline__ int uniform(int x) { return __reduce_max_sync(0xffffffffu, x); }

// Whether one of the values of the rows [from, to) of a tile in shared memory is a NaN or an infinity, as far as this
// thread (of 128) looks: 0 times it is not 0.
template <int D, bool BF16>
__device__ __forceinline__ bool any_strange(const uint8_t* v, int from, int to, int thread) {
  uint32_t sum = 0;
  auto add = [&](uint32_t x) {
    if constexpr (BF16) asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(sum) : "r"(x), "r"(0u));
    else asm("fma.rn.f16x2 %0, %1, %2, %0;" : "+r"(sum) : "r"(x), "r"(0u));
  };
  for (int e = from * 8 + thread; e < to * 8; e += 128)
#pragma unroll
    for (int c = 0; c < Cfg<D>::NCHUNK; ++c) {
      const uint4 x = *reinterpret_cast<const uint4*>(v + c * Cfg<D>::CHUNK_BYTES + e * 16);
      add(x.x);
      add(x.y);
      add(x.z);
      add(x.w);
    }
  return sum & 0x7fff7fffu;
}

// The product of a key tile whose values are not all numbers, with the weights that the tensor core would take: a
// thread adds to its row of O what the row sees, keys [from, to) of the tile. (A weight of 0 does not remove what
// is no number from the other rows of a tensor core's product.) Whatever the context's length: a call over 100000
// keys 1281 us, 1349 with one such value (BF16, D 128, 400 rows, 64 keys of the tile seen by some).
template <int D, bool BF16>
__device__ __noinline__ void own_product(uint32_t tP, uint32_t tO, const uint8_t* v, int from, int to, bool fresh) {
  const int first = __reduce_min_sync(0xffffffffu, to > from ? from : BN) & ~1;
  const int last = __reduce_max_sync(0xffffffffu, to > from ? to : 0);
#pragma unroll 1
  for (int c = 0; c < D / 32; ++c) {
    uint32_t o[32];
    tmem_ld32(tO + 32 * c, o);
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 32; ++i) o[i] = fresh ? 0u : o[i];
    const uint8_t* const at = v + c / 2 * Cfg<D>::CHUNK_BYTES;
#pragma unroll 1
    for (int key = first; key < last; ++key) {
      const uint32_t pair = tmem_ld1(tP + key / 2);
      tmem_wait_ld();
      const uint32_t half = key & 1 ? pair >> 16 : pair & 0xffffu;
      const float w = BF16 ? __uint_as_float(half << 16) : __half2float(__ushort_as_half(static_cast<unsigned short>(half)));
      if (key >= from && key < to) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const uint4 x = *reinterpret_cast<const uint4*>(at + key * 128 + (((c & 1) * 4 + u) ^ (key & 7)) * 16);
          const uint32_t y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 f = BF16 ? make_float2(__uint_as_float(y[i] << 16), __uint_as_float(y[i] & 0xffff0000u))
                                  : __half22float2(*reinterpret_cast<const __half2*>(&y[i]));
            o[8 * u + 2 * i] = __float_as_uint(fmaf(w, f.x, __uint_as_float(o[8 * u + 2 * i])));
            o[8 * u + 2 * i + 1] = __float_as_uint(fmaf(w, f.y, __uint_as_float(o[8 * u + 2 * i + 1])));
          }
        }
      }
      __syncwarp();
    }
    tmem_st32(tO + 32 * c, o);
  }
  tmem_wait_st();
}

template <int D, bool BF16, bool PREFIX>
__global__ void __launch_bounds__(NUM_THREADS, 1)
    tc_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
              const __grid_constant__ Params p, int qblocks, int64_t items, int after_prefix) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_dyn[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sb = smem_u32(smem);
  auto bar = [&](int i) -> uint32_t { return sb + C::OFF_BAR + 8 * i; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  Work* const works = reinterpret_cast<Work*>(smem + C::OFF_WORK);
  volatile Team* const teams = reinterpret_cast<volatile Team*>(smem + C::OFF_TEAM);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (PREFIX || !after_prefix) wait_before();  // nothing before this reads what other launches have written
  Planner<PREFIX> plan;
  if constexpr (PREFIX) {
    let_next();  // the suffix stage may come up
    plan.sh = p.suffix_rows > 0 ? share_out<NUM_THREADS, true>(p, SMS, BN, ROWS, halves(p))
                                : share_out<NUM_THREADS, false>(p, SMS, BN, ROWS, halves(p));
    if (static_cast<int>(blockIdx.x) >= plan.sh.ranges) return;  // the SM is the suffix stage's
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(bar(C::BAR_FULL + s), 1);
      mbar_init(bar(C::BAR_EMPTY + s), 1);
    }
    for (int t = 0; t < NQ; ++t) {
      mbar_init(bar(C::BAR_Q + t), BM);
      mbar_init(bar(C::BAR_S + t), 1);
      mbar_init(bar(C::BAR_P + t), BM);
      mbar_init(bar(C::BAR_O + t), 1);
      mbar_init(bar(C::BAR_TEAM + t), 4);
      teams[t].strange[0] = teams[t].strange[1] = teams[t].alone = 0;
    }
    mbar_init(bar(C::BAR_DONE), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(C::BAR_WORK + i), 1);
      mbar_init(bar(C::BAR_FREE + i), 10);  // the copying and the issuing warp, 8 softmax warps
    }
    mbar_init_fence();
  }
  if (warp == WARP_MMA) {
    tmem_alloc(smem_u32(tmem_slot), TMEM_COLS);
    tmem_relinquish();
  }
  if constexpr (PREFIX) {
    plan.u = plan.sh.u0;
    plan.u1 = plan.sh.u1;
    plan.first = plan.sh.first;
    plan.g = plan.sh.g;
    plan.fresh = true;
  } else {
    plan.item = blockIdx.x;
    plan.items = items;
    plan.qblocks = qblocks;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  auto fail = [&]() {
    if (p.status) atomicOr(p.status, STATUS_TIMEOUT);
  };
  // Piece i for a warp that takes part in it (all lanes); false: none, or a wait gave up.
  auto get_work = [&](int i, Work& w) {
    if (!warp_wait(bar(C::BAR_WORK + (i & 1)), (i >> 1) & 1)) {
      if (lane == 0) fail();
      return false;
    }
    w = works[i & 1];
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(C::BAR_FREE + (i & 1)));
    return w.state != 0;
  };

  if (warp >= 8) {
    setmaxnreg_dec<REG_OTHER>();
    if (warp == WARP_PLAN) {
      // ------------------------------------------------------------ the pieces, ahead of the others
      for (int i = 0;; ++i) {
        Work w{};
        const bool more = plan.next(p, w);
        if (!warp_wait(bar(C::BAR_FREE + (i & 1)), ((i >> 1) & 1) ^ 1)) {
          if (lane == 0) fail();
          break;
        }
        if (!more) w.state = 0;
        if (lane == 0) {
          works[i & 1] = w;
          mbar_arrive(bar(C::BAR_WORK + (i & 1)));
        }
        __syncwarp();
        if (!more) break;
      }
    } else if (warp == WARP_TMA) {
      // ------------------------------------------------------------ producer: a lane for each box of a tile
      const int box_rows = p.page_size < BN ? p.page_size : BN;
      const int boxes = BN / box_rows;
      int it = 0;
      bool ok = true;
      Work w{};
      if (lane == 0) {
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
      }
      auto load = [&](const CUtensorMap* m, int j) {  // key tile j into the next slot
        // the page is looked up before the wait: it costs a trip to L2
        const int key = j * BN + lane * box_rows, blk = key / p.page_size, in_page = key - blk * p.page_size;
        const int page = lane < boxes && key < w.to ? page_of(p, w.table, blk) : -1;  // -1: zero-filled box
        const int st = it % C::STAGES;
        if (!warp_wait(bar(C::BAR_EMPTY + st), ((it / C::STAGES) & 1) ^ 1)) return false;
        ++it;
        if (lane == 0) mbar_arrive_expect_tx(bar(C::BAR_FULL + st), C::TILE_BYTES);
        __syncwarp();
        // checked build: the box lands inside its chunk of the ring slot (a
        // skipped copy leaves the slot's barrier to time out)
        if (lane < boxes && range_in_bounds(p.status, lane * box_rows, box_rows, BN)) {
          for (int c = 0; c < C::NCHUNK; ++c)
            tma_load_4d(sb + C::OFF_KV + st * C::TILE_BYTES + c * C::CHUNK_BYTES + lane * box_rows * 128, m,
                        bar(C::BAR_FULL + st), c * 64, w.h, in_page, page);
        }
        __syncwarp();
        return true;
      };
      for (int i = 0; ok && get_work(i, w); ++i) {
        if (w.split) {  // in the order of the MMAs
          for (int j = 0; j <= w.n[0] && ok; ++j) {
            if (j < w.n[0]) ok = load(&tm_k, w.j0 + j);
            if (ok && j >= 1 && j - 1 < w.n[1]) ok = load(&tm_v, w.j0 + w.n[0] + j - 1);
            if (ok && j < w.n[1]) ok = load(&tm_k, w.j0 + w.n[0] + j);
            if (ok && j < w.n[0]) ok = load(&tm_v, w.j0 + j);
          }
        } else {
          const int nmax = max(w.n[0], w.n[1]);
          for (int j = 0; j < nmax && ok; ++j) ok = load(&tm_k, w.j0 + j) && load(&tm_v, w.j0 + j);
        }
      }
      if (!ok && lane == 0) fail();
      for (int st = 0; st < C::STAGES && st < it; ++st) {
        const int fills = (it - st + C::STAGES - 1) / C::STAGES;
        if (!warp_wait(bar(C::BAR_FULL + st), (fills - 1) & 1) && lane == 0) fail();
      }
    } else if (warp == WARP_MMA) {
      // ------------------------------------------------------------ MMA issuer
      // (the whole warp waits; one elected lane issues the MMAs and commits)
      constexpr uint32_t idesc_qk = make_idesc_f16(BF16, BM, BN, false);
      constexpr uint32_t idesc_pv = make_idesc_f16(BF16, BM, D, true);
      constexpr int ST = C::STAGES;
      const uint64_t dq0 = smem_desc(sb, 16, C::SBO, C::LAYOUT);
      const uint64_t dk0 = smem_desc(sb + C::OFF_KV, 16, C::SBO, C::LAYOUT);
      const uint64_t dv0 = smem_desc(sb + C::OFF_KV, C::CHUNK_BYTES, C::SBO, C::LAYOUT);
      constexpr uint32_t TILE16 = C::TILE_BYTES >> 4;
      constexpr uint32_t CHUNK16 = C::CHUNK_BYTES >> 4;
      constexpr uint32_t VSTEP16 = (16 * 128) >> 4;
      auto kstep = [](int k) -> uint32_t { return (k / 4) * CHUNK16 + (k % 4) * 2; };
      int it0 = 0;            // ring slots of the pieces before
      int done[NQ] = {0, 0};  // key tiles of each row tile in the pieces before
      int used[NQ] = {0, 0};  // pieces with such
      bool ok = true;
      Work w{};
      auto wait_full = [&](int idx) { return warp_wait(bar(C::BAR_FULL + idx % ST), (idx / ST) & 1); };
      // Values outside the unit's keys (tile j of the unit, in ring slot idx): whole rows, the swizzle stays inside them.
      auto fix_values = [&](int j, int idx) {
        const int lo = PREFIX ? 0 : w.lo - j * BN, hi = w.to - j * BN;  // its rows are [lo, hi)
        if (lo <= 0 && hi >= BN) return;
        uint8_t* const v = smem + C::OFF_KV + idx % ST * C::TILE_BYTES;
        auto clear = [&](int e) {
#pragma unroll
          for (int c = 0; c < C::NCHUNK; ++c) *reinterpret_cast<uint4*>(v + c * C::CHUNK_BYTES + e * 16) = make_uint4(0u, 0u, 0u, 0u);
        };
        if (!PREFIX && lo > 0) {
#pragma unroll 1
          for (int e = lane; e < min(lo, BN) * 8; e += 32) clear(e);
        }
        for (int e = max(hi, 0) * 8 + lane; e < BN * 8; e += 32) clear(e);
        fence_proxy_async_smem();
        __syncwarp();
      };
      auto issue_s = [&](int t, int idx) {
        const uint64_t a = dq0 + t * TILE16;
        const uint64_t b = dk0 + (idx % ST) * TILE16;
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < C::KSTEPS_QK; ++k)
            umma_ss(tmem + t * BN, a + kstep(k), b + kstep(k), idesc_qk, k > 0 ? 1u : 0u);
          umma_commit(bar(C::BAR_S + t));
        }
        __syncwarp();
      };
      auto issue_pv = [&](int t, int j, int idx, bool last, auto checked) {
        const uint64_t b = dv0 + (idx % ST) * TILE16;
        const uint32_t d = tmem + 256 + t * D;
        const uint32_t a = tmem + t * BN + C::COL_P;
        // the softmax warps may have added the product themselves (a loop of its own where they never do: one for both
        // costs the prefix stage 1%)
        if (decltype(checked)::value && uniform(teams[t].alone)) {
          if (last && elect_one()) umma_commit(bar(C::BAR_O + t));
        } else if (elect_one()) {
          umma_ts(d, a, b, idesc_pv, j > 0 ? 1u : 0u);
#pragma unroll
          for (int k = 1; k < C::KSTEPS_PV; ++k) umma_ts(d, a + k * 8, b + k * VSTEP16, idesc_pv, 1u);
          if (last) umma_commit(bar(C::BAR_O + t));
        }
        __syncwarp();
      };
      auto release = [&](int idx) {
        if (elect_one()) umma_commit(bar(C::BAR_EMPTY + idx % ST));
        __syncwarp();
      };
      auto wait_p = [&](int t, int j) { return warp_wait(bar(C::BAR_P + t), (done[t] + j) & 1); };
      for (int i = 0; ok && get_work(i, w); ++i) {
        // the loops below run in uniform registers, as the MMAs take their operands
        const int n0 = uniform(w.n[0]), n1 = uniform(w.n[1]), nmax = max(n0, n1);
        const bool split = uniform(w.split) != 0;
        for (int t = 0; t < NQ && ok; ++t)
          if ((t ? n1 : n0) > 0) {
            ok = warp_wait(bar(C::BAR_Q + t), used[t] & 1);
            ++used[t];
          }
        auto walk = [&](auto checked) {  // every wait is bounded
          if (split) {
            int idx = it0;
            for (int j = 0; j <= n0 && ok; ++j) {
              if (j < n0) {
                if (!(ok = wait_full(idx))) break;
                tc_fence_after();
                issue_s(0, idx);
                release(idx++);
              }
              if (j >= 1 && j - 1 < n1) {
                if (!(ok = wait_full(idx))) break;
                fix_values(w.j0 + n0 + j - 1, idx);
                if (!(ok = wait_p(1, j - 1))) break;
                tc_fence_after();
                issue_pv(1, j - 1, idx, j == n1, checked);
                release(idx++);
              }
              if (j < n1) {
                if (!(ok = wait_full(idx))) break;
                tc_fence_after();
                issue_s(1, idx);
                release(idx++);
              }
              if (j < n0) {
                if (!(ok = wait_full(idx))) break;
                fix_values(w.j0 + j, idx);
                if (!(ok = wait_p(0, j))) break;
                tc_fence_after();
                issue_pv(0, j, idx, j == n0 - 1, checked);
                release(idx++);
              }
            }
            it0 = idx;
          } else {
            for (int j = 0; j <= nmax && ok; ++j) {
              const int idx = it0 + 2 * j;
              if (j < nmax) {
                if (!(ok = wait_full(idx))) break;
                tc_fence_after();
                if (j < n0) issue_s(0, idx);
              }
              if (j >= 1 && j - 1 < n1) {
                if (j - 1 >= n0) {
                  if (!(ok = wait_full(idx - 1))) break;
                  fix_values(w.j0 + j - 1, idx - 1);
                }
                if (!(ok = wait_p(1, j - 1))) break;
                tc_fence_after();
                issue_pv(1, j - 1, idx - 1, j == n1, checked);
              }
              if (j >= 1) release(idx - 1);
              if (j < nmax) {
                if (j < n1) issue_s(1, idx);
                release(idx);
                if (j < n0) {
                  if (!(ok = wait_full(idx + 1))) break;
                  fix_values(w.j0 + j, idx + 1);
                  if (!(ok = wait_p(0, j))) break;
                  tc_fence_after();
                  issue_pv(0, j, idx + 1, j == n0 - 1, checked);
                }
              }
            }
            it0 += 2 * nmax;
          }
        };
        if (PREFIX && uniform(w.state) == 2) walk(std::false_type{});
        else walk(std::true_type{});
        done[0] += n0;
        done[1] += n1;
      }
      if (!ok && lane == 0) fail();
      if (elect_one()) umma_commit(bar(C::BAR_DONE));
      __syncwarp();
      if (!warp_wait(bar(C::BAR_DONE), 0) && lane == 0) fail();
    }
    __syncwarp();
  } else {
    // -------------------------------------------------------------- softmax
    setmaxnreg_inc<REG_SOFTMAX>();
    const int t = warp >> 2;
    const int row = ((warp & 3) << 5) + lane;
    const int64_t nrows = static_cast<int64_t>(p.num_queries) * p.Hq;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) << 5) << 16;
    const uint32_t tS = tmem + lane_off + t * BN;
    const uint32_t tP = tS + C::COL_P;
    const uint32_t tO = tmem + lane_off + 256 + t * D;
    const float sc = p.scale_log2;
    const int heads = p.Hq / p.Hkv;
    int done = 0, used = 0;  // key tiles and pieces before
    int it0 = 0;            // ring slots of the pieces before
    int met = 0;            // meetings of the row tile's four warps
    volatile Team& team = teams[t];
    bool failed = false, waited = false, alone = false;
    auto meet = [&]() {  // all lanes
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(C::BAR_TEAM + t));
      return warp_wait(bar(C::BAR_TEAM + t), met++ & 1);
    };
    for (int i = 0; !failed; ++i) {
      Work w{};
      if (!get_work(i, w)) break;
      const int pr = w.row0 + (w.split ? 0 : t * BM) + row;  // packed row: query * heads + head
      const int tq = pr / heads;
      const bool row_ok = tq < w.nq;
      const int64_t orow = row_ok ? static_cast<int64_t>(w.q_lo + tq) * p.Hq + w.h * heads + (pr - tq * heads) : 0;
      const bool row_in = row_ok && in_bounds(p.status, orow, nrows);
      const int n_t = w.n[t], jt = w.j0 + (w.split && t ? w.n[0] : 0);
      if (n_t > 0) {  // the thread's row of q, into the swizzled tile
        const uint4* const src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) + orow * D);
        uint8_t* const dst = smem + t * C::TILE_BYTES + row * 128;
        uint4 x[C::NCHUNK * 8];
#pragma unroll
        for (int k = 0; k < C::NCHUNK * 8; ++k) x[k] = row_in ? __ldg(src + k) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int k = 0; k < C::NCHUNK * 8; ++k)
          *reinterpret_cast<uint4*>(dst + k / 8 * C::CHUNK_BYTES + (((k % 8) ^ (row & 7)) << 4)) = x[k];
        fence_proxy_async_smem();
        tc_fence_before();
        mbar_arrive(bar(C::BAR_Q + t));
      }
      int lim = 0;  // keys that the row sees
      if (w.state == 2) {
        lim = w.to;
      } else if (row_ok) {
        const int q = w.q_lo + tq;
        lim = min(w.to, limit_of(p, PREFIX ? last_at_most(p.q_offsets, w.s0, w.s1, q) : w.s0, q));
      }
      const int least = __reduce_min_sync(0xffffffffu, row_ok ? lim : w.to);
      int least_t = w.to;  // of the row tile
      if (w.state != 2 && n_t > 0) {
        if (lane == 0) team.least[met & 1][warp & 3] = least;
        failed = !meet();
#pragma unroll
        for (int k = 0; k < 4; ++k) least_t = min(least_t, team.least[(met - 1) & 1][k]);
      }
      float m_run = -INFINITY, l_run = 0.f;
      for (int j = 0; j < n_t && !failed; ++j) {
        const bool ok = mbar_wait(bar(C::BAR_S + t), (done + j) & 1);
        if (__any_sync(0xffffffffu, !ok)) { failed = true; break; }
        tc_fence_after();
        // Values that a row of the tile does not see have to be numbers for the tensor core: where there are such keys
        // the four warps look through theirs. (Once S of a tile is there, so is what was in its values' slot before.)
        const int base = (jt + j) * BN;
        const int from = max(base, max(least_t, w.lo)), upto = min(base + BN, w.to);
        const uint8_t* values = nullptr;  // of the tile, if one of them is none
        if (from < upto) {
          const int idx = it0 + (!w.split ? 2 * j + 1 : t ? 4 * j + 3 + (j + 1 < w.n[0]) : 4 * j + 1 + (j < w.n[1]));
          const int slot = met & 1;
          values = smem + C::OFF_KV + idx % C::STAGES * C::TILE_BYTES;
          failed = !warp_wait(bar(C::BAR_FULL + idx % C::STAGES), (idx / C::STAGES) & 1);
          if (failed) break;
          const bool bad = any_strange<D, BF16>(values, from - base, upto - base, (warp & 3) * 32 + lane);
          if (__any_sync(0xffffffffu, bad) && lane == 0) team.strange[slot] = met + 1;
          failed = !meet();
          if (failed) break;
          if (team.strange[slot] != met) values = nullptr;
        }
        float s[128];
        {
          uint32_t sr[4][32];
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32(tS + 32 * c, sr[c]);
          tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < 128; ++k) s[k] = __uint_as_float(sr[k >> 5][k & 31]);
        }
        const int key0 = (jt + j) * BN;
        if (key0 + BN > least || key0 < w.lo) {
#pragma unroll
          for (int k = 0; k < 128; ++k) {
            const int key = key0 + k;
            if (key >= lim || key < w.lo) s[k] = -INFINITY;
          }
        }
        float c0 = fmax3(s[0], s[1], s[2]), c1 = fmax3(s[3], s[4], s[5]);
        float c2 = fmax3(s[6], s[7], s[8]), c3 = fmax3(s[9], s[10], s[11]);
#pragma unroll
        for (int k = 12; k < 124; k += 8) {
          c0 = fmax3(c0, s[k], s[k + 1]);
          c1 = fmax3(c1, s[k + 2], s[k + 3]);
          c2 = fmax3(c2, s[k + 4], s[k + 5]);
          c3 = fmax3(c3, s[k + 6], s[k + 7]);
        }
        c0 = fmax3(c0, s[124], s[125]);
        c1 = fmax3(c1, s[126], s[127]);
        const float m_tile = fmax3(c0, c1, fmaxf(c2, c3)) * sc;
        const bool need = m_tile > m_run + RESCALE_LOG2;
        float alpha = 1.f;
        if (need) {
          alpha = fast_exp2(m_run - m_tile);
          m_run = m_tile;
          l_run *= alpha;
        }
        const float neg_m = (m_run == -INFINITY) ? 0.f : -m_run;
        float2 sum_a = make_float2(0.f, 0.f), sum_b = make_float2(0.f, 0.f);
        // The product takes the weights rounded to the input type; their sum is of the unrounded ones. Error against 64
        // bits, relative to the output's norm, BF16: 2.2e-3 to 2.3e-3, of which 1.7e-3 are the output's own rounding (F16 2.7e-4,
        // 2.1e-4). As two numbers each, with a second product, the error is the output's rounding alone, and the calls take 21 to 36%
        // longer (96 rows behind 60001 keys 170 us, 140 as it is; 24 prompts behind 4096 220 and 161; 8 groups of 7 heads 76 and 60).
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          uint32_t pk[32];
#pragma unroll
          for (int c = 0; c < 32; c += 2) {
            const int k = 64 * hh + 2 * c;
            const float2 xa = ffma2(make_float2(s[k], s[k + 1]), make_float2(sc, sc), make_float2(neg_m, neg_m));
            const float2 xb = ffma2(make_float2(s[k + 2], s[k + 3]), make_float2(sc, sc), make_float2(neg_m, neg_m));
            const float2 pa = make_float2(fast_exp2(xa.x), fast_exp2(xa.y));
            const float2 pb = make_float2(fast_exp2(xb.x), fast_exp2(xb.y));
            sum_a = fadd2(sum_a, pa);
            sum_b = fadd2(sum_b, pb);
            pk[c] = pack2<BF16>(pa.x, pa.y);
            pk[c + 1] = pack2<BF16>(pb.x, pb.y);
          }
          tmem_st32(tP + 32 * hh, pk);
        }
        l_run += (sum_a.x + sum_a.y) + (sum_b.x + sum_b.y);
        if (j > 0 && __any_sync(0xffffffffu, need)) {
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tmem_ld32(tO + 32 * c, o);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 32; k += 2) {
              const float2 x = fmul2(make_float2(__uint_as_float(o[k]), __uint_as_float(o[k + 1])), make_float2(alpha, alpha));
              o[k] = __float_as_uint(x.x);
              o[k + 1] = __float_as_uint(x.y);
            }
            tmem_st32(tO + 32 * c, o);
          }
        }
        tmem_wait_st();
        if (values) own_product<D, BF16>(tP, tO, values, max(w.lo - key0, 0), min(lim - key0, BN), j == 0);
        if ((values != nullptr) != alone) {
          alone = values != nullptr;
          if (row == 0) team.alone = alone;
        }
        tc_fence_before();
        mbar_arrive(bar(C::BAR_P + t));
      }
      done += n_t;
      it0 += w.split ? 2 * (w.n[0] + w.n[1]) : 2 * max(w.n[0], w.n[1]);
      // -------------------------------------------------------------- epilogue
      const bool have = n_t > 0;
      if (!failed && have) {
        const bool ok = mbar_wait(bar(C::BAR_O + t), used & 1);
        ++used;
        if (__any_sync(0xffffffffu, !ok)) failed = true;
      }
      if (failed) {
        if (lane == 0) fail();
        break;
      }
      if (!w.split && w.row0 + t * BM >= w.nq * heads) continue;  // no rows of this tile
      tc_fence_after();
      if constexpr (PREFIX) {
        const int64_t at = (w.part + (w.split ? t : 0)) * nrows + orow;
        const bool ok = row_in && in_bounds(p.status, at, p.most_parts * nrows);
        float* const dst = p.o + at * D;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          if (have) {
            tmem_ld32(tO + 32 * c, o);
            tmem_wait_ld();
          } else {
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = 0u;
          }
          if (ok) {
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              float x[8];
#pragma unroll
              for (int k = 0; k < 8; ++k) x[k] = __uint_as_float(o[8 * u + k]);
              store8(dst + c * 32 + 8 * u, x);
            }
          }
        }
        if (ok) p.ml[at] = make_float2(have ? m_run : -INFINITY, l_run);
      } else {
        if (!waited) wait_before();  // the prefix's parts
        waited = true;
        const int parts = w.group >= 0 && row_in ? parts_of(p, w.group, w.q_lo + tq, pr - tq * heads, w.h) : 0;
        float M = have ? m_run : -INFINITY;
        for (int z = 0; z < parts; ++z) M = fmaxf(M, __ldcg(p.ml + z * nrows + orow).x);
        const bool any = M != -INFINITY;
        const float own = any ? fast_exp2(m_run - M) : 0.f;
        float sum = l_run * own;
        for (int z = 0; z < parts; ++z)
          if (any) {
            const float2 ml = __ldcg(p.ml + z * nrows + orow);
            sum = fmaf(ml.y, fast_exp2(ml.x - M), sum);
          }
        const bool live = sum > 0.f;
        const float inv = live ? 1.f / sum : __int_as_float(0x7fc00000);
        uint8_t* const dst = static_cast<uint8_t*>(p.out) + orow * D * 2;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          if (have) {
            tmem_ld32(tO + 32 * c, o);
            tmem_wait_ld();
          } else {
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = 0u;
          }
          if (row_in) {
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * own);
            for (int z = 0; z < parts && any; ++z) {
              const int64_t at = z * nrows + orow;
              const float f = fast_exp2(__ldcg(p.ml + at).x - M);
#pragma unroll
              for (int u = 0; u < 4; ++u) {
                float x[8];
                load8cg(x, p.o + at * D + c * 32 + 8 * u);
#pragma unroll
                for (int k = 0; k < 8; ++k) o[8 * u + k] = __float_as_uint(fmaf(f, x[k], __uint_as_float(o[8 * u + k])));
              }
            }
            uint32_t pk[16];
#pragma unroll
            for (int k = 0; k < 16; ++k)
              pk[k] = pack2<BF16>(__uint_as_float(o[2 * k]) * inv, __uint_as_float(o[2 * k + 1]) * inv);
#pragma unroll
            for (int u = 0; u < 4; ++u)
              reinterpret_cast<uint4*>(dst + c * 64)[u] = make_uint4(pk[4 * u], pk[4 * u + 1], pk[4 * u + 2], pk[4 * u + 3]);
          }
        }
        if (row_in && p.lse) p.lse[orow] = live ? (M + log2f(sum)) * LN2 : (sum == 0.f ? -INFINITY : sum);
      }
    }
    // the suffix stage does not end before the prefix's: the next call on the stream may use the workspace
    if constexpr (!PREFIX) {
      if (!waited) wait_before();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == WARP_MMA) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, TMEM_COLS);
  }
}

template <int D, bool BF16, bool PREFIX>
cudaError_t launch_d(EncodeTiledFn enc, const Params& p, bool after_prefix, cudaStream_t st) {
  const CUtensorMapDataType dt = BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  const cuuint32_t estride[4] = {1, 1, 1, 1};
  CUtensorMap tk, tv;  // k, v viewed as [pages, page_size, Hkv, D]
  const cuuint64_t gdim[4] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(p.Hkv),
                              static_cast<cuuint64_t>(p.page_size), static_cast<cuuint64_t>(p.num_pages)};
  const cuuint64_t gstride[3] = {static_cast<cuuint64_t>(D) * 2, static_cast<cuuint64_t>(p.Hkv) * D * 2,
                                 static_cast<cuuint64_t>(p.page_size) * p.Hkv * D * 2};
  const cuuint32_t box[4] = {64u, 1u, static_cast<cuuint32_t>(p.page_size < BN ? p.page_size : BN), 1u};
  for (int i = 0; i < 2; ++i)
    if (enc(i == 0 ? &tk : &tv, dt, 4, const_cast<void*>(i == 0 ? p.k : p.v), gdim, gstride, box, estride,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  auto kern = tc_kernel<D, BF16, PREFIX>;
  constexpr int smem = Cfg<D>::SMEM_BYTES;
  static std::atomic<unsigned long long> configured{0};
  const cudaError_t e = allow_smem(kern, smem, p.device, configured);
  if (e != cudaSuccess) return e;
  const int64_t heads = p.Hq / p.Hkv;
  const int64_t qblocks = (p.max_queries * heads + ROWS - 1) / ROWS;
  const int64_t items = p.num_seqs * qblocks * p.Hkv;
  const int64_t ctas = PREFIX ? SMS : std::min<int64_t>(items, SMS);
  if (ctas == 0) return cudaSuccess;
  return launch_early(kern, dim3(static_cast<unsigned>(ctas)), NUM_THREADS, smem, st, 0, tk, tv, p, static_cast<int>(qblocks),
                      items, after_prefix ? 1 : 0);
}

template <bool BF16, bool PREFIX>
cudaError_t launch(EncodeTiledFn enc, const Params& p, bool after_prefix, cudaStream_t st) {
  return p.D == 128 ? launch_d<128, BF16, PREFIX>(enc, p, after_prefix, st) : launch_d<64, BF16, PREFIX>(enc, p, after_prefix, st);
}

}  // namespace tc
}  // namespace prefix
}  // namespace attn
