// prefix_tc.cuh - both stages of attn_paged_prefix_fwd (prefix.cuh) for many rows, on the tcgen05
// tensor cores (F16/BF16, D in {64, 128}, page_size a multiple of 8 that divides 128 or a
// multiple of 128): the prefix of a group with more than 32 rows (queries x heads of a kv
// head), and the own keys of sequences with many new tokens.
//
// The pipeline is the dense forward's (attn_tc.cuh: 384 threads, two tiles of 128 rows that share
// every K/V tile, S and P in tensor memory, MMA order S_0 PV_1 S_1 PV_0, lazy rescale), with
//  - rows packed as row = query * heads + head, whatever the number of heads: each softmax
//    thread copies its own row of q into the swizzled tile (a TMA box would want heads
//    to divide 128);
//  - 128-key tiles gathered page by page, one TMA box each, from a 4-D view
//    [pages, page_size, Hkv, D] of the cache;
//  - values past the last key set to zero in shared memory before their product: a page's
//    unwritten rows may hold NaN, which a probability of 0 does not remove;
//  - prefix stage: a CTA takes one part of the keys (Item) for 256 rows and leaves (m, l, O);
//    suffix stage: a CTA takes all own keys of a sequence for 256 rows and joins them
//    with the prefix's parts.
#pragma once

#include <algorithm>

#include "prefix_rows.cuh"

namespace attn {
namespace prefix {
namespace tc {

constexpr int BM = 128;
constexpr int BN = 128;
constexpr int NQ = 2;
constexpr int ROWS = BM * NQ;
constexpr int NUM_THREADS = 384;
constexpr int WARP_TMA = 8, WARP_MMA = 9;
constexpr int TMEM_COLS = 512;
constexpr int REG_SOFTMAX = 200;
constexpr int REG_OTHER = 96;
constexpr float RESCALE_LOG2 = 8.0f;

template <int D>
struct Cfg {
  static constexpr int NCHUNK = D / 64;
  static constexpr int CHUNK_BYTES = BN * 128;
  static constexpr int TILE_BYTES = NCHUNK * CHUNK_BYTES;
  static constexpr int STAGES = D == 128 ? 4 : 8;
  static constexpr uint32_t LAYOUT = 2u;  // 128-byte swizzle
  static constexpr int SBO = 1024;
  static constexpr int KSTEPS_QK = D / 16;
  static constexpr int KSTEPS_PV = BN / 16;
  static constexpr int COL_P = 64;
  static constexpr int OFF_KV = NQ * TILE_BYTES;
  static constexpr int OFF_BAR = OFF_KV + STAGES * TILE_BYTES;
  static constexpr int BAR_FULL = 0, BAR_EMPTY = STAGES, BAR_Q = 2 * STAGES, BAR_S = BAR_Q + NQ;
  static constexpr int BAR_P = BAR_S + NQ, BAR_O = BAR_P + NQ, BAR_DONE = BAR_O + NQ;
  static constexpr int OFF_MISC = OFF_BAR + (BAR_DONE + 1) * 8;
  static constexpr int SMEM_BYTES = OFF_MISC + 16 + 1024;
};

struct Work {
  int s0, s1;         // the unit's sequences [s0, s1)
  int table;          // row of the table that names the pages
  int q_lo, nq, h;
  int64_t row0;       // first packed row
  int lo, to;         // keys [lo, to), of which tiles j0 .. j0 + n - 1
  int j0, n[NQ], nmax;
  int group, part, parts;
};

template <int D, bool BF16, bool PREFIX>
__global__ void __launch_bounds__(NUM_THREADS, 1)
    tc_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
              const __grid_constant__ Params p, int ctas, int qblocks, int* counters, int num_counters) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_dyn[];
  __shared__ rows::Item shared_item;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sb = smem_u32(smem);
  auto bar = [&](int i) -> uint32_t { return sb + C::OFF_BAR + 8 * i; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int heads = p.Hq / p.Hkv;
  if constexpr (PREFIX) {
    asm volatile("griddepcontrol.launch_dependents;");  // the suffix stage may come up: it waits before it reads
    for (int i = blockIdx.x * NUM_THREADS + threadIdx.x; i < num_counters; i += gridDim.x * NUM_THREADS) counters[i] = 0;
  }

  // -------------------------------------------------------------- the CTA's work
  Work w;
  if constexpr (PREFIX) {
    if (warp == 0) {
      const rows::Item x = rows::item_of(p, blockIdx.x, ctas, BN, ROWS);
      if (lane == 0) shared_item = x;
    }
    __syncthreads();
    const rows::Item it = shared_item;
    if (it.g < 0) return;
    group_range(p, it.g, w.s0, w.s1);
    const int pre = prefix_len(p, it.g);
    w.table = reader_of(p, w.s0, w.s1, pre);
    w.h = it.h;
    w.row0 = static_cast<int64_t>(it.rb) * ROWS;
    w.group = it.g;
    w.part = it.part;
    w.parts = it.parts;
    w.lo = 0;
    w.to = min(pre, seq_len(p, w.table));
    w.j0 = it.part * it.chunk;
    if (it.part == 0 && it.rb == 0 && it.h == 0 && threadIdx.x == 0) p.parts[it.g] = it.parts;
  } else {
    int item = blockIdx.x;
    w.h = item % p.Hkv;
    item /= p.Hkv;
    w.row0 = static_cast<int64_t>(qblocks - 1 - item % qblocks) * ROWS;  // the last blocks see the most keys and go first
    w.table = w.s0 = item / qblocks;
    w.s1 = w.s0 + 1;
    const rows::Own own = rows::own_of(p, w.s0);
    w.group = own.pre > 0 ? own.group : -1;
    w.lo = own.start;
    w.to = own.L;
    w.j0 = own.start / BN;
    w.part = w.parts = 0;
  }
  w.q_lo = query_at(p, w.s0);
  w.nq = max(query_at(p, w.s1) - w.q_lo, 0);
  const int64_t unit_rows = static_cast<int64_t>(w.nq) * heads;
  if (w.row0 >= unit_rows) {  // CTA-uniform
    // the suffix stage does not end before the prefix's: the next call on the stream may use the workspace
    if constexpr (!PREFIX) asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }
  w.nmax = 0;
#pragma unroll
  for (int t = 0; t < NQ; ++t) {
    const int64_t r0 = w.row0 + t * BM;
    w.n[t] = 0;
    if (r0 >= unit_rows) continue;
    int end = w.to;  // keys that the tile's rows see
    if constexpr (PREFIX) {
      end = static_cast<int>(min(static_cast<int64_t>(end), (static_cast<int64_t>(w.j0) + shared_item.chunk) * BN));
    } else if (p.causal && !p.positions) {
      const int64_t last_q = min(static_cast<int64_t>(w.nq) - 1, (r0 + BM - 1) / heads);
      end = static_cast<int>(min(static_cast<int64_t>(end), static_cast<int64_t>(w.to) - w.nq + last_q + 1));
    }
    w.n[t] = end > w.lo && end > w.j0 * BN ? (end + BN - 1) / BN - w.j0 : 0;
    w.nmax = max(w.nmax, w.n[t]);
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
    }
    mbar_init(bar(C::BAR_DONE), 1);
    mbar_init_fence();
  }
  if (warp == WARP_MMA) {
    tmem_alloc(smem_u32(tmem_slot), TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  auto fail = [&]() {
    if (p.status) atomicOr(p.status, STATUS_TIMEOUT);
  };

  if (warp >= 8) {
    setmaxnreg_dec<REG_OTHER>();
    if (warp == WARP_TMA && lane == 0) {
      // ------------------------------------------------------------ producer
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
      const int box_rows = p.page_size < BN ? p.page_size : BN;
      const int boxes = BN / box_rows;
      int it = 0;
      bool ok = true;
      for (int jj = 0; jj < w.nmax && ok; ++jj) {
        const int j = w.j0 + jj;  // key tile
        for (int kv = 0; kv < 2; ++kv, ++it) {
          const int st = it % C::STAGES;
          if (!mbar_wait(bar(C::BAR_EMPTY + st), ((it / C::STAGES) & 1) ^ 1)) { ok = false; break; }
          mbar_arrive_expect_tx(bar(C::BAR_FULL + st), C::TILE_BYTES);
          const CUtensorMap* m = kv == 0 ? &tm_k : &tm_v;
          for (int i = 0; i < boxes; ++i) {
            const int key = j * BN + i * box_rows;
            const int page = key < w.to ? page_of(p, w.table, key / p.page_size) : -1;  // -1: zero-filled box
            // checked build: the box lands inside its chunk of the ring slot (a
            // skipped copy leaves the slot's barrier to time out)
            if (!range_in_bounds(p.status, i * box_rows, box_rows, BN)) continue;
            for (int c = 0; c < C::NCHUNK; ++c)
              tma_load_4d(sb + C::OFF_KV + st * C::TILE_BYTES + c * C::CHUNK_BYTES + i * box_rows * 128, m,
                          bar(C::BAR_FULL + st), c * 64, w.h, key % p.page_size, page);
          }
        }
      }
      if (!ok) fail();
      for (int st = 0; st < C::STAGES && st < it; ++st) {
        const int fills = (it - st + C::STAGES - 1) / C::STAGES;
        if (!mbar_wait(bar(C::BAR_FULL + st), (fills - 1) & 1)) fail();
      }
    } else if (warp == WARP_MMA) {
      // ------------------------------------------------------------ MMA issuer
      // (the whole warp waits; one elected lane issues the MMAs and commits)
      constexpr uint32_t idesc_qk = make_idesc_f16(BF16, BM, BN, false);
      constexpr uint32_t idesc_pv = make_idesc_f16(BF16, BM, D, true);
      constexpr int ST = C::STAGES;
      const int n0 = w.n[0], n1 = w.n[1], nmax = w.nmax;
      bool ok = true;
      for (int t = 0; t < NQ && ok; ++t)
        if ((t ? n1 : n0) > 0 && !warp_wait(bar(C::BAR_Q + t), 0)) ok = false;
      const uint64_t dq0 = smem_desc(sb, 16, C::SBO, C::LAYOUT);
      const uint64_t dk0 = smem_desc(sb + C::OFF_KV, 16, C::SBO, C::LAYOUT);
      const uint64_t dv0 = smem_desc(sb + C::OFF_KV, C::CHUNK_BYTES, C::SBO, C::LAYOUT);
      constexpr uint32_t TILE16 = C::TILE_BYTES >> 4;
      constexpr uint32_t CHUNK16 = C::CHUNK_BYTES >> 4;
      constexpr uint32_t VSTEP16 = (16 * 128) >> 4;
      auto kstep = [](int k) -> uint32_t { return (k / 4) * CHUNK16 + (k % 4) * 2; };
      bool fix = nmax > 0 && static_cast<int64_t>(w.j0 + nmax) * BN > w.to;  // the last tile goes past the keys
      auto wait_full = [&](int idx) {
        if (!warp_wait(bar(C::BAR_FULL + idx % ST), (idx / ST) & 1)) return false;
        if (fix && idx == 2 * nmax - 1) {  // values past the last key: whole rows, the swizzle stays inside them
          fix = false;
          uint8_t* const v = smem + C::OFF_KV + idx % ST * C::TILE_BYTES;
          for (int e = max(w.to - (w.j0 + nmax - 1) * BN, 0) * 8 + lane; e < BN * 8; e += 32)
#pragma unroll
            for (int c = 0; c < C::NCHUNK; ++c) *reinterpret_cast<uint4*>(v + c * C::CHUNK_BYTES + e * 16) = make_uint4(0u, 0u, 0u, 0u);
          fence_proxy_async_smem();
          __syncwarp();
        }
        return true;
      };
      auto issue_s = [&](int t, int j) {
        const uint64_t a = dq0 + t * TILE16;
        const uint64_t b = dk0 + ((2 * j) % ST) * TILE16;
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < C::KSTEPS_QK; ++k)
            umma_ss(tmem + t * BN, a + kstep(k), b + kstep(k), idesc_qk, k > 0 ? 1u : 0u);
          umma_commit(bar(C::BAR_S + t));
        }
        __syncwarp();
      };
      auto issue_pv = [&](int t, int j) {
        const uint64_t b = dv0 + ((2 * j + 1) % ST) * TILE16;
        const uint32_t d = tmem + 256 + t * D;
        const uint32_t a = tmem + t * BN + C::COL_P;
        if (elect_one()) {
          umma_ts(d, a, b, idesc_pv, j > 0 ? 1u : 0u);
#pragma unroll
          for (int k = 1; k < C::KSTEPS_PV; ++k) umma_ts(d, a + k * 8, b + k * VSTEP16, idesc_pv, 1u);
          if (j == (t ? n1 : n0) - 1) umma_commit(bar(C::BAR_O + t));
        }
        __syncwarp();
      };
      for (int j = 0; j <= nmax && ok; ++j) {  // every wait is bounded
        if (j < nmax) {
          if (!wait_full(2 * j)) { ok = false; break; }
          tc_fence_after();
          if (j < n0) issue_s(0, j);
        }
        if (j >= 1 && j - 1 < n1) {
          if (j - 1 >= n0 && !wait_full(2 * (j - 1) + 1)) { ok = false; break; }
          if (!warp_wait(bar(C::BAR_P + 1), (j - 1) & 1)) { ok = false; break; }
          tc_fence_after();
          issue_pv(1, j - 1);
        }
        if (j >= 1) {
          if (elect_one()) umma_commit(bar(C::BAR_EMPTY + (2 * (j - 1) + 1) % ST));
          __syncwarp();
        }
        if (j < nmax) {
          if (j < n1) issue_s(1, j);
          if (elect_one()) umma_commit(bar(C::BAR_EMPTY + (2 * j) % ST));
          __syncwarp();
          if (j < n0) {
            if (!wait_full(2 * j + 1) || !warp_wait(bar(C::BAR_P + 0), j & 1)) { ok = false; break; }
            tc_fence_after();
            issue_pv(0, j);
          }
        }
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
    const int64_t pr = w.row0 + t * BM + row;  // packed row: query * heads + head
    const int tq = static_cast<int>(pr / heads);
    const bool row_ok = tq < w.nq;
    const int64_t orow = row_ok ? static_cast<int64_t>(w.q_lo + tq) * p.Hq + w.h * heads + (pr - static_cast<int64_t>(tq) * heads) : 0;
    const int64_t nrows = static_cast<int64_t>(p.num_queries) * p.Hq;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) << 5) << 16;
    const uint32_t tS = tmem + lane_off + t * BN;
    const uint32_t tP = tS + C::COL_P;
    const uint32_t tO = tmem + lane_off + 256 + t * D;
    const int n_t = t ? w.n[1] : w.n[0];
    const float sc = p.scale_log2;
    if (n_t > 0) {  // the thread's row of q, into the swizzled tile
      const bool in = row_ok && in_bounds(p.status, orow, nrows);
      const uint4* const src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) + orow * D);
      uint8_t* const dst = smem + t * C::TILE_BYTES + row * 128;
#pragma unroll
      for (int c = 0; c < C::NCHUNK; ++c) {
        uint4 x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = in ? __ldg(src + c * 8 + i) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int i = 0; i < 8; ++i) *reinterpret_cast<uint4*>(dst + c * C::CHUNK_BYTES + ((i ^ (row & 7)) << 4)) = x[i];
      }
      fence_proxy_async_smem();
      mbar_arrive(bar(C::BAR_Q + t));
    }
    int lim = 0;  // keys that the row sees
    if (row_ok) {
      const int i = w.q_lo + tq;
      lim = min(w.to, limit_of(p, PREFIX ? last_at_most(p.q_offsets, w.s0, w.s1, i) : w.s0, i));
    }
    const int least = __reduce_min_sync(0xffffffffu, row_ok ? lim : w.to);
    float m_run = -INFINITY, l_run = 0.f;
    bool failed = false;
    for (int j = 0; j < n_t; ++j) {
      const bool ok = mbar_wait(bar(C::BAR_S + t), j & 1);
      if (__any_sync(0xffffffffu, !ok)) { failed = true; break; }
      tc_fence_after();
      float s[128];
      {
        uint32_t sr[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(tS + 32 * c, sr[c]);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 128; ++i) s[i] = __uint_as_float(sr[i >> 5][i & 31]);
      }
      const int key0 = (w.j0 + j) * BN;
      if (key0 + BN > least || key0 < w.lo) {
#pragma unroll
        for (int i = 0; i < 128; ++i) {
          const int key = key0 + i;
          if (key >= lim || key < w.lo) s[i] = -INFINITY;
        }
      }
      float c0 = fmax3(s[0], s[1], s[2]), c1 = fmax3(s[3], s[4], s[5]);
      float c2 = fmax3(s[6], s[7], s[8]), c3 = fmax3(s[9], s[10], s[11]);
#pragma unroll
      for (int i = 12; i < 124; i += 8) {
        c0 = fmax3(c0, s[i], s[i + 1]);
        c1 = fmax3(c1, s[i + 2], s[i + 3]);
        c2 = fmax3(c2, s[i + 4], s[i + 5]);
        c3 = fmax3(c3, s[i + 6], s[i + 7]);
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
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        uint32_t pk[32];
#pragma unroll
        for (int c = 0; c < 32; c += 2) {
          const int i = 64 * hh + 2 * c;
          const float2 xa = ffma2(make_float2(s[i], s[i + 1]), make_float2(sc, sc), make_float2(neg_m, neg_m));
          const float2 xb = ffma2(make_float2(s[i + 2], s[i + 3]), make_float2(sc, sc), make_float2(neg_m, neg_m));
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
          for (int i = 0; i < 32; i += 2) {
            const float2 x = fmul2(make_float2(__uint_as_float(o[i]), __uint_as_float(o[i + 1])), make_float2(alpha, alpha));
            o[i] = __float_as_uint(x.x);
            o[i + 1] = __float_as_uint(x.y);
          }
          tmem_st32(tO + 32 * c, o);
        }
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(bar(C::BAR_P + t));
    }
    // ---------------------------------------------------------------- epilogue
    const bool have = n_t > 0;
    if (!failed && have) {
      const bool ok = mbar_wait(bar(C::BAR_O + t), 0);
      if (__any_sync(0xffffffffu, !ok)) failed = true;
    }
    if (failed) {
      if (lane == 0) fail();
    } else if (w.row0 + t * BM < unit_rows) {
      tc_fence_after();
      const bool row_in = row_ok && in_bounds(p.status, orow, nrows);
      if constexpr (PREFIX) {
        const int64_t at = w.part * nrows + orow;
        const bool ok = row_in && in_bounds(p.status, at, p.most_parts * nrows);
        float4* const dst = reinterpret_cast<float4*>(p.o) + at * (D / 4);
        if (have) {
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tmem_ld32(tO + 32 * c, o);
            tmem_wait_ld();
            if (ok) {
#pragma unroll
              for (int u = 0; u < 8; ++u)
                dst[c * 8 + u] = make_float4(__uint_as_float(o[4 * u]), __uint_as_float(o[4 * u + 1]),
                                             __uint_as_float(o[4 * u + 2]), __uint_as_float(o[4 * u + 3]));
            }
          }
        } else if (ok) {
          for (int u = 0; u < D / 4; ++u) dst[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        if (ok) p.ml[at] = make_float2(have ? m_run : -INFINITY, l_run);
      } else {
        asm volatile("griddepcontrol.wait;" ::: "memory");  // the prefix's parts
        const int parts = w.group >= 0 ? min(__ldcg(p.parts + w.group), p.most_parts) : 0;
        float M = have ? m_run : -INFINITY;
        for (int z = 0; z < parts; ++z)
          if (row_in) M = fmaxf(M, __ldcg(p.ml + z * nrows + orow).x);
        const float own = M == -INFINITY ? 0.f : fast_exp2(m_run - M);
        float sum = l_run * own;
        for (int z = 0; z < parts; ++z)
          if (row_in && M != -INFINITY) {
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
            for (int i = 0; i < 32; ++i) o[i] = 0u;
          }
          if (row_in) {
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * own);
            for (int z = 0; z < parts && M != -INFINITY; ++z) {
              const int64_t at = z * nrows + orow;
              const float f = fast_exp2(__ldcg(p.ml + at).x - M);
              const float4* const src = reinterpret_cast<const float4*>(p.o) + at * (D / 4) + c * 8;
#pragma unroll
              for (int u = 0; u < 8; ++u) {
                const float4 x = __ldcg(src + u);
                o[4 * u] = __float_as_uint(fmaf(f, x.x, __uint_as_float(o[4 * u])));
                o[4 * u + 1] = __float_as_uint(fmaf(f, x.y, __uint_as_float(o[4 * u + 1])));
                o[4 * u + 2] = __float_as_uint(fmaf(f, x.z, __uint_as_float(o[4 * u + 2])));
                o[4 * u + 3] = __float_as_uint(fmaf(f, x.w, __uint_as_float(o[4 * u + 3])));
              }
            }
            uint32_t pk[16];
#pragma unroll
            for (int i = 0; i < 16; ++i)
              pk[i] = pack2<BF16>(__uint_as_float(o[2 * i]) * inv, __uint_as_float(o[2 * i + 1]) * inv);
#pragma unroll
            for (int u = 0; u < 4; ++u)
              reinterpret_cast<uint4*>(dst + c * 64)[u] = make_uint4(pk[4 * u], pk[4 * u + 1], pk[4 * u + 2], pk[4 * u + 3]);
          }
        }
        if (row_in && p.lse) p.lse[orow] = live ? (M + log2f(sum)) * LN2 : (sum == 0.f ? -INFINITY : sum);
      }
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
cudaError_t launch_d(EncodeTiledFn enc, const Params& p, int* counters, int num_counters, cudaStream_t st) {
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
  // prefix stage: one item a CTA; cut or not, there are no more than this
  const int64_t ctas = PREFIX ? std::max<int64_t>(SMS, p.Hkv * ((p.num_queries * heads + ROWS - 1) / ROWS + p.num_groups))
                              : p.num_seqs * qblocks * p.Hkv;
  if (ctas == 0) return cudaSuccess;
  if (ctas > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(NUM_THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = PREFIX ? 0 : 1;
  return cudaLaunchKernelEx(&cfg, kern, tk, tv, p, SMS, static_cast<int>(qblocks), counters, num_counters);
}

template <bool BF16, bool PREFIX>
cudaError_t launch(EncodeTiledFn enc, const Params& p, int* counters, int num_counters, cudaStream_t st) {
  return p.D == 128 ? launch_d<128, BF16, PREFIX>(enc, p, counters, num_counters, st)
                    : launch_d<64, BF16, PREFIX>(enc, p, counters, num_counters, st);
}

}  // namespace tc
}  // namespace prefix
}  // namespace attn
