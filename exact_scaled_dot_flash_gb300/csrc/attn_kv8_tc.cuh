// attn_kv8_tc.cuh - attention over an 8-bit paged cache on the tcgen05 tensor
// cores, for calls with many rows (prompts and chunks of prompts; F16/BF16, D in
// {64, 128}, any page size).
//
// A CTA takes 256 packed rows (row = query * heads + head, the heads that share
// a kv head) of one sequence and kv head, as two tiles of 128, over all keys
// they see, 128 at a time:
//  - warps 8-11 convert. Each thread copies its share of a tile's codes ahead of
//    time (cp.async; it reads back only what it copied, so a page may end
//    anywhere and no barrier is needed), and writes them as F16, exactly, in the
//    128-byte swizzle that the tensor cores read (again, where it met one of
//    e4m3's two NaN codes); with K it leaves the tile's scales in shared memory.
//    A converted tile serves 256 rows;
//  - warp 12 issues S = Q K^T and O += P V in the order S_0 PV_1 S_1 PV_0, so
//    that each tile's softmax runs under the other's products;
//  - warps 0-7 own a row a thread: x = S ks scale in fp32, y = 2^(x - ref),
//    P = y vs rounded to F16 back into tensor memory, l += y. ref holds the
//    row's largest x + log2 vs, and moves only when that passes it by 2^8: the
//    row's largest P is 1 or more, whichever keys have the largest scores and
//    whichever the largest scales, and what F16 loses of those below 2^-14 is
//    small beside it. With a scale for each key, the largest score and the tile's
//    largest scale bound that sum where the tile's scales lie within a factor of
//    64 (such chunks, D 128, e4m3: 284 us, 316 with the sum for every key).
// The products are F16 for BF16 queries too: a row is brought into range by a
// power of two (see attn_kv8_decode.cuh).
// Where the row blocks do not fill the SMs (a few short chunks over long
// histories), their key tiles are cut into runs, one CTA each, whose unnormalised
// outputs merge_kernel combines.
// Bound: a step of 256 rows x 128 keys is 2048 cycles of the tensor pipe and some
// 3000 of shared memory (operands 1536, conversion 1024, scales), and takes some
// 4700: each row tile's softmax waits for its scores and the next products for
// its probabilities. 16 sequences, chunks of 128-512 tokens over 0.5k-4k keys,
// 32 / 8 heads, D 128, e4m3: 248 us, 756 TFLOP/s; 19 chunks of 512 over 4k: 1015.
// (Over a 16-bit cache, whose tiles need no conversion, the first take 180 us.)
#pragma once

#include <type_traits>

#include "kv8_fwd.h"
#include "kv8_ops.cuh"

namespace attn {
namespace kv8 {
namespace tc {

constexpr int BM = 128, BN = 128, NQ = 2;
constexpr int NUM_THREADS = 512;
constexpr int WARP_CONV = 8, CONV_WARPS = 4, WARP_MMA = 12;
constexpr int TMEM_COLS = 512;
// 512 threads start with 128 registers each: 2 x 128 x (REG_SOFTMAX + REG_OTHER) is
// the same sum. At D 128 the conversion of e4m3 spills with 64 (1.4% slower).
template <int D> constexpr int REG_SOFTMAX = D == 128 ? 184 : 192;
template <int D> constexpr int REG_OTHER = 256 - REG_SOFTMAX<D>;
constexpr float LN2 = 0.6931471805599453f;
constexpr float RESCALE_LOG2 = 8.0f;
constexpr float SPREAD = 64.f;
constexpr float SLACK_LOG2 = 7.f;   // a bound that takes the largest scale, below 2^vex, for one that is SPREAD times as small
constexpr float Y_RANGE = 80.f;     // y <= 2^(80 + 8 + 7): its sum over 2^31 keys is within fp32
constexpr float VS_LEAST = 8.271806125530277e-25f;  // 2^-Y_RANGE: smaller value scales count as this
constexpr float UNSEEN = -3e38f;    // reference of a row without keys: at the end of fp32's range, and finite

template <int D>
struct Cfg {
  static constexpr int NCHUNK = D / 64;                // 64 elements: one 128-byte row of the swizzle
  static constexpr int CHUNK_BYTES = BN * 128;
  static constexpr int TILE_BYTES = NCHUNK * CHUNK_BYTES;
  static constexpr int STAGES = 3;                     // converted tiles: K_j, V_j, K_j+1
  static constexpr int RAW = 3;                        // tiles of codes on their way
  static constexpr int RAW_BYTES = BN * D;
  static constexpr int SCALE_BYTES = 3 * BN * 4 + 32;  // ks, vs, log2 vs; the warps' largest and least vs
  static constexpr int OFF_KV = NQ * TILE_BYTES;
  static constexpr int OFF_RAW = OFF_KV + STAGES * TILE_BYTES;
  static constexpr int OFF_SCALE = OFF_RAW + RAW * RAW_BYTES;
  static constexpr int OFF_BAR = OFF_SCALE + 2 * SCALE_BYTES;
  static constexpr int BAR_FULL = 0, BAR_EMPTY = STAGES, BAR_Q = 2 * STAGES, BAR_S = BAR_Q + NQ;
  static constexpr int BAR_P = BAR_S + NQ, BAR_O = BAR_P + NQ, BAR_DONE = BAR_O + NQ;
  static constexpr int OFF_MISC = OFF_BAR + (BAR_DONE + 1) * 8;
  static constexpr int SMEM_BYTES = OFF_MISC + 16 + 1024;
  static_assert(SMEM_BYTES <= 227 * 1024);
  static constexpr int KSTEPS_QK = D / 16, KSTEPS_PV = BN / 16;
  static constexpr int COL_P = 64;
};

struct Work {
  int s, hk, sp, q_lo, nq, L;
  int j0;             // first key tile of the CTA's run
  int64_t row0;       // first packed row of the CTA
  int n[NQ], nmax;    // key tiles of each row tile
  int nfull[NQ];      // of which the first ones need no mask
};

// Item: kv head (fastest), run, row block, sequence.
__device__ __forceinline__ Work make_work(const FwdParams& p, int qblocks, int splits, int item) {
  Work w;
  const int heads = p.Hq / p.c.Hkv;
  w.hk = item % p.c.Hkv;
  item /= p.c.Hkv;
  w.sp = item % splits;
  item /= splits;
  // the last blocks of a sequence see the most keys and go first
  w.row0 = static_cast<int64_t>(qblocks - 1 - item % qblocks) * NQ * BM;
  w.s = item / qblocks;
  int hi;
  row_range(p.q_offsets, w.s, p.num_queries, w.q_lo, hi);
  w.nq = hi - w.q_lo;
  w.L = seq_len(p.c, w.s);
  w.nmax = 0;
#pragma unroll
  for (int t = 0; t < NQ; ++t) {
    const int64_t r0 = w.row0 + t * BM, rows = static_cast<int64_t>(w.nq) * heads;
    w.n[t] = w.nfull[t] = 0;
    if (r0 >= rows) continue;
    int64_t most = w.L, least = w.L;
    if (p.causal) {
      if (p.positions) {
        least = 0;  // any order: every tile is masked element by element
      } else {
        most = min(most, static_cast<int64_t>(w.L) - w.nq + min(static_cast<int64_t>(w.nq) - 1, (r0 + BM - 1) / heads) + 1);
        least = min(least, static_cast<int64_t>(w.L) - w.nq + r0 / heads + 1);
      }
    }
    w.n[t] = most > 0 ? static_cast<int>((most + BN - 1) / BN) : 0;
    w.nfull[t] = least > 0 ? static_cast<int>(least / BN) : 0;
    w.nmax = max(w.nmax, w.n[t]);
  }
  w.j0 = static_cast<int>(static_cast<int64_t>(w.nmax) * w.sp / splits);
  const int j1 = static_cast<int>(static_cast<int64_t>(w.nmax) * (w.sp + 1) / splits);
  w.nmax = j1 - w.j0;
#pragma unroll
  for (int t = 0; t < NQ; ++t) w.n[t] = max(0, min(w.n[t], j1) - w.j0);
  return w;
}

// Byte of 16-byte piece `c` (8 elements) of row r in a swizzled tile.
__device__ __forceinline__ uint32_t swizzled(int r, int c) {
  return (c >> 3) * (BN * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
}

// RUN: every 1, 4 or 16 keys share their scales (group, and so page_size, a
// multiple of it).
template <int D, int FMT, int RUN>
__global__ void __launch_bounds__(NUM_THREADS, 1) tc_kernel(const __grid_constant__ FwdParams p, int qblocks, int splits) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_dyn[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sb = smem_u32(smem);
  auto bar = [&](int i) -> uint32_t { return sb + C::OFF_BAR + 8 * i; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Cache& c = p.c;
  int* const status = c.status;
  const int heads = p.Hq / c.Hkv;
  const Work w = make_work(p, qblocks, splits, static_cast<int>(blockIdx.x));
  asm volatile("griddepcontrol.launch_dependents;");  // merge_kernel waits for this grid's end
  if (w.row0 >= static_cast<int64_t>(w.nq) * heads) return;  // no rows (CTA-uniform); rows without keys still get NaN

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(bar(C::BAR_FULL + s), CONV_WARPS * 32);
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
    if (status) atomicOr(status, STATUS_TIMEOUT);
  };

  if (warp >= WARP_CONV) {
    setmaxnreg_dec<REG_OTHER<D>>();
    if (warp < WARP_CONV + CONV_WARPS) {
      // ---------------------------------------------------------- conversion
      // Warp cw has keys 32 cw .. + 31 of a tile; a copy of the warp moves RPC
      // keys, D / 16 lanes each. Items: K_0 V_0 K_1 V_1 ... The lanes of a copy
      // are dealt out so that 8 neighbours, which a shared-memory store takes at
      // once, have 4 pieces each of two keys that differ in bit 0: 8 places of the
      // swizzle. The codes themselves lie in the lanes' order: a lane reads only
      // what it copied.
      constexpr int PIECES = D / 16, RPC = 32 / PIECES, COPIES = 32 / RPC;
      const int lpiece = (lane & 3) | (D == 128 ? (lane >> 1) & 4 : 0);
      const int lrow = D == 128 ? ((lane >> 2) & 1) | ((lane >> 3) & 2) : lane >> 2;
      const int cw = warp - WARP_CONV;
      const uint32_t step = static_cast<uint32_t>(c.Hkv) * D;
      const int64_t ntok = static_cast<int64_t>(c.num_pages) * c.page_size;
      const int64_t nscale = static_cast<int64_t>(c.num_pages) * c.Hkv * c.per;
      const uint8_t* const kb = p.k_codes + w.hk * D + lpiece * 16;
      const uint8_t* const vb = p.v_codes + w.hk * D + lpiece * 16;
      uint8_t* const raw = smem + C::OFF_RAW + cw * 32 * D;
      int tok = -1;        // the lane's key of the tile being copied, -1: zeros
      int64_t si = -1;     // its scales, -1: zeros
      float ks = 0.f, vs = 0.f, ks_next = 0.f, vs_next = 0.f;
      // The lane's key of the tile to copy next, and its page, which is read a
      // tile ahead of its use. Keys are looked up with K and used again for V.
      int key = w.j0 * BN + cw * 32 + lane, blk = key / c.page_size, row = key - blk * c.page_size;
      const int dblk = BN / c.page_size, drow = BN % c.page_size;
      const int32_t* const table = c.block_table + static_cast<size_t>(w.s) * c.max_pages;
      auto find_page = [&]() { return key < w.L && blk < c.max_pages ? __ldg(table + blk) : -1; };
      int page = find_page();
      auto look_up = [&]() {
        const bool ok = page >= 0 && page < c.num_pages && in_bounds(status, static_cast<int64_t>(page) * c.page_size + row, ntok);
        const int gi = c.group == 1 ? row : static_cast<int>(__umulhi(static_cast<uint32_t>(row), p.group_magic));
        tok = ok ? page * c.page_size + row : -1;
        si = ok ? (static_cast<int64_t>(page) * c.Hkv + w.hk) * c.per + gi : -1;
        if (si >= 0 && !in_bounds(status, si, nscale)) si = -1;
        key += BN;
        blk += dblk;
        row += drow;
        if (row >= c.page_size) {
          row -= c.page_size;
          ++blk;
        }
        page = find_page();
      };
      auto copy_item = [&](int it) {
        if (it < 2 * w.nmax) {
          if ((it & 1) == 0) {
            look_up();
            ks_next = si >= 0 ? __ldg(p.k_scale + si) : 0.f;
            vs_next = si >= 0 ? __ldg(p.v_scale + si) : 0.f;
          }
          const uint32_t at = smem_u32(raw) + (it % C::RAW) * C::RAW_BYTES;
          const uint8_t* const base = (it & 1) ? vb : kb;
#pragma unroll
          for (int i = 0; i < COPIES; ++i) {
            const int r = RPC * i + lrow;
            const int key = __shfl_sync(0xffffffffu, tok, r);
            copy16(at + (i * 32 + lane) * 16, base + static_cast<uint64_t>(static_cast<uint32_t>(max(key, 0))) * step,
                   key < 0 ? 0 : 16);
          }
        }
        copy_commit();
      };
      bool ok = true;
      copy_item(0);
      ks = ks_next;
      vs = vs_next;
      copy_item(1);
      for (int it = 0; it < 2 * w.nmax && ok; ++it) {
        const int st = it % C::STAGES, j = it >> 1;
        // the copies of item it + 2 take the place of item it - 1's, which this
        // thread has read; they bring the scales of tile j + 1 when it is K's turn
        copy_item(it + 2);
        copy_wait<2>();
        __syncwarp();
        if (!warp_wait(bar(C::BAR_EMPTY + st), ((it / C::STAGES) & 1) ^ 1)) { ok = false; break; }  // the whole warp
        const uint8_t* const src = raw + (it % C::RAW) * C::RAW_BYTES;
        uint8_t* const dst = smem + C::OFF_KV + st * C::TILE_BYTES;
        if ((it & 1) == 0) {
          // the softmax of tile j - 2 has read this slot: its P was used before
          // the converted tile that this one replaces (V_j-2) was released
          float* const sc = reinterpret_cast<float*>(smem + C::OFF_SCALE + (j & 1) * C::SCALE_BYTES);
          if (lane % RUN == 0) {
            sc[(cw * 32 + lane) / RUN] = ks * p.scale_log2;
            sc[BN + (cw * 32 + lane) / RUN] = vs;
            sc[2 * BN + (cw * 32 + lane) / RUN] = fmaxf(__log2f(vs), -Y_RANGE);  // a NaN counts as the least
          }
          if constexpr (RUN == 1) {
            // the bits of floats that are not negative are in their order; NaN does not
            // count, and keys behind the sequence's end are not among the least
            constexpr uint32_t MOST = 0x7f7fffffu;
            const uint32_t bits = __float_as_uint(vs);
            const bool there = (w.j0 + j) * BN + cw * 32 + lane < w.L;
            const uint32_t top = __reduce_max_sync(0xffffffffu, bits <= MOST ? bits : 0u);
            const uint32_t low = __reduce_min_sync(0xffffffffu, bits <= MOST && there ? bits : MOST);
            if (lane == 0) {
              sc[3 * BN + cw] = __uint_as_float(top);
              sc[3 * BN + CONV_WARPS + cw] = __uint_as_float(low);
            }
          }
        } else {
          ks = ks_next;
          vs = vs_next;
        }
        uint32_t bits = 0;  // a code leaves the low 7 bits of F16's mantissa clear, the NaN of 0x7f and 0xff sets them
#pragma unroll
        for (int i0 = 0; i0 < COPIES; i0 += 4) {
          uint4 x[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            x[i] = *reinterpret_cast<const uint4*>(src + ((i0 + i) * 32 + lane) * 16);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint4 a, b;
            pairs<FMT>(x[i].x, a.x, a.y);
            pairs<FMT>(x[i].y, a.z, a.w);
            pairs<FMT>(x[i].z, b.x, b.y);
            pairs<FMT>(x[i].w, b.z, b.w);
            if constexpr (FMT == FMT_E4M3) bits |= (a.x | a.y | a.z) | (a.w | b.x | b.y) | (b.z | b.w);
            const int r = cw * 32 + RPC * (i0 + i) + lrow;
            *reinterpret_cast<uint4*>(dst + swizzled(r, 2 * lpiece)) = a;
            *reinterpret_cast<uint4*>(dst + swizzled(r, 2 * lpiece + 1)) = b;
          }
        }
        if constexpr (FMT == FMT_E4M3) {
          if (bits & 0x007f007fu) {
#pragma unroll 1
            for (int i = 0; i < COPIES; ++i) {
              const uint4 x = *reinterpret_cast<const uint4*>(src + (i * 32 + lane) * 16);
              uint4 a, b;
              pairs<FMT, true>(x.x, a.x, a.y);
              pairs<FMT, true>(x.y, a.z, a.w);
              pairs<FMT, true>(x.z, b.x, b.y);
              pairs<FMT, true>(x.w, b.z, b.w);
              const int r = cw * 32 + RPC * i + lrow;
              *reinterpret_cast<uint4*>(dst + swizzled(r, 2 * lpiece)) = a;
              *reinterpret_cast<uint4*>(dst + swizzled(r, 2 * lpiece + 1)) = b;
            }
          }
        }
        fence_proxy_async_smem();
        mbar_arrive(bar(C::BAR_FULL + st));
      }
      copy_wait<0>();
      if (!ok && lane == 0) fail();
    } else if (warp == WARP_MMA) {
      // ---------------------------------------------------------- MMA issuer
      constexpr uint32_t idesc_qk = make_idesc_f16(false, BM, BN, false);
      constexpr uint32_t idesc_pv = make_idesc_f16(false, BM, D, true);
      constexpr int ST = C::STAGES;
      const int n0 = w.n[0], n1 = w.n[1], nmax = w.nmax;
      bool ok = true;
      for (int t = 0; t < NQ && ok; ++t)
        if ((t ? n1 : n0) > 0 && !warp_wait(bar(C::BAR_Q + t), 0)) ok = false;
      const uint64_t dq0 = smem_desc(sb, 16, 1024, 2u);
      const uint64_t dk0 = smem_desc(sb + C::OFF_KV, 16, 1024, 2u);
      const uint64_t dv0 = smem_desc(sb + C::OFF_KV, C::CHUNK_BYTES, 1024, 2u);
      constexpr uint32_t TILE16 = C::TILE_BYTES >> 4, CHUNK16 = C::CHUNK_BYTES >> 4, VSTEP16 = (16 * 128) >> 4;
      auto kstep = [](int k) -> uint32_t { return (k / 4) * CHUNK16 + (k % 4) * 2; };
      auto wait_full = [&](int idx) { return warp_wait(bar(C::BAR_FULL + idx % ST), (idx / ST) & 1); };
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
      for (int j = 0; j <= nmax && ok; ++j) {
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
    // ------------------------------------------------------------ softmax
    setmaxnreg_inc<REG_SOFTMAX<D>>();
    const int t = warp >> 2;
    const int row = ((warp & 3) << 5) + lane;
    const int64_t pr = w.row0 + t * BM + row;
    const int tq = static_cast<int>(pr / heads);
    const bool row_ok = tq < w.nq;
    const int64_t orow = row_ok ? static_cast<int64_t>(w.q_lo + tq) * p.Hq + w.hk * heads + (pr - static_cast<int64_t>(tq) * heads) : 0;
    const int64_t nrows = static_cast<int64_t>(p.num_queries) * p.Hq;
    const bool row_in = row_ok && in_bounds(status, orow, nrows);
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) << 5) << 16;
    const uint32_t tS = tmem + lane_off + t * BN;
    const uint32_t tP = tS + C::COL_P;
    const uint32_t tO = tmem + lane_off + 256 + t * D;
    const int n_t = t ? w.n[1] : w.n[0];
    const int nfull_t = t ? w.nfull[1] : w.nfull[0];
    // the thread's row of Q, as F16
    float back = 1.f;
    if (n_t > 0) {
      const uint4* const src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) + orow * D);
      uint4 x[D / 8];
#pragma unroll
      for (int i = 0; i < D / 8; ++i) x[i] = row_in ? __ldg(src + i) : make_uint4(0u, 0u, 0u, 0u);
      if (p.bf16) {
        uint32_t* const y = reinterpret_cast<uint32_t*>(x);
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < D / 2; ++i) top = fmaxf(top, finite_top(y[i]));
        const float f = f16_range(top, back);
#pragma unroll
        for (int i = 0; i < D / 2; ++i)
          y[i] = pack2<false>(__uint_as_float(y[i] << 16) * f, __uint_as_float(y[i] & 0xffff0000u) * f);
      }
#pragma unroll
      for (int i = 0; i < D / 8; ++i) *reinterpret_cast<uint4*>(smem + t * C::TILE_BYTES + swizzled(row, i)) = x[i];
      fence_proxy_async_smem();
      mbar_arrive(bar(C::BAR_Q + t));
    }
    int pos = -1;
    if (row_ok)
      pos = p.positions ? (in_bounds(status, w.q_lo + tq, p.num_queries) ? __ldg(p.positions + w.q_lo + tq) : -1)
                        : w.L - w.nq + tq;
    // last key the row sees; a position far below 0 must not pass 2^31 in the difference to a tile's first key
    const int lim = p.causal ? max(min(pos, w.L - 1), -1) : (row_ok ? w.L - 1 : -1);
    float ref = UNSEEN, l_run = 0.f;
    bool failed = false;
    for (int j = 0; j < n_t; ++j) {
      const bool ok = mbar_wait(bar(C::BAR_S + t), j & 1);
      if (__any_sync(0xffffffffu, !ok)) { failed = true; break; }
      tc_fence_after();
      const float4* const sk = reinterpret_cast<const float4*>(smem + C::OFF_SCALE + (j & 1) * C::SCALE_BYTES);
      const float4 *const sv = sk + BN / 4, *const sl = sv + BN / 4;
      // s: products times k_scale; with runs the products alone
      float s[128];
      {
        uint32_t sr[4][32];
#pragma unroll
        for (int i = 0; i < 4; ++i) tmem_ld32(tS + 32 * i, sr[i]);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const uint32_t* const x = &sr[i >> 3][(4 * i) & 31];
          float2 a = make_float2(__uint_as_float(x[0]), __uint_as_float(x[1]));
          float2 b = make_float2(__uint_as_float(x[2]), __uint_as_float(x[3]));
          if constexpr (RUN == 1) {
            const float4 k = sk[i];
            a = fmul2(a, make_float2(k.x, k.y));
            b = fmul2(b, make_float2(k.z, k.w));
          }
          s[4 * i] = a.x; s[4 * i + 1] = a.y; s[4 * i + 2] = b.x; s[4 * i + 3] = b.y;
        }
      }
      const bool masked = w.j0 + j >= nfull_t;
      if (masked) {
        const int end = lim - (w.j0 + j) * BN;
        asm volatile("");  // a branch, not 256 predicated instructions in every tile
#pragma unroll
        for (int i = 0; i < 128; ++i)
          if (i > end) s[i] = -INFINITY;
      }
      float c0 = -INFINITY, c1 = c0, c2 = c0, c3 = c0;
      if constexpr (RUN > 1) {  // scales are not negative: the largest product of a run gives its largest score
        auto run4 = [&](int i) { return fmaxf(fmax3(s[i], s[i + 1], s[i + 2]), s[i + 3]); };
        auto run = [&](int r) {
          if constexpr (RUN == 4) return run4(4 * r);
          else return fmaxf(fmax3(run4(16 * r), run4(16 * r + 4), run4(16 * r + 8)), run4(16 * r + 12));
        };
#pragma unroll
        for (int i = 0; i < BN / RUN / 4; ++i) {
          const float4 k = sk[i];
          const float4 e = sl[i];
          c0 = fmaxf(c0, fmaf(run(4 * i) * k.x, back, e.x));
          c1 = fmaxf(c1, fmaf(run(4 * i + 1) * k.y, back, e.y));
          c2 = fmaxf(c2, fmaf(run(4 * i + 2) * k.z, back, e.z));
          c3 = fmaxf(c3, fmaf(run(4 * i + 3) * k.w, back, e.w));
        }
      } else {
        const float4 vt = sl[BN / 4], vl = sl[BN / 4 + 1];
        const float vtop = fmaxf(fmax3(vt.x, vt.y, vt.z), vt.w), vlow = fminf(fminf(vl.x, vl.y), fminf(vl.z, vl.w));
        if (vtop > fmaxf(vlow, VS_LEAST) * SPREAD) {  // the same for the CTA's threads
          asm volatile("");
          const float2 b2 = make_float2(back, back);
#pragma unroll
          for (int i = 0; i < 128; i += 4) {
            const float4 e = sl[i / 4];
            const float2 xa = ffma2(make_float2(s[i], s[i + 1]), b2, make_float2(e.x, e.y));
            const float2 xb = ffma2(make_float2(s[i + 2], s[i + 3]), b2, make_float2(e.z, e.w));
            c0 = fmax3(c0, xa.x, xa.y);
            c1 = fmax3(c1, xb.x, xb.y);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 128; i += 8) {
            c0 = fmax3(c0, s[i], s[i + 1]);
            c1 = fmax3(c1, s[i + 2], s[i + 3]);
            c2 = fmax3(c2, s[i + 4], s[i + 5]);
            c3 = fmax3(c3, s[i + 6], s[i + 7]);
          }
          const float vex = static_cast<float>(static_cast<int>(__float_as_uint(vtop) >> 23) - 126);  // vtop < 2^vex
          c0 = fmax3(c0, c1, fmaxf(c2, c3)) * back + fmaxf(vex, -Y_RANGE);
          c1 = c2 = c3 = -INFINITY;
        }
      }
      const float x_tile = fmax3(c0, c1, fmaxf(c2, c3)) - (RUN == 1 ? SLACK_LOG2 : 0.f);
      const bool need = x_tile > ref + RESCALE_LOG2;
      float alpha = 1.f;
      if (need) {
        alpha = fast_exp2(ref - x_tile);
        ref = x_tile;
        l_run *= alpha;
      }
      const float neg = -ref;
      float2 sum_a = make_float2(0.f, 0.f), sum_b = make_float2(0.f, 0.f);
      auto probabilities = [&](auto mask) {
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          uint32_t pk[32];
#pragma unroll
          for (int i2 = 0; i2 < 32; i2 += 2) {
            const int i = 64 * hh + 2 * i2;
            float4 v;
            float kb = back;
            if constexpr (RUN > 1) {
              auto pick = [&](const float4* f) {  // of the run that key i lies in
                const float4 x = f[i / RUN / 4];
                return i / RUN % 4 == 0 ? x.x : i / RUN % 4 == 1 ? x.y : i / RUN % 4 == 2 ? x.z : x.w;
              };
              kb *= pick(sk);
              const float vr = pick(sv);
              v = make_float4(vr, vr, vr, vr);
            } else {
              v = sv[i >> 2];
            }
            float2 xa = ffma2(make_float2(s[i], s[i + 1]), make_float2(kb, kb), make_float2(neg, neg));
            float2 xb = ffma2(make_float2(s[i + 2], s[i + 3]), make_float2(kb, kb), make_float2(neg, neg));
            if constexpr (RUN > 1 && decltype(mask)::value) {
              xa.x = s[i] == -INFINITY ? -INFINITY : xa.x;
              xa.y = s[i + 1] == -INFINITY ? -INFINITY : xa.y;
              xb.x = s[i + 2] == -INFINITY ? -INFINITY : xb.x;
              xb.y = s[i + 3] == -INFINITY ? -INFINITY : xb.y;
            }
            const float2 ya = make_float2(fast_exp2(xa.x), fast_exp2(xa.y));
            const float2 yb = make_float2(fast_exp2(xb.x), fast_exp2(xb.y));
            sum_a = fadd2(sum_a, ya);
            sum_b = fadd2(sum_b, yb);
            float2 za = fmul2(ya, make_float2(v.x, v.y)), zb = fmul2(yb, make_float2(v.z, v.w));
            if constexpr (decltype(mask)::value) {  // a masked key may have any scale
              za.x = s[i] == -INFINITY ? 0.f : za.x;
              za.y = s[i + 1] == -INFINITY ? 0.f : za.y;
              zb.x = s[i + 2] == -INFINITY ? 0.f : zb.x;
              zb.y = s[i + 3] == -INFINITY ? 0.f : zb.y;
            }
            pk[i2] = pack2<false>(za.x, za.y);
            pk[i2 + 1] = pack2<false>(zb.x, zb.y);
          }
          tmem_st32(tP + 32 * hh, pk);
        }
      };
      if (masked) probabilities(std::true_type());
      else probabilities(std::false_type());
      l_run += (sum_a.x + sum_a.y) + (sum_b.x + sum_b.y);
      if (j > 0 && __any_sync(0xffffffffu, need)) {
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          uint32_t o[32];
          tmem_ld32(tO + 32 * i, o);
          tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < 32; k += 2) {
            const float2 x = fmul2(make_float2(__uint_as_float(o[k]), __uint_as_float(o[k + 1])), make_float2(alpha, alpha));
            o[k] = __float_as_uint(x.x);
            o[k + 1] = __float_as_uint(x.y);
          }
          tmem_st32(tO + 32 * i, o);
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
    } else if (w.row0 + t * BM < static_cast<int64_t>(w.nq) * heads) {
      tc_fence_after();
      const bool live = have && l_run > 0.f;
      const float inv = splits > 1 ? 1.f : live ? 1.f / l_run : __int_as_float(0x7fc00000);
      const int64_t prow = static_cast<int64_t>(w.sp) * nrows + orow;  // of the run's partials
      uint8_t* const dst = static_cast<uint8_t*>(p.out) + orow * D * 2;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        uint32_t o[32];
        if (have) {
          tmem_ld32(tO + 32 * i, o);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = 0u;
        }
        if (row_in && splits > 1) {
          if (have && in_bounds(status, prow, splits * nrows)) {
            float4* const part = static_cast<float4*>(p.ws) + prow * (D / 4) + i * 8;
#pragma unroll
            for (int u = 0; u < 8; ++u)
              part[u] = make_float4(__uint_as_float(o[4 * u]), __uint_as_float(o[4 * u + 1]), __uint_as_float(o[4 * u + 2]),
                                    __uint_as_float(o[4 * u + 3]));
          }
        } else if (row_in) {
          uint32_t pk[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const float2 x = fmul2(make_float2(__uint_as_float(o[2 * k]), __uint_as_float(o[2 * k + 1])), make_float2(inv, inv));
            pk[k] = pack_out(p.bf16, x.x, x.y);
          }
#pragma unroll
          for (int u = 0; u < 4; ++u)
            reinterpret_cast<uint4*>(dst + i * 64)[u] = make_uint4(pk[4 * u], pk[4 * u + 1], pk[4 * u + 2], pk[4 * u + 3]);
        }
      }
      if (splits > 1) {
        if (row_in && in_bounds(status, prow, splits * nrows))
          reinterpret_cast<float2*>(static_cast<float4*>(p.ws) + splits * nrows * (D / 4))[prow] =
              make_float2(l_run == 0.f ? -INFINITY : ref, l_run);
      } else if (row_in && p.lse) p.lse[orow] = live ? (ref + log2f(l_run)) * LN2 : (l_run == 0.f ? -INFINITY : l_run);
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

// A warp combines the runs of one row: partials (ref, l, O) of `splits` runs.
constexpr int MERGE_WARPS = 8;

template <int D>
__global__ void __launch_bounds__(MERGE_WARPS * 32) merge_kernel(const __grid_constant__ FwdParams p, int qblocks, int splits) {
  const Work w = make_work(p, qblocks, 1, static_cast<int>(blockIdx.x));
  const int heads = p.Hq / p.c.Hkv, lane = threadIdx.x & 31;
  const int64_t pr = w.row0 + static_cast<int64_t>(blockIdx.y) * MERGE_WARPS + (threadIdx.x >> 5);
  asm volatile("griddepcontrol.wait;" ::: "memory");  // also without rows: this grid ends after tc_kernel's
  if (pr >= static_cast<int64_t>(w.nq) * heads) return;
  const int tq = static_cast<int>(pr / heads);
  const int64_t orow = static_cast<int64_t>(w.q_lo + tq) * p.Hq + w.hk * heads + (pr - static_cast<int64_t>(tq) * heads);
  const int64_t nrows = static_cast<int64_t>(p.num_queries) * p.Hq;
  if (!in_bounds(p.c.status, orow, nrows)) return;
  const float4* const wo = static_cast<const float4*>(p.ws);
  const float2* const wml = reinterpret_cast<const float2*>(wo + splits * nrows * (D / 4));
  const float2 ml = lane < splits ? wml[lane * nrows + orow] : make_float2(-INFINITY, 0.f);
  float M = ml.x;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  const bool has_keys = ml.x != -INFINITY;  // a run without keys wrote no output
  const unsigned runs = __ballot_sync(0xffffffffu, has_keys);
  const float f = has_keys ? fast_exp2(ml.x - M) : 0.f;
  float sum = f == 0.f ? 0.f : f * ml.y;
  if (ml.y != ml.y) sum = ml.y;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  constexpr int V = D / 32;  // floats of a lane
  float acc[V] = {};
#pragma unroll 4
  for (int s = 0; s < splits; ++s) {
    const float fs = __shfl_sync(0xffffffffu, f, s);
    if (!(runs >> s & 1)) continue;  // warp-uniform; a weight of 0 is added too: 0 * NaN
    const float* const src = reinterpret_cast<const float*>(wo) + (s * nrows + orow) * D + lane * V;
#pragma unroll
    for (int k = 0; k < V; ++k) acc[k] = fmaf(fs, src[k], acc[k]);
  }
  const bool live = sum > 0.f;
  const float inv = live ? 1.f / sum : __int_as_float(0x7fc00000);
  uint32_t* const dst = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + orow * D) + lane * V / 2;
#pragma unroll
  for (int k = 0; k < V; k += 2) dst[k / 2] = pack_out(p.bf16, acc[k] * inv, acc[k + 1] * inv);
  if (p.lse && lane == 0) p.lse[orow] = live ? (M + log2f(sum)) * LN2 : (sum == 0.f ? -INFINITY : sum);
}

template <int D, int FMT, int RUN>
cudaError_t launch_run(const FwdParams& p, cudaStream_t st) {
  const int64_t qblocks = tc_qblocks(p.max_queries, p.Hq / p.c.Hkv);
  const int splits = tc_splits(p.c.num_seqs, p.c.Hkv, qblocks, p.c.max_pages, p.c.page_size);
  const int64_t blocks = static_cast<int64_t>(p.c.num_seqs) * qblocks * p.c.Hkv;
  if (blocks == 0) return cudaSuccess;
  if (blocks * splits > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  auto kern = tc_kernel<D, FMT, RUN>;
  constexpr int smem = Cfg<D>::SMEM_BYTES;
  static std::atomic<unsigned long long> configured{0};
  cudaError_t e = allow_smem(kern, smem, p.device, configured);
  if (e != cudaSuccess) return e;
  kern<<<static_cast<unsigned>(blocks * splits), NUM_THREADS, smem, st>>>(p, static_cast<int>(qblocks), splits);
  e = cudaGetLastError();
  if (e != cudaSuccess || splits == 1) return e;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks), NQ * BM / MERGE_WARPS);
  cfg.blockDim = dim3(MERGE_WARPS * 32);
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, merge_kernel<D>, p, static_cast<int>(qblocks), splits);
}

template <int D, int FMT>
cudaError_t launch_d(const FwdParams& p, cudaStream_t st) {
  // Scales are read once a run: 16 or 4 instead of 64 vector loads for a row and
  // tile (the chunks above: 257 us with runs of 4, 241 of 16).
  return p.c.group % 16 == 0  ? launch_run<D, FMT, 16>(p, st)
         : p.c.group % 4 == 0 ? launch_run<D, FMT, 4>(p, st)
                              : launch_run<D, FMT, 1>(p, st);
}

}  // namespace tc

template <int FMT>
cudaError_t launch_tc(const FwdParams& p, cudaStream_t st) {
  return p.c.D == 128 ? tc::launch_d<128, FMT>(p, st) : tc::launch_d<64, FMT>(p, st);
}

}  // namespace kv8
}  // namespace attn
