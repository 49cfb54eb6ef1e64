// attn_kv8_decode.cuh - attention over an 8-bit paged cache for calls with few
// rows (queries x heads of a kv head, at most 32 a CTA and 64 a call): decode
// steps and drafted tokens (F16/BF16, D in {64, 128}).
//
// Measured: 64 sequences of 1k-8k keys, 32 / 8 heads, D 128, e4m3: 112 us, 5.75 TB/s
// (85% of the copy bandwidth); one row of 130k keys, int8: 61 us, 4.4 TB/s; 35 rows
// of 12 sequences: 82 us, 1.7 TB/s (two row groups convert the codes twice; the
// instructions are the bound from 16 rows on; 25 to 32 rows at D 128 spill).
//
// Bound: the bytes of the codes, read once for all the rows of a kv head. At
// the copy bandwidth an SM is fed 21 bytes a cycle, and each byte has to become
// a 16-bit operand, so what the kernel economises is instructions and
// shared-memory traffic per byte:
//  - a warp streams its own 32-key tiles through two buffers of cp.async copies in
//    shared memory (no barrier between warps), reads each code once into
//    registers, converts it there and feeds it to mma.sync as the A operand: 2
//    bytes of shared-memory traffic for a byte of cache (a 16-bit tcgen05 operand
//    would be written once and read twice, 6 bytes of it), and 8 columns for the
//    query rows instead of 128;
//  - S^T = K Q^T (keys x rows), then O^T = V^T P^T. The order of the head's
//    elements inside a 16-element step of S^T, and of the rows of O^T, is free,
//    so that a lane's operands are 16 consecutive bytes of one key; V^T wants
//    two keys in one register, which the byte permutation of the conversion
//    gives without an instruction of its own; P^T is S^T transposed, one
//    movmatrix for 8 keys x 8 rows;
//  - the products are F16 whatever the type of q: every code is exact in F16, a
//    BF16 query is brought to F16's range by a power of two for its row (what
//    falls below 2^-24 there is 2^-40 of the row's largest element), and the
//    probabilities get 11 bits instead of 8. Codes convert exactly: int8 by
//    placing the byte, offset by 128, under the exponent of 1024 and
//    subtracting; e4m3 by the conversion instruction (its two NaN codes: a
//    warp that meets a NaN takes its keys again);
//  - k_scale enters the score in fp32, v_scale the probability before it is
//    rounded. A row has one reference exponent for both: with y = 2^(x - ref),
//    l = sum y and P' = y v_scale, and ref moves up when a P' passes 2^8 (one vote
//    a tile instead of a reduction), to bring the largest p v_scale so far near 1.
//    What F16 loses below 2^-14 is then small beside the largest term of the sum,
//    whatever the scales of other keys.
//
// Work: the keys of all sequences, in blocks of 128 (32 a warp), are cut into
// ranges, one for each group of Hkv CTAs (one CTA a head, side by side, since
// their codes lie side by side). A CTA walks the sequences of its range;
// a sequence wholly inside it is written out, a cut one as a partial (m, l, O).
// The CTA that finishes a cut sequence's last part (a counter that zero_kernel
// has cleared) combines all of them, in the order of the ranges, whichever CTA
// that is: the result does not depend on who came last. Sequences of at most 512
// keys are not cut: a CTA each (and head), no counters, no workspace.
#pragma once

#include <type_traits>

#include "kv8_fwd.h"
#include "kv8_ops.cuh"

namespace attn {
namespace kv8 {
namespace dec {

constexpr int WARPS = 4;
constexpr int THREADS = WARPS * 32;
constexpr int TILE_KEYS = 32;
constexpr int BLOCK_KEYS = TILE_KEYS * WARPS;
constexpr float LN2 = 0.6931471805599453f;
constexpr float Y_RANGE = 80.f;     // y <= 2^80: below it a row of tiny value scales still fills F16
constexpr float UNSEEN = -3e38f;    // reference of a row without keys: its first one passes every range

__device__ __forceinline__ int blocks_of(int nq, int L) {
  return nq > 0 ? max(1, (L + BLOCK_KEYS - 1) / BLOCK_KEYS) : 0;  // without keys: one, for the NaN rows
}

__device__ __forceinline__ int blocks_of(const FwdParams& p, int s) {
  int lo, hi;
  row_range(p.q_offsets, s, p.num_queries, lo, hi);
  return blocks_of(hi - lo, seq_len(p.c, s));
}

// First block of range r.
__device__ __forceinline__ int64_t cut(int64_t total, int r, int ranges) { return total * r / ranges; }

// Blocks of all sequences; the sequence s that the first block of a range lies in,
// and that sequence's first block.
struct Place {
  int64_t total, at;
  int s;
};

// The whole CTA calls it.
__device__ __forceinline__ Place locate(const FwdParams& p, int range, int ranges, int64_t& u0, int64_t& u1) {
  constexpr int N = THREADS;
  __shared__ int64_t warp_sum[N / 32];
  __shared__ int64_t found_at;
  __shared__ int found_s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (p.c.num_seqs + N - 1) / N;
  const int s0 = min(tid * per, p.c.num_seqs), s1 = min(s0 + per, p.c.num_seqs);
  int64_t mine = 0;
  for (int s = s0; s < s1; ++s) mine += blocks_of(p, s);
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  if (lane == 31) warp_sum[warp] = incl;
  if (tid == 0) {
    found_at = 0;
    found_s = 0;
  }
  __syncthreads();
  int64_t before = incl - mine, total = 0;
#pragma unroll
  for (int w = 0; w < N / 32; ++w) {
    if (w < warp) before += warp_sum[w];
    total += warp_sum[w];
  }
  u0 = cut(total, range, ranges);
  u1 = cut(total, range + 1, ranges);
  if (u0 >= before && u0 < before + mine) {
    int s = s0;
    int64_t at = before;
    for (; s < s1; ++s) {
      const int n = blocks_of(p, s);
      if (u0 < at + n) break;
      at += n;
    }
    found_at = at;
    found_s = s;
  }
  __syncthreads();
  return Place{total, found_at, found_s};
}

// ------------------------------------------------------------------ operands
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

// Where 16-byte piece `c` of row r of a tile is kept (in pieces), so that the
// lanes of a read fall on different banks: K is read as rows 4 (g/2) + g%2 and
// pieces 4 i + t, V as rows 4 t + i and pieces (D 64: half pieces) g.
template <int D>
__device__ __forceinline__ int k_piece(int r, int c) {
  return D == 128 ? r * 8 + (c ^ ((r & 1) << 2)) : r * 4 + c;
}
template <int D>
__device__ __forceinline__ int v_piece(int r, int c) {
  return D == 128 ? r * 8 + (c ^ ((r >> 1) & 6)) : ((r & ~1) | ((r ^ (r >> 2)) & 1)) * 4 + (c ^ ((r >> 2) & 2));
}

template <int D, int NT>
struct Shared {
  static constexpr int STAGES = 2;
  static constexpr int TILE = TILE_KEYS * D;           // K or V codes of a tile
  static constexpr int STAGE = 2 * TILE + 8 * TILE_KEYS;  // both, and their scales
  static constexpr int RING = WARPS * STAGES * STAGE;
  static constexpr int ROW = D + 4;
  static constexpr int O = WARPS * 8 * NT * ROW * 4;   // partial outputs of the warps, in the ring's place
  static constexpr int OFF_ML = RING > O ? RING : O;
  static constexpr int OFF_QF = OFF_ML + WARPS * 8 * NT * 8;
  static constexpr int OFF_Q = OFF_QF + 8 * NT * 4;    // query operands, in the lanes' order
  static constexpr int BYTES = OFF_Q + NT * (D / 16) * 32 * 8;
};

// Rows of a call: `rows` in all, in blockIdx.y groups of 8 NT; a slot of the
// workspace holds all groups (slot_rows).
template <int D, int FMT, int NT>
__global__ void __launch_bounds__(THREADS, NT <= 2 ? 3 : 2)
    decode_kernel(const __grid_constant__ FwdParams p, int ranges, int aligned, int slot_rows, int64_t ml_offset,
                  int* counters) {
  constexpr int KS = D / 16;    // 16-element steps of a head
  constexpr int KB = D / 64;    // 64-byte pieces of a key
  constexpr int VW = D / 32;    // words of V a lane holds of one key
  constexpr int ROWS = 8 * NT;
  using SH = Shared<D, NT>;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ bool last_part;
  float* const so = reinterpret_cast<float*>(smem);
  float2* const sml = reinterpret_cast<float2*>(smem + SH::OFF_ML);
  float* const sqf = reinterpret_cast<float*>(smem + SH::OFF_QF);  // the rows' inverse powers of two
  uint2* const sq = reinterpret_cast<uint2*>(smem + SH::OFF_Q);

  const Cache& c = p.c;
  int* const status = c.status;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int h = blockIdx.x % c.Hkv, range = blockIdx.x / c.Hkv;
  const int row_lo = blockIdx.y * ROWS;
  const int heads = p.Hq / c.Hkv;
  const bool bf16 = p.bf16;
  const uint32_t step = static_cast<uint32_t>(c.Hkv) * D;  // bytes from token to token
  const int64_t ntok = static_cast<int64_t>(c.num_pages) * c.page_size;
  const int64_t nscale = static_cast<int64_t>(c.num_pages) * c.Hkv * c.per;
  const int64_t nrows = static_cast<int64_t>(p.num_queries) * p.Hq;
  constexpr int PIECES = D / 16;             // 16-byte pieces of a key
  constexpr int RPC = 32 / PIECES;           // keys that one copy of the warp covers
  const uint8_t* const kb = p.k_codes + h * D + lane % PIECES * 16;
  const uint8_t* const vb = p.v_codes + h * D + lane % PIECES * 16;
  uint8_t* const ring = smem + (threadIdx.x >> 5) * SH::STAGES * SH::STAGE;
  const uint32_t ring_at = smem_u32(ring);
  const bool tiles_in_page = c.page_size % TILE_KEYS == 0;
  const int dblk = BLOCK_KEYS / c.page_size, drow = BLOCK_KEYS % c.page_size;

  int64_t u0 = 0, u1 = 0;
  Place pl{0, 0, range};
  if (aligned) u1 = blocks_of(p, range);  // the range is one sequence
  else pl = locate(p, range, ranges, u0, u1);
  int s = pl.s;
  int b = static_cast<int>(u0 - pl.at);
  for (int64_t u = u0; u < u1; ++s, b = 0) {
    int q_lo, q_hi;
    row_range(p.q_offsets, s, p.num_queries, q_lo, q_hi);
    const int nq = q_hi - q_lo, L = seq_len(c, s);
    const int nb = blocks_of(nq, L);
    if (nb == 0) continue;
    const int take = static_cast<int>(min(static_cast<int64_t>(nb - b), u1 - u));
    const bool first = u == u0, whole = take == nb;
    u += take;
    const int R = static_cast<int>(min(static_cast<int64_t>(nq) * heads - row_lo, static_cast<int64_t>(ROWS)));
    if (R <= 0) continue;  // CTA-uniform
    auto row_at = [&](int row) {  // row of the call's [queries, Hq]
      const int q = (row_lo + row) / heads;
      return static_cast<int64_t>(q_lo + q) * p.Hq + h * heads + (row_lo + row - q * heads);
    };

    // ------------------------------------------------ query rows
    // Row 8 w + g by warp w, its elements in the lanes' order: lane t holds
    // elements 64 i + 16 t .. + 15, two registers for each of 4 steps.
    if (warp < NT) {
      uint32_t r[KB][8];
      const int row = 8 * warp + g;
#pragma unroll
      for (int i = 0; i < KB; ++i) {
        uint4 x = make_uint4(0u, 0u, 0u, 0u), y = x;
        if (row < R) {
          const int64_t at = row_at(row);
          if (in_bounds(status, at, nrows)) {
            const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) + at * D + i * 64 + t * 16);
            x = __ldg(src);
            y = __ldg(src + 1);
          }
        }
        r[i][0] = x.x; r[i][1] = x.y; r[i][2] = x.z; r[i][3] = x.w;
        r[i][4] = y.x; r[i][5] = y.y; r[i][6] = y.z; r[i][7] = y.w;
      }
      float back = 1.f;
      if (bf16) {
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < KB; ++i)
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            top = fmaxf(top, finite_top(r[i][k]));
          }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const float f = f16_range(top, back);
#pragma unroll
        for (int i = 0; i < KB; ++i)
#pragma unroll
          for (int k = 0; k < 8; ++k)
            r[i][k] = pack2<false>(__uint_as_float(r[i][k] << 16) * f, __uint_as_float(r[i][k] & 0xffff0000u) * f);
      }
      if (t == 0) sqf[row] = back;
#pragma unroll
      for (int i = 0; i < KB; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) sq[(warp * KS + 4 * i + k) * 32 + lane] = make_uint2(r[i][2 * k], r[i][2 * k + 1]);
    }
    __syncthreads();
    uint32_t qf[NT == 1 ? KS : 1][2];
    if constexpr (NT == 1) {
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        const uint2 w = sq[k * 32 + lane];
        qf[k][0] = w.x;
        qf[k][1] = w.y;
      }
    }
    int lim[NT][2];     // last key that the lane's rows (8 i + 2 t, + 1) see
    float back[NT][2];  // and their inverse powers of two
    int least = L - 1, most = -1;
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = 8 * i + 2 * t + e;
        back[i][e] = sqf[row];
        int x = -1;
        if (row < R) {
          x = L - 1;
          if (p.causal) {
            const int q = (row_lo + row) / heads;
            const int pos = p.positions ? (in_bounds(status, q_lo + q, p.num_queries) ? __ldg(p.positions + q_lo + q) : -1)
                                        : L - nq + q;
            x = min(x, pos);
          }
          least = min(least, x);
          most = max(most, x);
        }
        lim[i][e] = x;
      }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      least = min(least, __shfl_xor_sync(0xffffffffu, least, o));
      most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
    }

    // ------------------------------------------------ keys
    // Of a row: y = 2^(x - ref) for a score x (log2 units), l the lane's part of
    // the sum of y, acc the sum of P' = y v_scale times the codes.
    float ref[NT][2], l[NT][2], acc[KS][NT][4];
    auto stream = [&](auto every) {
      constexpr bool EVERY = decltype(every)::value;
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        ref[i][0] = ref[i][1] = UNSEEN;
        l[i][0] = l[i][1] = 0.f;
#pragma unroll
        for (int k = 0; k < KS; ++k) acc[k][i][0] = acc[k][i][1] = acc[k][i][2] = acc[k][i][3] = 0.f;
      }
      // Lane (g, t): keys ka and ka + 2 of each 16 of a tile in S^T, 4 t .. 4 t + 3 in V^T
      const int ka = 4 * (g >> 1) + (g & 1);
      const int last_key = min(most + 1, (b + take) * BLOCK_KEYS);
      int key0 = b * BLOCK_KEYS + warp * TILE_KEYS;
      // The tile to copy next; a lane has one of its keys. The page is looked up
      // one tile ahead of the copy.
      int ckey = key0, blk = key0 / c.page_size, row0 = key0 - blk * c.page_size;
      auto find_page = [&]() {
        if (ckey + lane >= L) return -1;
        return page_of(c, s, tiles_in_page ? blk : blk + (row0 + lane) / c.page_size);
      };
      int page = find_page();
      auto copy_tile = [&](int stage) {
        if (ckey < last_key) {
          int row = row0 + lane;
          if (!tiles_in_page) row %= c.page_size;
          const int tok = page * c.page_size + row;
          const bool ok = page >= 0 && in_bounds(status, tok, ntok);
          const int mine = ok ? tok : -1;  // -1: zeros
          const int gi = c.group == 1 ? row : static_cast<int>(__umulhi(static_cast<uint32_t>(row), p.group_magic));
          const int64_t si = ok ? (static_cast<int64_t>(page) * c.Hkv + h) * c.per + gi : 0;
          const int bytes = ok && in_bounds(status, si, nscale) ? 4 : 0;
          const uint32_t at = ring_at + stage * SH::STAGE;
          copy4(at + 2 * SH::TILE + lane * 4, p.k_scale + (bytes ? si : 0), bytes);
          copy4(at + 2 * SH::TILE + 4 * TILE_KEYS + lane * 4, p.v_scale + (bytes ? si : 0), bytes);
#pragma unroll
          for (int j = 0; j < TILE_KEYS / RPC; ++j) {
            const int r = RPC * j + lane / PIECES;
            const int key = __shfl_sync(0xffffffffu, mine, r), n = key < 0 ? 0 : 16;
            const uint64_t off = static_cast<uint64_t>(static_cast<uint32_t>(max(key, 0))) * step;
            copy16(at + k_piece<D>(r, lane % PIECES) * 16, kb + off, n);
            copy16(at + SH::TILE + v_piece<D>(r, lane % PIECES) * 16, vb + off, n);
          }
        }
        copy_commit();
        ckey += BLOCK_KEYS;
        blk += dblk;
        row0 += drow;
        if (row0 >= c.page_size) {
          row0 -= c.page_size;
          ++blk;
        }
        page = find_page();
      };
#pragma unroll
      for (int i = 0; i < SH::STAGES - 1; ++i) copy_tile(i);
      int stage = 0;
      for (; key0 < last_key; key0 += BLOCK_KEYS) {
        copy_wait<SH::STAGES - 2>();
        __syncwarp();  // the tile's copies of every lane; and every lane is done with the tile before
        copy_tile(stage == 0 ? SH::STAGES - 1 : stage - 1);
        const uint8_t* const at = ring + stage * SH::STAGE;
        stage = stage == SH::STAGES - 1 ? 0 : stage + 1;
        const float* const scales = reinterpret_cast<const float*>(at + 2 * SH::TILE);
        float sc[2][NT][4], vs[2][2];
        const bool masked = key0 + TILE_KEYS - 1 > least;
#pragma unroll
        for (int u = 0; u < 2; ++u) {  // 16 keys
          uint32_t kr[2][KB * 4];
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int i = 0; i < KB; ++i) {
              const uint4 x = reinterpret_cast<const uint4*>(at)[k_piece<D>(16 * u + ka + 2 * e, 4 * i + t)];
              kr[e][4 * i] = x.x; kr[e][4 * i + 1] = x.y; kr[e][4 * i + 2] = x.z; kr[e][4 * i + 3] = x.w;
            }
#pragma unroll
          for (int i = 0; i < NT; ++i) sc[u][i][0] = sc[u][i][1] = sc[u][i][2] = sc[u][i][3] = 0.f;
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            uint32_t a0, a1, a2, a3;
            pairs<FMT, EVERY>(kr[0][k], a0, a2);
            pairs<FMT, EVERY>(kr[1][k], a1, a3);
#pragma unroll
            for (int i = 0; i < NT; ++i) {
              if constexpr (NT == 1) {
                mma16816(sc[u][i], a0, a1, a2, a3, qf[k][0], qf[k][1]);
              } else {
                const uint2 w = sq[(i * KS + k) * 32 + lane];
                mma16816(sc[u][i], a0, a1, a2, a3, w.x, w.y);
              }
            }
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float f = scales[16 * u + ka + 2 * e] * p.scale_log2;
            vs[u][e] = scales[TILE_KEYS + 16 * u + ka + 2 * e];
#pragma unroll
            for (int i = 0; i < NT; ++i) {
              sc[u][i][2 * e] *= f;
              sc[u][i][2 * e + 1] *= f;
            }
          }
          if (masked) {
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (key0 + 16 * u + ka + (e & 2) > lim[i][e & 1]) sc[u][i][e] = -INFINITY;
          }
        }
        // y and P' against the rows' references
        float z[2][NT][4], d[NT][2];
        auto against = [&](int i) {
#pragma unroll
          for (int e = 0; e < 2; ++e) d[i][e] = 0.f;
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float y = fast_exp2(fmaf(sc[u][i][e], back[i][e & 1], -ref[i][e & 1]));
              d[i][e & 1] += y;
              z[u][i][e] = y * vs[u][e >> 1];
            }
        };
        float big = 0.f;
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          against(i);
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            big = fmax3(big, z[u][i][0], z[u][i][1]);
            big = fmax3(big, z[u][i][2], z[u][i][3]);
          }
          // y itself past 2^88: value scales so small that P' does not show it
          constexpr float DOWN = 8.271806125530277e-25f;  // 2^-80
          big = fmax3(big, d[i][0] * DOWN, d[i][1] * DOWN);
        }
        if (__any_sync(0xffffffffu, big > 256.f)) {
#pragma unroll
          for (int i = 0; i < NT; ++i) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float x = fmaxf(fmaxf(sc[0][i][e], sc[0][i][2 + e]), fmaxf(sc[1][i][e], sc[1][i][2 + e]));
#pragma unroll
              for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
              const bool none = x == -INFINITY;
              x = none ? 0.f : x * back[i][e];
              float w = 0.f;  // the largest p v_scale of the tile, p relative to x
#pragma unroll
              for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int a = 0; a < 2; ++a)
                  w = fmaxf(w, fast_exp2(fmaf(sc[u][i][2 * a + e], back[i][e], -x)) * vs[u][a]);
#pragma unroll
              for (int o = 4; o < 32; o <<= 1) w = fmaxf(w, __shfl_xor_sync(0xffffffffu, w, o));
              // w < 2^ex
              const int ex = static_cast<int>(__float_as_uint(w) >> 23) - 126;
              const float n = none ? ref[i][e] : fmaxf(ref[i][e], x + fmaxf(static_cast<float>(ex), -Y_RANGE));
              const float f = fast_exp2(ref[i][e] - n);
              ref[i][e] = n;
              l[i][e] *= f;
#pragma unroll
              for (int k = 0; k < KS; ++k) {
                acc[k][i][e] *= f;
                acc[k][i][2 + e] *= f;
              }
            }
            against(i);
          }
        }
        uint32_t pf[2][NT][2];
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          l[i][0] += d[i][0];
          l[i][1] += d[i][1];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            if (masked) {  // a masked key may have any scale
#pragma unroll
              for (int e = 0; e < 4; ++e) z[u][i][e] = sc[u][i][e] == -INFINITY ? 0.f : z[u][i][e];
            }
            pf[u][i][0] = transpose8x8(pack2<false>(z[u][i][0], z[u][i][1]));
            pf[u][i][1] = transpose8x8(pack2<false>(z[u][i][2], z[u][i][3]));
          }
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          uint32_t vr[4][VW];
          const uint8_t* const va = at + SH::TILE;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if constexpr (D == 128) {
              const uint4 x = reinterpret_cast<const uint4*>(va)[v_piece<D>(16 * u + 4 * t + i, g)];
              vr[i][0] = x.x; vr[i][1] = x.y; vr[i][2] = x.z; vr[i][3] = x.w;
            } else {
              const uint2 x = reinterpret_cast<const uint2*>(va)[v_piece<D>(16 * u + 4 * t + i, g >> 1) * 2 + (g & 1)];
              vr[i][0] = x.x; vr[i][1] = x.y;
            }
          }
#pragma unroll
          for (int w = 0; w < VW; ++w) {
            // keys 0, 1 and 2, 3 of the lane interleaved: two steps' operands
            uint32_t a[2][4];
            pairs<FMT, EVERY>(__byte_perm(vr[0][w], vr[1][w], 0x5140), a[0][0], a[0][1]);
            pairs<FMT, EVERY>(__byte_perm(vr[2][w], vr[3][w], 0x5140), a[0][2], a[0][3]);
            pairs<FMT, EVERY>(__byte_perm(vr[0][w], vr[1][w], 0x7362), a[1][0], a[1][1]);
            pairs<FMT, EVERY>(__byte_perm(vr[2][w], vr[3][w], 0x7362), a[1][2], a[1][3]);
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
              for (int i = 0; i < NT; ++i)
                mma16816(acc[2 * w + k][i], a[k][0], a[k][1], a[k][2], a[k][3], pf[u][i][0], pf[u][i][1]);
          }
        }
      }
    };
    stream(std::false_type());
    if constexpr (FMT == FMT_E4M3) {
      // A NaN in a sum may come of a code 0x7f or 0xff, of a key that some row of the
      // warp sees or of a masked one's value: the warp's keys once more, with every
      // code as what it stands for. (A NaN of the query or of a scale stays one.)
      bool nan = false;
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        nan |= l[i][0] != l[i][0] || l[i][1] != l[i][1];
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int e = 0; e < 4; ++e) nan |= acc[k][i][e] != acc[k][i][e];
      }
      if (__any_sync(0xffffffffu, nan)) {
        __syncwarp();  // every lane is done with the ring
        stream(std::true_type());
      }
    }
    copy_wait<0>();
    __syncthreads();  // the ring's place takes the warps' parts

    // ------------------------------------------------ the warps' parts
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l[i][e] += __shfl_xor_sync(0xffffffffu, l[i][e], o);
        const int row = 8 * i + 2 * t + e;
        // a warp without keys has no reference
        if (g == 0) sml[warp * ROWS + row] = make_float2(l[i][e] == 0.f ? -INFINITY : ref[i][e], l[i][e]);
        float* const o = so + (warp * ROWS + row) * SH::ROW + g * (D / 8);
#pragma unroll
        for (int k = 0; k < KS; ++k) *reinterpret_cast<float2*>(o + 2 * k) = make_float2(acc[k][i][e], acc[k][i][2 + e]);
      }
    __syncthreads();
    const int64_t slot = 2ll * blockIdx.x + (first ? 0 : 1), nslot = 2ll * ranges * c.Hkv * slot_rows;
    for (int e = threadIdx.x; e < R * (D / 4); e += THREADS) {
      const int row = e / (D / 4), d4 = e - row * (D / 4);
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) M = fmaxf(M, sml[w * ROWS + row].x);
      float sum = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < WARPS; ++w) {
        const float2 ml = sml[w * ROWS + row];
        const float f = M == -INFINITY ? 0.f : fast_exp2(ml.x - M);
        const float4 x = *reinterpret_cast<const float4*>(so + (w * ROWS + row) * SH::ROW + 4 * d4);
        sum = fmaf(f, ml.y, sum);
        o.x = fmaf(f, x.x, o.x);
        o.y = fmaf(f, x.y, o.y);
        o.z = fmaf(f, x.z, o.z);
        o.w = fmaf(f, x.w, o.w);
      }
      if (whole) {
        const bool live = sum > 0.f;
        const float inv = live ? 1.f / sum : __int_as_float(0x7fc00000);
        const int64_t at = row_at(row);
        if (!in_bounds(status, at, nrows)) continue;
        reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at * D)[d4] =
            make_uint2(pack_out(bf16, o.x * inv, o.y * inv), pack_out(bf16, o.z * inv, o.w * inv));
        if (p.lse && d4 == 0) p.lse[at] = live ? (M + log2f(sum)) * LN2 : (sum == 0.f ? -INFINITY : sum);
      } else {
        const int64_t at = slot * slot_rows + row_lo + row;
        if (!in_bounds(status, at, nslot)) continue;
        reinterpret_cast<float4*>(p.ws)[at * (D / 4) + d4] = o;
        if (d4 == 0) reinterpret_cast<float2*>(static_cast<uint8_t*>(p.ws) + ml_offset)[at] = make_float2(M, sum);
      }
    }
    if (!whole) {
      // the ranges rf .. rl hold the sequence's blocks
      const int64_t begin = u - take - b, end = begin + nb;
      const int rf = static_cast<int>(((begin + 1) * ranges + pl.total - 1) / pl.total) - 1;  // last with cut(rf) <= begin
      const int rl = static_cast<int>((end * ranges + pl.total - 1) / pl.total) - 1;          // first with cut(rl + 1) >= end
      const bool gaps = pl.total < ranges;  // some ranges are empty, the others have a block each
      const int parts = gaps ? nb : rl - rf + 1;
      __threadfence();
      __syncthreads();
      if (threadIdx.x == 0) {
        asm volatile("griddepcontrol.wait;" ::: "memory");  // the counters are zero
        const int64_t n = (static_cast<int64_t>(rf) * c.Hkv + h) * gridDim.y + blockIdx.y;
        last_part = in_bounds(status, n, static_cast<int64_t>(ranges) * c.Hkv * gridDim.y) && atomicAdd(counters + n, 1) == parts - 1;
      }
      __syncthreads();
      if (last_part) {
        __threadfence();
        const float4* const wo = static_cast<const float4*>(p.ws);
        const float2* const wml = reinterpret_cast<const float2*>(static_cast<const uint8_t*>(p.ws) + ml_offset);
        constexpr int G = D / 4, TEAMS = THREADS / G, BATCH = 8;  // parts read together: each read is a trip to L2
        const int g4 = threadIdx.x % G, team = threadIdx.x / G;
        const int share = R >= TEAMS ? 1 : TEAMS / R;  // teams of a row, added up in order
        const int at_once = TEAMS / share;
        const bool starts_late = begin > cut(pl.total, rf, ranges);
        for (int base = 0; base < R; base += at_once) {
          const int row = base + team / share, part0 = team % share;
          const bool mine = row < R && team / share < at_once;
          float M = -INFINITY, sum = 0.f;
          float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
          auto add = [&](float2 ml, float4 x) {
            const float n = fmaxf(M, ml.x);
            const float f = n == -INFINITY ? 0.f : fast_exp2(M - n), e = n == -INFINITY ? 0.f : fast_exp2(ml.x - n);
            M = n;
            sum = sum * f + ml.y * e;
            o = make_float4(o.x * f + x.x * e, o.y * f + x.y * e, o.z * f + x.z * e, o.w * f + x.w * e);
          };
          for (int r0 = rf + part0; mine && r0 <= rl; r0 += share * BATCH) {
            float2 ml[BATCH];
            float4 x[BATCH];
#pragma unroll
            for (int k = 0; k < BATCH; ++k) {
              const int r = r0 + k * share;
              const int64_t at = (2ll * (static_cast<int64_t>(r) * c.Hkv + h) + (r == rf && starts_late ? 1 : 0)) * slot_rows + row_lo + row;
              const bool part = r <= rl && !(gaps && cut(pl.total, r, ranges) == cut(pl.total, r + 1, ranges)) &&
                                in_bounds(status, at, nslot);
              ml[k] = part ? __ldcg(wml + at) : make_float2(-INFINITY, 0.f);
              x[k] = part ? __ldcg(wo + at * G + g4) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
#pragma unroll
            for (int k = 0; k < BATCH; ++k) add(ml[k], x[k]);
          }
          if (share > 1) {
            __syncthreads();
            reinterpret_cast<float4*>(so)[team * G + g4] = o;
            if (g4 == 0) sml[team] = make_float2(M, sum);
            __syncthreads();
            if (mine && part0 == 0)
              for (int i = 1; i < share; ++i) add(sml[team + i], reinterpret_cast<const float4*>(so)[(team + i) * G + g4]);
          }
          if (!mine || part0 != 0) continue;
          const bool live = sum > 0.f;
          const float inv = live ? 1.f / sum : __int_as_float(0x7fc00000);
          const int64_t at = row_at(row);
          if (!in_bounds(status, at, nrows)) continue;
          reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at * D)[g4] =
              make_uint2(pack_out(bf16, o.x * inv, o.y * inv), pack_out(bf16, o.z * inv, o.w * inv));
          if (p.lse && g4 == 0) p.lse[at] = live ? (M + log2f(sum)) * LN2 : (sum == 0.f ? -INFINITY : sum);
        }
      }
    }
    __syncthreads();
  }
  // a grid that cut no sequence does not end before zero_kernel either: the next
  // one on the stream may use the workspace
  if (threadIdx.x == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Clears the counters of the cut sequences.
static __global__ void zero_kernel(int* counters, int n) {
  asm volatile("griddepcontrol.launch_dependents;");  // the decode kernel may come up; it waits before it counts
  for (int i = threadIdx.x; i < n; i += blockDim.x) counters[i] = 0;
}

template <int D, int FMT, int NT>
cudaError_t launch_nt(const FwdParams& p, const DecodePlan& plan, cudaStream_t st) {
  auto kern = decode_kernel<D, FMT, NT>;
  constexpr int smem = Shared<D, NT>::BYTES;
  static std::atomic<unsigned long long> configured{0};
  cudaError_t e = allow_smem(kern, smem, p.device, configured);
  if (e != cudaSuccess) return e;
  const unsigned ctas = static_cast<unsigned>(plan.ranges) * p.c.Hkv;
  const int64_t ml = plan.ml_offset(p.c.Hkv, D);
  int* const counters = reinterpret_cast<int*>(static_cast<uint8_t*>(p.ws) + plan.counter_offset(p.c.Hkv, D));
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(ctas, plan.row_groups);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  if (plan.cuts()) {
    zero_kernel<<<1, 512, 0, st>>>(counters, static_cast<int>(ctas) * plan.row_groups);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
  }
  return cudaLaunchKernelEx(&cfg, kern, p, plan.ranges, plan.aligned, plan.slot_rows(), ml, counters);
}

template <int D, int FMT>
cudaError_t launch_d(const FwdParams& p, const DecodePlan& plan, cudaStream_t st) {
  switch (plan.nt) {
    case 1: return launch_nt<D, FMT, 1>(p, plan, st);
    case 2: return launch_nt<D, FMT, 2>(p, plan, st);
    case 3: return launch_nt<D, FMT, 3>(p, plan, st);
    default: return launch_nt<D, FMT, 4>(p, plan, st);
  }
}

}  // namespace dec

template <int FMT>
cudaError_t launch_decode(const FwdParams& p, const DecodePlan& plan, cudaStream_t st) {
  return p.c.D == 128 ? dec::launch_d<128, FMT>(p, plan, st) : dec::launch_d<64, FMT>(p, plan, st);
}

}  // namespace kv8
}  // namespace attn
