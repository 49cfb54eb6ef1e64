// prefix_rows.cuh - both stages of attn_paged_prefix_fwd (prefix.cuh) for few rows, at most 32
// a CTA: decode steps and drafted tokens behind a prefix, and the prefixes of small
// groups (F16/BF16, D in {64, 128}, any page size).
//
// Measured: own keys of 64 sequences, 100-2000 tokens each, 32/8 heads, D 128, BF16, by themselves: 54 us, 5.1 TB/s
// (76% of the copy bandwidth); behind 8192 shared keys the whole call 75 us.
// Bound: the bytes of the keys and values, read once for all the rows of a kv head; then the latency
// of a unit's beginning (metadata, query, page, first keys: a trip to L2 or beyond each) and of the join.
// A warp streams its own 16-key tiles through buffers of cp.async copies in shared memory,
// without a barrier between warps:
//  - S^T = K Q^T (keys x rows), then O^T = V^T P^T, by mma.sync with the cache as the A
//    operand, so that 8 columns hold the rows instead of 16 or 128; K by ldmatrix, V by its
//    transposing form, P^T from S^T by one movmatrix for 8 keys x 8 rows;
//  - a row has a reference exponent: y = 2^(x - ref), and ref moves up only when a y passes
//    2^15 (one vote a tile instead of a reduction), to bring the largest y to 2^8;
//  - up to 16 rows a CTA, a probability meets the values as two numbers of the input type, one below it and
//    what that left (both above 0: the sum of their products with an infinite value is that infinity): a second
//    mma with the operand that is there already (64 sequences with 8 rows a kv
//    head 78.0 us, 77.2 with the rounded one alone; with 16 rows 91.5 and 86.7; 4 rows, F16, error against
//    64 bits 2.1e-4, the output's own rounding, instead of 2.5e-4 to 2.9e-4). With 32 rows it costs 11-20%
//    (148 us, 124 without), and the roundings of many rows average out: there it is the rounded one alone.
//
// Suffix stage: the keys of all sequences, in blocks of 32 (16 a warp), are cut into ranges
// of equal length, one for each group of Hkv CTAs (one a head, side by side). A CTA walks the
// units (sequences) of its range and leaves a part for each row; join_kernel joins a
// row's parts, those of its prefix first, then those of the ranges in their order.
// Prefix stage: blocks of 32 keys for 8 NT rows and a head, shared out as prefix.cuh says. Groups of more rows
// come here too where prefix_tc.cuh does not take the page size, and read their prefix once for every 32 of
// them (384 rows a head behind 8192 keys: 123 us with pages of 48 or 96 tokens, 49 with 64).
#pragma once

#include "prefix.cuh"

namespace attn {
namespace prefix {
namespace rows {

constexpr int TILE = 16;                  // keys of a warp's tile
constexpr float UNSEEN = -3.40282347e38f; // reference of a row without keys, the least number: a first score above it passes every range

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
template <bool BF16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (BF16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int D, int NT>
struct Shared {
  static constexpr int ROWS = 8 * NT;
  static constexpr int STAGES = D == 128 && NT <= 2 ? 2 : 3;
  static constexpr int TILE_BYTES = TILE * D * 2;             // K or V
  static constexpr int RING = WARPS * STAGES * 2 * TILE_BYTES;
  static constexpr int ROW = D + 4;
  static constexpr int O = WARPS * ROWS * ROW * 4;            // the warps' outputs, in the ring's place
  static constexpr int OFF_ML = RING > O ? RING : O;
  static constexpr int OFF_LIM = OFF_ML + WARPS * ROWS * 8;
  static constexpr int OFF_Q = OFF_LIM + ROWS * 4;            // query operands, in the lanes' order
  static constexpr int BYTES = OFF_Q + NT * (D / 16) * 32 * 8;
};

template <bool BF16>
__device__ __forceinline__ float2 unpack2(uint32_t u) {
  if constexpr (BF16) return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
  else return __half22float2(*reinterpret_cast<const __half2*>(&u));
}

// Two weights of 0 or more as numbers of the type below them, so that what is left of a weight above 0 is above 0 too: a
// part of 0 or less would make NaN of an infinite value. F16 stays half a step away: the rest then has a
// number from a weight of 2^-12 on (a row's largest one is 2^8 at least).
template <bool BF16>
__device__ __forceinline__ uint32_t pack2_below(float lo, float hi) {
  constexpr float LESS = BF16 ? 0x1.fffffcp-1f : 0x1.ffep-1f;  // 1 - 2^-23, 1 - 2^-12
  const float2 x = fmul2(make_float2(lo, hi), make_float2(LESS, LESS));
  uint32_t d;
  if constexpr (BF16) asm("cvt.rz.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(x.y), "f"(x.x));
  else asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(x.y), "f"(x.x));
  return d;
}

// Whether a pair holds a NaN or an infinity: all bits of an exponent set.
template <bool BF16>
__device__ __forceinline__ bool not_finite(uint32_t pair) {
  constexpr uint32_t LO = BF16 ? 0x7f80u : 0x7c00u, HI = LO << 16;
  return (pair & LO) == LO || (pair & HI) == HI;
}

// A CTA's piece of a unit: rows (queries from q_lo on, `nq` of them, times heads; row_lo the
// first of R rows), keys [from, to), read through row `table` of the table.
struct Piece {
  int q_lo, row_lo, R, h, table, from, to;
};

// The parts of the softmax of the piece's rows: streams the keys and leaves the warps'
// parts in shared memory (so, sml). The whole CTA calls it. lims: keys each row sees.
template <int D, bool BF16, int NT>
__device__ __forceinline__ void stream(const Params& p, const Piece& w, uint8_t* smem) {
  constexpr int KS = D / 16;       // 16-element steps of a head
  constexpr int ROWS = 8 * NT;
  constexpr bool BOTH = NT <= 2;   // probabilities as two numbers
  using SH = Shared<D, NT>;
  constexpr int STAGES = SH::STAGES;
  float* const so = reinterpret_cast<float*>(smem);
  float2* const sml = reinterpret_cast<float2*>(smem + SH::OFF_ML);
  const int* const lims = reinterpret_cast<const int*>(smem + SH::OFF_LIM);
  uint2* const sq = reinterpret_cast<uint2*>(smem + SH::OFF_Q);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int heads = p.Hq / p.Hkv;
  int* const status = p.status;
  const int64_t nrows = static_cast<int64_t>(p.num_queries) * p.Hq;

  // What the first products need comes of three trips to L2 or beyond: the page of the first keys,
  // looked up for every key that may be seen, flies with the query's elements.
  constexpr int PIECES = D / 8;          // 16-byte pieces of a key
  constexpr int RPC = 32 / PIECES;       // keys that one copy of the warp covers
  const uint32_t ring = smem_u32(smem) + warp * STAGES * 2 * SH::TILE_BYTES;
  const int64_t ntok = static_cast<int64_t>(p.num_pages) * p.page_size;
  const int64_t step = static_cast<int64_t>(p.Hkv) * D * 2;  // bytes from token to token
  const uint8_t* const kb = static_cast<const uint8_t*>(p.k) + (w.h * D + lane % PIECES * 8) * 2;
  const uint8_t* const vb = static_cast<const uint8_t*>(p.v) + (w.h * D + lane % PIECES * 8) * 2;
  // The lane's key of the tile to copy next: its block and the row in it.
  int ckey = w.from + warp * TILE + (lane & (TILE - 1));
  const int tile0 = w.from + warp * TILE;
  int cfirst = tile0;
  int blk = ckey / p.page_size, row = ckey - blk * p.page_size;
  const int dblk = BLOCK / p.page_size, drow = BLOCK - dblk * p.page_size;
  auto find_page = [&]() { return ckey < w.to ? page_of(p, w.table, blk) : -1; };
  int page = find_page();
  // query operands: of 8 rows by warp: lane (g, t) holds elements 16 k + 2 t, + 1 and + 8, + 9 of row g
  for (int i = warp; i < NT; i += WARPS) {
    const int row = 8 * i + g;
    const uint32_t* src = nullptr;
    if (row < w.R) {
      const int q = (w.row_lo + row) / heads;
      const int64_t at = static_cast<int64_t>(w.q_lo + q) * p.Hq + w.h * heads + (w.row_lo + row - q * heads);
      if (in_bounds(status, at, nrows)) src = reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(p.q) + at * D);
    }
    uint2 x[KS];
#pragma unroll
    for (int k = 0; k < KS; ++k) x[k] = src ? make_uint2(__ldg(src + 8 * k + t), __ldg(src + 8 * k + 4 + t)) : make_uint2(0u, 0u);
#pragma unroll
    for (int k = 0; k < KS; ++k) sq[(i * KS + k) * 32 + lane] = x[k];
  }
  __syncthreads();
  uint2 qf[NT == 1 ? KS : 1];
  if constexpr (NT == 1) {
#pragma unroll
    for (int k = 0; k < KS; ++k) qf[k] = sq[k * 32 + lane];
  }
  int lim[NT][2];  // keys that the lane's rows (8 i + 2 t, + 1) see
  int least = w.to, most = 0;
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int row = 8 * i + 2 * t + e;
      lim[i][e] = min(lims[row], w.to);
      if (row < w.R) {
        least = min(least, lim[i][e]);
        most = max(most, lim[i][e]);
      }
    }
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    least = min(least, __shfl_xor_sync(0xffffffffu, least, o));
    most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
  }

  float ref[NT][2], l[NT][2], acc[KS][NT][4];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    ref[i][0] = ref[i][1] = UNSEEN;
    l[i][0] = l[i][1] = 0.f;
#pragma unroll
    for (int k = 0; k < KS; ++k) acc[k][i][0] = acc[k][i][1] = acc[k][i][2] = acc[k][i][3] = 0.f;
  }
  int64_t mine = -1;  // its row of the cache; -1: zeros
  auto copy_half = [&](uint32_t at, const uint8_t* from) {  // K or V of the tile at cfirst
    if (cfirst < most) {
#pragma unroll
      for (int j = 0; j < TILE / RPC; ++j) {
        const int r = RPC * j + lane / PIECES, c = lane % PIECES;
        const int64_t key = __shfl_sync(0xffffffffu, mine, r);
        copy16(at + (r * PIECES + (c ^ (r & 7))) * 16, from + (key < 0 ? 0 : key) * step, key < 0 ? 0 : 16);
      }
    }
    copy_commit();
  };
  auto copy_keys = [&](int stage) {
    const int64_t tok = static_cast<int64_t>(page) * p.page_size + row;
    mine = page >= 0 && ckey < most && in_bounds(status, tok, ntok) ? tok : -1;
    copy_half(ring + stage * 2 * SH::TILE_BYTES, kb);
  };
  auto copy_values = [&](int stage) {  // of the same tile; then on to the next one, whose page is looked up ahead
    copy_half(ring + stage * 2 * SH::TILE_BYTES + SH::TILE_BYTES, vb);
    cfirst += BLOCK;
    ckey += BLOCK;
    blk += dblk;
    row += drow;
    if (row >= p.page_size) {
      row -= p.page_size;
      ++blk;
    }
    page = find_page();
  };
  // K and V of a tile are copies of their own: the place of K is free, and filled again, while V waits
#pragma unroll
  for (int i = 0; i < STAGES; ++i) {
    copy_keys(i);
    copy_values(i);
  }
  int stage = 0;
  // ldmatrix addresses: K rows (lane & 15), piece 2 k + lane / 16; V rows (lane & 7) + 8 (lane / 16), piece 2 k + lane / 8 % 2
  const int kr = lane & 15, vr = (lane & 7) + ((lane >> 4) << 3);
  for (int key0 = tile0; key0 < most; key0 += BLOCK) {
    copy_wait<2 * STAGES - 1>();
    __syncwarp();  // the tile's keys by every lane
    const uint32_t ka = ring + stage * 2 * SH::TILE_BYTES, va = ka + SH::TILE_BYTES;
    float sc[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i) sc[i][0] = sc[i][1] = sc[i][2] = sc[i][3] = 0.f;
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      uint32_t a[4];
      ldsm4(a, ka + (kr * PIECES + ((2 * k + (lane >> 4)) ^ (kr & 7))) * 16);
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        if constexpr (NT == 1) {
          mma16816<BF16>(sc[i], a, qf[k].x, qf[k].y);
        } else {
          const uint2 b = sq[(i * KS + k) * 32 + lane];
          mma16816<BF16>(sc[i], a, b.x, b.y);
        }
      }
    }
    __syncwarp();  // every lane has read them
    copy_keys(stage);
    const bool masked = key0 + TILE > least;
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        sc[i][e] *= p.scale_log2;
        if (masked && key0 + g + (e & 2) * 4 >= lim[i][e & 1]) sc[i][e] = -INFINITY;
      }
    float y[NT][4], big = 0.f;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
#pragma unroll
      for (int e = 0; e < 4; ++e) y[i][e] = fast_exp2(sc[i][e] - ref[i][e & 1]);
      big = fmax3(big, y[i][0], y[i][1]);
      big = fmax3(big, y[i][2], y[i][3]);
    }
    if (__any_sync(0xffffffffu, big > 32768.f)) {
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x = fmaxf(sc[i][e], sc[i][2 + e]);
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
          const float n = x == -INFINITY ? ref[i][e] : fmaxf(ref[i][e], x - 8.f);
          const float f = fast_exp2(ref[i][e] - n);
          ref[i][e] = n;
          l[i][e] *= f;
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            acc[k][i][e] *= f;
            acc[k][i][2 + e] *= f;
          }
          y[i][e] = fast_exp2(sc[i][e] - n);
          y[i][2 + e] = fast_exp2(sc[i][2 + e] - n);
        }
    }
    uint32_t pf[NT][2], pl[BOTH ? NT : 1][2];  // in the input type, and what that left
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      l[i][0] += y[i][0] + y[i][2];
      l[i][1] += y[i][1] + y[i][3];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float a = y[i][2 * e], b = y[i][2 * e + 1];
        const uint32_t hi = BOTH ? pack2_below<BF16>(a, b) : pack2<BF16>(a, b);
        pf[i][e] = transpose8x8(hi);
        if constexpr (BOTH) {
          const float2 back = unpack2<BF16>(hi);
          pl[i][e] = transpose8x8(pack2<BF16>(a - back.x, b - back.y));
        }
      }
    }
    copy_wait<2 * STAGES - 1>();
    __syncwarp();  // its values
    bool strange = false;  // a value that is no number, in a tile that some row sees a part of
    if (masked) {
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        uint32_t a[4];
        ldsm4_t(a, va + (vr * PIECES + ((2 * k + ((lane >> 3) & 1)) ^ (vr & 7))) * 16);
#pragma unroll
        for (int e = 0; e < 4; ++e) strange |= not_finite<BF16>(a[e]);
      }
      strange = __any_sync(0xffffffffu, strange);
    }
    if (!strange) {
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        uint32_t a[4];
        ldsm4_t(a, va + (vr * PIECES + ((2 * k + ((lane >> 3) & 1)) ^ (vr & 7))) * 16);
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          if constexpr (BOTH) mma16816<BF16>(acc[k][i], a, pl[i][0], pl[i][1]);
          mma16816<BF16>(acc[k][i], a, pf[i][0], pf[i][1]);
        }
      }
    } else {
      // 0 times it is not 0: a row at a time, with zeros in the place of what that row does not see
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll 1
        for (int n = 0; n < 8; ++n) {
          const int sees = min(lims[8 * i + n], w.to) - key0;
          const uint32_t b0 = g == n ? pf[i][0] : 0u, b1 = g == n ? pf[i][1] : 0u;
          auto keep = [&](uint32_t x, int key) {  // of the pair of keys from `key` on
            return (key < sees ? x & 0xffffu : 0u) | (key + 1 < sees ? x & 0xffff0000u : 0u);
          };
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            uint32_t a[4];
            ldsm4_t(a, va + (vr * PIECES + ((2 * k + ((lane >> 3) & 1)) ^ (vr & 7))) * 16);
            a[0] = keep(a[0], 2 * t);
            a[1] = keep(a[1], 2 * t);
            a[2] = keep(a[2], 8 + 2 * t);
            a[3] = keep(a[3], 8 + 2 * t);
            // the other rows' columns get 0 times what this row sees, which may be no number: they keep theirs
            float d[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) d[e] = acc[k][i][e];
            if constexpr (BOTH) mma16816<BF16>(d, a, g == n ? pl[i][0] : 0u, g == n ? pl[i][1] : 0u);
            mma16816<BF16>(d, a, b0, b1);
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (2 * t + (e & 1) == n) acc[k][i][e] = d[e];
          }
        }
    }
    __syncwarp();
    copy_values(stage);
    stage = stage == STAGES - 1 ? 0 : stage + 1;
  }
  copy_wait<0>();
  __syncthreads();  // the ring's place takes the warps' parts
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) l[i][e] += __shfl_xor_sync(0xffffffffu, l[i][e], o);
      const int r = 8 * i + 2 * t + e;
      // a warp without keys has no reference
      if (g == 0) sml[warp * ROWS + r] = make_float2(l[i][e] == 0.f ? -INFINITY : ref[i][e], l[i][e]);
      float* const o = so + (warp * ROWS + r) * SH::ROW + g;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        o[16 * k] = acc[k][i][e];
        o[16 * k + 8] = acc[k][i][2 + e];
      }
    }
  __syncthreads();
}

// A row's running part: 4 elements of O, relative to 2^M.
struct Part {
  float M = -INFINITY, sum = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  __device__ __forceinline__ void add(float2 ml, float4 x) {
    const float n = fmaxf(M, ml.x);
    const float f = n == -INFINITY ? 0.f : fast_exp2(M - n), e = n == -INFINITY ? 0.f : fast_exp2(ml.x - n);
    M = n;
    sum = sum * f + ml.y * e;
    o = make_float4(o.x * f + x.x * e, o.y * f + x.y * e, o.z * f + x.z * e, o.w * f + x.w * e);
  }
};

// Of row r of the piece, elements 4 d4 ..: the warps' parts together.
template <int D, int NT>
__device__ __forceinline__ Part of_warps(const uint8_t* smem, int r, int d4) {
  constexpr int ROWS = 8 * NT;
  using SH = Shared<D, NT>;
  const float* const so = reinterpret_cast<const float*>(smem);
  const float2* const sml = reinterpret_cast<const float2*>(smem + SH::OFF_ML);
  Part a;
#pragma unroll
  for (int w = 0; w < WARPS; ++w)
    a.add(sml[w * ROWS + r], *reinterpret_cast<const float4*>(so + (w * ROWS + r) * SH::ROW + 4 * d4));
  return a;
}

// ------------------------------------------------------------------ prefix stage
// Each row's limit of a group's rows (row_lo on), into shared memory.
__device__ __forceinline__ void group_limits(const Params& p, int a, int b, int q_lo, int row_lo, int R, int rows, int* lims) {
  const int heads = p.Hq / p.Hkv;
  for (int r = threadIdx.x; r < rows; r += blockDim.x) {
    int x = 0;
    if (r < R) {
      const int i = q_lo + (row_lo + r) / heads;
      x = limit_of(p, last_at_most(p.q_offsets, a, b, i), i);
    }
    lims[r] = x;
  }
}

template <int D, bool BF16, int NT>
__global__ void __launch_bounds__(THREADS, ctas_of_sm(D, NT)) prefix_kernel(const __grid_constant__ Params p) {
  wait_before();
  let_next();  // the suffix stage runs beside this one
  constexpr int ROWS = 8 * NT;
  extern __shared__ __align__(16) uint8_t smem[];
  using SH = Shared<D, NT>;
  const Share sh = share_out<THREADS, false>(p, gridDim.x, BLOCK, ROWS, false);
  const int heads = p.Hq / p.Hkv;
  int64_t u = sh.u0, first = sh.first;
  for (int g = sh.g; u < sh.u1; ++g) {
    const Rec rec = rec_of(p, g, BLOCK, ROWS, false);
    const int64_t n = blocks_of(p, rec);
    if (u >= first + n) {
      first += n;
      continue;
    }
    int a, b;
    group_range(p, g, a, b);
    const int pre = prefix_len(p, g), table = reader_of(p, a, b, pre);
    int q_lo;
    const int64_t rows = static_cast<int64_t>(queries_of(p, a, b, p.max_group_queries, q_lo)) * heads;
    while (u < sh.u1 && u < first + n) {
      const int unit = static_cast<int>((u - first) / rec.nb), k0 = static_cast<int>(u - first - static_cast<int64_t>(unit) * rec.nb);
      const int take = static_cast<int>(min(static_cast<int64_t>(rec.nb - k0), sh.u1 - u));
      const int part = static_cast<int>(blockIdx.x) - range_of(u - k0, sh.total, sh.ranges);
      u += take;
      Piece w;
      w.q_lo = q_lo;
      w.row_lo = unit / p.Hkv * ROWS;
      w.R = static_cast<int>(min(rows - w.row_lo, static_cast<int64_t>(ROWS)));
      w.h = unit % p.Hkv;
      w.table = table;
      w.from = k0 * BLOCK;
      w.to = min(pre, w.from + take * BLOCK);
      group_limits(p, a, b, q_lo, w.row_lo, w.R, ROWS, reinterpret_cast<int*>(smem + SH::OFF_LIM));
      stream<D, BF16, NT>(p, w, smem);
      const int64_t nrows = static_cast<int64_t>(p.num_queries) * p.Hq;
      for (int e = threadIdx.x; e < w.R * (D / 4); e += THREADS) {
        const int r = e / (D / 4), d4 = e - r * (D / 4);
        const Part x = of_warps<D, NT>(smem, r, d4);
        const int q = (w.row_lo + r) / heads;
        const int64_t at = part * nrows + static_cast<int64_t>(w.q_lo + q) * p.Hq + w.h * heads + (w.row_lo + r - q * heads);
        if (!in_bounds(p.status, at, p.most_parts * nrows)) continue;
        reinterpret_cast<float4*>(p.o)[at * (D / 4) + d4] = x.o;
        if (d4 == 0) p.ml[at] = make_float2(x.M, x.sum);
      }
      __syncthreads();
    }
    first += n;
  }
}

// ------------------------------------------------------------------ suffix stage
__device__ __forceinline__ int key_blocks(int n) { return max(1, (n + BLOCK - 1) / BLOCK); }  // without keys: one

__device__ __forceinline__ int row_blocks(const Params& p, int nq, int rows) {
  return static_cast<int>((static_cast<int64_t>(nq) * (p.Hq / p.Hkv) + rows - 1) / rows);
}

// Blocks in the order (sequence, row block, key block). The whole CTA calls it.
struct Place {
  int64_t total, at;  // blocks of all; first block of the unit that range begins in
  int s, rb, ranges;
};

template <int ROWS>
__device__ __forceinline__ Place locate(const Params& p, int range, int ranges, int least, int64_t& u0, int64_t& u1) {
  __shared__ int64_t warp_sum[THREADS / 32];
  __shared__ int64_t found_at;
  __shared__ int found_s, units;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (p.num_seqs + THREADS - 1) / THREADS;
  const int s0 = min(tid * per, p.num_seqs), s1 = min(s0 + per, p.num_seqs);
  auto blocks = [&](int s, int& rbs) -> int64_t {
    const int end = query_at(p, s + 1), L = seq_len(p, s), q_lo = query_at(p, s);  // read together
    const Own o = own_of(p, s, L);
    const int nq = min(max(end - q_lo, 0), p.max_queries);
    rbs = row_blocks(p, nq, ROWS);
    return nq > 0 ? static_cast<int64_t>(key_blocks(o.L - o.start)) * rbs : 0;
  };
  int64_t mine = 0;
  int my_units = 0, rbs;
  for (int s = s0; s < s1; ++s) {
    mine += blocks(s, rbs);
    my_units += rbs;
  }
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  if (lane == 31) warp_sum[warp] = incl;
  if (tid == 0) found_at = found_s = units = 0;
  __syncthreads();
  my_units = __reduce_add_sync(0xffffffffu, my_units);
  if (lane == 0) atomicAdd(&units, my_units);
  __syncthreads();
  int64_t before = incl - mine, total = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < warp) before += warp_sum[w];
    total += warp_sum[w];
  }
  Place pl;
  pl.total = total;
  // one for each unit, and no more than leave `least` blocks to each where units are cut
  const int64_t most = max(static_cast<int64_t>(units), total / least);
  pl.ranges = static_cast<int>(max(static_cast<int64_t>(1), min(static_cast<int64_t>(ranges), most)));
  u0 = range < pl.ranges ? cut(total, range, pl.ranges) : total;
  u1 = range < pl.ranges ? cut(total, range + 1, pl.ranges) : total;
  if (blockIdx.x == 0 || (u0 >= before && u0 < before + mine)) {
    int64_t at = before;
    for (int s = s0; s < s1; ++s) {
      const int64_t n = blocks(s, rbs);
      if (u0 >= at && u0 < at + n) {
        found_at = at;
        found_s = s;
      }
      if (blockIdx.x == 0) p.suffix_first[s] = at;
      at += n;
    }
  }
  if (blockIdx.x == 0 && tid == 0) *p.suffix_head = Head{total, pl.ranges, ROWS};
  __syncthreads();
  pl.s = found_s;
  pl.at = found_at;
  return pl;
}

template <int D, bool BF16, int NT>
__global__ void __launch_bounds__(THREADS, ctas_of_sm(D, NT))
    suffix_kernel(const __grid_constant__ Params p, int ranges, int least, int after_prefix) {
  // After the prefix stage nothing is waited for: what this one reads was complete before that began.
  if (!after_prefix) wait_before();
  let_next();
  constexpr int ROWS = 8 * NT, G = D / 4;
  extern __shared__ __align__(16) uint8_t smem[];
  using SH = Shared<D, NT>;
  const int h = blockIdx.x % p.Hkv, range = blockIdx.x / p.Hkv;
  const int heads = p.Hq / p.Hkv;
  int64_t u0, u1;
  const Place pl = locate<ROWS>(p, range, ranges, least, u0, u1);
  int64_t begin = pl.at;  // first block of the sequence
  Own own{};
  int q_lo = 0, nq = 0, s = pl.s;
  auto look = [&](int i) {  // sequence i
    nq = queries_of(p, i, i + 1, p.max_queries, q_lo);
    own = own_of(p, i);
  };
  if (u0 < u1) look(s);
  for (int64_t u = u0; u < u1; ++s) {
    if (s != pl.s) look(s);
    if (nq <= 0) continue;
    const int nb = key_blocks(own.L - own.start), rbs = row_blocks(p, nq, ROWS);
    for (int rb = static_cast<int>((u - begin) / nb); rb < rbs && u < u1; ++rb) {
      const int64_t first = begin + static_cast<int64_t>(rb) * nb;  // of the unit
      const int b = static_cast<int>(u - first);
      const int take = static_cast<int>(min(static_cast<int64_t>(nb - b), u1 - u));
      const bool starts = u == u0, whole = take == nb;
      u += take;
      Piece w;
      w.q_lo = q_lo;
      w.row_lo = rb * ROWS;
      w.R = static_cast<int>(min(static_cast<int64_t>(nq) * heads - w.row_lo, static_cast<int64_t>(ROWS)));
      w.h = h;
      w.table = s;
      w.from = own.start + b * BLOCK;
      w.to = min(own.L, w.from + take * BLOCK);
      auto row_at = [&](int r) {
        const int q = (w.row_lo + r) / heads;
        return static_cast<int64_t>(q_lo + q) * p.Hq + h * heads + (w.row_lo + r - q * heads);
      };
      int* const lims = reinterpret_cast<int*>(smem + SH::OFF_LIM);
      for (int r = threadIdx.x; r < ROWS; r += THREADS)
        lims[r] = r < w.R ? limit_of(p, s, q_lo + (w.row_lo + r) / heads) : 0;
      stream<D, BF16, NT>(p, w, smem);
      const int64_t slot = 2ll * blockIdx.x + (starts ? 0 : 1);
      const int64_t rows = whole ? static_cast<int64_t>(p.num_queries) * p.Hq : 2ll * ranges * p.Hkv * ROWS;
      float4* const to = reinterpret_cast<float4*>(whole ? p.own_o : p.cut_o);
      float2* const to_ml = whole ? p.own_ml : p.cut_ml;
      for (int e = threadIdx.x; e < w.R * G; e += THREADS) {
        const int r = e / G, d4 = e - r * G;
        const Part x = of_warps<D, NT>(smem, r, d4);
        const int64_t at = whole ? row_at(r) : slot * ROWS + r;
        if (!in_bounds(p.status, at, rows)) continue;
        to[at * G + d4] = x.o;
        if (d4 == 0) to_ml[at] = make_float2(x.M, x.sum);
      }
      __syncthreads();
    }
    begin += static_cast<int64_t>(nb) * rbs;
  }
  // the stage does not end before the prefix's: the next launch waits for this one
  if (blockIdx.x == 0 && after_prefix) wait_before();
}

// ------------------------------------------------------------------ the parts together
constexpr int JOIN_THREADS = 256;

// A thread takes 4 elements of a row. What it reads of the metadata it reads before it waits for
// the stages: its CTA may be on its SM long before they end. A thread without a row of a sequence waits too: the
// next launch may own the workspace, and a call may have no such row at all.
template <int D, bool BF16>
__global__ void __launch_bounds__(JOIN_THREADS) join_kernel(const __grid_constant__ Params p) {
  constexpr int G = D / 4, BATCH = 8;  // parts read together: each read is a trip to L2
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (JOIN_THREADS / G) + threadIdx.x / G;
  const int d4 = threadIdx.x % G;
  const int64_t rows = static_cast<int64_t>(p.num_queries) * p.Hq;
  if (row >= rows) {
    wait_before();
    return;
  }
  const int query = static_cast<int>(row / p.Hq), head = static_cast<int>(row - static_cast<int64_t>(query) * p.Hq);
  const int heads = p.Hq / p.Hkv, h = head / heads, hr = head - h * heads;
  // the query's sequence: in a decode step the one of its own number
  int s = min(query, p.num_seqs - 1);
  if (query < query_at(p, s) || query >= query_at(p, s + 1)) s = last_at_most(p.q_offsets, 0, p.num_seqs, query);
  int q_lo;
  const int nq = queries_of(p, s, s + 1, p.max_queries, q_lo);
  if (query < q_lo || query >= q_lo + nq) {  // of no sequence
    wait_before();
    return;
  }
  const Own own = own_of(p, s);
  const int nb = key_blocks(own.L - own.start);
  const int64_t local = static_cast<int64_t>(query - q_lo) * heads + hr;
  const int rb = static_cast<int>(local / p.suffix_rows), r = static_cast<int>(local - static_cast<int64_t>(rb) * p.suffix_rows);
  wait_before();
  const int64_t total = __ldcg(reinterpret_cast<const long long*>(&p.suffix_head->total));
  const int ranges = __ldcg(&p.suffix_head->ranges);
  const int64_t first = __ldcg(reinterpret_cast<const long long*>(p.suffix_first + s)) + static_cast<int64_t>(rb) * nb;
  const int n = own.pre > 0 ? parts_of(p, own.group, query, hr, h) : 0;  // of the prefix
  const int rf = range_of(first, total, ranges), rl = range_of(first + nb - 1, total, ranges);
  const int late = first > cut(total, rf, ranges) ? 1 : 0;
  const int64_t slots = 2ll * p.suffix_ranges * p.Hkv * p.suffix_rows;
  Part x;
  for (int z0 = 0; z0 < n + rl - rf + 1; z0 += BATCH) {
    float2 ml[BATCH];
    float4 y[BATCH];
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      const int z = z0 + k, c = rf + z - n;  // part of the prefix, or range
      const float2* m = p.ml;
      const float* o = p.o;
      int64_t at = z * rows + row, most = p.most_parts * rows;
      if (z >= n) {
        const bool one = rf == rl;
        m = one ? p.own_ml : p.cut_ml;
        o = one ? p.own_o : p.cut_o;
        at = one ? row : (2ll * (static_cast<int64_t>(c) * p.Hkv + h) + (c == rf ? late : 0)) * p.suffix_rows + r;
        most = one ? rows : slots;
      }
      const bool is = (z < n || c <= rl) && in_bounds(p.status, at, most);
      ml[k] = is ? __ldcg(m + at) : make_float2(-INFINITY, 0.f);
      y[k] = is ? __ldcg(reinterpret_cast<const float4*>(o) + at * G + d4) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int k = 0; k < BATCH; ++k) x.add(ml[k], y[k]);
  }
  const bool live = x.sum > 0.f;
  const float inv = live ? 1.f / x.sum : __int_as_float(0x7fc00000);
  reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + row * D)[d4] =
      make_uint2(pack2<BF16>(x.o.x * inv, x.o.y * inv), pack2<BF16>(x.o.z * inv, x.o.w * inv));
  if (p.lse && d4 == 0) p.lse[row] = live ? (x.M + log2f(x.sum)) * LN2 : (x.sum == 0.f ? -INFINITY : x.sum);
}

// ------------------------------------------------------------------ launches
template <int D, bool BF16, int NT>
cudaError_t launch_prefix_nt(const Params& p, cudaStream_t st) {
  auto kern = prefix_kernel<D, BF16, NT>;
  constexpr int smem = Shared<D, NT>::BYTES;
  static std::atomic<unsigned long long> configured{0};
  const cudaError_t e = allow_smem(kern, smem, p.device, configured);
  return e != cudaSuccess ? e : launch_early(kern, dim3(SMS * ctas_of_sm(D, NT)), THREADS, smem, st, 0, p);
}

template <int D, bool BF16, int NT>
cudaError_t launch_suffix_nt(const Params& p, bool after_prefix, cudaStream_t st) {
  auto kern = suffix_kernel<D, BF16, NT>;
  constexpr int smem = Shared<D, NT>::BYTES;
  static std::atomic<unsigned long long> configured{0};
  const cudaError_t e = allow_smem(kern, smem, p.device, configured);
  if (e != cudaSuccess) return e;
  return launch_early(kern, dim3(static_cast<unsigned>(p.suffix_ranges) * p.Hkv), THREADS, smem, st, 0, p, p.suffix_ranges,
                      LEAST_BLOCKS, after_prefix ? 1 : 0);
}

template <int D, bool BF16>
cudaError_t launch_join_d(const Params& p, cudaStream_t st) {
  const int64_t rows = static_cast<int64_t>(p.num_queries) * p.Hq, per = JOIN_THREADS / (D / 4);
  if ((rows + per - 1) / per > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  return launch_early(join_kernel<D, BF16>, dim3(static_cast<unsigned>((rows + per - 1) / per)), JOIN_THREADS, 0, st, 0, p);
}

#define ATTN_NT(F, NT, ...)                                        \
  (p.D == 128 ? (NT == 1   ? F<128, BF16, 1>(__VA_ARGS__)          \
                 : NT == 2 ? F<128, BF16, 2>(__VA_ARGS__)          \
                 : NT == 3 ? F<128, BF16, 3>(__VA_ARGS__)          \
                           : F<128, BF16, 4>(__VA_ARGS__))         \
              : (NT == 1   ? F<64, BF16, 1>(__VA_ARGS__)           \
                 : NT == 2 ? F<64, BF16, 2>(__VA_ARGS__)           \
                 : NT == 3 ? F<64, BF16, 3>(__VA_ARGS__)           \
                           : F<64, BF16, 4>(__VA_ARGS__)))

template <bool BF16>
cudaError_t launch_prefix(const Params& p, int nt, cudaStream_t st) {
  return ATTN_NT(launch_prefix_nt, nt, p, st);
}

template <bool BF16>
cudaError_t launch_suffix(const Params& p, int nt, bool after_prefix, cudaStream_t st) {
  return ATTN_NT(launch_suffix_nt, nt, p, after_prefix, st);
}

template <bool BF16>
cudaError_t launch_join(const Params& p, cudaStream_t st) {
  return p.D == 128 ? launch_join_d<128, BF16>(p, st) : launch_join_d<64, BF16>(p, st);
}
#undef ATTN_NT

}  // namespace rows
}  // namespace prefix
}  // namespace attn
