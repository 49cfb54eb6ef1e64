// attn_kv8_decode.cuh - attention over an 8-bit paged cache for calls with few
// rows (queries x heads of a kv head, at most 32): decode steps and drafted
// tokens (F16/BF16, D in {64, 128}).
//
// Bound: the bytes of the codes, read once for all the rows of a kv head. At
// the copy bandwidth an SM is fed 21 bytes a cycle, and each byte has to become
// a 16-bit operand, so what the kernel economises is instructions and
// shared-memory traffic per byte:
//  - the codes go from global memory to registers and, converted there, into
//    mma.sync as the A operand (a 16-key tile of a warp); nothing is staged in
//    shared memory (a tcgen05 operand would be written once and read twice, 6
//    bytes of shared-memory traffic for a byte of cache) and a tile has 8
//    columns for the query rows instead of 128;
//  - S^T = K Q^T (keys x rows), then O^T = V^T P^T. The order of the head's
//    elements inside a 16-element step of S^T, and of the rows of O^T, is free,
//    so that a lane's operands are 16 consecutive bytes of one key; V^T wants
//    two keys in one register, which the byte permutation of the conversion
//    gives without an instruction of its own; P^T is S^T transposed, one
//    movmatrix for 8 keys x 8 rows;
//  - codes convert exactly: int8 by placing the byte under the exponent of 128
//    (BF16, its sign bit apart) or 1024 (F16) and subtracting, e4m3 by moving
//    its 7 low bits to the top of exponent and mantissa, which leaves a power of
//    two (BF16: 2^-120, multiplied out; F16: 2^-8, folded into the scales);
//  - k_scale enters the score in fp32, v_scale the probability before it is
//    rounded to 16 bits. In F16 that product is kept within the type by dividing
//    by a running power of two that is at least every v_scale seen;
//  - the running maximum moves only when a score exceeds it by 2^8 (one vote a
//    tile instead of a reduction).
//
// Work: the keys of all sequences, in blocks of 128 (16 a warp), are cut into
// equal ranges, one for each group of Hkv CTAs (one CTA a head, side by side,
// since their codes lie side by side). A CTA walks the sequences of its range;
// a sequence wholly inside it is written out, a cut one as a partial (m, l, O)
// that merge_kernel combines in order. Uneven lengths cost nothing and there
// are no atomics.
#pragma once

#include "kv8_fwd.h"

namespace attn {
namespace kv8 {
namespace dec {

constexpr int WARPS = 8;
constexpr int THREADS = WARPS * 32;
constexpr int BLOCK_KEYS = 16 * WARPS;
constexpr float LN2 = 0.6931471805599453f;
constexpr float RESCALE_LOG2 = 8.0f;

__device__ __forceinline__ int blocks_of(int nq, int L) {
  return nq > 0 ? max(1, (L + BLOCK_KEYS - 1) / BLOCK_KEYS) : 0;  // without keys: one, for the NaN rows
}

__device__ __forceinline__ int blocks_of(const FwdParams& p, int s) {
  int lo, hi;
  row_range(p.q_offsets, s, p.num_queries, lo, hi);
  return blocks_of(hi - lo, seq_len(p.c, s));
}

// Where block u lies: sequence, block inside it; and the number of all blocks.
struct Place {
  int64_t total;
  int64_t at;  // first block of sequence s
  int s;
};

// The whole CTA (THREADS threads) calls it. `range` of `ranges`; the first or
// the last block of the range is located.
__device__ __forceinline__ Place locate(const FwdParams& p, int range, int ranges, bool last, int64_t& u0, int64_t& u1) {
  __shared__ int64_t warp_sum[WARPS];
  __shared__ int64_t found_at;
  __shared__ int found_s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (p.c.num_seqs + THREADS - 1) / THREADS;
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
  for (int w = 0; w < WARPS; ++w) {
    if (w < warp) before += warp_sum[w];
    total += warp_sum[w];
  }
  u0 = total * range / ranges;
  u1 = total * (range + 1) / ranges;
  const int64_t u = last ? u1 - 1 : u0;
  if (u >= before && u < before + mine) {
    int s = s0;
    int64_t at = before;
    for (; s < s1; ++s) {
      const int n = blocks_of(p, s);
      if (u < at + n) break;
      at += n;
    }
    found_at = at;
    found_s = s;
  }
  __syncthreads();
  return Place{total, found_at, found_s};
}

// ------------------------------------------------------------------ operands
template <bool BF16>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  if constexpr (BF16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

// Two codes as a 16-bit pair: byte `i` of x in the low half, byte `j` of y in
// the high half. F16 e4m3 pairs are 2^-8 of their values (CODE_SCALE).
template <bool BF16, int FMT>
__device__ __forceinline__ uint32_t pair(uint32_t x, uint32_t y, int i, int j) {
  const uint32_t t = __byte_perm(x, y, i | (i << 4) | ((4 + j) << 8) | ((4 + j) << 12));
  if constexpr (FMT == FMT_INT8) {
    if constexpr (BF16) {
      const uint32_t low = (t & 0x007f007fu) | 0x43004300u, sign = (t & 0x00800080u) | 0x43004300u;  // 128 + b, 128 + 128 s
      uint32_t r;
      asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(low), "r"(sign));
      return r;
    } else {
      const uint32_t u = (t & 0x00ff00ffu) ^ 0x64806480u;  // 1024 + (c + 128)
      uint32_t r;
      asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(u), "r"(0x64806480u));
      return r;
    }
  } else if constexpr (BF16) {
    const uint32_t u = (t & 0x80008000u) | ((t >> 4) & 0x07f007f0u);
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(u), "r"(0x7b807b80u));  // 2^120
    return r;
  } else {
    return (t & 0x80008000u) | ((t >> 1) & 0x3f803f80u);
  }
}

template <bool BF16, int FMT>
__device__ __forceinline__ constexpr float code_scale() {
  return !BF16 && FMT == FMT_E4M3 ? 256.f : 1.f;
}

// D / 8 bytes of one key that a lane holds of V, D / 4 of K (words)
template <int N>
__device__ __forceinline__ void load_words(uint32_t* r, const uint8_t* at) {
  if constexpr (N == 2) {
    const uint2 u = __ldg(reinterpret_cast<const uint2*>(at));
    r[0] = u.x; r[1] = u.y;
  } else {
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(at));
    r[0] = u.x; r[1] = u.y; r[2] = u.z; r[3] = u.w;
  }
}

template <int D, int NT>
struct Shared {
  static constexpr int ROW = D + 4;
  static constexpr int O = WARPS * 8 * NT * ROW * 4;  // partial outputs of the warps
  static constexpr int ML = WARPS * 8 * NT * 8;
  static constexpr int Q = NT > 1 ? NT * (D / 16) * 32 * 8 : 0;  // query operands, in fragment order
  static constexpr int BYTES = O + ML + Q;
};

template <int D, bool BF16, int FMT, int NT>
__global__ void __launch_bounds__(THREADS, NT == 1 ? 2 : 1)
    decode_kernel(const __grid_constant__ FwdParams p, int ranges, int64_t ml_offset) {
  constexpr int KS = D / 16;    // 16-element steps of a head
  constexpr int KB = D / 64;    // 64-byte pieces of a key
  constexpr int VW = D / 32;    // words of V a lane holds of one key
  constexpr int ROWS = 8 * NT;
  using SH = Shared<D, NT>;
  extern __shared__ __align__(16) uint8_t smem[];
  float* const so = reinterpret_cast<float*>(smem);
  float2* const sml = reinterpret_cast<float2*>(smem + SH::O);
  uint2* const sq = reinterpret_cast<uint2*>(smem + SH::O + SH::ML);

  const Cache& c = p.c;
  int* const status = c.status;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int h = blockIdx.x % c.Hkv, range = blockIdx.x / c.Hkv;
  const int heads = p.Hq / c.Hkv;
  const size_t step = static_cast<size_t>(c.Hkv) * D;  // bytes from token to token
  const int64_t ntok = static_cast<int64_t>(c.num_pages) * c.page_size;
  const int64_t nscale = static_cast<int64_t>(c.num_pages) * c.Hkv * c.per;
  const int64_t nrows = static_cast<int64_t>(p.num_queries) * p.Hq;
  const uint8_t* const kb = p.k_codes + h * D;
  const uint8_t* const vb = p.v_codes + h * D;
  const bool tiles_in_page = c.page_size % 16 == 0;

  int64_t u0, u1;
  const Place pl = locate(p, range, ranges, false, u0, u1);
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
    const int R = static_cast<int>(min(static_cast<int64_t>(nq) * heads, static_cast<int64_t>(ROWS)));

    // ------------------------------------------------ query rows
    uint32_t qf[NT == 1 ? KS : 1][2];
    auto load_q = [&](int row, int piece, uint32_t (&r)[8]) {  // 16 elements at 64 piece + 16 t
      uint4 x = make_uint4(0u, 0u, 0u, 0u), y = x;
      if (row < R) {
        const int64_t at = static_cast<int64_t>(q_lo + row / heads) * p.Hq + h * heads + row % heads;
        if (in_bounds(status, at, nrows)) {
          const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) + at * D + piece * 64 + t * 16);
          x = __ldg(src);
          y = __ldg(src + 1);
        }
      }
      r[0] = x.x; r[1] = x.y; r[2] = x.z; r[3] = x.w;
      r[4] = y.x; r[5] = y.y; r[6] = y.z; r[7] = y.w;
    };
    if constexpr (NT == 1) {
#pragma unroll
      for (int i = 0; i < KB; ++i) {
        uint32_t r[8];
        load_q(g, i, r);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          qf[4 * i + k][0] = r[2 * k];
          qf[4 * i + k][1] = r[2 * k + 1];
        }
      }
    } else {
      if (warp < NT) {
#pragma unroll
        for (int i = 0; i < KB; ++i) {
          uint32_t r[8];
          load_q(8 * warp + g, i, r);
#pragma unroll
          for (int k = 0; k < 4; ++k) sq[(warp * KS + 4 * i + k) * 32 + lane] = make_uint2(r[2 * k], r[2 * k + 1]);
        }
      }
      __syncthreads();
    }
    int lim[NT][2];  // last key that the lane's rows (8 i + 2 t, + 1) see
    int least = L - 1, most = -1;
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = 8 * i + 2 * t + e;
        int x = -1;
        if (row < R) {
          x = L - 1;
          if (p.causal) {
            const int q = row / heads;
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
    float m[NT][2], l[NT][2], acc[KS][NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      m[i][0] = m[i][1] = -INFINITY;
      l[i][0] = l[i][1] = 0.f;
#pragma unroll
      for (int k = 0; k < KS; ++k) acc[k][i][0] = acc[k][i][1] = acc[k][i][2] = acc[k][i][3] = 0.f;
    }
    float top = 1.17549435e-38f, itop = 8.5070592e37f;  // F16: the power of two that P' is relative to, its inverse
    // Lane (g, t): keys ka and ka + 2 of a tile in S^T; keys 4 t .. 4 t + 3 in V^T
    const int ka = 4 * (g >> 1) + (g & 1);
    // token (page * page_size + row) of keys j and j + 2, -1 for zeros
    auto tokens = [&](int key0, int& x, int& y) {
      if (tiles_in_page) {
        const int blk = key0 / c.page_size;
        const int page = key0 < L ? page_of(c, s, blk) : -1;
        const int base = page * c.page_size + (key0 - blk * c.page_size) + ka;
        x = page >= 0 && key0 + ka < L ? base : -1;
        y = page >= 0 && key0 + ka + 2 < L ? base + 2 : -1;
      } else {
        auto one = [&](int j) {
          if (j >= L) return -1;
          const int blk = j / c.page_size, page = page_of(c, s, blk);
          return page >= 0 ? page * c.page_size + (j - blk * c.page_size) : -1;
        };
        x = one(key0 + ka);
        y = one(key0 + ka + 2);
      }
    };
    uint32_t kr[2][KB * 4], vr[4][VW];
    float ks[2], vs[2];
    auto load_k = [&](int x, int y) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int tok = e ? y : x;
        const bool ok = tok >= 0 && in_bounds(status, tok, ntok);
        const uint8_t* at = kb + (ok ? static_cast<size_t>(tok) * step : 0) + t * 16;
#pragma unroll
        for (int i = 0; i < KB; ++i) load_words<4>(&kr[e][4 * i], at + 64 * i);
        ks[e] = vs[e] = 0.f;
        if (ok) {
          const int page = tok / c.page_size;
          const size_t si = scale_index(c, page, tok - page * c.page_size, h);
          if (in_bounds(status, static_cast<int64_t>(si), nscale)) {
            ks[e] = __ldg(p.k_scale + si) * (p.scale_log2 * code_scale<BF16, FMT>());
            vs[e] = __ldg(p.v_scale + si) * code_scale<BF16, FMT>();
          }
        }
      }
    };
    auto load_v = [&](int x, int y) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int tok = __shfl_sync(0xffffffffu, i < 2 ? x : y, (2 * t + (i & 1)) * 4);
        const bool ok = tok >= 0 && in_bounds(status, tok, ntok);
        load_words<VW>(vr[i], vb + (ok ? static_cast<size_t>(tok) * step : 0) + g * (D / 8));
      }
    };
    const int key_end = most + 1;
    const int last_key = min(key_end, (b + take) * BLOCK_KEYS);
    int key0 = b * BLOCK_KEYS + warp * 16;
    int nx, ny;  // tokens of the tile to load next
    if (key0 < last_key) {
      tokens(key0, nx, ny);
      load_k(nx, ny);
      load_v(nx, ny);
    }
    for (; key0 < last_key; key0 += BLOCK_KEYS) {
      const bool more = key0 + BLOCK_KEYS < last_key;
      if (more) tokens(key0 + BLOCK_KEYS, nx, ny);
      float sc[NT][4];
#pragma unroll
      for (int i = 0; i < NT; ++i) sc[i][0] = sc[i][1] = sc[i][2] = sc[i][3] = 0.f;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        const uint32_t a0 = pair<BF16, FMT>(kr[0][k], kr[0][k], 0, 1), a1 = pair<BF16, FMT>(kr[1][k], kr[1][k], 0, 1);
        const uint32_t a2 = pair<BF16, FMT>(kr[0][k], kr[0][k], 2, 3), a3 = pair<BF16, FMT>(kr[1][k], kr[1][k], 2, 3);
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          uint32_t b0, b1;
          if constexpr (NT == 1) {
            b0 = qf[k][0];
            b1 = qf[k][1];
          } else {
            const uint2 w = sq[(i * KS + k) * 32 + lane];
            b0 = w.x;
            b1 = w.y;
          }
          mma16816<BF16>(sc[i], a0, a1, a2, a3, b0, b1);
        }
      }
      const float k0 = ks[0], k1 = ks[1], v0 = vs[0], v1 = vs[1];
      if (more) load_k(nx, ny);

      // scores (log2 units) of keys key0 + ka and + 2
      const bool masked = key0 + 15 > least;
      bool grow = false;
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        sc[i][0] *= k0;
        sc[i][1] *= k0;
        sc[i][2] *= k1;
        sc[i][3] *= k1;
        if (masked) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            if (key0 + ka > lim[i][e]) sc[i][e] = -INFINITY;
            if (key0 + ka + 2 > lim[i][e]) sc[i][2 + e] = -INFINITY;
          }
        }
        grow = grow || fmaxf(sc[i][0], sc[i][2]) > m[i][0] + RESCALE_LOG2 ||
               fmaxf(sc[i][1], sc[i][3]) > m[i][1] + RESCALE_LOG2;
      }
      if constexpr (!BF16) grow = grow || fmaxf(v0, v1) > top;
      if (__any_sync(0xffffffffu, grow)) {
        float ratio = 1.f;
        if constexpr (!BF16) {
          float x = fmaxf(v0, v1);
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
          if (x > top) {  // the power of two above x (or 2^126)
            const float n = __uint_as_float(min((__float_as_uint(x) & 0x7f800000u) + 0x00800000u, 0x7e800000u));
            ratio = top / n;
            top = n;
            itop = 1.f / n;
          }
        }
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float x = fmaxf(sc[i][e], sc[i][2 + e]);
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
            const float n = fmaxf(m[i][e], x);
            const float alpha = n == -INFINITY ? 1.f : fast_exp2(m[i][e] - n);
            m[i][e] = n;
            l[i][e] *= alpha;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
              acc[k][i][e] *= alpha * ratio;
              acc[k][i][2 + e] *= alpha * ratio;
            }
          }
      }
      const float w0 = BF16 ? v0 : v0 * itop, w1 = BF16 ? v1 : v1 * itop;
      uint32_t pf[NT][2];
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        float x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float n = m[i][e & 1];
          const float y = fast_exp2(sc[i][e] - (n == -INFINITY ? 0.f : n));
          l[i][e & 1] += y;
          // a masked key may have any scale
          x[e] = masked && sc[i][e] == -INFINITY ? 0.f : y * (e < 2 ? w0 : w1);
        }
        pf[i][0] = transpose8x8(pack2<BF16>(x[0], x[1]));
        pf[i][1] = transpose8x8(pack2<BF16>(x[2], x[3]));
      }
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        const int w = k / 2, o = (k & 1) * 2;  // bytes 2 k and 2 k + 1 of the lane's
        const uint32_t a0 = pair<BF16, FMT>(vr[0][w], vr[1][w], o, o), a1 = pair<BF16, FMT>(vr[0][w], vr[1][w], o + 1, o + 1);
        const uint32_t a2 = pair<BF16, FMT>(vr[2][w], vr[3][w], o, o), a3 = pair<BF16, FMT>(vr[2][w], vr[3][w], o + 1, o + 1);
#pragma unroll
        for (int i = 0; i < NT; ++i) mma16816<BF16>(acc[k][i], a0, a1, a2, a3, pf[i][0], pf[i][1]);
      }
      if (more) load_v(nx, ny);
    }

    // ------------------------------------------------ the warps' parts
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l[i][e] += __shfl_xor_sync(0xffffffffu, l[i][e], o);
        const int row = 8 * i + 2 * t + e;
        if (g == 0) sml[warp * ROWS + row] = make_float2(m[i][e], l[i][e]);
        float* const o = so + (warp * ROWS + row) * SH::ROW + g * (D / 8);
#pragma unroll
        for (int k = 0; k < KS; ++k)
          *reinterpret_cast<float2*>(o + 2 * k) = make_float2(BF16 ? acc[k][i][e] : acc[k][i][e] * top,
                                                              BF16 ? acc[k][i][2 + e] : acc[k][i][2 + e] * top);
      }
    __syncthreads();
    const int64_t slot = 2ll * blockIdx.x + (first ? 0 : 1);
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
        const int64_t at = static_cast<int64_t>(q_lo + row / heads) * p.Hq + h * heads + row % heads;
        if (!in_bounds(status, at, nrows)) continue;
        reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at * D)[d4] =
            make_uint2(pack2<BF16>(o.x * inv, o.y * inv), pack2<BF16>(o.z * inv, o.w * inv));
        if (p.lse && d4 == 0) p.lse[at] = live ? (M + log2f(sum)) * LN2 : (sum == 0.f ? -INFINITY : sum);
      } else {
        const int64_t at = slot * ROWS + row;
        if (!in_bounds(status, at, 2ll * ranges * c.Hkv * ROWS)) continue;
        reinterpret_cast<float4*>(p.ws)[at * (D / 4) + d4] = o;
        if (d4 == 0) reinterpret_cast<float2*>(static_cast<uint8_t*>(p.ws) + ml_offset)[at] = make_float2(M, sum);
      }
    }
    __syncthreads();
  }
}

// A CTA (range, head; blockIdx.y: row) combines the parts of the sequence that
// begins in the range and goes on past it: its own last slot, then the first
// slot of the ranges after it.
template <int D, bool BF16>
__global__ void __launch_bounds__(THREADS) merge_kernel(const __grid_constant__ FwdParams p, int ranges, int ROWS,
                                                        int64_t ml_offset) {
  constexpr int G = D / 4;
  __shared__ float4 so[WARPS * 32 / G][G];
  __shared__ float2 sml[WARPS * 32 / G];
  const Cache& c = p.c;
  const int h = blockIdx.x % c.Hkv, range = blockIdx.x / c.Hkv, row = blockIdx.y;
  int64_t u0, u1;
  const Place pl = locate(p, range, ranges, true, u0, u1);
  if (u1 <= u0 || pl.at < u0) return;  // CTA-uniform, as every return below
  int q_lo, q_hi;
  row_range(p.q_offsets, pl.s, p.num_queries, q_lo, q_hi);
  const int heads = p.Hq / c.Hkv;
  const int64_t end = pl.at + blocks_of(q_hi - q_lo, seq_len(c, pl.s));
  if (end <= u1 || row >= static_cast<int64_t>(q_hi - q_lo) * heads) return;
  int last = range;  // the range that holds the sequence's last block
  while (pl.total * (last + 1) / ranges < end) ++last;
  const float4* const wo = static_cast<const float4*>(p.ws);
  const float2* const wml = reinterpret_cast<const float2*>(static_cast<const uint8_t*>(p.ws) + ml_offset);
  const int g = threadIdx.x % G, part0 = threadIdx.x / G, parts = THREADS / G;
  float M = -INFINITY, sum = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int r = range + part0; r <= last; r += parts) {
    const int64_t a = pl.total * r / ranges, b = pl.total * (r + 1) / ranges;
    if (a == b) continue;
    const int64_t at = (2ll * (static_cast<int64_t>(r) * c.Hkv + h) + (r == range && pl.at > u0 ? 1 : 0)) * ROWS + row;
    if (!in_bounds(c.status, at, 2ll * ranges * c.Hkv * ROWS)) continue;
    const float2 ml = wml[at];
    const float4 x = wo[at * G + g];
    const float n = fmaxf(M, ml.x);
    const float f = n == -INFINITY ? 0.f : fast_exp2(M - n), e = n == -INFINITY ? 0.f : fast_exp2(ml.x - n);
    M = n;
    sum = sum * f + ml.y * e;
    o = make_float4(o.x * f + x.x * e, o.y * f + x.y * e, o.z * f + x.z * e, o.w * f + x.w * e);
  }
  so[part0][g] = o;
  if (g == 0) sml[part0] = make_float2(M, sum);
  __syncthreads();
  if (part0 != 0) return;
  for (int i = 1; i < parts; ++i) {
    const float2 ml = sml[i];
    const float4 x = so[i][g];
    const float n = fmaxf(M, ml.x);
    const float f = n == -INFINITY ? 0.f : fast_exp2(M - n), e = n == -INFINITY ? 0.f : fast_exp2(ml.x - n);
    M = n;
    sum = sum * f + ml.y * e;
    o = make_float4(o.x * f + x.x * e, o.y * f + x.y * e, o.z * f + x.z * e, o.w * f + x.w * e);
  }
  const bool live = sum > 0.f;
  const float inv = live ? 1.f / sum : __int_as_float(0x7fc00000);
  const int64_t at = static_cast<int64_t>(q_lo + row / heads) * p.Hq + h * heads + row % heads;
  if (!in_bounds(c.status, at, static_cast<int64_t>(p.num_queries) * p.Hq)) return;
  reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at * D)[g] =
      make_uint2(pack2<BF16>(o.x * inv, o.y * inv), pack2<BF16>(o.z * inv, o.w * inv));
  if (p.lse && g == 0) p.lse[at] = live ? (M + log2f(sum)) * LN2 : (sum == 0.f ? -INFINITY : sum);
}

template <int D, bool BF16, int FMT, int NT>
cudaError_t launch_nt(const FwdParams& p, int ranges, cudaStream_t st) {
  auto kern = decode_kernel<D, BF16, FMT, NT>;
  constexpr int smem = Shared<D, NT>::BYTES;
  cudaError_t e = cudaSuccess;
  if (smem > 48 * 1024) e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const DecodeLayout lay{2ll * ranges * p.c.Hkv, 8 * NT};
  const unsigned ctas = static_cast<unsigned>(ranges) * p.c.Hkv;
  kern<<<ctas, THREADS, smem, st>>>(p, ranges, lay.ml_offset(D));
  e = cudaGetLastError();
  if (e != cudaSuccess || ranges == 1) return e;
  const int rows = min(p.max_queries * (p.Hq / p.c.Hkv), 8 * NT);
  merge_kernel<D, BF16><<<dim3(ctas, rows), THREADS, 0, st>>>(p, ranges, 8 * NT, lay.ml_offset(D));
  return cudaGetLastError();
}

template <int D, bool BF16, int FMT>
cudaError_t launch_d(const FwdParams& p, int ranges, cudaStream_t st) {
  const int64_t rows = static_cast<int64_t>(p.max_queries) * (p.Hq / p.c.Hkv);
  if (rows <= 8) return launch_nt<D, BF16, FMT, 1>(p, ranges, st);
  if (rows <= 16) return launch_nt<D, BF16, FMT, 2>(p, ranges, st);
  return launch_nt<D, BF16, FMT, 4>(p, ranges, st);
}

}  // namespace dec

template <bool BF16>
cudaError_t launch_decode(const FwdParams& p, int fmt, cudaStream_t st) {
  const int ranges = decode_ranges(p.c.num_seqs, p.c.Hkv, p.c.max_pages, p.c.page_size);
  if (fmt == FMT_INT8)
    return p.c.D == 128 ? dec::launch_d<128, BF16, FMT_INT8>(p, ranges, st) : dec::launch_d<64, BF16, FMT_INT8>(p, ranges, st);
  return p.c.D == 128 ? dec::launch_d<128, BF16, FMT_E4M3>(p, ranges, st) : dec::launch_d<64, BF16, FMT_E4M3>(p, ranges, st);
}

}  // namespace kv8
}  // namespace attn
