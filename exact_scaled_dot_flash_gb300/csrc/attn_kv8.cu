// attn_kv8.cu - writing keys and values into an 8-bit paged cache, and reading
// the cache back (layout and codes: kv8.cuh).
//
// Write. The n new tokens of sequence s are its last: positions L - n .. L - 1.
// A group is `group` consecutive tokens of one page with one scale per head.
// For every group that receives a token, with a = max |x| over the new tokens
// in it:
//   int8: t = fl32(a / 127);   e4m3: t = the least power of two >= a / 448,
// not below 2^-100. If the group begins with tokens of an earlier call, its
// scale may only grow, S = max(S_old, t), and when it does their codes become
// the nearest code of c * S_old / S; else S = t. New codes are the nearest code
// of x / S, ties to the even code, exactly: an fp32 quotient can be rounded
// onto a tie, so the int8 code is settled by its residual x - r S, which fp32
// holds exactly (see nearest8), and the e4m3 scale, a power of two, divides
// exactly (a float format gains nothing from a finer scale; one that another
// program left in a part-filled group divides with its remainder). A NaN or infinity
// among the new tokens makes the group's scale NaN: the group then reads as
// NaN until a call writes its first token again.
// Bytes: the new tokens are read once and one byte written for each element. 32
// prompts of 500-2000 tokens, 8 heads, D 128, F16 to e4m3: 52 us, to int8: 58 us (37
// by bytes); instructions are the bound (74% of the issue slots). From F32: 78 and 82
// (62 by bytes).
//
// Read. Row i of sequence s is its token starts[s] + i; value = code * scale,
// rounded once to the output type. Bound by the bytes: 640M elements to F32 490 us,
// 6.5 TB/s, 98% of the copy bandwidth.
#include <math.h>

#include <type_traits>

#include "attn.h"
#include "host_checks.h"
#include "kv8.cuh"
#include "simt.cuh"

namespace attn {
namespace kv8 {

constexpr int THREADS = 256;
constexpr int WRITE_UNITS = 8;

struct WriteParams {
  Cache c;
  int num_tokens;
  const int32_t* off;    // [num_seqs + 1] rows of each sequence's new tokens
  const void* x[2];      // k, v
  int64_t xt[2], xh[2];  // token and head strides (elements)
  uint8_t* codes[2];
  float* scales[2];
};

// ------------------------------------------------------------------ element access
// 8 elements as they lie in memory (16-bit types: 4 registers).
template <int DT>
struct Raw8 {
  uint4 w[DT == 0 ? 2 : 1];
};

template <int DT, bool VEC>
__device__ __forceinline__ Raw8<DT> load_raw(const uint8_t* at) {
  Raw8<DT> r;
  if constexpr (VEC) {
#pragma unroll
    for (int k = 0; k < (DT == 0 ? 2 : 1); ++k) r.w[k] = __ldg(reinterpret_cast<const uint4*>(at) + k);
  } else {
    using E = std::conditional_t<DT == 0, uint32_t, uint16_t>;
    E* const e = reinterpret_cast<E*>(r.w);
#pragma unroll
    for (int k = 0; k < 8; ++k) e[k] = __ldg(reinterpret_cast<const E*>(at) + k);
  }
  return r;
}

template <int DT>
__device__ __forceinline__ void expand(const Raw8<DT>& r, float (&x)[8]) {
  if constexpr (DT == 0) {
    const float* const f = reinterpret_cast<const float*>(r.w);
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = f[k];
  } else {
    const uint32_t* const w = reinterpret_cast<const uint32_t*>(r.w);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 f = DT == 1 ? __half22float2(*reinterpret_cast<const __half2*>(w + k))
                               : make_float2(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xffff0000u));
      x[2 * k] = f.x;
      x[2 * k + 1] = f.y;
    }
  }
}

// The integer nearest to x / s (ties to even), |x| <= 127 s up to rounding.
// r = rint(x * (1/s)) is off by at most one; d = x - r s is exact (for r != 0
// it is a multiple of s's last place of at most 24 bits), so comparing |d| with
// s / 2 decides it.
__device__ __forceinline__ int nearest8(float x, float s, float inv) {
  float r = rintf(x * inv);
  const float d = fmaf(-r, s, x), h = 0.5f * s;
  const float step = d > 0.f ? 1.f : -1.f;
  if (fabsf(d) > h || (fabsf(d) == h && (static_cast<int>(r) & 1))) r += step;
  return static_cast<int>(fminf(fmaxf(r, -127.f), 127.f));
}

// Four of them: rounded by the addition of 1.5 * 2^23, whose sum holds the
// integer in its low byte; only where a residual reaches s / 2 are they settled
// one by one.
__device__ __forceinline__ uint32_t nearest8x4(const float* x, float s, float inv) {
  constexpr float ROUND = 12582912.f;
  float q[4], worst = 0.f;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    q[k] = fmaf(x[k], inv, ROUND);
    worst = fmaxf(worst, fabsf(fmaf(ROUND - q[k], s, x[k])));
  }
  if (worst >= 0.5f * s) {
    uint32_t w = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) w |= (static_cast<uint32_t>(nearest8(x[k], s, inv)) & 0xffu) << (8 * k);
    return w;
  }
  const uint32_t lo = __byte_perm(__float_as_uint(q[0]), __float_as_uint(q[1]), 0x0040);
  const uint32_t hi = __byte_perm(__float_as_uint(q[2]), __float_as_uint(q[3]), 0x0040);
  return __byte_perm(lo, hi, 0x5410);
}

// max(|a|, |b|), a NaN if either is one.
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// Running maximum of |x| over raw vectors, NaN once one was met; an infinity
// stays. 16-bit types keep two halves of a register.
template <int DT>
struct AbsMax {
  uint32_t m = 0;
  __device__ __forceinline__ void add(const Raw8<DT>& r) {
    const uint32_t* const w = reinterpret_cast<const uint32_t*>(r.w);
    if constexpr (DT == 0) {
#pragma unroll
      for (int k = 0; k < 8; ++k) m = __float_as_uint(max_nan(__uint_as_float(m), __uint_as_float(w[k] & 0x7fffffffu)));
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if constexpr (DT == 1) asm("max.NaN.f16x2 %0, %0, %1;" : "+r"(m) : "r"(w[k] & 0x7fff7fffu));
        else asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(w[k] & 0x7fff7fffu));
      }
    }
  }
  __device__ __forceinline__ float value() const {
    if constexpr (DT == 0) return __uint_as_float(m);
    else if constexpr (DT == 1) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&m));
      return max_nan(f.x, f.y);
    } else {
      return max_nan(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
    }
  }
};

// The 4 e4m3 codes nearest to q.
__device__ __forceinline__ uint32_t e4m3x4(const float* q) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(q[1]), "f"(q[0]));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(q[3]), "f"(q[2]));
  return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

__device__ __forceinline__ bool power_of_two(float s) { return (__float_as_uint(s) & 0x7fffffu) == 0; }

// q, off the exact value by d's sign and less than its own last place: cut towards
// zero, with the lowest bit set for what was cut away, so that the conversion to
// fewer bits is the only rounding.
__device__ __forceinline__ float cut_odd(float q, float d) {
  const uint32_t b = __float_as_uint(q);
  return d == 0.f || q == 0.f ? q : __uint_as_float((b - ((d < 0.f) != (q < 0.f) ? 1u : 0u)) | 1u);
}

// The e4m3 codes nearest to x / s for any s, ties to even. The remainder x - q s is
// exact wherever q could be a border of two codes (q has 5 bits then).
__device__ __forceinline__ uint32_t e4m3x4_over(const float* x, float s) {
  float q[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    q[k] = __fdiv_rn(x[k], s);
    q[k] = cut_odd(q[k], fmaf(-q[k], s, x[k]));
  }
  return e4m3x4(q);
}

template <int FMT>
__device__ __forceinline__ uint32_t encode4(const float* x, float s, float inv) {
  if constexpr (FMT == FMT_INT8) {
    return nearest8x4(x, s, inv);
  } else {
    const float q[4] = {x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv};
    return e4m3x4(q);
  }
}

// Codes of c * s_old / s for s > s_old. int8: the fp32 product is within 2^-15 of
// the quotient (|c| <= 128); only one that lies that near a tie is settled in
// fp64. e4m3: s > s_old is a power of two (the writer's), the ratio exact.
template <int FMT>
__device__ __forceinline__ uint32_t recode4(uint32_t w, float s_old, float s) {
  const float4 v = decode4<FMT>(w);
  const float c[4] = {v.x, v.y, v.z, v.w};
  const float ratio = s_old / s;
  if constexpr (FMT == FMT_INT8) {
    uint32_t o = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float q = c[k] * ratio;
      float r = rintf(q);
      if (fabsf(fabsf(q - r) - 0.5f) < 6.103515625e-5f)
        r = static_cast<float>(rint(static_cast<double>(c[k]) * static_cast<double>(s_old) / static_cast<double>(s)));
      o |= (static_cast<uint32_t>(static_cast<int>(r)) & 0xffu) << (8 * k);
    }
    return o;
  } else {
    float q[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float p = c[k] * ratio;
      q[k] = cut_odd(p, fmaf(c[k], ratio, -p));
    }
    return e4m3x4(q);
  }
}

template <int FMT>
__device__ __forceinline__ float scale_of(float amax) {
  if constexpr (FMT == FMT_INT8) {
    return fmaxf(__fdiv_rn(amax, 127.f), SCALE_FLOOR);
  } else {
    const uint32_t b = __float_as_uint(amax);  // amax = 1.m 2^(e - 127); 448 = 1.75 * 2^8
    int e = static_cast<int>(b >> 23) - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
    e = max(e, 27);  // 2^-100
    return __uint_as_float(static_cast<uint32_t>(e) << 23);
  }
}

// ------------------------------------------------------------------ write
// Work items ("slots") of sequence s: one for each group its new tokens may
// touch, from base(s) = off[s] / group + 2 s on. n tokens touch at most
// floor((n + group - 2) / group) + 1 <= floor(n / group) + 2 groups, so the
// slots of different sequences never meet, and base is monotone: the sequence
// of a slot is found by a search that reads 128 offsets at a time.
__device__ __forceinline__ int seq_of_slot(const int32_t* off, int num_seqs, int group, int num_tokens, int slot,
                                           int lane) {
  int lo = 0, n = num_seqs;  // the answer is in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 127) / 128;
    int o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int64_t at = static_cast<int64_t>(32 * k + lane) * step;
      o[k] = at < n ? __ldg(off + lo + at) : 0;
    }
    int last = -1;  // starts at or before the slot
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int64_t at = static_cast<int64_t>(32 * k + lane) * step;
      const bool in = at < n && static_cast<int64_t>(min(max(o[k], 0), num_tokens) / group) + 2 * (lo + at) <= slot;
      const unsigned m = __ballot_sync(0xffffffffu, in);
      if (m) last = 32 * k + 31 - __clz(m);
    }
    const int end = lo + n;
    lo += max(last, 0) * step;
    n = min(step, end - lo);
  }
  return lo;
}

// TPU threads (a warp, or the CTA) hold one unit: a (slot, head, k or v). The
// elements are kept in registers between the maximum and the codes, KEEP
// vectors of 8 a thread, as they lie in memory: as fp32 they left room for half
// the CTAs, and a CTA is a chain of dependent reads (offsets, lengths, table,
// tokens) that only other CTAs hide. A larger group reads the rest a second time.
template <int DT, int FMT, bool VEC, int TPU>
__global__ void __launch_bounds__(THREADS, DT == 0 ? 2 : 4) write_kernel(const __grid_constant__ WriteParams p, int units) {
  constexpr int KEEP = 4;
  __shared__ float red[THREADS / 32];
  const Cache& c = p.c;
  const int lane = threadIdx.x & 31;
  const int tu = threadIdx.x % TPU;
  // units of this thread: head, then k / v, side by side and `units` in turn
  constexpr int SIDE = THREADS / TPU;
  const int unit0 = blockIdx.y * SIDE * units + threadIdx.x / TPU;
  if (unit0 >= 2 * c.Hkv) return;  // a whole warp (TPU 32) or no thread (TPU 256) returns
  const int slot = blockIdx.x;
  const int s = seq_of_slot(p.off, c.num_seqs, c.group, p.num_tokens, slot, lane);
  int lo, hi;
  row_range(p.off, s, p.num_tokens, lo, hi);
  const int n = hi - lo, L = seq_len(c, s);
  const int64_t first = static_cast<int64_t>(max(L - n, 0));  // tokens before position 0 are not written
  const int64_t nth = static_cast<int64_t>(slot) - (lo / c.group + 2ll * s);  // group of the sequence's new tokens
  const int64_t g0 = (first / c.group + nth) * c.group;                       // its first position
  if (n <= 0 || nth < 0 || g0 >= L) return;
  const int page = page_of(c, s, static_cast<int>(g0 / c.page_size));
  if (page < 0) return;
  const int row0 = static_cast<int>(g0 % c.page_size);
  const int held = static_cast<int>(max(first - g0, static_cast<int64_t>(0)));  // tokens of earlier calls
  const int m = static_cast<int>(min(static_cast<int64_t>(c.group), L - g0)) - held;  // new tokens
  const int64_t x0 = lo + (g0 + held - (static_cast<int64_t>(L) - n));  // row of the first of them
  const int vpt = c.D >> 3, sh = __ffs(vpt) - 1;  // vectors of a token
  // The thread's vectors of a unit: column `col` of tokens t0, t0 + tinc, ... (TPU
  // is a multiple of vpt): an addition from one to the next.
  const int t0 = tu >> sh, col = tu & (vpt - 1), tinc = TPU >> sh;
  const int64_t cstep = static_cast<int64_t>(c.Hkv) * c.D;
  const int64_t ncode8 = static_cast<int64_t>(c.num_pages) * c.page_size * c.Hkv * vpt;
  const int64_t nscale = static_cast<int64_t>(c.num_pages) * c.Hkv * c.per;
  constexpr int ES = DT == 0 ? 4 : 2;
  auto source = [&](int unit) {  // of the thread's first vector
    const int kv = unit >= c.Hkv ? 1 : 0, h = unit - kv * c.Hkv;
    return static_cast<const uint8_t*>(p.x[kv]) + ((x0 + t0) * p.xt[kv] + h * p.xh[kv] + col * 8) * ES;
  };
  auto stride = [&](int unit) { return p.xt[unit >= c.Hkv ? 1 : 0] * (tinc * ES); };
  Raw8<DT> next[KEEP];
  auto fetch = [&](int unit) {
    const uint8_t* at = source(unit);
    const int64_t inc = stride(unit);
#pragma unroll
    for (int i = 0; i < KEEP; ++i, at += inc)
      if (t0 + i * tinc < m) next[i] = load_raw<DT, VEC>(at);
  };
  fetch(unit0);
  uint32_t odd = 0;  // units whose scale is no power of two (e4m3)
  for (int u = 0; u < units; ++u) {
    const int unit = unit0 + u * SIDE;
    if (unit >= 2 * c.Hkv) break;
    const int kv = unit >= c.Hkv ? 1 : 0, h = unit - kv * c.Hkv;
    Raw8<DT> keep[KEEP];
#pragma unroll
    for (int i = 0; i < KEEP; ++i) keep[i] = next[i];
    if (u + 1 < units && unit + SIDE < 2 * c.Hkv) fetch(unit + SIDE);  // on their way under this unit's work
    AbsMax<DT> most;
#pragma unroll
    for (int i = 0; i < KEEP; ++i)
      if (t0 + i * tinc < m) most.add(keep[i]);
    if (t0 + KEEP * tinc < m) {  // what the registers do not keep
      const int64_t inc = stride(unit);
      const uint8_t* at = source(unit) + KEEP * inc;
      for (int t = t0 + KEEP * tinc; t < m; t += tinc, at += inc) most.add(load_raw<DT, VEC>(at));
    }
    float amax = most.value();
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if constexpr (TPU > 32) {
      if (lane == 0) red[threadIdx.x >> 5] = amax;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < TPU / 32; ++w) amax = max_nan(amax, red[w]);
    }
    const size_t si = scale_index(c, page, row0, h);
    if (!in_bounds(c.status, static_cast<int64_t>(si), nscale)) return;  // the same for all of the unit's threads
    float* const sc = p.scales[kv] + si;
    float sn = amax < INFINITY ? scale_of<FMT>(amax) : __int_as_float(0x7fc00000);
    float so = 0.f;
    if (held > 0) {
      so = *sc;
      sn = (so != so || sn != sn) ? __int_as_float(0x7fc00000) : fmaxf(so, sn);
    }
    if constexpr (TPU > 32) __syncthreads();  // every thread has read the old scale
    else __syncwarp();
    if (tu == 0) *sc = sn;
    const size_t cbase = ((static_cast<size_t>(page) * c.page_size + row0) * c.Hkv + h) * c.D;
    // of the group's token `held` + t0
    uint8_t* const dst = p.codes[kv] + cbase + (held + t0) * cstep + col * 8;
    const int64_t dinc = tinc * cstep;
    const float inv = 1.f / sn;
    auto inside = [&](const uint8_t* at) { return in_bounds(c.status, (at - p.codes[kv]) >> 3, ncode8); };
    auto put = [&](uint8_t* at, const Raw8<DT>& r) {
      float v[8];
      expand<DT>(r, v);
      if (!inside(at)) return;
      // a group without a scale (NaN) gets zero codes
      *reinterpret_cast<uint2*>(at) =
          sn == sn ? make_uint2(encode4<FMT>(v, sn, inv), encode4<FMT>(v + 4, sn, inv)) : make_uint2(0u, 0u);
    };
#pragma unroll
    for (int i = 0; i < KEEP; ++i)
      if (t0 + i * tinc < m) put(dst + i * dinc, keep[i]);
    if (t0 + KEEP * tinc < m) {
      const int64_t inc = stride(unit);
      const uint8_t* at = source(unit) + KEEP * inc;
      uint8_t* to = dst + KEEP * dinc;
      for (int t = t0 + KEEP * tinc; t < m; t += tinc, at += inc, to += dinc) put(to, load_raw<DT, VEC>(at));
    }
    if (held > 0 && sn > so) {  // the codes of earlier calls, at the larger scale
      uint8_t* at = dst - held * cstep;
      for (int t = t0; t < held; t += tinc, at += dinc) {
        if (!inside(at)) continue;
        const uint2 w = *reinterpret_cast<const uint2*>(at);
        *reinterpret_cast<uint2*>(at) = make_uint2(recode4<FMT>(w.x, so, sn), recode4<FMT>(w.y, so, sn));
      }
    }
    if (FMT == FMT_E4M3 && sn == sn && !power_of_two(sn)) odd |= 1u << u;
  }
  if (FMT == FMT_E4M3 && odd) {  // the same for all of a unit's threads; only where held > 0
    // part-filled groups whose scale is another program's: the new tokens once more
    if constexpr (TPU > 32) __syncthreads();  // the scales are written
    else __syncwarp();
    for (; odd; odd &= odd - 1) {
      const int unit = unit0 + (__ffs(odd) - 1) * SIDE;
      const int kv = unit >= c.Hkv ? 1 : 0, h = unit - kv * c.Hkv;
      const float sn = p.scales[kv][scale_index(c, page, row0, h)];
      const uint8_t* at = source(unit);
      uint8_t* to = p.codes[kv] + ((static_cast<size_t>(page) * c.page_size + row0) * c.Hkv + h) * c.D +
                    (held + t0) * cstep + col * 8;
      for (int t = t0; t < m; t += tinc, at += stride(unit), to += tinc * cstep) {
        float v[8];
        expand<DT>(load_raw<DT, VEC>(at), v);
        if (in_bounds(c.status, (to - p.codes[kv]) >> 3, ncode8))
          *reinterpret_cast<uint2*>(to) = make_uint2(e4m3x4_over(v, sn), e4m3x4_over(v + 4, sn));
      }
    }
  }
}

template <int DT, int FMT, bool VEC>
cudaError_t launch_write(const WriteParams& p, cudaStream_t st) {
  const unsigned slots = static_cast<unsigned>(p.num_tokens / p.c.group + 2 * p.c.num_seqs);
  // A warp keeps up to 1024 elements of a unit in registers, the CTA 8192. What
  // counts is the tokens that a unit gets: at most a group, and about those of a
  // sequence (64 sequences of one token, group 16: 6 us by warps, 16 us by CTAs).
  const int64_t tokens = (static_cast<int64_t>(p.num_tokens) + p.c.num_seqs - 1) / p.c.num_seqs;
  if (min(static_cast<int64_t>(p.c.group), tokens) * p.c.D <= 1024) {
    constexpr int SIDE = THREADS / 32;
    write_kernel<DT, FMT, VEC, 32><<<dim3(slots, (2 * p.c.Hkv + SIDE - 1) / SIDE), THREADS, 0, st>>>(p, 1);
  } else {
    // a CTA that takes several heads in turn finds its tokens once for all of
    // them; where that leaves two CTAs an SM (32 prompts and reading them back:
    // 94 us, 114 one by one; 8: 32 and 36; 4, too few: 21 and 19; 1: 15 and 9)
    const int units = static_cast<int64_t>(slots) * 2 * p.c.Hkv >= 2ll * SMS * WRITE_UNITS ? WRITE_UNITS : 1;
    write_kernel<DT, FMT, VEC, THREADS><<<dim3(slots, (2 * p.c.Hkv + units - 1) / units), THREADS, 0, st>>>(p, units);
  }
  return cudaGetLastError();
}

// ------------------------------------------------------------------ read
struct ReadParams {
  Cache c;
  int num_rows;
  const int32_t* off;     // [num_seqs + 1] output rows of each sequence
  const int32_t* starts;  // [num_seqs] first token of each sequence, or nullptr (0)
  const uint8_t* codes[2];
  const float* scales[2];
  void* out[2];
};

constexpr int READ_ROWS = 8;  // output rows of a CTA

// Codes of a thread and step: 16, but 4 for F32, so that the lanes' 16-byte
// stores lie side by side (640M elements: 492 us; 576 us with 8, 788 us with 16).
template <int DT>
constexpr int READ_PIECE = DT == 0 ? 4 : 16;
template <int DT>
using ReadWord = std::conditional_t<READ_PIECE<DT> == 4, uint32_t, uint4>;

template <int DT, int FMT>
__device__ __forceinline__ void store_piece(void* out, size_t o, ReadWord<DT> w, float s) {
  if constexpr (DT == 0) {
    const float4 v = decode4<FMT>(w);
    reinterpret_cast<float4*>(out)[o] = make_float4(v.x * s, v.y * s, v.z * s, v.w * s);
  } else {
    const uint32_t* const c = reinterpret_cast<const uint32_t*>(&w);
    uint32_t r[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float4 v = decode4<FMT>(c[k]);
      r[2 * k] = pack2<DT == 2>(v.x * s, v.y * s);
      r[2 * k + 1] = pack2<DT == 2>(v.z * s, v.w * s);
    }
    reinterpret_cast<uint4*>(out)[2 * o] = make_uint4(r[0], r[1], r[2], r[3]);
    reinterpret_cast<uint4*>(out)[2 * o + 1] = make_uint4(r[4], r[5], r[6], r[7]);
  }
}

// A CTA finds its rows' places in the cache once; then a thread keeps its
// piece of a row (all heads side by side) and goes through the rows, the codes
// of k and v in flight together.
template <int DT, int FMT>
__global__ void __launch_bounds__(THREADS) read_kernel(const __grid_constant__ ReadParams p) {
  __shared__ int64_t code_s[READ_ROWS], scale_s[READ_ROWS];  // token, and its scale of head 0; -1: zeros; -2: no row
  const Cache& c = p.c;
  const int r0 = blockIdx.x * READ_ROWS;
  if (threadIdx.x < READ_ROWS) {
    const int r = r0 + threadIdx.x;
    int64_t code = -2, scale = 0;
    if (r < p.num_rows) {
      int lo = 0, hi = c.num_seqs;  // the last sequence that starts at or before r
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(p.off + mid) <= r) lo = mid;
        else hi = mid;
      }
      int a, b;
      row_range(p.off, lo, p.num_rows, a, b);
      if (r >= a && r < b) {
        const int64_t pos = static_cast<int64_t>(p.starts ? __ldg(p.starts + lo) : 0) + (r - a);
        code = -1;
        if (pos >= 0 && pos < seq_len(c, lo)) {
          const int page = page_of(c, lo, static_cast<int>(pos / c.page_size));
          const int row = static_cast<int>(pos % c.page_size);
          if (page >= 0) {
            code = static_cast<int64_t>(page) * c.page_size + row;
            scale = static_cast<int64_t>(scale_index(c, page, row, 0));
          }
        }
      }
    }
    code_s[threadIdx.x] = code;
    scale_s[threadIdx.x] = scale;
  }
  __syncthreads();
  const int per_row = c.Hkv * (c.D / READ_PIECE<DT>), sh = __ffs(c.D / READ_PIECE<DT>) - 1;  // pieces of a row
  const int64_t ncode = static_cast<int64_t>(c.num_pages) * c.page_size * per_row;
  const int64_t nscale = static_cast<int64_t>(c.num_pages) * c.Hkv * c.per;
  const int64_t nout = static_cast<int64_t>(p.num_rows) * per_row;
  const int side = per_row < THREADS ? THREADS / per_row : 1;  // rows side by side
  const int first = per_row < THREADS ? threadIdx.x / per_row : 0;
  if (first >= side) return;
  for (int i = threadIdx.x - first * per_row; i < per_row; i += THREADS) {
    const int64_t hs = static_cast<int64_t>(i >> sh) * c.per;
#pragma unroll 2
    for (int r = first; r < READ_ROWS; r += side) {
      const int64_t code = code_s[r];
      if (code == -2) continue;
      ReadWord<DT> k{}, v{};
      float a = 0.f, b = 0.f;
      if (code >= 0) {
        const int64_t ci = code * per_row + i, si = scale_s[r] + hs;
        if (in_bounds(c.status, ci, ncode) && in_bounds(c.status, si, nscale)) {
          k = __ldg(reinterpret_cast<const ReadWord<DT>*>(p.codes[0]) + ci);
          v = __ldg(reinterpret_cast<const ReadWord<DT>*>(p.codes[1]) + ci);
          a = __ldg(p.scales[0] + si);
          b = __ldg(p.scales[1] + si);
        }
      }
      const int64_t o = static_cast<int64_t>(r0 + r) * per_row + i;
      if (!in_bounds(c.status, o, nout)) continue;
      store_piece<DT, FMT>(p.out[0], o, k, a);
      store_piece<DT, FMT>(p.out[1], o, v, b);
    }
  }
}

template <int DT, int FMT>
cudaError_t launch_read(const ReadParams& p, cudaStream_t st) {
  read_kernel<DT, FMT><<<(p.num_rows + READ_ROWS - 1) / READ_ROWS, THREADS, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace kv8
}  // namespace attn

namespace {

using attn::aligned;
using attn::Buf;
using attn::meet;
using attn::kv8::Cache;

// Shape checks shared by the cache's entries; fills `c` but for its pointers.
int check_cache(const attn_kv8_cache_t* cache, int num_seqs, int max_pages, Cache& c) {
  if (!cache) return ATTN_ERR_NULL;
  const attn_kv8_cache_t& s = *cache;
  if (s.format != ATTN_KV8_INT8 && s.format != ATTN_KV8_E4M3) return ATTN_ERR_DTYPE;
  if (s.num_pages < 0 || s.page_size <= 0 || s.Hkv <= 0 || s.D <= 0 || s.group <= 0 || s.page_size % s.group != 0 ||
      num_seqs < 0 || max_pages < 0 || static_cast<int64_t>(max_pages) * s.page_size > 0x7fffffffLL ||
      s.Hkv > 32767)
    return ATTN_ERR_SHAPE;
  // extents stay far inside 64 bits
  if (static_cast<double>(s.num_pages) * s.page_size * s.Hkv * s.D > 1e16 ||
      static_cast<double>(num_seqs) * max_pages > 1e16)
    return ATTN_ERR_SHAPE;
  if (!(s.D == 16 || s.D == 32 || s.D == 64 || s.D == 128)) return ATTN_ERR_HEAD_DIM;
  c.num_pages = s.num_pages;
  c.page_size = s.page_size;
  c.Hkv = s.Hkv;
  c.D = s.D;
  c.group = s.group;
  c.per = s.page_size / s.group;
  c.num_seqs = num_seqs;
  c.max_pages = max_pages;
  return ATTN_OK;
}

int64_t code_bytes(const Cache& c) { return static_cast<int64_t>(c.num_pages) * c.page_size * c.Hkv * c.D; }
int64_t scale_bytes(const Cache& c) { return static_cast<int64_t>(c.num_pages) * c.Hkv * c.per * 4; }

}  // namespace

extern "C" int attn_kv8_write(const attn_kv8_cache_t* cache, int num_seqs, int max_pages, int num_tokens,
                              const void* k, const void* v, const int64_t* k_strides, const int64_t* v_strides,
                              const int32_t* block_table, const int32_t* seq_lens, const int32_t* tok_offsets,
                              attn_dtype_t dtype, void* k_cache, void* v_cache, float* k_scale, float* v_scale,
                              void* stream) {
  if (dtype != ATTN_F32 && dtype != ATTN_F16 && dtype != ATTN_BF16) return ATTN_ERR_DTYPE;
  attn::kv8::WriteParams p{};
  if (const int rc = check_cache(cache, num_seqs, max_pages, p.c)) return rc;
  if (num_tokens < 0) return ATTN_ERR_SHAPE;
  if (!k_strides || !v_strides) return ATTN_ERR_NULL;
  for (const int64_t* st : {k_strides, v_strides})
    for (int j = 0; j < 2; ++j)
      if (st[j] < 0 || st[j] > (1ll << 28)) return ATTN_ERR_SHAPE;
  if (static_cast<int64_t>(num_tokens) / p.c.group + 2ll * num_seqs > 0x7fffffffLL) return ATTN_ERR_SHAPE;
  if (num_tokens == 0 || num_seqs == 0 || max_pages == 0 || p.c.num_pages == 0) return ATTN_OK;
  if (!k || !v || !block_table || !seq_lens || !tok_offsets || !k_cache || !v_cache || !k_scale || !v_scale)
    return ATTN_ERR_NULL;
  const int es = dtype == ATTN_F32 ? 4 : 2;
  if (!aligned(k, es) || !aligned(v, es) || !aligned(k_cache, 16) || !aligned(v_cache, 16)) return ATTN_ERR_ALIGN;
  for (const void* pi : {static_cast<const void*>(block_table), static_cast<const void*>(seq_lens),
                         static_cast<const void*>(tok_offsets), static_cast<const void*>(k_scale),
                         static_cast<const void*>(v_scale)})
    if (!aligned(pi, 4)) return ATTN_ERR_ALIGN;
  const Cache& c = p.c;
  auto extent = [&](const int64_t* st) { return ((num_tokens - 1ll) * st[0] + (c.Hkv - 1ll) * st[1] + c.D) * es; };
  const Buf outs[] = {{k_cache, code_bytes(c)}, {v_cache, code_bytes(c)}, {k_scale, scale_bytes(c)}, {v_scale, scale_bytes(c)}};
  const Buf ins[] = {{k, extent(k_strides)}, {v, extent(v_strides)},
                     {block_table, static_cast<int64_t>(num_seqs) * max_pages * 4},
                     {seq_lens, num_seqs * 4ll}, {tok_offsets, (num_seqs + 1ll) * 4}};
  for (int i = 0; i < 4; ++i) {
    for (int j = 0; j < i; ++j)
      if (meet(outs[i], outs[j])) return ATTN_ERR_OVERLAP;
    for (const Buf& b : ins)
      if (meet(outs[i], b)) return ATTN_ERR_OVERLAP;
  }
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return attn::record_cuda_error(e);
  p.c.block_table = block_table;
  p.c.seq_lens = seq_lens;
  p.c.status = attn::status_word(dev);
  p.num_tokens = num_tokens;
  p.off = tok_offsets;
  p.x[0] = k;
  p.x[1] = v;
  for (int i = 0; i < 2; ++i) {
    const int64_t* st = i ? v_strides : k_strides;
    p.xt[i] = st[0];
    p.xh[i] = st[1];
  }
  p.codes[0] = static_cast<uint8_t*>(k_cache);
  p.codes[1] = static_cast<uint8_t*>(v_cache);
  p.scales[0] = k_scale;
  p.scales[1] = v_scale;
  // 8-element loads need rows that start on their boundary
  bool vec = aligned(k, 16) && aligned(v, 16);
  for (int i = 0; i < 2; ++i)
    vec = vec && (num_tokens == 1 || p.xt[i] % 8 == 0) && (c.Hkv == 1 || p.xh[i] % 8 == 0);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool i8 = cache->format == ATTN_KV8_INT8;
  using namespace attn::kv8;
#define ATTN_WRITE(DT)                                                                              \
  (i8 ? (vec ? launch_write<DT, FMT_INT8, true>(p, st) : launch_write<DT, FMT_INT8, false>(p, st)) \
      : (vec ? launch_write<DT, FMT_E4M3, true>(p, st) : launch_write<DT, FMT_E4M3, false>(p, st)))
  e = dtype == ATTN_F32 ? ATTN_WRITE(0) : dtype == ATTN_F16 ? ATTN_WRITE(1) : ATTN_WRITE(2);
#undef ATTN_WRITE
  return e == cudaSuccess ? ATTN_OK : attn::record_cuda_error(e);
}

extern "C" int attn_kv8_read(const attn_kv8_cache_t* cache, int num_seqs, int max_pages, int num_rows,
                             const void* k_cache, const void* v_cache, const float* k_scale, const float* v_scale,
                             const int32_t* block_table, const int32_t* seq_lens, const int32_t* row_offsets,
                             const int32_t* starts, attn_dtype_t dtype, void* k_out, void* v_out, void* stream) {
  if (dtype != ATTN_F32 && dtype != ATTN_F16 && dtype != ATTN_BF16) return ATTN_ERR_DTYPE;
  attn::kv8::ReadParams p{};
  if (const int rc = check_cache(cache, num_seqs, max_pages, p.c)) return rc;
  if (num_rows < 0 || num_rows > 0x7fffff00) return ATTN_ERR_SHAPE;
  if (num_rows == 0 || num_seqs == 0) return ATTN_OK;
  const Cache& c = p.c;
  if (!seq_lens || !row_offsets || !k_out || !v_out || (max_pages > 0 && !block_table) ||
      (c.num_pages > 0 && (!k_cache || !v_cache || !k_scale || !v_scale)))
    return ATTN_ERR_NULL;
  for (const void* pi : {k_cache, v_cache, static_cast<const void*>(k_out), static_cast<const void*>(v_out)})
    if (!aligned(pi, 16)) return ATTN_ERR_ALIGN;
  for (const void* pi : {static_cast<const void*>(block_table), static_cast<const void*>(seq_lens),
                         static_cast<const void*>(row_offsets), static_cast<const void*>(starts),
                         static_cast<const void*>(k_scale), static_cast<const void*>(v_scale)})
    if (!aligned(pi, 4)) return ATTN_ERR_ALIGN;
  const int64_t out_bytes = static_cast<int64_t>(num_rows) * c.Hkv * c.D * (dtype == ATTN_F32 ? 4 : 2);
  const Buf outs[] = {{k_out, out_bytes}, {v_out, out_bytes}};
  const Buf ins[] = {{k_cache, code_bytes(c)}, {v_cache, code_bytes(c)}, {k_scale, scale_bytes(c)},
                     {v_scale, scale_bytes(c)}, {block_table, static_cast<int64_t>(num_seqs) * max_pages * 4},
                     {seq_lens, num_seqs * 4ll}, {row_offsets, (num_seqs + 1ll) * 4},
                     {starts, starts ? num_seqs * 4ll : 0}};
  for (const Buf& o : outs)
    for (const Buf& b : ins)
      if (meet(o, b)) return ATTN_ERR_OVERLAP;
  if (meet(outs[0], outs[1])) return ATTN_ERR_OVERLAP;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return attn::record_cuda_error(e);
  p.c.block_table = block_table;
  p.c.seq_lens = seq_lens;
  p.c.status = attn::status_word(dev);
  p.num_rows = num_rows;
  p.off = row_offsets;
  p.starts = starts;
  p.codes[0] = static_cast<const uint8_t*>(k_cache);
  p.codes[1] = static_cast<const uint8_t*>(v_cache);
  p.scales[0] = k_scale;
  p.scales[1] = v_scale;
  p.out[0] = k_out;
  p.out[1] = v_out;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool i8 = cache->format == ATTN_KV8_INT8;
  using namespace attn::kv8;
#define ATTN_READ(DT) (i8 ? launch_read<DT, FMT_INT8>(p, st) : launch_read<DT, FMT_E4M3>(p, st))
  e = dtype == ATTN_F32 ? ATTN_READ(0) : dtype == ATTN_F16 ? ATTN_READ(1) : ATTN_READ(2);
#undef ATTN_READ
  return e == cudaSuccess ? ATTN_OK : attn::record_cuda_error(e);
}
