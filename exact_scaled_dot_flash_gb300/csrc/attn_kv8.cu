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
// exactly (a float format gains nothing from a finer scale). A NaN or infinity
// among the new tokens makes the group's scale NaN: the group then reads as
// NaN until a call writes its first token again.
// Bytes: the new tokens are read once and one byte written for each element.
//
// Read. Row i of sequence s is its token starts[s] + i; value = code * scale,
// rounded once to the output type.
#include <math.h>

#include "attn.h"
#include "kv8.cuh"
#include "simt.cuh"

namespace attn {
namespace kv8 {

constexpr int THREADS = 256;

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
template <int DT, bool VEC>
__device__ __forceinline__ void load8x(const void* base, int64_t i, float (&x)[8]) {
  if constexpr (VEC) {
    float4 a, b;
    simt::load8<DT>(base, static_cast<size_t>(i) >> 3, a, b);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if constexpr (DT == 0) x[k] = __ldg(static_cast<const float*>(base) + i + k);
      else if constexpr (DT == 1) x[k] = __half2float(__ldg(static_cast<const __half*>(base) + i + k));
      else x[k] = __bfloat162float(__ldg(static_cast<const __nv_bfloat16*>(base) + i + k));
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

template <int FMT>
__device__ __forceinline__ uint32_t encode4(const float* x, float s, float inv) {
  if constexpr (FMT == FMT_INT8) {
    uint32_t w = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) w |= (static_cast<uint32_t>(nearest8(x[k], s, inv)) & 0xffu) << (8 * k);
    return w;
  } else {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(x[1] * inv), "f"(x[0] * inv));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(x[3] * inv), "f"(x[2] * inv));
    return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
  }
}

// Codes of c * s_old / s for s > s_old. The fp32 product is within 2^-15 of the
// quotient (|c| <= 128); only one that lies that near a tie is settled in fp64.
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
    return encode4<FMT>(c, s, ratio);
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
// of a slot is found by a search that reads 32 offsets at a time.
__device__ __forceinline__ int seq_of_slot(const int32_t* off, int num_seqs, int group, int num_tokens, int slot,
                                           int lane) {
  int lo = 0, n = num_seqs;  // the answer is in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32;
    bool at = false;
    if (lane * step < n) {
      const int i = lo + lane * step;
      const int o = min(max(__ldg(off + i), 0), num_tokens);
      at = static_cast<int64_t>(o / group) + 2ll * i <= slot;
    }
    const unsigned m = __ballot_sync(0xffffffffu, at);
    const int last = m ? 31 - __clz(m) : 0;
    const int end = lo + n;
    lo += last * step;
    n = min(step, end - lo);
  }
  return lo;
}

// TPU threads (a warp, or the CTA) hold one unit: a (slot, head, k or v). The
// elements are kept in registers between the maximum and the codes, KEEP
// vectors of 8 a thread; a larger group reads the rest a second time.
template <int DT, int FMT, bool VEC, int TPU>
__global__ void __launch_bounds__(THREADS) write_kernel(const __grid_constant__ WriteParams p) {
  constexpr int KEEP = 4;
  __shared__ float red[THREADS / 32];
  const Cache& c = p.c;
  const int lane = threadIdx.x & 31;
  const int tu = threadIdx.x % TPU;
  const int unit = blockIdx.y * (THREADS / TPU) + threadIdx.x / TPU;  // head, then k / v
  if (unit >= 2 * c.Hkv) return;  // a whole warp (TPU 32) or no thread (TPU 256) returns
  const int kv = unit >= c.Hkv ? 1 : 0, h = unit - kv * c.Hkv;
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
  const int nv = m * vpt;
  const void* const x = p.x[kv];
  const int64_t xbase = x0 * p.xt[kv] + h * p.xh[kv];

  float keep[KEEP][8];
  float amax = 0.f;
  bool odd = false;  // a NaN or an infinity
  auto look = [&](const float (&v)[8]) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float a = fabsf(v[k]);
      odd = odd || !(a < INFINITY);
      amax = fmaxf(amax, a);
    }
  };
#pragma unroll
  for (int i = 0; i < KEEP; ++i) {
    const int e = tu + i * TPU;
    if (e < nv) load8x<DT, VEC>(x, xbase + (e >> sh) * p.xt[kv] + (e & (vpt - 1)) * 8, keep[i]);
  }
#pragma unroll
  for (int i = 0; i < KEEP; ++i)
    if (tu + i * TPU < nv) look(keep[i]);
  for (int e = tu + KEEP * TPU; e < nv; e += TPU) {
    float v[8];
    load8x<DT, VEC>(x, xbase + (e >> sh) * p.xt[kv] + (e & (vpt - 1)) * 8, v);
    look(v);
  }
  if (odd) amax = INFINITY;  // no finite value reaches it
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if constexpr (TPU > 32) {
    if (lane == 0) red[threadIdx.x >> 5] = amax;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < TPU / 32; ++w) amax = fmaxf(amax, red[w]);
  }
  const size_t si = scale_index(c, page, row0, h);
  const int64_t nscale = static_cast<int64_t>(c.num_pages) * c.Hkv * c.per;
  if (!in_bounds(c.status, static_cast<int64_t>(si), nscale)) return;
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
  const size_t cstep = static_cast<size_t>(c.Hkv) * c.D;
  const int64_t ncode8 = static_cast<int64_t>(c.num_pages) * c.page_size * c.Hkv * vpt;
  uint8_t* const codes = p.codes[kv];
  auto slot8 = [&](int token, int col) { return reinterpret_cast<uint2*>(codes + cbase + token * cstep + col * 8); };
  const float inv = 1.f / sn;
  auto put = [&](int e, const float (&v)[8]) {
    const int t = held + (e >> sh), col = e & (vpt - 1);
    if (!in_bounds(c.status, static_cast<int64_t>((cbase + t * cstep) >> 3) + col, ncode8)) return;
    // a group without a scale (NaN) gets zero codes
    *slot8(t, col) = sn == sn ? make_uint2(encode4<FMT>(v, sn, inv), encode4<FMT>(v + 4, sn, inv)) : make_uint2(0u, 0u);
  };
  if (held > 0 && sn > so) {  // the codes of earlier calls, at the larger scale
    for (int e = tu; e < held * vpt; e += TPU) {
      const int t = e >> sh, col = e & (vpt - 1);
      if (!in_bounds(c.status, static_cast<int64_t>((cbase + t * cstep) >> 3) + col, ncode8)) continue;
      uint2* const at = slot8(t, col);
      const uint2 w = *at;
      *at = make_uint2(recode4<FMT>(w.x, so, sn), recode4<FMT>(w.y, so, sn));
    }
  }
#pragma unroll
  for (int i = 0; i < KEEP; ++i) {
    const int e = tu + i * TPU;
    if (e < nv) put(e, keep[i]);
  }
  for (int e = tu + KEEP * TPU; e < nv; e += TPU) {
    float v[8];
    load8x<DT, VEC>(x, xbase + (e >> sh) * p.xt[kv] + (e & (vpt - 1)) * 8, v);
    put(e, v);
  }
}

template <int DT, int FMT, bool VEC>
cudaError_t launch_write(const WriteParams& p, cudaStream_t st) {
  const unsigned slots = static_cast<unsigned>(p.num_tokens / p.c.group + 2 * p.c.num_seqs);
  // a warp keeps up to 1024 elements of a unit in registers, the CTA 8192
  if (p.c.group * p.c.D <= 1024) {
    constexpr int U = THREADS / 32;
    write_kernel<DT, FMT, VEC, 32><<<dim3(slots, (2 * p.c.Hkv + U - 1) / U), THREADS, 0, st>>>(p);
  } else {
    write_kernel<DT, FMT, VEC, THREADS><<<dim3(slots, 2 * p.c.Hkv), THREADS, 0, st>>>(p);
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

// A CTA finds its rows' places in the cache once, then moves their heads side
// by side: 8 codes in, 8 values out a thread and step.
template <int DT, int FMT>
__global__ void __launch_bounds__(THREADS) read_kernel(const __grid_constant__ ReadParams p) {
  __shared__ int page_s[READ_ROWS], row_s[READ_ROWS];
  const Cache& c = p.c;
  const int r0 = blockIdx.x * READ_ROWS;
  if (threadIdx.x < READ_ROWS) {
    const int r = r0 + threadIdx.x;
    int page = -2, row = 0;  // -2: a row of no sequence, left alone; -1: zeros
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
        page = -1;
        if (pos >= 0 && pos < seq_len(c, lo)) {
          page = page_of(c, lo, static_cast<int>(pos / c.page_size));
          row = static_cast<int>(pos % c.page_size);
        }
      }
    }
    page_s[threadIdx.x] = page;
    row_s[threadIdx.x] = row;
  }
  __syncthreads();
  const int vpt = c.D >> 3, sh = __ffs(vpt) - 1;
  const int per_row = c.Hkv * vpt;
  const int64_t ncode8 = static_cast<int64_t>(c.num_pages) * c.page_size * per_row;
  const int64_t nscale = static_cast<int64_t>(c.num_pages) * c.Hkv * c.per;
  const int64_t nout8 = static_cast<int64_t>(p.num_rows) * per_row;
  for (int e = threadIdx.x; e < READ_ROWS * per_row; e += THREADS) {
    const int r = e / per_row, i = e - r * per_row;
    const int page = page_s[r];
    if (page == -2) continue;
    const int row = row_s[r], h = i >> sh;
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
      if (page >= 0) {
        const size_t ci = (static_cast<size_t>(page) * c.page_size + row) * per_row + i;
        const size_t si = scale_index(c, page, row, h);
        if (in_bounds(c.status, static_cast<int64_t>(ci), ncode8) &&
            in_bounds(c.status, static_cast<int64_t>(si), nscale)) {
          const uint2 w = __ldg(reinterpret_cast<const uint2*>(p.codes[kv]) + ci);
          const float s = __ldg(p.scales[kv] + si);
          a = decode4<FMT>(w.x);
          b = decode4<FMT>(w.y);
          a.x *= s; a.y *= s; a.z *= s; a.w *= s;
          b.x *= s; b.y *= s; b.z *= s; b.w *= s;
        }
      }
      const size_t o = static_cast<size_t>(r0 + r) * per_row + i;
      if (!in_bounds(c.status, static_cast<int64_t>(o), nout8)) continue;
      simt::store4<DT>(p.out[kv], 2 * o, a);
      simt::store4<DT>(p.out[kv], 2 * o + 1, b);
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

using attn::kv8::Cache;

struct Buf {
  const void* p;
  int64_t n;
};

bool meet(const Buf& a, const Buf& b) {
  if (!a.p || !b.p || a.n <= 0 || b.n <= 0) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x < y + static_cast<uintptr_t>(b.n) && y < x + static_cast<uintptr_t>(a.n);
}

bool aligned(const void* p, int to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }

// Shape checks shared by the cache's entries; fills `c` but for its pointers.
int check_cache(const attn_kv8_cache_t* cache, int num_seqs, int max_pages, Cache& c) {
  if (!cache) return ATTN_ERR_NULL;
  const attn_kv8_cache_t& s = *cache;
  if (s.format != ATTN_KV8_INT8 && s.format != ATTN_KV8_E4M3) return ATTN_ERR_DTYPE;
  if (s.num_pages < 0 || s.page_size <= 0 || s.Hkv <= 0 || s.D <= 0 || s.group <= 0 || s.page_size % s.group != 0 ||
      num_seqs < 0 || max_pages < 0 || static_cast<int64_t>(max_pages) * s.page_size > 0x7fffffffLL ||
      s.Hkv > 32767)
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
