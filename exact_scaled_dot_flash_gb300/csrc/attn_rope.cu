// attn_rope.cu - rotary positions of queries and keys, and their gradient.
//
// Pair i of a head (elements i and i + rot/2, or 2i and 2i + 1) is turned by
// the angle a = position * inv_freq[i] and multiplied by mscale; elements from
// `rot` on are copied. The turn is linear and orthogonal up to mscale, so the
// gradient is the turn by -a with the same factor (inverse = 1).
//
// Angles: of a far position only the fraction of a turn matters, and fp32
// loses it (position 10^6 leaves an error of 0.06 rad). inv_freq / 2 pi is
// taken once as a 64-bit fraction of a turn, F = frac(f) 2^64; position * F
// modulo 2^64 is then the exact fraction of the product with F, for every int32
// position, and its upper 32 bits as a signed number are the angle in half
// turns, in [-1, 1), which sincospi takes without any range reduction. f itself
// is off by 2^-52 of it (the product in double and its constant): an angle by
// position * inv_freq * 2^-52, 5e-7 at the last position and inv_freq 1.
//
// Bytes: every element is read once and written once, and nothing else counts:
// the angles of a token are computed once for all its heads, in shared memory,
// while the first vectors are on their way. A thread moves 16-byte vectors. The
// addresses of a CTA's rows are computed once, in shared memory: with every
// thread working out its own for every 16 bytes, the instructions were the bound
// (72 us for 8191 tokens of 40 F16 heads, D 128). For the 16-bit types, whose
// vectors take twice the conversions, many threads with one vector each beat few
// with several in flight (F16, 8 CTAs an SM and 1: 36.5 us, 4.6 TB/s; 4 and 4: 49
// us; the 32 registers of a thread hold an F16 item, of a BF16 one 40-72 bytes spill);
// for F32 it is the other way round (16384 tokens of 64 heads: 160 us, 6.7 TB/s,
// with 4 vectors and 2 tokens a CTA, 171 us as the 16-bit types).
#include <math.h>

#include <algorithm>

#include "attn.h"
#include "host_checks.h"
#include "params.h"
#include "ptx.cuh"

namespace attn {
namespace rope {

constexpr int THREADS = 256;

constexpr int MAX_ROWS = 512;  // (token, head) rows of a CTA

struct Side {  // queries or keys
  const void* in;
  void* out;
  int copy_tail;
  int64_t ib, it, ih, ob, ot, oh;  // batch, token and head strides (elements)
};

struct Params {
  int B, S, D, rot, Hq, H;  // H: heads of queries and keys together
  int64_t pos_batch;  // 0 or S: one row of positions for all, or one each
  const int32_t* pos;
  const double* freq;
  float mscale;
  int inverse, tok, heads;  // tokens and heads of a CTA (blockIdx.y: which heads)
  Side side[2];
};

// VEC: elements of 16 bytes; BATCH: vectors a thread has in flight; CTAS: of an
// SM; TOKENS: of a CTA, where there are many.
template <int DT> struct Elem;
template <> struct Elem<0> { using T = float; static constexpr int VEC = 4, BATCH = 4, CTAS = 4, TOKENS = 2; };
template <> struct Elem<1> { using T = __half; static constexpr int VEC = 8, BATCH = 1, CTAS = 8, TOKENS = 4; };
template <> struct Elem<2> { using T = __nv_bfloat16; static constexpr int VEC = 8, BATCH = 1, CTAS = 8, TOKENS = 4; };

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f(float& y, float x) { y = x; }
__device__ __forceinline__ void from_f(__half& y, float x) { y = __float2half_rn(x); }
__device__ __forceinline__ void from_f(__nv_bfloat16& y, float x) { y = __float2bfloat16_rn(x); }

// N elements moved as one access (16 bytes, or one element).
template <typename T, int N>
struct alignas(N * sizeof(T)) Vec {
  T x[N];
};

// Items of a head: pairs of vectors (halves) or single vectors (interleaved),
// then the vectors of the copied tail. N = 1: elements instead of vectors
// (interleaved: pairs), for rows that 16-byte accesses do not fit. A thread keeps
// its item and goes through the CTA's rows (token, head).
template <int DT, bool HALVES, int N>
__global__ void __launch_bounds__(THREADS, Elem<DT>::CTAS) rope_kernel(const __grid_constant__ Params p) {
  using T = typename Elem<DT>::T;
  using V = Vec<T, N>;
  constexpr int BATCH = Elem<DT>::BATCH;
  constexpr int M = HALVES || N > 1 ? N : 2;  // elements of the first access
  using V1 = Vec<T, M>;                       // (not one access where N is 1)
  extern __shared__ float2 cs[];              // [tok][rot / 2] cos, sin times mscale
  __shared__ struct { const T* in; T* out; } row_s[MAX_ROWS];
  __shared__ int16_t tok_s[MAX_ROWS];         // token, + 256 if the tail is copied
  const int half = p.rot >> 1;
  const int64_t total = static_cast<int64_t>(p.B) * p.S;
  const int64_t tok0 = static_cast<int64_t>(blockIdx.x) * p.tok;
  const int ntok = static_cast<int>(min(static_cast<int64_t>(p.tok), total - tok0));
  const int h0 = blockIdx.y * p.heads, nh = min(p.heads, p.H - h0);
  const int nrow = ntok * nh;
  for (int r = threadIdx.x; r < nrow; r += THREADS) {
    const int t = r / nh, h = h0 + r - t * nh, sd = h >= p.Hq ? 1 : 0, hh = h - sd * p.Hq;
    const int64_t g = tok0 + t, b = p.B == 1 ? 0 : g / p.S, q = g - b * p.S;
    const Side& s = p.side[sd];
    row_s[r].in = static_cast<const T*>(s.in) + b * s.ib + q * s.it + hh * s.ih;
    row_s[r].out = static_cast<T*>(s.out) + b * s.ob + q * s.ot + hh * s.oh;
    tok_s[r] = static_cast<int16_t>(t + (s.copy_tail ? 256 : 0));
  }
  __syncthreads();

  const int turn = HALVES ? half / N : (N > 1 ? p.rot / N : half);
  const int items = turn + (p.side[0].copy_tail | p.side[1].copy_tail ? (p.D - p.rot) / N : 0);
  const int per = items < THREADS ? THREADS / items : 1;  // rows side by side in the CTA
  const int r0 = items < THREADS ? threadIdx.x / items : 0;
  const int rows = r0 < per ? nrow : 0;
  const int first = threadIdx.x - r0 * items;
  V1 x[BATCH];
  V y[BATCH];
  auto load = [&](int item, int r) {
#pragma unroll
    for (int u = 0; u < BATCH; ++u) {
      if (r + u * per >= rows) break;
      const auto w = row_s[r + u * per];
      if (item >= turn) {
        y[u] = *reinterpret_cast<const V*>(w.in + p.rot + (item - turn) * N);
      } else if constexpr (HALVES) {
        x[u] = *reinterpret_cast<const V1*>(w.in + item * N);
        y[u] = *reinterpret_cast<const V*>(w.in + half + item * N);
      } else if constexpr (N > 1) {
        x[u] = *reinterpret_cast<const V1*>(w.in + item * N);
      } else {
        x[u].x[0] = w.in[2 * item];
        x[u].x[1] = w.in[2 * item + 1];
      }
    }
  };
  auto finish = [&](int item, int r) {
#pragma unroll
    for (int u = 0; u < BATCH; ++u) {
      if (r + u * per >= rows) break;
      const auto w = row_s[r + u * per];
      const int tok = tok_s[r + u * per];
      const float2* const c = cs + (tok & 255) * half;
      if (item >= turn) {
        if (tok & 256) *reinterpret_cast<V*>(w.out + p.rot + (item - turn) * N) = y[u];
      } else if constexpr (HALVES) {
#pragma unroll
        for (int k = 0; k < N; ++k) {
          const float a = to_f(x[u].x[k]), b = to_f(y[u].x[k]);
          const float2 f = c[item * N + k];
          from_f(x[u].x[k], a * f.x - b * f.y);
          from_f(y[u].x[k], b * f.x + a * f.y);
        }
        *reinterpret_cast<V1*>(w.out + item * N) = x[u];
        *reinterpret_cast<V*>(w.out + half + item * N) = y[u];
      } else {
#pragma unroll
        for (int k = 0; k < M; k += 2) {
          const float a = to_f(x[u].x[k]), b = to_f(x[u].x[k + 1]);
          const float2 f = c[(item * M + k) >> 1];
          from_f(x[u].x[k], a * f.x - b * f.y);
          from_f(x[u].x[k + 1], b * f.x + a * f.y);
        }
        if constexpr (N > 1) {
          *reinterpret_cast<V1*>(w.out + item * N) = x[u];
        } else {
          w.out[2 * item] = x[u].x[0];
          w.out[2 * item + 1] = x[u].x[1];
        }
      }
    }
  };
  if (first < items) load(first, r0);
  for (int e = threadIdx.x; e < ntok * half; e += THREADS) {
    constexpr double INV_2PI = 0.15915494309189533577;
    const int t = e / half, i = e - t * half;
    const int64_t g = tok0 + t;
    const int64_t pos = __ldg(p.pos + (p.pos_batch || p.B == 1 ? g : g % p.S));
    const double f = __ldg(p.freq + i) * INV_2PI;
    const uint64_t F = __double2ull_rd((f - floor(f)) * 18446744073709551616.0);
    const int32_t top = static_cast<int32_t>(static_cast<uint32_t>((static_cast<uint64_t>(pos) * F) >> 32));
    float sn, cn;
    sincospif(static_cast<float>(top) * 4.656612873077393e-10f, &sn, &cn);  // 2^-31
    cs[e] = make_float2(cn * p.mscale, (p.inverse ? -sn : sn) * p.mscale);
  }
  __syncthreads();
  for (int item = first; item < items; item += THREADS) {
    for (int r = r0; r < rows; r += BATCH * per) {
      if (item != first || r != r0) load(item, r);
      finish(item, r);
    }
  }
}

template <int DT>
cudaError_t launch_dt(const Params& p, bool halves, bool vec, dim3 grid, cudaStream_t st) {
  constexpr int N = Elem<DT>::VEC;
  const size_t smem = static_cast<size_t>(p.tok) * (p.rot / 2) * sizeof(float2);
  if (halves) {
    if (vec) rope_kernel<DT, true, N><<<grid, THREADS, smem, st>>>(p);
    else rope_kernel<DT, true, 1><<<grid, THREADS, smem, st>>>(p);
  } else {
    if (vec) rope_kernel<DT, false, N><<<grid, THREADS, smem, st>>>(p);
    else rope_kernel<DT, false, 1><<<grid, THREADS, smem, st>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace rope
}  // namespace attn

namespace {

using attn::rope::Params;
using attn::rope::Side;

struct Span {  // what a strided tensor may touch, in bytes
  uintptr_t p;
  int64_t token, row, all;  // token stride, extent of one token's heads, extent of everything
  int64_t batch, one;       // batch stride, extent of one batch
};

Span span_of(const void* p, int64_t B, int64_t S, int64_t H, int64_t D, const int64_t* st, int es) {
  Span s;
  s.p = reinterpret_cast<uintptr_t>(p);
  s.token = st[1] * es;
  s.row = ((H - 1) * st[2] + D) * es;
  s.batch = st[0] * es;
  s.one = ((S - 1) * st[1] + (H - 1) * st[2] + D) * es;
  s.all = ((B - 1) * st[0] + (S - 1) * st[1] + (H - 1) * st[2] + D) * es;
  return s;
}

// Whether pieces of na bytes every `period` from a on and of nb bytes from b on lie apart.
bool apart_modulo(uintptr_t a, int64_t na, uintptr_t b, int64_t nb, int64_t period) {
  if (period <= 0 || na > period || nb > period) return false;
  const int64_t diff = static_cast<int64_t>(b) - static_cast<int64_t>(a);
  const int64_t d = ((diff % period) + period) % period;
  return d >= na && d + nb <= period;
}

// Whether two strided tensors may share an element. Slices of one fused
// projection interleave without sharing any: tokens the same stride apart
// (batches too, as multiples of it), and rows that lie apart modulo it; or
// batches the same stride apart, and all of a batch apart modulo that (the
// heads of one dense tensor).
bool spans_meet(const Span& a, const Span& b, bool batches_fit) {
  if (a.p + a.all <= b.p || b.p + b.all <= a.p) return false;
  if (batches_fit && a.token == b.token && apart_modulo(a.p, a.row, b.p, b.row, a.token)) return false;
  return a.batch != b.batch || !apart_modulo(a.p, a.one, b.p, b.one, a.batch);
}

// No two (batch, token, head) rows of a written tensor may share an element:
// the axes, from the smallest stride up, each step over what lies below.
bool rows_apart(int64_t B, int64_t S, int64_t H, int64_t D, const int64_t* st) {
  struct Axis { int64_t n, stride; } ax[3] = {{B, st[0]}, {S, st[1]}, {H, st[2]}};
  std::sort(ax, ax + 3, [](const Axis& x, const Axis& y) { return x.stride < y.stride; });
  int64_t below = D;
  for (const Axis& a : ax) {
    if (a.n <= 1) continue;
    if (a.stride < below) return false;
    below = (a.n - 1) * a.stride + below;
  }
  return true;
}

}  // namespace

extern "C" int attn_rope(const attn_rope_shape_t* shape, const void* q, const void* k, const int32_t* positions,
                         const double* inv_freq, int layout, int inverse, float mscale, attn_dtype_t dtype,
                         void* q_out, void* k_out, void* stream) {
  if (!shape) return ATTN_ERR_NULL;
  const attn_rope_shape_t s = *shape;
  if (dtype != ATTN_F32 && dtype != ATTN_F16 && dtype != ATTN_BF16) return ATTN_ERR_DTYPE;
  if (s.B < 0 || s.S < 0 || s.Hq <= 0 || s.Hk < 0 || s.D <= 0 || s.D > ATTN_ROPE_MAX_D || s.rot <= 0 ||
      s.rot > s.D || (s.rot & 1) || (layout != ATTN_ROPE_HALF && layout != ATTN_ROPE_INTERLEAVED) ||
      (inverse != 0 && inverse != 1) || (s.pos_batch_stride != 0 && s.pos_batch_stride != s.S))
    return ATTN_ERR_SHAPE;
  if (!isfinite(mscale)) return ATTN_ERR_SCALE;
  const int nside = s.Hk > 0 ? 2 : 1;
  const int64_t* st[4] = {s.q_strides, s.q_out_strides, s.k_strides, s.k_out_strides};
  const int heads[4] = {s.Hq, s.Hq, s.Hk, s.Hk};
  for (int i = 0; i < 2 * nside; ++i) {
    for (int j = 0; j < 3; ++j)
      if (st[i][j] < 0) return ATTN_ERR_SHAPE;
    // extents stay far inside 64 bits
    if (static_cast<double>(s.B) * st[i][0] + static_cast<double>(s.S) * st[i][1] +
            static_cast<double>(heads[i]) * st[i][2] > 1e17)
      return ATTN_ERR_SHAPE;
  }
  const int64_t tokens = static_cast<int64_t>(s.B) * s.S;
  if (tokens == 0) return ATTN_OK;
  if (tokens > 0x7fffffffLL || (static_cast<int64_t>(s.Hq) + s.Hk) * 64 > 0x7fffffffLL) return ATTN_ERR_SHAPE;
  if (!q || !q_out || !positions || !inv_freq || (s.Hk > 0 && (!k || !k_out))) return ATTN_ERR_NULL;
  const int es = dtype == ATTN_F32 ? 4 : 2;
  const void* ptr[4] = {q, q_out, k, k_out};
  Span sp[4];
  bool fit = true, vec = (s.D * es) % 16 == 0;
  for (int i = 0; i < 2 * nside; ++i) {
    if (reinterpret_cast<uintptr_t>(ptr[i]) % es) return ATTN_ERR_ALIGN;
    if ((i & 1) && !rows_apart(s.B, s.S, heads[i], s.D, st[i])) return ATTN_ERR_OVERLAP;
    sp[i] = span_of(ptr[i], s.B, s.S, heads[i], s.D, st[i], es);
    fit = fit && (s.B == 1 || (st[i][1] > 0 && st[i][0] % st[i][1] == 0));
    vec = vec && reinterpret_cast<uintptr_t>(ptr[i]) % 16 == 0;
    const int n[3] = {s.B, s.S, heads[i]};
    for (int j = 0; j < 3; ++j) vec = vec && (n[j] == 1 || (st[i][j] * es) % 16 == 0);
  }
  if ((reinterpret_cast<uintptr_t>(positions) & 3u) || (reinterpret_cast<uintptr_t>(inv_freq) & 7u))
    return ATTN_ERR_ALIGN;
  bool in_place[2] = {false, false};
  for (int i = 0; i < nside; ++i) {
    in_place[i] = ptr[2 * i] == ptr[2 * i + 1];
    for (int j = 0; j < 3; ++j) in_place[i] = in_place[i] && st[2 * i][j] == st[2 * i + 1][j];
  }
  Span meta[2];
  const int64_t meta_bytes[2] = {(s.pos_batch_stride ? tokens : s.S) * 4, s.rot / 2 * 8};
  for (int i = 0; i < 2; ++i) {
    meta[i].p = reinterpret_cast<uintptr_t>(i == 0 ? static_cast<const void*>(positions) : inv_freq);
    meta[i].token = meta[i].batch = 0;
    meta[i].row = meta[i].one = meta[i].all = meta_bytes[i];
  }
  for (int o = 1; o < 2 * nside; o += 2) {  // each output against every other tensor
    for (int i = 0; i < 2 * nside; ++i)
      if (i != o && !(i == o - 1 && in_place[o / 2]) && spans_meet(sp[o], sp[i], fit)) return ATTN_ERR_OVERLAP;
    for (const Span& m : meta)
      if (spans_meet(sp[o], m, false)) return ATTN_ERR_OVERLAP;
  }

  Params p{};
  p.B = s.B;
  p.S = s.S;
  p.D = s.D;
  p.rot = s.rot;
  p.pos_batch = s.pos_batch_stride;
  p.pos = positions;
  p.freq = inv_freq;
  p.mscale = mscale;
  p.inverse = inverse;
  for (int i = 0; i < nside; ++i) {
    const int64_t *a = st[2 * i], *b = st[2 * i + 1];
    p.side[i] = Side{ptr[2 * i], const_cast<void*>(ptr[2 * i + 1]), in_place[i] ? 0 : 1, a[0], a[1], a[2], b[0], b[1], b[2]};
  }
  p.Hq = s.Hq;
  p.H = s.Hq + (nside == 2 ? s.Hk : 0);
  const bool halves = layout == ATTN_ROPE_HALF;
  const int n = dtype == ATTN_F32 ? 4 : 8;
  vec = vec && (halves ? s.rot / 2 : s.rot) % n == 0 && (s.D - s.rot) % n == 0;
  // A CTA takes several tokens when that still leaves several CTAs for each SM;
  // with few tokens the heads of one are dealt to up to 8 CTAs (64 tokens of 40
  // heads: 2.9 us by two each, 3.4 by one).
  const int several = dtype == ATTN_F32 ? attn::rope::Elem<0>::TOKENS : attn::rope::Elem<2>::TOKENS;
  p.tok = tokens >= attn::SMS * 16 && p.H * several <= attn::rope::MAX_ROWS ? several : 1;
  const int64_t want = std::min<int64_t>({2 * attn::SMS / tokens, 8, (p.H + 7) / 8});
  const int64_t least = (static_cast<int64_t>(p.H) * p.tok + attn::rope::MAX_ROWS - 1) / attn::rope::MAX_ROWS;
  const int split = static_cast<int>(std::max(want, least));
  if (split > 65535) return ATTN_ERR_SHAPE;
  p.heads = (p.H + split - 1) / split;
  const dim3 grid(static_cast<unsigned>((tokens + p.tok - 1) / p.tok), static_cast<unsigned>((p.H + p.heads - 1) / p.heads));
  cudaError_t e;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  if (dtype == ATTN_F32) e = attn::rope::launch_dt<0>(p, halves, vec, grid, cs);
  else if (dtype == ATTN_F16) e = attn::rope::launch_dt<1>(p, halves, vec, grid, cs);
  else e = attn::rope::launch_dt<2>(p, halves, vec, grid, cs);
  return e == cudaSuccess ? ATTN_OK : attn::record_cuda_error(e);
}
