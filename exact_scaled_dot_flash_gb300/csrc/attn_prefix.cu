// attn_prefix.cu - attention of sequences that share a prefix: the entry point, and the
// fp32 FMA kernel of its two stages (prefix.cuh).
//
// A CTA takes 64 rows of a unit and kv head, 4 threads a row; 32 keys at a time are
// staged in shared memory as fp32.
#include <math.h>

#include <algorithm>
#include <initializer_list>

#include "attn.h"
#include "prefix.cuh"
#include "simt.cuh"

namespace attn {
namespace prefix {

using simt::axpy4;
using simt::dot4;
using simt::load4;
using simt::store4;

constexpr int ROWS = 64;
constexpr int THREADS = 256;
constexpr int KT = 32;

// Parts of a prefix of `pre` keys, 128 keys or more each.
__device__ __forceinline__ int parts_of_simt(const Params& p, int pre) { return min(p.most_parts, (pre + 127) / 128); }

template <int D, int DT, bool PREFIX>
__global__ void __launch_bounds__(THREADS) simt_kernel(const __grid_constant__ Params p) {
  constexpr int G = D / 4;
  constexpr int GPT = G / 4;
  __shared__ float4 ks[KT][G];
  __shared__ float4 vs[KT][G];
  int* const st = p.status;
  const int tid = threadIdx.x, part = tid & 3, rl = tid >> 2;
  const int unit = blockIdx.x / p.Hkv, hk = blockIdx.x - unit * p.Hkv;
  const int heads = p.Hq / p.Hkv;
  int a = unit, b = unit + 1, group = unit;  // members
  if constexpr (PREFIX) group_range(p, unit, a, b);
  else group = group_of(p, unit);
  const int pre = group >= 0 ? prefix_len(p, group) : 0;
  const int parts = pre > 0 ? parts_of_simt(p, pre) : 0;
  if constexpr (PREFIX) {
    if (static_cast<int>(blockIdx.z) >= parts) return;
  }
  if (a >= b) return;
  int q_lo;
  const int nq = queries_of(p, a, b, PREFIX ? p.max_group_queries : p.max_queries, q_lo);
  const int64_t r = static_cast<int64_t>(blockIdx.y) * ROWS + rl;
  if (static_cast<int64_t>(blockIdx.y) * ROWS >= static_cast<int64_t>(nq) * heads) return;  // CTA-uniform
  const int tq = static_cast<int>(r / heads), h = hk * heads + static_cast<int>(r - static_cast<int64_t>(tq) * heads);
  const bool row_ok = tq < nq;
  const int t = q_lo + (row_ok ? tq : 0);
  int s = a;  // the row's sequence
  if constexpr (PREFIX) s = last_at_most(p.q_offsets, a, b, t);
  int lim = row_ok ? limit_of(p, s, t) : 0;
  int from = 0, to, row;  // keys of this CTA, and the table's row that names them
  if constexpr (PREFIX) {
    row = reader_of(p, a, b, pre);
    const int64_t tiles = (pre + KT - 1) / KT;
    from = static_cast<int>(tiles * blockIdx.z / parts) * KT;
    to = min(pre, static_cast<int>(tiles * (blockIdx.z + 1) / parts) * KT);
    lim = min(lim, to);
  } else {
    row = s;
    to = seq_len(p, s);
    from = min(pre, to);
  }
  const int64_t nq4 = static_cast<int64_t>(p.num_queries) * p.Hq * G;
  const int64_t nk4 = static_cast<int64_t>(p.num_pages) * p.page_size * p.Hkv * G;
  const int64_t lrow = static_cast<int64_t>(t) * p.Hq + h;
  const int64_t qrow = lrow * G;
  float4 qr[GPT], acc[GPT];
#pragma unroll
  for (int i = 0; i < GPT; ++i) {
    qr[i] = row_ok ? load4<DT>(p.q, qrow + part + 4 * i, nq4, st) : make_float4(0.f, 0.f, 0.f, 0.f);
    acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  float m_run = -INFINITY, l_run = 0.f;
  for (int key0 = from; key0 < to; key0 += KT) {
    if (__syncthreads_and(key0 >= lim)) break;  // no row sees a key from here on
    for (int e = tid; e < KT * G; e += THREADS) {
      const int kr = e / G, c = e - (e / G) * G;
      const int j = key0 + kr;
      float4 kv = make_float4(0.f, 0.f, 0.f, 0.f), vv = kv;
      if (j < to) {
        const int page = page_of(p, row, j / p.page_size);
        if (page >= 0) {
          const int64_t idx = ((static_cast<int64_t>(page) * p.page_size + j % p.page_size) * p.Hkv + hk) * G + c;
          kv = load4<DT>(p.k, idx, nk4, st);
          vv = load4<DT>(p.v, idx, nk4, st);
        }
      }
      ks[kr][c] = kv;
      vs[kr][c] = vv;
    }
    __syncthreads();
    float sreg[KT];
#pragma unroll
    for (int c = 0; c < KT; ++c) {
      float d = 0.f;
#pragma unroll
      for (int i = 0; i < GPT; ++i) d = dot4(qr[i], ks[c][part + 4 * i], d);
      d += __shfl_xor_sync(0xffffffffu, d, 1);
      d += __shfl_xor_sync(0xffffffffu, d, 2);
      sreg[c] = key0 + c < lim ? d * p.scale_log2 : -INFINITY;
    }
    float mx = sreg[0];
#pragma unroll
    for (int c = 1; c < KT; ++c) mx = fmaxf(mx, sreg[c]);
    const float m_new = fmaxf(m_run, mx);
    const float m_use = m_new == -INFINITY ? 0.f : m_new;
    const float alpha = fast_exp2(m_run - m_use);
    float sum = 0.f;
#pragma unroll
    for (int c = 0; c < KT; ++c) {
      sreg[c] = fast_exp2(sreg[c] - m_use);
      sum += sreg[c];
    }
    l_run = l_run * alpha + sum;
    m_run = m_new;
#pragma unroll
    for (int i = 0; i < GPT; ++i) {
      float4 x = acc[i];
      x.x *= alpha; x.y *= alpha; x.z *= alpha; x.w *= alpha;
#pragma unroll
      for (int c = 0; c < KT; ++c)
        if (key0 + c < lim) x = axpy4(sreg[c], vs[c][part + 4 * i], x);  // an unseen key may hold anything
      acc[i] = x;
    }
  }
  const int64_t rows = static_cast<int64_t>(p.num_queries) * p.Hq;
  if constexpr (PREFIX) {
    const int64_t at = blockIdx.z * rows + lrow;
    if (!row_ok || !in_bounds(st, at, p.most_parts * rows)) return;
#pragma unroll
    for (int i = 0; i < GPT; ++i) reinterpret_cast<float4*>(p.o)[at * G + part + 4 * i] = acc[i];
    if (part == 0) p.ml[at] = make_float2(m_run, l_run);
  } else {
    if (!row_ok || !in_bounds(st, lrow, rows)) return;
    constexpr int BATCH = 4;  // parts read together: each read is a trip to L2
    for (int z0 = 0; z0 < parts; z0 += BATCH) {
      float2 ml[BATCH];
      float4 y[BATCH][GPT];
#pragma unroll
      for (int z = 0; z < BATCH; ++z) {
        const int64_t at = (z0 + z) * rows + lrow;
        const bool is = z0 + z < parts && in_bounds(st, at, p.most_parts * rows);
        ml[z] = is ? __ldcg(p.ml + at) : make_float2(-INFINITY, 0.f);
#pragma unroll
        for (int i = 0; i < GPT; ++i)
          y[z][i] = is ? __ldcg(reinterpret_cast<const float4*>(p.o) + at * G + part + 4 * i) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int z = 0; z < BATCH; ++z) {
        const float m = fmaxf(m_run, ml[z].x);
        if (m == -INFINITY) continue;
        const float f = fast_exp2(m_run - m), e = fast_exp2(ml[z].x - m);
        m_run = m;
        l_run = l_run * f + ml[z].y * e;
#pragma unroll
        for (int i = 0; i < GPT; ++i) {
          float4 x = acc[i];
          x.x *= f; x.y *= f; x.z *= f; x.w *= f;
          acc[i] = axpy4(e, y[z][i], x);
        }
      }
    }
    const bool live = l_run > 0.f;
    const float inv = live ? 1.f / l_run : __int_as_float(0x7fc00000);
#pragma unroll
    for (int i = 0; i < GPT; ++i)
      store4<DT>(p.out, qrow + part + 4 * i, nq4, st, make_float4(acc[i].x * inv, acc[i].y * inv, acc[i].z * inv, acc[i].w * inv));
    if (p.lse && part == 0) p.lse[lrow] = live ? (m_run + log2f(l_run)) * LN2 : (l_run == 0.f ? -INFINITY : l_run);
  }
}

template <int D, int DT>
cudaError_t launch_simt(const Params& p, cudaStream_t st) {
  const int heads = p.Hq / p.Hkv;
  auto blocks = [&](int queries) { return static_cast<unsigned>((static_cast<int64_t>(queries) * heads + ROWS - 1) / ROWS); };
  if (p.num_groups > 0 && p.max_group_queries > 0) {
    const dim3 grid(static_cast<unsigned>(p.num_groups) * p.Hkv, blocks(p.max_group_queries), static_cast<unsigned>(p.most_parts));
    simt_kernel<D, DT, true><<<grid, THREADS, 0, st>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  const dim3 grid(static_cast<unsigned>(p.num_seqs) * p.Hkv, blocks(p.max_queries));
  simt_kernel<D, DT, false><<<grid, THREADS, 0, st>>>(p);
  return cudaGetLastError();
}

template <int DT>
cudaError_t launch_dt(const Params& p, cudaStream_t st) {
  switch (p.D) {
    case 16: return launch_simt<16, DT>(p, st);
    case 32: return launch_simt<32, DT>(p, st);
    case 64: return launch_simt<64, DT>(p, st);
    default: return launch_simt<128, DT>(p, st);
  }
}

}  // namespace prefix
}  // namespace attn

namespace {

using attn::aligned;
using attn::Buf;
using attn::meet;

int check_shape(const attn_paged_shape_t& s, int num_groups, int max_group_queries) {
  if (s.num_seqs < 0 || s.num_queries < 0 || s.Hq <= 0 || s.Hkv <= 0 || s.D <= 0 || s.page_size <= 0 ||
      s.num_pages < 0 || s.max_pages < 0 || s.max_queries < 0 || s.Hq % s.Hkv != 0 || num_groups < 0 ||
      max_group_queries < 0 || s.num_seqs > 1 << 30 || num_groups > 1 << 30)
    return ATTN_ERR_SHAPE;
  if (!(s.D == 16 || s.D == 32 || s.D == 64 || s.D == 128)) return ATTN_ERR_HEAD_DIM;
  const int heads = s.Hq / s.Hkv;
  if (static_cast<int64_t>(s.num_seqs) * s.Hkv > 0x7fffffffLL || static_cast<int64_t>(num_groups) * s.Hkv > 0x7fffffffLL ||
      (static_cast<int64_t>(s.max_queries) * heads + 63) / 64 > 65535 ||
      (static_cast<int64_t>(max_group_queries) * heads + 63) / 64 > 65535 ||
      static_cast<int64_t>(s.max_pages) * s.page_size > 0x7fff0000LL)
    return ATTN_ERR_SHAPE;
  // extents stay far inside 64 bits
  const double tokens = static_cast<double>(s.num_pages) * s.page_size;
  if (tokens * s.Hkv * s.D > 1e16 || static_cast<double>(s.num_queries) * s.Hq * s.D > 1e15 ||
      static_cast<double>(s.num_seqs) * s.max_pages > 1e16)
    return ATTN_ERR_SHAPE;
  return ATTN_OK;
}

// Shapes of the 16-bit kernels for few rows, and of those for many.
bool takes_rows(const attn_paged_shape_t& s) { return (s.D == 64 || s.D == 128) && s.num_pages > 0; }
bool takes_tc(const attn_paged_shape_t& s) {
  return takes_rows(s) && s.page_size % 8 == 0 && (128 % s.page_size == 0 || s.page_size % 128 == 0);
}

// How a call runs and lays out its workspace.
struct Plan {
  int most_parts = 1;                 // parts of a row's prefix
  bool alone = false;                 // 16-bit kernels: no prefix stage
  bool prefix_tc = false, suffix_tc = false;  // the kernel for many rows
  int prefix_nt = 0, suffix_nt = 0;   // that for few: 8-row groups of a CTA
  int ranges = 0;                     // of the suffix stage
  int64_t ml_offset = 0, o_offset = 0, bytes = 0;
  int64_t head_offset = 0, first_offset = 0, own_ml_offset = 0, own_o_offset = 0, cut_ml_offset = 0, cut_o_offset = 0;
};

Plan plan_of(const attn_paged_shape_t& s, int num_groups, int max_group_queries) {
  using namespace attn::prefix;
  Plan d;
  const int64_t heads = s.Hq / s.Hkv, rows = static_cast<int64_t>(s.num_queries) * s.Hq;
  const int64_t group_rows = std::min(max_group_queries, s.num_queries) * heads;
  const int64_t seq_rows = std::min(s.max_queries, s.num_queries) * heads;
  d.prefix_tc = group_rows > 32 && takes_tc(s) && s.Hkv * ((s.num_queries * heads + 255) / 256 + num_groups) <= 0x7fffffffLL;
  d.suffix_tc = seq_rows > 32 && takes_tc(s) && s.num_seqs * s.Hkv * ((seq_rows + 255) / 256) <= 0x7fffffffLL;
  // Up to 8 MB of keys and values, counted for every sequence by itself, are 2 us of streaming: reading the
  // prefix once costs a launch and a stage more (4 rows over 201 + 40 keys: 14.4 us on the GPU and 34 us for the
  // call with it, 13.5 and 27 without).
  d.alone = takes_rows(s) && !d.suffix_tc &&
            static_cast<int64_t>(s.num_seqs) * s.max_pages * s.page_size <= (8ll << 20) / (4ll * s.Hkv * s.D);
  // With many rows the prefix stage packs rows of several sequences into its row blocks and fills every SM, but
  // each row's part goes out in FP32 and comes back, and a stage more comes up: of a pass over 256 rows, 1.85 us a
  // key tile of D 128, that is 17 us beside 40 us once (the stages run one after another here, unlike those that
  // prefix.cuh's constants are of). Without it a sequence's own row blocks run over all its keys, in whole
  // rounds of the SMs. 32/8 heads, us with the stage and without, BF16 with D 128: 4 sequences of 32 queries behind
  // 8192 tokens 65 and 106, 24 of 64 211 and 236, 8 of 128 145 and 121, 24 of 512 1346 and 1292; behind 1024 tokens
  // 46 and 25, 84 and 53, 58 and 30, 438 and 298. F16 with D 64, where the constants of D 128 choose the faster way
  // too: 46 and 92, 158 and 197, 111 and 102, 1123 and 1060; 35 and 21, 62 and 43, 45 and 25, 330 and 233. The
  // table's width stands for the lengths, and groups of one size for the call's.
  if (d.prefix_tc && d.suffix_tc) {
    const double tiles = 1.85 * s.max_pages * s.page_size / 128;
    const int64_t own = s.num_seqs * s.Hkv * ((seq_rows + 255) / 256), rounds = (own + attn::SMS - 1) / attn::SMS;
    const int64_t of_group = (s.num_queries * heads + 256ll * num_groups - 1) / (256ll * std::max(1, num_groups));
    const int64_t packed = s.Hkv * num_groups * of_group;
    d.alone = 8 + rounds * (tiles + 4) <= 40 + (tiles + 17) * packed / attn::SMS;
  }
  d.prefix_nt = rows::nt_of(group_rows);
  d.suffix_nt = rows::nt_of(seq_rows);
  // Room for as many parts of a row's prefix as its group's CTAs can leave (two each where they split
  // their keys), within 64 MB where that is enough for MIN_PARTS, or for one (FP32) of rows that 16 bits
  // take alone; a call uses what the device settles on.
  const int64_t ctas = static_cast<int64_t>(attn::SMS) * (d.prefix_tc ? 1 : rows::ctas_of_sm(s.D, d.prefix_nt));
  const int64_t units = s.Hkv * (num_groups == 1 ? std::max<int64_t>(1, (group_rows + 255) / 256) : 1);
  const int64_t room = (64ll << 20) / std::max<int64_t>(1, rows * (4 * s.D + 8));
  d.most_parts = static_cast<int>(std::max<int64_t>(d.alone ? 1 : MIN_PARTS, std::min<int64_t>({MAX_PARTS, 2 * (ctas + units - 1) / units, room})));
  const int suffix_ctas = attn::SMS * rows::ctas_of_sm(s.D, d.suffix_nt);
  d.ranges = std::max(1, suffix_ctas / s.Hkv);
  auto up = [](int64_t n) { return (n + 31) / 32 * 32; };  // the parts move in 32 bytes
  const int64_t parts = num_groups > 0 && max_group_queries > 0 ? d.most_parts : 0;
  const int64_t slots = 2ll * d.ranges * s.Hkv * 8 * d.suffix_nt;
  d.ml_offset = up(sizeof(Head) + num_groups * sizeof(Rec));
  d.o_offset = up(d.ml_offset + parts * rows * 8);
  d.bytes = up(d.o_offset + parts * rows * s.D * 4);
  if (takes_rows(s) && !d.suffix_tc) {
    d.head_offset = d.bytes;
    d.first_offset = d.head_offset + sizeof(Head);
    d.own_ml_offset = up(d.first_offset + s.num_seqs * 8ll);
    d.own_o_offset = up(d.own_ml_offset + rows * 8);
    d.cut_ml_offset = d.own_o_offset + rows * s.D * 4;
    d.cut_o_offset = up(d.cut_ml_offset + slots * 8);
    d.bytes = d.cut_o_offset + slots * s.D * 4;
  }
  d.bytes += 16;  // it begins at the next 32 bytes
  return d;
}

}  // namespace

extern "C" int attn_paged_prefix_workspace_bytes(const attn_paged_shape_t* shape, int num_groups, int max_group_queries,
                                                 size_t* bytes) {
  if (!shape || !bytes) return ATTN_ERR_NULL;
  if (const int rc = check_shape(*shape, num_groups, max_group_queries)) return rc;
  *bytes = static_cast<size_t>(plan_of(*shape, num_groups, max_group_queries).bytes);
  return ATTN_OK;
}

extern "C" int attn_paged_prefix_fwd(const attn_paged_shape_t* shape, int num_groups, int max_group_queries, const void* q,
                                     const void* k_cache, const void* v_cache, const int32_t* block_table,
                                     const int32_t* seq_lens, const int32_t* q_offsets, const int32_t* positions,
                                     const int32_t* group_offsets, const int32_t* prefix_lens, int causal, float scale,
                                     attn_dtype_t dtype, void* workspace, size_t workspace_bytes, void* out, float* lse,
                                     void* stream) {
  if (!shape) return ATTN_ERR_NULL;
  const attn_paged_shape_t s = *shape;
  if (dtype != ATTN_F32 && dtype != ATTN_F16 && dtype != ATTN_BF16) return ATTN_ERR_DTYPE;
  if (const int rc = check_shape(s, num_groups, max_group_queries)) return rc;
  if (causal != 0 && causal != 1) return ATTN_ERR_MASK;
  if (!(scale > 0.f) || !isfinite(scale)) return ATTN_ERR_SCALE;
  if (s.num_queries == 0 || s.num_seqs == 0 || s.max_queries == 0) return ATTN_OK;
  if (!q || !out || !seq_lens || !q_offsets || (s.max_pages > 0 && !block_table) ||
      (s.num_pages > 0 && (!k_cache || !v_cache)) || (num_groups > 0 && (!group_offsets || !prefix_lens)))
    return ATTN_ERR_NULL;
  for (const void* p : {q, k_cache, v_cache, static_cast<const void*>(out)})
    if (!aligned(p, 16)) return ATTN_ERR_ALIGN;
  const int64_t es = dtype == ATTN_F32 ? 4 : 2;
  const int64_t q_bytes = static_cast<int64_t>(s.num_queries) * s.Hq * s.D * es;
  const int64_t cache_bytes = static_cast<int64_t>(s.num_pages) * s.page_size * s.Hkv * s.D * es;
  const Plan plan = plan_of(s, num_groups, max_group_queries);
  if (plan.bytes > 0) {
    if (!workspace || workspace_bytes < static_cast<size_t>(plan.bytes)) return ATTN_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return ATTN_ERR_ALIGN;
  }
  const Buf outs[] = {{out, q_bytes}, {lse, lse ? static_cast<int64_t>(s.num_queries) * s.Hq * 4 : 0}, {workspace, plan.bytes}};
  const Buf ins[] = {{q, q_bytes}, {k_cache, cache_bytes}, {v_cache, cache_bytes},
                     {block_table, static_cast<int64_t>(s.num_seqs) * s.max_pages * 4}, {seq_lens, s.num_seqs * 4ll},
                     {q_offsets, (s.num_seqs + 1ll) * 4}, {positions, positions ? s.num_queries * 4ll : 0},
                     {group_offsets, (num_groups + 1ll) * 4}, {prefix_lens, num_groups * 4ll}};
  for (int i = 3; i < 9; ++i)
    if (!aligned(ins[i].p, 4)) return ATTN_ERR_ALIGN;
  if (!aligned(lse, 4)) return ATTN_ERR_ALIGN;
  for (int i = 0; i < 3; ++i) {
    for (int j = 0; j < i; ++j)
      if (meet(outs[i], outs[j])) return ATTN_ERR_OVERLAP;
    for (const Buf& b : ins)
      if (meet(outs[i], b)) return ATTN_ERR_OVERLAP;
  }
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return attn::record_cuda_error(e);
  attn::prefix::Params p{};
  p.num_seqs = s.num_seqs;
  p.num_queries = s.num_queries;
  p.num_groups = max_group_queries > 0 ? num_groups : 0;
  p.Hq = s.Hq;
  p.Hkv = s.Hkv;
  p.D = s.D;
  p.page_size = s.page_size;
  p.num_pages = s.num_pages;
  p.max_pages = s.max_pages;
  p.max_queries = std::min(s.max_queries, s.num_queries);
  p.max_group_queries = std::min(max_group_queries, s.num_queries);
  p.causal = causal;
  p.device = dev;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.block_table = block_table;
  p.seq_lens = seq_lens;
  p.q_offsets = q_offsets;
  p.positions = positions;
  p.group_offsets = group_offsets;
  p.prefix_lens = prefix_lens;
  p.q = q;
  p.k = k_cache;
  p.v = v_cache;
  p.out = out;
  p.lse = lse;
  p.status = attn::status_word(dev);
  p.most_parts = plan.most_parts;
  uint8_t* const ws = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(workspace) + 31) / 32 * 32);
  p.head = reinterpret_cast<attn::prefix::Head*>(ws);
  p.rec = reinterpret_cast<attn::prefix::Rec*>(p.head + 1);
  p.ml = reinterpret_cast<float2*>(ws + plan.ml_offset);
  p.o = reinterpret_cast<float*>(ws + plan.o_offset);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype != ATTN_F32 && takes_rows(s)) {
    if (!plan.suffix_tc) {
      p.suffix_rows = 8 * plan.suffix_nt;
      p.suffix_ranges = plan.ranges;
      p.suffix_head = reinterpret_cast<attn::prefix::Head*>(ws + plan.head_offset);
      p.suffix_first = reinterpret_cast<int64_t*>(ws + plan.first_offset);
      p.own_ml = reinterpret_cast<float2*>(ws + plan.own_ml_offset);
      p.own_o = reinterpret_cast<float*>(ws + plan.own_o_offset);
      p.cut_ml = reinterpret_cast<float2*>(ws + plan.cut_ml_offset);
      p.cut_o = reinterpret_cast<float*>(ws + plan.cut_o_offset);
    }
    const bool bf16 = dtype == ATTN_BF16;
    using namespace attn::prefix::rows;
    using attn::prefix::tc::launch;
    attn::EncodeTiledFn enc = nullptr;
    if (plan.prefix_tc || plan.suffix_tc) {
      enc = attn::encode_tiled();
      if (!enc) return attn::record_cuda_error(cudaErrorNotSupported);
    }
    if (plan.alone) p.num_groups = 0;
    const bool shared = p.num_groups > 0;
    if (shared) {
      if (plan.prefix_tc) e = bf16 ? launch<true, true>(enc, p, false, st) : launch<false, true>(enc, p, false, st);
      else e = bf16 ? launch_prefix<true>(p, plan.prefix_nt, st) : launch_prefix<false>(p, plan.prefix_nt, st);
      if (e != cudaSuccess) return attn::record_cuda_error(e);
    }
    if (plan.suffix_tc) {
      e = bf16 ? launch<true, false>(enc, p, shared, st) : launch<false, false>(enc, p, shared, st);
    } else {
      e = bf16 ? launch_suffix<true>(p, plan.suffix_nt, shared, st) : launch_suffix<false>(p, plan.suffix_nt, shared, st);
      if (e == cudaSuccess) e = bf16 ? launch_join<true>(p, st) : launch_join<false>(p, st);
    }
    return e == cudaSuccess ? ATTN_OK : attn::record_cuda_error(e);
  }
  e = dtype == ATTN_F32 ? attn::prefix::launch_dt<0>(p, st)
      : dtype == ATTN_F16 ? attn::prefix::launch_dt<1>(p, st) : attn::prefix::launch_dt<2>(p, st);
  return e == cudaSuccess ? ATTN_OK : attn::record_cuda_error(e);
}
