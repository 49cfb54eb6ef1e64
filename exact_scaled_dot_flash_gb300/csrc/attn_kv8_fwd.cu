// attn_kv8_fwd.cu - attention of packed queries over an 8-bit paged cache: the
// entry point, and the fp32 FMA kernel that takes the calls the tensor-core
// kernels (attn_kv8_decode.cuh, attn_kv8_tc.cuh) do not: F32, D in {16, 32}.
//
// Per query row i (a query and a head) and visible key j of its sequence, with
// the codes kc, vc and the scales ks, vs of the cache (kv8.cuh):
//   s_ij = scale * ks_j * (q_i . kc_j),   o_i = sum_j softmax_j(s_i) vs_j vc_j.
// Paging, packed queries, positions, the causal mask, rows that see no key (NaN,
// lse -inf) and pages outside the cache (zero keys and values) are those of
// attn_paged_fwd.
#include <math.h>

#include <initializer_list>

#include "attn.h"
#include "host_checks.h"
#include "kv8_fwd.h"
#include "simt.cuh"

namespace attn {
namespace kv8 {

using simt::axpy4;
using simt::dot4;
using simt::load4;
using simt::store4;

constexpr int ROWS = 64;
constexpr int THREADS = 256;
constexpr int KT = 32;
constexpr float LN2 = 0.6931471805599453f;

// CTA = one (sequence, kv head) and 64 rows, 4 threads a row; 32 keys at a time
// are decoded, scaled and staged in shared memory as fp32.
template <int D, int DT, int FMT>
__global__ void __launch_bounds__(THREADS) simt_kernel(const __grid_constant__ FwdParams p) {
  constexpr int G = D / 4;
  constexpr int GPT = G / 4;
  __shared__ float4 ks[KT][G];
  __shared__ float4 vs[KT][G];
  const Cache& c = p.c;
  int* const st = c.status;
  const int tid = threadIdx.x, part = tid & 3, rl = tid >> 2;
  const int s = blockIdx.x / c.Hkv, hk = blockIdx.x - s * c.Hkv;
  const int heads = p.Hq / c.Hkv;
  int q_lo, q_hi;
  row_range(p.q_offsets, s, p.num_queries, q_lo, q_hi);
  const int nq = q_hi - q_lo;
  const int64_t r = static_cast<int64_t>(blockIdx.y) * ROWS + rl;  // row = (query, head of the kv head)
  if (static_cast<int64_t>(blockIdx.y) * ROWS >= static_cast<int64_t>(nq) * heads) return;  // CTA-uniform
  const int tq = static_cast<int>(r / heads);
  const int h = hk * heads + static_cast<int>(r - static_cast<int64_t>(tq) * heads);
  const bool row_ok = tq < nq;
  const int t = q_lo + (row_ok ? tq : 0);
  const int L = seq_len(c, s);
  const size_t nq4 = static_cast<size_t>(p.num_queries) * p.Hq * G;
  const int64_t ncode4 = static_cast<int64_t>(c.num_pages) * c.page_size * c.Hkv * G;
  const int64_t nscale = static_cast<int64_t>(c.num_pages) * c.Hkv * c.per;
  const int64_t nrows = static_cast<int64_t>(p.num_queries) * p.Hq;
  const int64_t pos = p.positions ? __ldg(p.positions + t) : L - nq + tq;
  const int key_hi_row = p.causal ? static_cast<int>(min(static_cast<int64_t>(L), pos + 1)) : L;
  int key_hi = L;  // keys any row of this CTA may see
  if (p.causal && !p.positions) {
    const int64_t last = min(static_cast<int64_t>(nq) - 1, (static_cast<int64_t>(blockIdx.y) * ROWS + ROWS - 1) / heads);
    key_hi = static_cast<int>(min(static_cast<int64_t>(L), L - nq + last + 1));
  }
  const size_t qrow = (static_cast<size_t>(t) * p.Hq + h) * G;
  float4 qr[GPT], acc[GPT];
#pragma unroll
  for (int i = 0; i < GPT; ++i) {
    qr[i] = row_ok ? load4<DT>(p.q, qrow + part + 4 * i, nq4, st) : make_float4(0.f, 0.f, 0.f, 0.f);
    acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  float m_run = -INFINITY, l_run = 0.f;
  for (int64_t tile0 = 0; tile0 < key_hi; tile0 += KT) {  // 64 bits: key_hi may be 2^31 - 1
    const int key0 = static_cast<int>(tile0);
    __syncthreads();
    for (int e = tid; e < KT * G; e += THREADS) {
      const int kr = e / G, col = e - kr * G;
      const int j = key0 + kr;
      float4 kv = make_float4(0.f, 0.f, 0.f, 0.f), vv = kv;
      const int page = j < key_hi ? page_of(c, s, j / c.page_size) : -1;
      if (page >= 0) {
        const int row = j % c.page_size;
        const size_t ci = ((static_cast<size_t>(page) * c.page_size + row) * c.Hkv + hk) * G + col;
        const size_t si = scale_index(c, page, row, hk);
        if (in_bounds(st, static_cast<int64_t>(ci), ncode4) && in_bounds(st, static_cast<int64_t>(si), nscale)) {
          const float a = __ldg(p.k_scale + si), b = __ldg(p.v_scale + si);
          kv = decode4<FMT>(__ldg(reinterpret_cast<const uint32_t*>(p.k_codes) + ci));
          vv = decode4<FMT>(__ldg(reinterpret_cast<const uint32_t*>(p.v_codes) + ci));
          kv = make_float4(kv.x * a, kv.y * a, kv.z * a, kv.w * a);
          vv = make_float4(vv.x * b, vv.y * b, vv.z * b, vv.w * b);
        }
      }
      ks[kr][col] = kv;
      vs[kr][col] = vv;
    }
    __syncthreads();
    float sreg[KT];
#pragma unroll
    for (int k = 0; k < KT; ++k) {
      float d = 0.f;
#pragma unroll
      for (int i = 0; i < GPT; ++i) d = dot4(qr[i], ks[k][part + 4 * i], d);
      d += __shfl_xor_sync(0xffffffffu, d, 1);
      d += __shfl_xor_sync(0xffffffffu, d, 2);
      sreg[k] = (row_ok && key0 + k < key_hi_row) ? d * p.scale_log2 : -INFINITY;
    }
    float mx = sreg[0];
#pragma unroll
    for (int k = 1; k < KT; ++k) mx = fmaxf(mx, sreg[k]);
    const float m_new = fmaxf(m_run, mx);
    const float m_use = m_new == -INFINITY ? 0.f : m_new;
    const float alpha = fast_exp2(m_run - m_use);
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < KT; ++k) {
      sreg[k] = fast_exp2(sreg[k] - m_use);
      sum += sreg[k];
    }
    l_run = l_run * alpha + sum;
    m_run = m_new;
#pragma unroll
    for (int i = 0; i < GPT; ++i) {
      float4 a = acc[i];
      a.x *= alpha; a.y *= alpha; a.z *= alpha; a.w *= alpha;
#pragma unroll
      for (int k = 0; k < KT; ++k) {
        // a key that this row does not see may hold anything (a NaN scale):
        // its value must not meet the zero probability
        if (key0 + k < key_hi_row) a = axpy4(sreg[k], vs[k][part + 4 * i], a);
      }
      acc[i] = a;
    }
  }
  if (!row_ok) return;
  const bool live = l_run > 0.f;
  const float inv = live ? 1.f / l_run : __int_as_float(0x7fc00000);
#pragma unroll
  for (int i = 0; i < GPT; ++i) {
    const float4 a = acc[i];
    store4<DT>(p.out, qrow + part + 4 * i, nq4, st, make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv));
  }
  const int64_t lrow = static_cast<int64_t>(t) * p.Hq + h;
  if (p.lse && part == 0 && in_bounds(st, lrow, nrows))
    p.lse[lrow] = live ? (m_run + log2f(l_run)) * LN2 : (l_run == 0.f ? -INFINITY : l_run);
}

template <int DT, int FMT>
cudaError_t launch_simt(const FwdParams& p, cudaStream_t st) {
  const int64_t ry = (static_cast<int64_t>(p.max_queries) * (p.Hq / p.c.Hkv) + ROWS - 1) / ROWS;
  const dim3 grid(static_cast<unsigned>(p.c.num_seqs) * p.c.Hkv, static_cast<unsigned>(ry > 0 ? ry : 1));
  switch (p.c.D) {
    case 16: simt_kernel<16, DT, FMT><<<grid, THREADS, 0, st>>>(p); break;
    case 32: simt_kernel<32, DT, FMT><<<grid, THREADS, 0, st>>>(p); break;
    case 64: simt_kernel<64, DT, FMT><<<grid, THREADS, 0, st>>>(p); break;
    default: simt_kernel<128, DT, FMT><<<grid, THREADS, 0, st>>>(p); break;
  }
  return cudaGetLastError();
}

}  // namespace kv8
}  // namespace attn

namespace {

using attn::aligned;
using attn::Buf;
using attn::meet;

int check_shape(const attn_paged_shape_t& s) {
  if (s.num_seqs < 0 || s.num_queries < 0 || s.Hq <= 0 || s.Hkv <= 0 || s.D <= 0 || s.page_size <= 0 ||
      s.num_pages < 0 || s.max_pages < 0 || s.max_queries < 0 || s.Hq % s.Hkv != 0)
    return ATTN_ERR_SHAPE;
  if (!(s.D == 16 || s.D == 32 || s.D == 64 || s.D == 128)) return ATTN_ERR_HEAD_DIM;
  if (static_cast<int64_t>(s.num_seqs) * s.Hkv > 0x7fffffffLL ||
      (static_cast<int64_t>(s.max_queries) * (s.Hq / s.Hkv) + 63) / 64 > 65535 ||
      static_cast<int64_t>(s.max_pages) * s.page_size > 0x7fffffffLL)
    return ATTN_ERR_SHAPE;
  // extents stay far inside 64 bits
  const double tokens = static_cast<double>(s.num_pages) * s.page_size;
  if (tokens * s.Hkv * s.D > 1e16 || static_cast<double>(s.num_queries) * s.Hq * s.D > 1e16 ||
      static_cast<double>(s.num_seqs) * s.max_pages > 1e16)
    return ATTN_ERR_SHAPE;
  return ATTN_OK;
}

// Shapes of the 16-bit kernels on the tensor cores. Their token numbers (page *
// page_size + row) are 32-bit, their row / group a 32-bit multiplication.
bool takes_tensor(const attn_paged_shape_t& s) {
  return (s.D == 64 || s.D == 128) && s.max_queries > 0 && s.num_pages > 0 && s.num_seqs > 0 &&
         static_cast<int64_t>(s.num_pages) * s.page_size <= 0x7fffffffLL && s.page_size < 65536 && s.Hkv <= 65535 &&
         static_cast<int64_t>(s.max_pages) * s.page_size <= 0x7fff0000LL;
}

// The kernel that shares out the keys; the other tensor-core kernel takes the rest.
bool takes_decode(const attn_paged_shape_t& s) {
  return takes_tensor(s) &&
         attn::kv8::decode_takes(s.num_seqs, s.Hkv, s.Hq / s.Hkv, s.max_queries, s.max_pages, s.page_size);
}

attn::kv8::DecodePlan plan_of(const attn_paged_shape_t& s) {
  return attn::kv8::decode_plan(s.num_seqs, s.Hkv, s.Hq / s.Hkv, s.max_queries, s.max_pages, s.page_size);
}

}  // namespace

extern "C" int attn_paged_kv8_workspace_bytes(const attn_paged_shape_t* shape, size_t* bytes) {
  if (!shape || !bytes) return ATTN_ERR_NULL;
  if (const int rc = check_shape(*shape)) return rc;
  const attn_paged_shape_t& s = *shape;
  *bytes = 0;
  if (takes_decode(s)) {
    *bytes = static_cast<size_t>(plan_of(s).bytes(s.Hkv, s.D));
  } else if (takes_tensor(s)) {
    const int splits = attn::kv8::tc_splits(s.num_seqs, s.Hkv, attn::kv8::tc_qblocks(s.max_queries, s.Hq / s.Hkv),
                                            s.max_pages, s.page_size);
    if (splits > 1) *bytes = static_cast<size_t>(splits) * s.num_queries * s.Hq * (s.D * 4 + 8);
  }
  return ATTN_OK;
}

extern "C" int attn_paged_kv8_fwd(const attn_paged_shape_t* shape, int group, int format, const void* q,
                                  const void* k_cache, const void* v_cache, const float* k_scale,
                                  const float* v_scale, const int32_t* block_table, const int32_t* seq_lens,
                                  const int32_t* q_offsets, const int32_t* positions, int causal, float scale,
                                  attn_dtype_t dtype, void* workspace, size_t workspace_bytes, void* out, float* lse,
                                  void* stream) {
  if (!shape) return ATTN_ERR_NULL;
  const attn_paged_shape_t s = *shape;
  if (dtype != ATTN_F32 && dtype != ATTN_F16 && dtype != ATTN_BF16) return ATTN_ERR_DTYPE;
  if (format != ATTN_KV8_INT8 && format != ATTN_KV8_E4M3) return ATTN_ERR_DTYPE;
  if (const int rc = check_shape(s)) return rc;
  if (group <= 0 || s.page_size % group != 0) return ATTN_ERR_SHAPE;
  if (causal != 0 && causal != 1) return ATTN_ERR_MASK;
  if (!(scale > 0.f) || !isfinite(scale)) return ATTN_ERR_SCALE;
  if (s.num_queries == 0 || s.num_seqs == 0) return ATTN_OK;
  if (!q || !out || !seq_lens || !q_offsets || (s.max_pages > 0 && !block_table) ||
      (s.num_pages > 0 && (!k_cache || !v_cache || !k_scale || !v_scale)))
    return ATTN_ERR_NULL;
  for (const void* p : {q, k_cache, v_cache, static_cast<const void*>(out)})
    if (!aligned(p, 16)) return ATTN_ERR_ALIGN;
  for (const void* p : {static_cast<const void*>(block_table), static_cast<const void*>(seq_lens),
                        static_cast<const void*>(q_offsets), static_cast<const void*>(positions),
                        static_cast<const void*>(k_scale), static_cast<const void*>(v_scale),
                        static_cast<const void*>(lse)})
    if (!aligned(p, 4)) return ATTN_ERR_ALIGN;
  size_t need = 0;
  attn_paged_kv8_workspace_bytes(shape, &need);
  if (need > 0) {
    if (!workspace || workspace_bytes < need) return ATTN_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return ATTN_ERR_ALIGN;
  }
  const int64_t q_bytes = static_cast<int64_t>(s.num_queries) * s.Hq * s.D * (dtype == ATTN_F32 ? 4 : 2);
  const int64_t code_bytes = static_cast<int64_t>(s.num_pages) * s.page_size * s.Hkv * s.D;
  const int64_t scale_bytes = static_cast<int64_t>(s.num_pages) * s.Hkv * (s.page_size / group) * 4;
  const Buf outs[] = {{out, q_bytes}, {lse, lse ? static_cast<int64_t>(s.num_queries) * s.Hq * 4 : 0},
                      {workspace, static_cast<int64_t>(need)}};
  const Buf ins[] = {{q, q_bytes}, {k_cache, code_bytes}, {v_cache, code_bytes}, {k_scale, scale_bytes},
                     {v_scale, scale_bytes}, {block_table, static_cast<int64_t>(s.num_seqs) * s.max_pages * 4},
                     {seq_lens, s.num_seqs * 4ll}, {q_offsets, (s.num_seqs + 1ll) * 4},
                     {positions, positions ? s.num_queries * 4ll : 0}};
  for (int i = 0; i < 3; ++i) {
    for (int j = 0; j < i; ++j)
      if (meet(outs[i], outs[j])) return ATTN_ERR_OVERLAP;
    for (const Buf& b : ins)
      if (meet(outs[i], b)) return ATTN_ERR_OVERLAP;
  }
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return attn::record_cuda_error(e);
  attn::kv8::FwdParams p{};
  p.c.num_pages = s.num_pages;
  p.c.page_size = s.page_size;
  p.c.Hkv = s.Hkv;
  p.c.D = s.D;
  p.c.group = group;
  p.c.per = s.page_size / group;
  p.c.num_seqs = s.num_seqs;
  p.c.max_pages = s.max_pages;
  p.c.block_table = block_table;
  p.c.seq_lens = seq_lens;
  p.c.status = attn::status_word(dev);
  p.Hq = s.Hq;
  p.num_queries = s.num_queries;
  p.max_queries = s.max_queries;
  p.causal = causal;
  p.device = dev;
  p.bf16 = dtype == ATTN_BF16;
  p.group_magic = group > 1 ? static_cast<uint32_t>((1ull << 32) / group + 1) : 0u;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.q_offsets = q_offsets;
  p.positions = positions;
  p.q = q;
  p.k_codes = static_cast<const uint8_t*>(k_cache);
  p.v_codes = static_cast<const uint8_t*>(v_cache);
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.out = out;
  p.lse = lse;
  p.ws = workspace;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool i8 = format == ATTN_KV8_INT8;
  using namespace attn::kv8;
  if (dtype != ATTN_F32 && takes_decode(s)) {
    const DecodePlan plan = plan_of(s);
    e = i8 ? launch_decode<FMT_INT8>(p, plan, st) : launch_decode<FMT_E4M3>(p, plan, st);
    return e == cudaSuccess ? ATTN_OK : attn::record_cuda_error(e);
  }
  if (dtype != ATTN_F32 && takes_tensor(s)) {
    e = i8 ? launch_tc<FMT_INT8>(p, st) : launch_tc<FMT_E4M3>(p, st);
    return e == cudaSuccess ? ATTN_OK : attn::record_cuda_error(e);
  }
#define ATTN_FWD(DT) (i8 ? launch_simt<DT, FMT_INT8>(p, st) : launch_simt<DT, FMT_E4M3>(p, st))
  e = dtype == ATTN_F32 ? ATTN_FWD(0) : dtype == ATTN_F16 ? ATTN_FWD(1) : ATTN_FWD(2);
#undef ATTN_FWD
  return e == cudaSuccess ? ATTN_OK : attn::record_cuda_error(e);
}
