// kv8_ops.cuh - operands of the 16-bit kernels over an 8-bit cache: codes as F16,
// queries in F16's range, asynchronous copies.
#pragma once

#include "kv8.cuh"

namespace attn {
namespace kv8 {

// The 4 codes of a word as two F16 pairs: bytes 0, 1 and bytes 2, 3. The
// conversion instruction makes NaN of the e4m3 codes 0x7f and 0xff, which stand
// for +-480: the kernels look for a NaN among what they made of a tile, and
// convert it again with EVERY. EVERY places the code's 7 bits in the top of F16's
// exponent and mantissa, the value times 2^(7 - 15), subnormals included, and
// multiplies by 2^8, exactly: 5 instructions for a pair instead of 1.
template <int FMT, bool EVERY = false>
__device__ __forceinline__ void pairs(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (FMT == FMT_INT8) {
    const uint32_t u = w ^ 0x80808080u;  // c + 128
    const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);  // 1024 + (c + 128)
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(a), "r"(0x64806480u));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(b), "r"(0x64806480u));
  } else if constexpr (EVERY) {
    auto one = [](uint32_t p) {  // a code in the high byte of each half
      uint32_t r;
      asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"((p & 0x80008000u) | ((p & 0x7f007f00u) >> 1)), "r"(0x5c005c00u));
      return r;
    };
    lo = one(__byte_perm(w, 0u, 0x1404));
    hi = one(__byte_perm(w, 0u, 0x3424));
  } else {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  }
}

// 16 or 4 bytes global -> shared; `bytes` of them (0: zeros are written).
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Power of two 2^e as fp32, e in [-126, 127].
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// A pair of outputs in the type of q.
__device__ __forceinline__ uint32_t pack_out(bool bf16, float a, float b) {
  return bf16 ? pack2<true>(a, b) : pack2<false>(a, b);
}

// The factor that brings a row of BF16 whose largest finite magnitude is `top` to
// F16 (that element to [2^14, 2^15)), and its inverse.
__device__ __forceinline__ float f16_range(float top, float& back) {
  const int e = min(max(14 + 127 - static_cast<int>(__float_as_uint(top) >> 23), -126), 126);
  back = pow2(-e);
  return pow2(e);
}

// Largest finite magnitude of a BF16 pair.
__device__ __forceinline__ float finite_top(uint32_t pair) {
  const float lo = fabsf(__uint_as_float(pair << 16)), hi = fabsf(__uint_as_float(pair & 0xffff0000u));
  return fmaxf(lo < INFINITY ? lo : 0.f, hi < INFINITY ? hi : 0.f);
}

}  // namespace kv8
}  // namespace attn
