// host_checks.h - what the entry points of the 8-bit cache and of rotary positions
// share on the host.
#pragma once

#include <stdint.h>

namespace attn {

constexpr int SMS = 152;  // of the GPU that these kernels are built for

struct Buf {
  const void* p;
  int64_t n;
};

inline bool meet(const Buf& a, const Buf& b) {
  if (!a.p || !b.p || a.n <= 0 || b.n <= 0) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x < y + static_cast<uintptr_t>(b.n) && y < x + static_cast<uintptr_t>(a.n);
}

inline bool aligned(const void* p, int to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }

}  // namespace attn
