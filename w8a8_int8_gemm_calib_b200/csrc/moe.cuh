// moe.cuh -- what the row steps of the routing share (moe.cu, combine.cu).
#pragma once

#include <stdint.h>

#include "sq_device.cuh"
#include "sq_internal.h"

namespace sq {

constexpr int kRowThreads = 256;

// the sorted row of assignment (t, c), or -1
__device__ __forceinline__ int64_t place(const MoeArgs& a, int64_t t, int c) {
  if (c >= a.top_k || !in_bounds(t * a.top_k + c, 1, a.T * a.top_k, a.status)) return -1;
  const int64_t r = __ldcg(a.pos + t * a.top_k + c);
  return r >= 0 && r < a.R ? r : -1;
}

// threads of a block that covers n pieces of a row
inline unsigned row_threads(int64_t n) {
  return n >= kRowThreads ? (unsigned)kRowThreads : (unsigned)((n + 31) / 32 * 32);
}

}  // namespace sq
