// tree_common.cuh -- shared by the operators on trees of drafted tokens: the rows of a sequence and the check of an
// accepted path.
#pragma once

#include "common.cuh"
#include "kernels.h"

namespace ink {
namespace {   // each kernel's translation unit has its own copy (internal linkage)

// Parent of the token at place i of its sequence, -1 for a child of the history.
__device__ __forceinline__ int tree_parent(const int32_t* parents, int i, uint32_t* err) {
  const int p = __ldg(parents + i);
  if (p >= -1 && p < i) return p;
  record_error(err, INK_DEVERR_BAD_TREE);
  return -1;
}

// Length of the accepted path of a sequence of n drafted tokens, 0 if it is none; by a whole warp.
__device__ __forceinline__ int tree_path(const int32_t* path, int m, int max_path, int n, int lane, uint32_t* err) {
  bool ok = m >= 0 && m <= max_path;
  for (int j = lane; ok && j < m; j += 32) {
    const int i = __ldg(path + j);
    ok = i < n && i > (j > 0 ? __ldg(path + max(j - 1, 0)) : -1);
  }
  ok = __all_sync(0xffffffffu, ok);
  if (!ok && lane == 0) record_error(err, INK_DEVERR_BAD_TREE);
  return ok ? m : 0;
}

// The last b with cu_q[b] <= t < cu_q[B] = end (-1: t lies outside), by a whole warp: 32 offsets a step.
__device__ __forceinline__ int tree_find_seq_warp(const int32_t* cu_q, int B, int end, int t, int lane) {
  if (t >= end || t < __ldg(cu_q)) return -1;
  int lo = 0, n = B;   // the answer is among lo .. lo + n - 1
  while (n > 1) {
    const int step = (n + 31) >> 5;
    const bool le = lane * step < n && __ldg(cu_q + lo + lane * step) <= t;
    const uint32_t m = __ballot_sync(0xffffffffu, le);
    const int k = m ? 31 - __clz(m) : 0;
    const int last = lo + n;
    lo += k * step;
    n = min(step, last - lo);
  }
  return lo;
}

}  // namespace
}  // namespace ink
