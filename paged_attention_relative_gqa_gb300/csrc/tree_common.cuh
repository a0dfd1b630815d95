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
    ok = i < n && i > (j > 0 ? __ldg(path + j - 1) : -1);
  }
  ok = __all_sync(0xffffffffu, ok);
  if (!ok && lane == 0) record_error(err, INK_DEVERR_BAD_TREE);
  return ok ? m : 0;
}

// The last b with cu_q[b] <= t < cu_q[B] (-1: t lies outside).
__device__ __forceinline__ int tree_find_seq(const int32_t* cu_q, int B, int t) {
  if (t < __ldg(cu_q) || t >= __ldg(cu_q + B)) return -1;
  int lo = 0, hi = B;   // cu_q[lo] <= t < cu_q[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(cu_q + mid) <= t) lo = mid; else hi = mid;
  }
  return lo;
}

}  // namespace
}  // namespace ink
