// masked_common.cuh -- shared by the masked prefill and decode: the visible keys of a token and the
// capped score.
#pragma once

#include "common.cuh"
#include "kernels.h"

namespace ink {
namespace {   // each kernel's translation unit has its own copy (internal linkage)

constexpr float LN2 = 0.6931471805599453f;

// Visible keys [lo, hi) of token t at position p of a sequence of length L (hi <= lo: none).
__device__ __forceinline__ void token_keys(const MaskedArgs& a, int t, int p, int L, int& lo, int& hi) {
  lo = a.key_begin ? max(__ldg(a.key_begin + t), 0) : 0;
  if (a.W > 0) lo = max(lo, p - a.W + 1);
  hi = a.key_end ? __ldg(a.key_end + t) : p + 1;
  hi = max(0, min(hi, (int)min((long long)L, (long long)a.max_pages << a.log2_page)));
}

// 1 / x with the hardware approximation; 1 / infinity = 0.
__device__ __forceinline__ float fast_rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The score in units of log 2 from the raw product x = <q, K[k]>.  With C the cap:
//   CAP 0: x scale.
//   CAP 1: C tanh(x scale / C) = C (1 - 2 / (1 + 2^(k1 x))), off by about 2^-23 C: for caps up to
//          SOFTCAP_PLAIN.
//   CAP 2: the same, and below C / 4 the odd series of tanh up to the 7th power, whose relative
//          error stays below 2^-21 there: for caps so large that 2^-23 C would count.
template <int CAP>
__device__ __forceinline__ float score_log2(const MaskedArgs& a, float x) {
  if constexpr (CAP == 0) return x * a.scale_log2;
  float s = fmaf(fast_rcp(1.f + fast_exp2(x * a.cap_k1)), -2.f * a.cap_log2, a.cap_log2);
  if constexpr (CAP == 2) {
    const float u = x * a.cap_inv, u2 = u * u;
    const float w = fmaf(fmaf(fmaf(u2, -17.f / 315.f, 2.f / 15.f), u2, -1.f / 3.f), u2, 1.f) * u * a.cap_log2;
    s = fabsf(u) < 0.25f ? w : s;
  }
  return s;
}

}  // namespace
}  // namespace ink
