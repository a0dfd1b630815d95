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

// The score in units of log 2 from the raw product x = <q, K[k]>: x scale, or with a cap C
// C tanh(y), y = x scale / C:
//   |y| <= 1   y T(y^2), T the polynomial of degree 6 with the least relative error against
//              tanh(y) / y (an exchange iteration; 2^-24.2, 2^-22.6 when evaluated in fp32)
//   beyond     1 - 2 / (1 + 2^(k1 x)), off by about 2^-23
// (The prefill takes whole tiles by polynomials where it can.)
constexpr int CAP_TERMS = 7;
__device__ __forceinline__ constexpr float cap_term(int i) {
  return i == 0 ? 0.99999994f : i == 1 ? -0.3333284f : i == 2 ? 0.13325204f : i == 3 ? -0.05345703f
       : i == 4 ? 0.02028998f : i == 5 ? -0.006203379f : 0.0010410226f;
}

template <bool CAP>
__device__ __forceinline__ float score_log2(const MaskedArgs& a, float x) {
  if constexpr (!CAP) return x * a.scale_log2;
  const float y = x * a.cap_inv, u = y * y;
  float t = cap_term(CAP_TERMS - 1);
#pragma unroll
  for (int i = CAP_TERMS - 2; i >= 0; --i) t = fmaf(t, u, cap_term(i));
  const float far = fmaf(fast_rcp(1.f + fast_exp2(x * a.cap_k1)), -2.f * a.cap_log2, a.cap_log2);
  return fabsf(y) <= 1.f ? t * y * a.cap_log2 : far;
}

}  // namespace
}  // namespace ink
