// masked_simple.cu -- masked attention over the paged cache, one warp per (token, query head).
//
// s_k = cap(sm_scale <q, K[k]>) - slope |p - k| over the token's visible keys, cap(x) = c tanh(x / c);
// out = softmax(s) V, lse = log sum exp(s).  32 keys at a time: a lane scores one key, the warp
// keeps the running maximum and sum, and each lane adds up D / 32 output channels.  A key that is
// not visible, or whose page lies outside the pool, is never read.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "kernels.h"

namespace ink {
namespace {

constexpr int MS_WARPS = 8;

template <int D>
__global__ void __launch_bounds__(MS_WARPS * 32) masked_simple_kernel(const MaskedArgs a) {
  __shared__ float qs[MS_WARPS][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long w = (long long)blockIdx.x * MS_WARPS + warp;
  if (w >= (long long)a.T * a.Hq) return;
  const int t = (int)(w / a.Hq), h = (int)(w - (long long)t * a.Hq), g = h / a.G;
  int b = t, p = 0, L;
  bool empty = false;
  if (a.cu_q) {
    if (t < __ldg(a.cu_q) || t >= __ldg(a.cu_q + a.B)) return;
    int lo = 0, hi = a.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (__ldg(a.cu_q + mid) <= t) lo = mid; else hi = mid;
    }
    b = lo;
    const int c0 = __ldg(a.cu_q + b), c1 = __ldg(a.cu_q + b + 1);
    L = __ldg(a.seq_lens + b);
    if (c0 < 0 || c1 > a.T) {
      if (lane == 0) record_error(a.err, INK_DEVERR_BAD_ROWS);
      return;
    }
    if (c1 - c0 > L) {
      if (lane == 0) record_error(a.err, INK_DEVERR_QLEN_EXCEEDS_KV);
      empty = true;
    }
    p = L - (c1 - c0) + (t - c0);
  } else {
    L = __ldg(a.seq_lens + b);
    p = L - 1;
    empty = L <= 0;
  }
  const long long reach = (long long)a.max_pages << a.log2_page;
  if (!empty && L > reach && lane == 0) record_error(a.err, INK_DEVERR_PAGE_OUT_OF_RANGE);
  int k0 = a.key_begin ? max(__ldg(a.key_begin + t), 0) : 0;
  if (a.W > 0) k0 = max(k0, p - a.W + 1);
  int k1 = a.key_end ? __ldg(a.key_end + t) : p + 1;
  k1 = min(k1, (int)min((long long)L, reach));
  if (empty) k1 = k0;
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + ((size_t)t * a.Hq + h) * D;
  for (int d = lane; d < D; d += 32) qs[warp][d] = __bfloat162float(q[d]);
  __syncwarp();
  const float slope = a.slopes ? __ldg(a.slopes + h) : 0.f;
  float m = -INFINITY, l = 0.f, o[D / 32];
#pragma unroll
  for (int i = 0; i < D / 32; ++i) o[i] = 0.f;
  for (int c = k0; c < k1; c += 32) {
    const int k = c + lane;
    float s = -INFINITY;
    long long row = -1;
    if (k < k1) {
      const int page = __ldg(a.block_table + (size_t)b * a.max_pages + (k >> a.log2_page));
      if (page < 0 || page >= a.num_pages) {
        record_error(a.err, INK_DEVERR_PAGE_OUT_OF_RANGE);
      } else {
        row = (((long long)page * a.Hkv + g) << a.log2_page) + (k & ((1 << a.log2_page) - 1));
        const __nv_bfloat16* kr = static_cast<const __nv_bfloat16*>(a.k) + row * D;
        float x = 0.f;
        for (int d = 0; d < D; ++d) x = fmaf(qs[warp][d], __bfloat162float(kr[d]), x);
        x *= a.sm_scale;
        if (a.softcap > 0.f) x = a.softcap * tanhf(x / a.softcap);
        s = x - slope * fabsf((float)(p - k));
      }
    }
    float mx = s;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
    const float mn = fmaxf(m, mx);
    const float mu = mn == -INFINITY ? 0.f : mn;
    const float f = expf(m - mu), pr = row >= 0 ? expf(s - mu) : 0.f;
    m = mn;
    l = l * f + pr;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) o[i] *= f;
    for (int j = 0; j < 32; ++j) {
      const float pj = __shfl_sync(0xffffffffu, pr, j);
      const long long rj = __shfl_sync(0xffffffffu, row, j);
      if (rj < 0) continue;
      const __nv_bfloat16* vr = static_cast<const __nv_bfloat16*>(a.v) + rj * D;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) o[i] = fmaf(pj, __bfloat162float(vr[lane + 32 * i]), o[i]);
    }
  }
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
  const float inv = l > 0.f ? 1.f / l : 0.f;
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + ((size_t)t * a.Hq + h) * D;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) out[lane + 32 * i] = __float2bfloat16(l == 0.f ? 0.f : o[i] * inv);
  if (a.lse && lane == 0) a.lse[(size_t)t * a.Hq + h] = l == 0.f ? -INFINITY : m + logf(l);
}

}  // namespace

cudaError_t launch_masked_simple(const MaskedArgs& a, int head_dim, cudaStream_t stream) {
  const long long warps = (long long)a.T * a.Hq;
  const int grid = (int)((warps + MS_WARPS - 1) / MS_WARPS);
  if (head_dim == 128) masked_simple_kernel<128><<<grid, MS_WARPS * 32, 0, stream>>>(a);
  else masked_simple_kernel<64><<<grid, MS_WARPS * 32, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace ink
