// tree.cu -- attention of drafted tokens over the paged cache: every token sees its sequence's history and the
// drafted tokens on its way to the root.
//
//   x = sm_scale <q[t,h], K[k]>,  d = |p - pos(k)|,  s = cap(x) - slope_h d + rel[t,h,min(d, E - 1)]
//   out = softmax(s) V,  lse = log sum exp(s)
//
// A warp per (token, head): a key at a time, the running maximum and sum of its softmax, D / 32 channels a lane.
#include "masked_common.cuh"

namespace ink {
namespace {

template <int D>
__global__ void __launch_bounds__(128) tree_kernel(const TreeArgs a) {
  constexpr int C = D / 32;   // channels of a lane
  const int lane = threadIdx.x & 31;
  const long long row = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (row >= (long long)a.T * a.Hq) return;
  const int t = (int)(row / a.Hq), h = (int)(row - (long long)t * a.Hq), kvh = h / a.G;
  if (t >= __ldg(a.cu_q + a.B) || t < __ldg(a.cu_q)) return;
  int lo = 0, hi = a.B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(a.cu_q + mid) <= t) lo = mid; else hi = mid;
  }
  const int b = lo, c0 = __ldg(a.cu_q + b), c1 = __ldg(a.cu_q + b + 1), n = c1 - c0, L = __ldg(a.seq_lens + b);
  if (c0 < 0 || c1 > a.T || t >= c1) {
    if (lane == 0) record_error(a.err, INK_DEVERR_BAD_ROWS);
    return;
  }
  const int H = L - n;
  const bool bad = n > L || n > 32 * a.words;
  if (bad && lane == 0) record_error(a.err, n > L ? INK_DEVERR_QLEN_EXCEEDS_KV : INK_DEVERR_QLEN_EXCEEDS_MAX);
  const int p = max(__ldg(a.positions + t), H);
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + row * D + lane * C;
  float qv[C], o[C], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    qv[c] = __bfloat162float(q[c]);
    o[c] = 0.f;
  }
  const float slope2 = a.slopes ? __ldg(a.slopes + h) * LOG2E : 0.f;
  for (int k = a.W > 0 ? min(max(0, p - a.W + 1), H) : 0; !bad && k < L; ++k) {
    int pos = k;
    if (k >= H) {
      const int j = k - H;
      if (!((__ldg(a.ancestors + (size_t)t * a.words + (j >> 5)) >> (j & 31)) & 1u)) continue;
      pos = max(__ldg(a.positions + c0 + j), H);
      if (a.W > 0 && p - pos >= a.W) continue;
    }
    const int pi = k >> a.log2_page;
    const int page = pi < a.max_pages ? __ldg(a.block_table + (size_t)b * a.max_pages + pi) : -1;
    if (page < 0 || page >= a.num_pages) {
      if (lane == 0) record_error(a.err, INK_DEVERR_PAGE_OUT_OF_RANGE);
      continue;
    }
    const size_t kr = ((((size_t)page * a.Hkv + kvh) << a.log2_page) + (k & ((1 << a.log2_page) - 1))) * D + lane * C;
    const __nv_bfloat16* kp = static_cast<const __nv_bfloat16*>(a.k) + kr;
    const __nv_bfloat16* vp = static_cast<const __nv_bfloat16*>(a.v) + kr;
    float x = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) x = fmaf(qv[c], __bfloat162float(kp[c]), x);
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) x += __shfl_xor_sync(0xffffffffu, x, w);
    float s = x * a.scale_log2;
    if (a.softcap != 0.f) s = a.cap_log2 * tanhf(x * a.cap_inv);
    const int d = p > pos ? p - pos : pos - p;
    s = fmaf(-slope2, (float)d, s);
    if (a.rel) {
      const size_t at = (size_t)row * a.E + min(d, a.E - 1);
      s = fmaf(a.rel_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.rel)[at]) : static_cast<const float*>(a.rel)[at], LOG2E, s);
    }
    const float mn = fmaxf(m, s), f = m == -INFINITY ? 0.f : exp2f(m - mn), w = mn == -INFINITY ? 0.f : exp2f(s - mn);
    m = mn;
    l = l * f + w;
#pragma unroll
    for (int c = 0; c < C; ++c) o[c] = fmaf(w, __bfloat162float(vp[c]), o[c] * f);
  }
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + row * D + lane * C;
#pragma unroll
  for (int c = 0; c < C; ++c) out[c] = __float2bfloat16(l == 0.f ? 0.f : o[c] / l);
  if (a.lse && lane == 0) a.lse[row] = l == 0.f ? -INFINITY : m * LN2 + logf(l);
}

}  // namespace

cudaError_t launch_tree(const TreeArgs& a, int head_dim, cudaStream_t stream) {
  const long long blocks = ((long long)a.T * a.Hq + 3) / 4;
  if (head_dim == 128) tree_kernel<128><<<(int)blocks, 128, 0, stream>>>(a);
  else tree_kernel<64><<<(int)blocks, 128, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace ink
