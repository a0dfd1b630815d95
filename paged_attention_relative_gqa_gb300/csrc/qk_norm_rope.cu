// qk_norm_rope.cu -- RMS norm of every query and key head, rotation by the token's position, and
// the write of K and V into the paged caches, in one pass over the rows of the projection.
//
// For a head x of D channels at position p:
//     y = x * (mean(x^2) + eps)^(-1/2) * w
//     a' = c (a cos(p f) - b sin(p f)),  b' = c (b cos(p f) + a sin(p f))
// for each pair (a, b) of the first rot_dim channels with frequency f (halves: channels i and
// i + rot_dim / 2; interleaved: 2 i and 2 i + 1), all in fp32, one rounding to bf16 at the store.
//
// Bytes bound it: every row is read once and written once.  A warp takes one token and runs over
// its head rows, LPR = D / 8 lanes to a row (16 bytes a lane, 512 contiguous bytes a warp and
// pass), the next NB passes on their way while NB are worked on.  The angles depend on the token
// alone: a warp takes the sine and cosine of each pair once (a pair a lane) and folds them and the
// weights into two factors per channel, which stay in registers over all heads of q or k.  A token's
// passes are cut over several warps when there are few tokens (decode).  In the half layout the
// partner channels sit rot_dim / 16 lanes away and come by shuffle as raw bf16 (4 registers for
// 8 channels), normed with the partner's weights.
//
// Measured (GPU time alone): 34,500 tokens of 64 + 2 x 8 heads of 128 (1.4 GB) 211 us, 6.7 TB/s, as fast as a copy;
// 5,161 tokens of 40 + 2 x 8 heads of 128, half of the channels rotated, 31 us, 4.8 TB/s: there a warp's serial start
// (offsets, length, angles, page) and the 2 to 4 passes it has on their way show; 64 tokens of a decode 5 us, one token
// 3 us (a launch).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace ink {
namespace {

constexpr int NR_THREADS = 256;
constexpr int NR_BLOCKS = 3;   // blocks an SM has registers for

__device__ __forceinline__ void unpack_bf16x8(const uint4 r, float (&f)[8]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

// cos and sin of p * f, p any non-negative int32.  In turns, in fixed point (the idea of Payne and Hanek's
// "Radian reduction for trigonometric functions": only what is left of whole turns is kept): g = f / (2 pi) modulo 1 in
// 64 bits, from f's 24 digits and 2^66 / (2 pi) rounded to 64 bits; p g modulo 1 is then the low 64
// bits of a product of integers.  Cutting g off costs p 2^-64 <= 2^-33 of a turn, the constant's
// rounding p f 2^-68, cutting the turn to 32 bits 2^-32 and its float 2^-26: the error does not grow with
// the position.  (Two-float products, 1 % faster, were off by 2^-18 of a turn near 2^31.)
__device__ __forceinline__ void turn(int p, float f, float scale, float& c, float& s) {
  constexpr uint32_t HI = 0xA2F9836Eu, LO = 0x4E44152Au;   // 2^66 / (2 pi)
  const uint32_t u = __float_as_uint(f);
  const uint32_t m = (u & 0x7FFFFFu) | 0x800000u;              // |f| = m 2^(e - 150) (a denormal f is next to none)
  const uint32_t down = 152u - ((u >> 23) & 0xFFu);            // g = m 2^66 / (2 pi) / 2^down
  const unsigned long long low = (unsigned long long)m * LO;
  const unsigned long long high = (unsigned long long)m * HI + (low >> 32);
  const uint32_t w0 = (uint32_t)low, w1 = (uint32_t)high, w2 = (uint32_t)(high >> 32);
  const uint32_t x0 = down < 32 ? w0 : down < 64 ? w1 : w2, x1 = down < 32 ? w1 : down < 64 ? w2 : 0u;
  const uint32_t x2 = down < 32 ? w2 : 0u;
  uint32_t g0 = __funnelshift_r(x0, x1, down), g1 = __funnelshift_r(x1, x2, down);
  if (down - 1u >= 95u) {                                      // |f| >= 2^25, or so small that nothing turns
    const uint32_t up = 0u - down;                             // (after 2^32: of the lower 64 bits)
    const unsigned long long g = up < 64 ? ((high << 32) | w0) << up : 0ull;
    g0 = (uint32_t)g;
    g1 = (uint32_t)(g >> 32);
  }
  const int top = (int)(__umulhi((uint32_t)p, g0) + (uint32_t)p * g1);   // p g in [-1/2, 1/2) of a turn, times 2^32
  // (an infinite or NaN frequency gives NaN)
  const float r = fmaf(f, 0.f, (float)top * ((u >> 31) ? -0x1p-31f : 0x1p-31f));
  float cs, sn;
  sincospif(r, &sn, &cs);
  c = cs * scale;
  s = sn * scale;
}

// The last b with cu_q[b] <= t < cu_q[B] = end (-1: t lies outside), by a whole warp: 32 offsets a step.
__device__ __forceinline__ int find_seq_warp(const int32_t* cu_q, int B, int end, int t, int lane) {
  if (t >= end || t < __ldg(cu_q)) return -1;
  int lo = 0, n = B;   // the answer is among lo .. lo + n - 1
  while (n > 1) {
    const int step = (n + 31) >> 5;
    const int i = lo + lane * step;
    const bool le = lane * step < n && __ldg(cu_q + i) <= t;
    const uint32_t m = __ballot_sync(0xffffffffu, le);
    const int k = m ? 31 - __clz(m) : 0;
    const int last = lo + n;
    lo += k * step;
    n = min(step, last - lo);
  }
  return lo;
}

// LAYOUT 0: no rotation, 1: halves, 2: interleaved
template <int D, int LAYOUT>
__global__ void __launch_bounds__(NR_THREADS, NR_BLOCKS) qk_norm_rope_kernel(const NormRopeArgs a) {
  constexpr int LPR = D / 8;          // lanes per row
  constexpr int RPP = 32 / LPR;       // rows per pass
  // Passes loaded together, the next as many on their way.  Four, but two where the rotation of halves
  // needs the registers (20,000 tokens of 16 + 2 x 2 heads of 64: 43 against 36 us; norm alone, 34,500
  // tokens of 64 + 2 x 8 heads of 128: 211 against 229 us).
  constexpr int NB = LAYOUT == 1 ? 2 : 4;
  const int lane = threadIdx.x & 31;
  const long long gw = (long long)blockIdx.x * (NR_THREADS / 32) + (threadIdx.x >> 5);
  const int t = (int)(gw / a.nchunks);
  if (t >= a.T) return;
  const int pass0 = (int)(gw - (long long)t * a.nchunks) * a.chunk;
  const int pass1 = min(pass0 + a.chunk, a.passes);
  const int lr = lane % LPR, rip = lane / LPR;
  const int d = lr * 8;

  uint4 ahead[NB];   // the next batch of passes
  // passes q .. q + NB - 1 of section sec, up to its pass `end`
  auto load = [&](int sec, int q, int end) {
    const uint16_t* src = a.x[sec] + (size_t)t * a.x_stride[sec] + d;
#pragma unroll
    for (int k = 0; k < NB; ++k) {
      const int h = (q + k) * RPP + rip;
      ahead[k] = make_uint4(0, 0, 0, 0);
      if (q + k < end && h < a.H[sec]) ahead[k] = *reinterpret_cast<const uint4*>(src + (size_t)h * D);
    }
  };
  // this warp's passes of section sec
  auto span = [&](int sec, int& q0, int& q1) {
    const int nq = (a.H[0] + RPP - 1) / RPP, nkv = (a.H[1] + RPP - 1) / RPP;
    const int base = sec == 0 ? 0 : sec == 1 ? nq : nq + nkv;
    q0 = max(pass0 - base, 0);
    q1 = min(pass1 - base, sec == 0 ? nq : nkv);
  };
  // the first rows need nothing but the token: they are on their way while its request is looked up
  int first = 0;
  {
    int q0, q1;
    for (span(0, q0, q1); q0 >= q1; span(++first, q0, q1)) {}
    load(first, q0, q1);
  }

  const int end = __ldg(a.cu_q + a.B);
  // (by the first row's warp too: requests that lie behind the last row have none)
  if (end > a.T && t == 0 && lane == 0) record_error(a.err, INK_DEVERR_BAD_ROWS);
  const int b = find_seq_warp(a.cu_q, a.B, end, t, lane);
  if (b < 0) return;                  // a row of no request
  const int c0 = __ldg(a.cu_q + b), c1 = __ldg(a.cu_q + b + 1), n = c1 - c0, L = __ldg(a.seq_lens + b);
  if (c0 < 0 || c1 > a.T || t >= c1) {   // rows outside [0, T), or offsets that do not increase
    if (lane == 0) record_error(a.err, INK_DEVERR_BAD_ROWS);
    return;
  }
  if (n > L) {
    if (lane == 0) record_error(a.err, INK_DEVERR_QLEN_EXCEEDS_KV);
    return;
  }
  const int p = L - n + (t - c0);     // in [0, L)

  const int hl = a.rot_dim >> 4;      // halves: lanes of half the rotated channels
  const bool turned = LAYOUT != 0 && d < a.rot_dim;
  // cos and sin of every pair, each taken by one lane, in shared memory until a section needs them
  __shared__ float2 turns[LAYOUT != 0 ? NR_THREADS / 32 : 1][LAYOUT != 0 ? D / 2 : 1];
  float2* mine = turns[LAYOUT != 0 ? threadIdx.x >> 5 : 0];
  if constexpr (LAYOUT != 0) {
    for (int f = lane; f < a.rot_dim / 2; f += 32) {
      float c, sn;
      turn(p, __ldg(a.inv_freq + f), a.rot_scale, c, sn);
      mine[f] = make_float2(c, sn);
    }
    __syncwarp();
  }
  const int partner = LAYOUT == 1 && turned ? (lr < hl ? lr + hl : lr - hl) : lr;

#pragma unroll 1
  for (int sec = first; sec < 3; ++sec) {
    const int H = a.H[sec];
    int q0, q1;
    span(sec, q0, q1);
    if (q0 >= q1) continue;
    if (sec != first) load(sec, q0, q1);
    uint16_t* dst;                    // row h goes to dst + h * step
    long long step;
    if (sec == 0) {
      dst = a.q_out + (size_t)t * H * D;
      step = D;
    } else {
      const int pi = p >> a.log2_page;
      const int page = pi < a.max_pages ? __ldg(a.block_table + (size_t)b * a.max_pages + pi) : -1;
      if (page < 0 || page >= a.num_pages) {
        if (lane == 0) record_error(a.err, INK_DEVERR_PAGE_OUT_OF_RANGE);
        continue;
      }
      step = (long long)D << a.log2_page;
      dst = a.cache[sec - 1] + (size_t)page * H * step + (size_t)(p & ((1 << a.log2_page) - 1)) * D;
    }
    const float* wsrc = sec < 2 ? a.w[sec] : nullptr;
    // y = r (x A + x' B) with the mean square's r, the pair's other channel x' and
    //   halves: A = w cos, B = w' (-+ sin);  interleaved: the same with x' in the same lane
    float A[8], B[LAYOUT != 0 ? 8 : 1];
#pragma unroll
    for (int e = 0; e < 8; ++e) A[e] = 1.f;
    if (wsrc) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const float4 f = __ldg(reinterpret_cast<const float4*>(wsrc + d) + x);
        A[4 * x] = f.x; A[4 * x + 1] = f.y; A[4 * x + 2] = f.z; A[4 * x + 3] = f.w;
      }
    }
    if (LAYOUT != 0 && turned && sec < 2) {
#pragma unroll
      for (int e = 0; e < (LAYOUT == 1 ? 8 : 4); ++e) {
        if constexpr (LAYOUT == 1) {   // first half: a cos - b sin; second: b cos + a sin
          const float2 t2 = mine[(lr < hl ? lr : lr - hl) * 8 + e];
          B[e] = (wsrc ? __ldg(wsrc + partner * 8 + e) : 1.f) * (lr < hl ? -t2.y : t2.y);
          A[e] *= t2.x;
        } else if constexpr (LAYOUT == 2) {
          const float2 t2 = mine[lr * 4 + e];
          B[2 * e] = -A[2 * e + 1] * t2.y;
          B[2 * e + 1] = A[2 * e] * t2.y;
          A[2 * e] *= t2.x;
          A[2 * e + 1] *= t2.x;
        }
      }
    }
    uint4 raw[NB];
#pragma unroll 1
    for (int q = q0; q < q1; q += NB) {
#pragma unroll
      for (int k = 0; k < NB; ++k) raw[k] = ahead[k];
      if (q + NB < q1) load(sec, q + NB, q1);
#pragma unroll
      for (int k = 0; k < NB; ++k) {
        if (q + k >= q1) break;       // the same for the whole warp
        const int h = (q + k) * RPP + rip;
        uint4 res = raw[k];
        if (sec < 2) {
          float x[8], y[8];
          unpack_bf16x8(raw[k], x);
          float r = 1.f;
          if (wsrc) {
            float ss = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            r = rsqrtf(fmaf(ss, 1.f / D, a.eps));
          }
          if constexpr (LAYOUT == 1) {
            const int from = rip * LPR + partner;
            uint4 other;
            other.x = __shfl_sync(0xffffffffu, raw[k].x, from);
            other.y = __shfl_sync(0xffffffffu, raw[k].y, from);
            other.z = __shfl_sync(0xffffffffu, raw[k].z, from);
            other.w = __shfl_sync(0xffffffffu, raw[k].w, from);
            float z[8];
            unpack_bf16x8(other, z);
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = r * (turned ? fmaf(z[e], B[e], x[e] * A[e]) : x[e] * A[e]);
          } else if constexpr (LAYOUT == 2) {
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = r * (turned ? fmaf(x[e ^ 1], B[e], x[e] * A[e]) : x[e] * A[e]);
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = r * (x[e] * A[e]);
          }
          res = make_uint4(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]), pack_bf16(y[4], y[5]), pack_bf16(y[6], y[7]));
        }
        if (h < H) *reinterpret_cast<uint4*>(dst + (size_t)h * step + d) = res;
      }
    }
  }
}

template <int D>
cudaError_t launch_t(const NormRopeArgs& a, int layout, cudaStream_t stream) {
  const long long warps = (long long)a.T * a.nchunks;
  const long long blocks = (warps + NR_THREADS / 32 - 1) / (NR_THREADS / 32);
  if (blocks >= (1ll << 31)) return cudaErrorInvalidConfiguration;
  const int grid = (int)blocks;
  if (layout == 0) qk_norm_rope_kernel<D, 0><<<grid, NR_THREADS, 0, stream>>>(a);
  else if (layout == 1) qk_norm_rope_kernel<D, 1><<<grid, NR_THREADS, 0, stream>>>(a);
  else qk_norm_rope_kernel<D, 2><<<grid, NR_THREADS, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_qk_norm_rope(NormRopeArgs& a, int head_dim, bool interleaved, int num_sms, cudaStream_t stream) {
  const int rpp = 32 / (head_dim / 8);
  a.passes = (a.H[0] + rpp - 1) / rpp + 2 * ((a.H[1] + rpp - 1) / rpp);
  // One warp per token when that already fills the machine (about 32 warps an SM); with fewer
  // tokens a token's passes are cut over more warps, down to one pass each.
  const long long want = (long long)num_sms * 32;
  long long cut = a.T > 0 ? (want + a.T - 1) / a.T : 1;
  cut = std::max(1ll, std::min<long long>(cut, a.passes));
  a.chunk = (int)((a.passes + cut - 1) / cut);
  a.nchunks = (a.passes + a.chunk - 1) / a.chunk;
  const int layout = a.rot_dim == 0 ? 0 : interleaved ? 2 : 1;
  return head_dim == 128 ? launch_t<128>(a, layout, stream) : launch_t<64>(a, layout, stream);
}

}  // namespace ink
