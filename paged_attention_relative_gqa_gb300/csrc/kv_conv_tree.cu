// kv_conv_tree.cu -- the short convolution of K and V for a tree of drafted tokens, and the convolution state behind
// the path that was accepted.
//
//     y_i = sum_{d < ks} w[ks - 1 - d] * x[ancestor of i at distance d]      (d = 0: the token itself)
// with the rows of the carried state, newest first, as the ancestors of a root.  The terms are summed in fp32 from the
// oldest row on, as the convolution of a step without drafted tokens sums them; one rounding to bf16 at the store.
//
// Bytes would bound it (rows in, rows out); a step's trees are few rows, so what it takes is a launch, a chain of cold
// reads (offsets, length, page and parents, then the rows) and the taps.  A block takes a run of tokens and 256 vectors of 8
// channels of K and V side by side: the taps stay in registers over its tokens, so few blocks with many tokens read them
// seldom, and one wave of blocks is the least that fills the machine.  A warp looks a token up while the others' taps come in;
// the next token's rows are on their way while one's are summed.  A row is read by its token and by up to ks - 1 generations of
// children, which sit next to it in the packed rows and so find it in L1 or L2.
//
// Measured (GPU time alone): 1,700 tokens of 64 trees, 2 x 16 heads of 128, 4 taps (28 MB) 14.7 us cold, 11.6 from L2;
// with as many blocks as gave four an SM in more than one wave 19.4, the taps taken thread by thread 15.1.  The state 3.1 us.
#include <algorithm>

#include "tree_common.cuh"

namespace ink {
namespace {

constexpr int CT_THREADS = 256;
constexpr int CT_TOKENS = 16;    // most tokens of a block

// Blocks an SM: what the taps and two tokens' rows leave registers for.
constexpr int ct_blocks(int ks) { return ks <= 4 ? 3 : ks <= 6 ? 2 : 1; }

__device__ __forceinline__ void ct_unpack(const uint4 r, float (&f)[8]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

template <int KS>
__global__ void __launch_bounds__(CT_THREADS, ct_blocks(KS)) kv_conv_tree_kernel(const TreeConvArgs a, int tokens) {
  __shared__ int from[CT_TOKENS][KS];   // row of the ancestor at distance d; ~r: row r of the states
  __shared__ int page[CT_TOKENS], slot[CT_TOKENS];
  const int t0 = blockIdx.x * tokens, nt = min(tokens, a.T - t0);
  const int vec = blockIdx.y * CT_THREADS + threadIdx.x;   // of K, then of V
  const int z = vec >= a.nvec, v = vec - z * a.nvec;
  const bool mine = vec < 2 * a.nvec;
  const int col = v * 8, g = col / a.D, d = col - g * a.D;
  const int lane = threadIdx.x & 31;
  // The taps of a thread's 8 channels lie 32 KS bytes from its neighbour's.  A warp loads them side by side and hands
  // them out through shared memory, four channels at a time, padded to an odd number of 16-byte units.
  float w[KS][8];
  {
    constexpr int UNITS = KS | 1;
    __shared__ float4 stage[CT_THREADS / 32][32 * UNITS];
    float4* st = stage[threadIdx.x >> 5];
    const int first = vec - lane;   // the warp's vectors lie in K, then in V
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (h) __syncwarp();
#pragma unroll
      for (int q = 0; q < KS; ++q) {
        const int i = q * 32 + lane, at = i / KS, to = first + at;
        if (to < 2 * a.nvec) {
          const int kv = to >= a.nvec;
          st[at * UNITS + i % KS] =
              __ldg(reinterpret_cast<const float4*>(a.w[kv]) + ((size_t)(to - kv * a.nvec) * 2 + h) * KS + i % KS);
        }
      }
      __syncwarp();
      float flat[4 * KS];
#pragma unroll
      for (int q = 0; q < KS; ++q) {
        const float4 f = mine ? st[lane * UNITS + q] : make_float4(0.f, 0.f, 0.f, 0.f);
        flat[4 * q] = f.x; flat[4 * q + 1] = f.y; flat[4 * q + 2] = f.z; flat[4 * q + 3] = f.w;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int j = 0; j < KS; ++j) w[j][4 * h + e] = flat[e * KS + j];
    }
  }
  // a warp looks a token up: 32 offsets a step to find its sequence, then its page and its ancestors
  for (int x = threadIdx.x >> 5; x < nt; x += CT_THREADS / 32) {
    const int t = t0 + x;
    const bool tell = blockIdx.y == 0 && lane == 0;   // one of the blocks reports
    int to = -1, at = 0;
    const int end = __ldg(a.cu_q + a.B);
    const int b = tree_find_seq_warp(a.cu_q, a.B, end, t, lane);
    if (b >= 0) {
      const int c0 = __ldg(a.cu_q + b), c1 = __ldg(a.cu_q + b + 1), L = __ldg(a.seq_lens + b), n = c1 - c0;
      if (c0 < 0 || c1 > a.T || t >= c1) {
        if (tell) record_error(a.err, INK_DEVERR_BAD_ROWS);
      } else if (n > L) {
        if (tell) record_error(a.err, INK_DEVERR_QLEN_EXCEEDS_KV);
      } else {
        const int key = L - n + t - c0, pi = key >> a.log2_page;
        const int page_id = pi < a.max_pages ? __ldg(a.block_table + (size_t)b * a.max_pages + min(pi, a.max_pages - 1)) : -1;
        int node = t - c0, back = KS - 2;   // the state's newest row is the parent of a root
#pragma unroll
        for (int i = 0; i < KS; ++i) {
          int r;
          if (node >= 0) {
            r = c0 + node;
            if (i + 1 < KS) node = tree_parent(a.parents + c0, node, a.err);
          } else {
            r = ~(b * (KS - 1) + back--);
          }
          if (lane == 0) from[x][i] = r;
        }
        at = key & ((1 << a.log2_page) - 1);
        if (page_id >= 0 && page_id < a.num_pages) to = page_id;
        else if (tell) record_error(a.err, INK_DEVERR_PAGE_OUT_OF_RANGE);
      }
    } else if (tell && t == 0 && end > a.T) {
      record_error(a.err, INK_DEVERR_BAD_ROWS);
    }
    if (lane == 0) {
      page[x] = to;
      slot[x] = at;
    }
  }
  __syncthreads();
  if (!mine) return;
  const int row = a.nvec * 8;
  auto load = [&](int x, uint4 (&raw)[KS]) {   // the rows of token x (nothing of a token that has no page)
    if (x >= nt || page[x] < 0) return;
#pragma unroll
    for (int i = 0; i < KS; ++i) {
      const int r = from[x][i];
      raw[i] = __ldg(reinterpret_cast<const uint4*>(r >= 0 ? a.x[z] + (size_t)r * row + col : a.st_in[z] + (size_t)~r * row + col));
    }
  };
  uint4 next[KS];
  load(0, next);
  for (int x = 0; x < nt; ++x) {
    uint4 raw[KS];
#pragma unroll
    for (int i = 0; i < KS; ++i) raw[i] = next[i];
    load(x + 1, next);   // on their way while these are summed
    if (page[x] < 0) continue;
    float y[8];
#pragma unroll
    for (int i = KS - 1; i >= 0; --i) {
      float f[8];
      ct_unpack(raw[i], f);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = i == KS - 1 ? w[0][e] * f[e] : fmaf(w[KS - 1 - i][e], f[e], y[e]);
    }
    const size_t to = ((((size_t)page[x] * (row / a.D) + g) << a.log2_page) + slot[x]) * a.D + d;
    *reinterpret_cast<uint4*>(a.cache[z] + to) =
        make_uint4(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]), pack_bf16(y[4], y[5]), pack_bf16(y[6], y[7]));
  }
}

// A block takes a sequence and 256 vectors of K and V side by side; its first warp checks the path.
template <int KS>
__global__ void __launch_bounds__(CT_THREADS) kv_conv_state_tree_kernel(const TreeConvArgs a) {
  __shared__ int from[KS > 1 ? KS - 1 : 1];   // row of the step; ~r: row r of the states
  const int b = blockIdx.x;
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    const int c0 = __ldg(a.cu_q + b), c1 = __ldg(a.cu_q + b + 1);
    const int32_t* path = a.path + (size_t)b * a.max_path;
    int m = 0;
    if (c0 < 0 || c1 > a.T || c1 < c0) {
      if (lane == 0) record_error(a.err, INK_DEVERR_BAD_ROWS);
    } else {
      m = tree_path(path, __ldg(a.path_lens + b), a.max_path, c1 - c0, lane, a.err);
    }
    // row r of the new state is row m + r of the old one and the path's rows side by side
    if (lane < KS - 1) from[lane] = m + lane < KS - 1 ? ~(b * (KS - 1) + m + lane)
                                                          : c0 + __ldg(path + max(m + lane - (KS - 1), 0));
  }
  __syncthreads();
  const int vec = blockIdx.y * CT_THREADS + threadIdx.x;
  if (vec >= 2 * a.nvec) return;
  const int z = vec >= a.nvec, col = (vec - z * a.nvec) * 8, row = a.nvec * 8;
  uint4 x[KS > 1 ? KS - 1 : 1];
#pragma unroll
  for (int r = 0; r < KS - 1; ++r) {
    const int f = from[r];
    x[r] = __ldg(reinterpret_cast<const uint4*>(f >= 0 ? a.x[z] + (size_t)f * row + col : a.st_in[z] + (size_t)~f * row + col));
  }
#pragma unroll
  for (int r = 0; r < KS - 1; ++r)
    *reinterpret_cast<uint4*>(a.st_out[z] + ((size_t)b * (KS - 1) + r) * row + col) = x[r];
}

template <int KS>
cudaError_t launch_state_t(const TreeConvArgs& a, cudaStream_t stream) {
  kv_conv_state_tree_kernel<KS><<<dim3(a.B, (2 * a.nvec + CT_THREADS - 1) / CT_THREADS), CT_THREADS, 0, stream>>>(a);
  return cudaGetLastError();
}

template <int KS>
cudaError_t launch_conv_t(const TreeConvArgs& a, int num_sms, cudaStream_t stream) {
  const int cols = (2 * a.nvec + CT_THREADS - 1) / CT_THREADS;
  // as few tokens a block as one wave of ct_blocks(KS) blocks an SM holds: they share the loads of the taps, but follow one another
  const long long fit = std::max(1ll, (long long)ct_blocks(KS) * num_sms / cols);
  const int tokens = (int)std::min<long long>(CT_TOKENS, (a.T + fit - 1) / fit);
  kv_conv_tree_kernel<KS><<<dim3((a.T + tokens - 1) / tokens, cols), CT_THREADS, 0, stream>>>(a, tokens);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_conv_tree(const TreeConvArgs& a, int kernel_size, int num_sms, cudaStream_t stream) {
  switch (kernel_size) {
    case 1: return launch_conv_t<1>(a, num_sms, stream);
    case 2: return launch_conv_t<2>(a, num_sms, stream);
    case 3: return launch_conv_t<3>(a, num_sms, stream);
    case 4: return launch_conv_t<4>(a, num_sms, stream);
    case 5: return launch_conv_t<5>(a, num_sms, stream);
    case 6: return launch_conv_t<6>(a, num_sms, stream);
    case 7: return launch_conv_t<7>(a, num_sms, stream);
    case 8: return launch_conv_t<8>(a, num_sms, stream);
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_kv_conv_state_tree(const TreeConvArgs& a, int kernel_size, cudaStream_t stream) {
  switch (kernel_size) {
    case 2: return launch_state_t<2>(a, stream);
    case 3: return launch_state_t<3>(a, stream);
    case 4: return launch_state_t<4>(a, stream);
    case 5: return launch_state_t<5>(a, stream);
    case 6: return launch_state_t<6>(a, stream);
    case 7: return launch_state_t<7>(a, stream);
    case 8: return launch_state_t<8>(a, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace ink
