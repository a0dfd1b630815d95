// kv_conv_tree.cu -- the short convolution of K and V for a tree of drafted tokens, and the convolution state behind
// the path that was accepted.
//
//     y_i = sum_{d < ks} w[ks - 1 - d] * x[ancestor of i at distance d]      (d = 0: the token itself)
// with the rows of the carried state, newest first, as the ancestors of a root.  The terms are summed in fp32 from the
// oldest row on, as the convolution of a step without drafted tokens sums them; one rounding to bf16 at the store.
//
// Bytes bound it: rows in, rows out, and the taps.  A row is read by its token and by up to ks - 1 generations of children, which
// sit next to it in the packed rows and so find it in L1 or L2.  A block takes a few tokens and 256 vectors of
// 8 channels of K and V side by side; who the ancestors are, and where the row goes, is found once per token by
// one thread and kept in shared memory, while the other threads load their channels' taps.
#include <algorithm>

#include "tree_common.cuh"

namespace ink {
namespace {

constexpr int CT_THREADS = 256;
constexpr int CT_TOKENS = 8;     // most tokens of a block

__device__ __forceinline__ void ct_unpack(const uint4 r, float (&f)[8]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

template <int KS>
__global__ void __launch_bounds__(CT_THREADS) kv_conv_tree_kernel(const TreeConvArgs a, int tokens) {
  __shared__ int from[CT_TOKENS][KS];   // row of the ancestor at distance d; ~r: row r of the states
  __shared__ int page[CT_TOKENS], slot[CT_TOKENS];
  const int t0 = blockIdx.x * tokens, nt = min(tokens, a.T - t0);
  const int vec = blockIdx.y * CT_THREADS + threadIdx.x;   // of K, then of V
  const int z = vec >= a.nvec, v = vec - z * a.nvec;
  const bool mine = vec < 2 * a.nvec;
  const int col = v * 8, g = col / a.D, d = col - g * a.D;
  float w[KS][8];
  if (mine) {
    float flat[8 * KS];
    const float4* wp = reinterpret_cast<const float4*>(a.w[z] + (size_t)col * KS);
#pragma unroll
    for (int q = 0; q < 2 * KS; ++q) {
      const float4 f = __ldg(wp + q);
      flat[4 * q] = f.x; flat[4 * q + 1] = f.y; flat[4 * q + 2] = f.z; flat[4 * q + 3] = f.w;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
#pragma unroll
      for (int j = 0; j < KS; ++j) w[j][e] = flat[e * KS + j];
  }
  if ((int)threadIdx.x < nt) {
    const int x = threadIdx.x, t = t0 + x;
    const bool tell = blockIdx.y == 0;   // one of the blocks reports
    int to = -1, at = 0;
    const int b = tree_find_seq(a.cu_q, a.B, t);
    if (b >= 0) {
      const int c0 = __ldg(a.cu_q + b), c1 = __ldg(a.cu_q + b + 1), L = __ldg(a.seq_lens + b), n = c1 - c0;
      if (c0 < 0 || c1 > a.T || t >= c1) {
        if (tell) record_error(a.err, INK_DEVERR_BAD_ROWS);
      } else if (n > L) {
        if (tell) record_error(a.err, INK_DEVERR_QLEN_EXCEEDS_KV);
      } else {
        const int key = L - n + t - c0, pi = key >> a.log2_page;
        to = pi < a.max_pages ? __ldg(a.block_table + (size_t)b * a.max_pages + pi) : -1;
        at = key & ((1 << a.log2_page) - 1);
        if (to < 0 || to >= a.num_pages) {
          to = -1;
          if (tell) record_error(a.err, INK_DEVERR_PAGE_OUT_OF_RANGE);
        }
        int node = t - c0, back = KS - 2;   // the state's newest row is the parent of a root
#pragma unroll
        for (int i = 0; i < KS; ++i) {
          if (node >= 0) {
            from[x][i] = c0 + node;
            if (i + 1 < KS) node = tree_parent(a.parents + c0, node, a.err);
          } else {
            from[x][i] = ~(b * (KS - 1) + back--);
          }
        }
      }
    } else if (tell && t == 0 && __ldg(a.cu_q + a.B) > a.T) {
      record_error(a.err, INK_DEVERR_BAD_ROWS);
    }
    page[x] = to;
    slot[x] = at;
  }
  __syncthreads();
  if (!mine) return;
  const int row = a.nvec * 8;
  for (int x = 0; x < nt; ++x) {
    if (page[x] < 0) continue;
    uint4 raw[KS];
#pragma unroll
    for (int i = 0; i < KS; ++i) {
      const int r = from[x][i];
      raw[i] = __ldg(reinterpret_cast<const uint4*>(r >= 0 ? a.x[z] + (size_t)r * row + col : a.st_in[z] + (size_t)~r * row + col));
    }
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
    if (lane < KS - 1) from[lane] = m + lane < KS - 1 ? ~(b * (KS - 1) + m + lane) : c0 + __ldg(path + m + lane - (KS - 1));
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
  // as many tokens a block (they share the taps' loads) as leave four blocks an SM
  const long long per = (long long)a.T * cols / (4ll * num_sms);
  const int tokens = (int)std::max(1ll, std::min<long long>(CT_TOKENS, per));
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
