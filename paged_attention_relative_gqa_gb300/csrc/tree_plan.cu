// tree_plan.cu -- the two ends of a step that checks trees of drafted tokens: positions and visible tokens from the
// parents, and the move of the accepted path's K and V rows.
//
// Plan: token i sees the drafted tokens on its way to the root.  With S_0(i) = {i} and u_0(i) its parent,
//     S_{s+1}(i) = S_s(i) + S_s(u_s(i)),   u_{s+1}(i) = u_s(u_s(i))
// doubles the way covered in every step, so a tree of depth d takes log2(d) steps; the depth is |S| - 1.  A block takes a
// sequence, its sets (a bit per token) and pointers twice in shared memory, read from one copy and
// written to the other.  Latency bounds it: a launch and a chain of three loads (one tree 2.9 us of GPU time alone, 128 trees of
// up to 64 tokens 3.7; 32 of up to 512 take 43 us, chains of them 61: with 16 words a token lanes meet on two banks).
//
// Commit: row path[j] of a sequence goes to row j, in place.  The path increases, so path[j] >= j, and what is
// written while rows j0 .. j1 - 1 move lies below all that is read for rows from j1 on: a warp takes the rows in order,
// a batch of loads, then the batch's stores.  Bytes bound it, read and written once in rows of 2 D bytes, but a path moves few of
// them and the chain of loads in front of them (lengths, path, table) is longer (one layer 3.0 us of GPU time alone; 11 layers, 64
// paths in trees of up to 32 tokens, 8 heads of 128, 6.0 us).
#include <algorithm>

#include "tree_common.cuh"

namespace ink {
namespace {

__global__ void __launch_bounds__(256) tree_plan_kernel(const TreePlanArgs a) {
  extern __shared__ uint32_t sets[];   // [2][n][words], then pointers [2][n]
  const int b = blockIdx.x;
  const int c0 = __ldg(a.cu_q + b), c1 = __ldg(a.cu_q + b + 1), L = __ldg(a.seq_lens + b);
  if (c0 < 0 || c1 > a.T || c1 < c0) {
    if (threadIdx.x == 0) record_error(a.err, INK_DEVERR_BAD_ROWS);
    return;
  }
  const int n = c1 - c0, cap = 32 * a.words;
  if (n > cap || n > L) {
    if (threadIdx.x == 0) record_error(a.err, n > L ? INK_DEVERR_QLEN_EXCEEDS_KV : INK_DEVERR_QLEN_EXCEEDS_MAX);
    return;
  }
  uint32_t* set[2] = {sets, sets + cap * a.words};
  int* up[2] = {reinterpret_cast<int*>(sets + 2 * cap * a.words), reinterpret_cast<int*>(sets + 2 * cap * a.words) + cap};
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    up[0][i] = tree_parent(a.parents + c0, i, a.err);
    for (int w = 0; w < a.words; ++w) set[0][i * a.words + w] = w == i >> 5 ? 1u << (i & 31) : 0u;
  }
  __syncthreads();
  int now = 0;
  for (int step = 1; step < n; step *= 2, now ^= 1) {
    int more = 0;
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
      const int u = up[now][i], v = u >= 0 ? up[now][u] : -1;
      for (int w = 0; w < a.words; ++w)
        set[now ^ 1][i * a.words + w] = set[now][i * a.words + w] | (u >= 0 ? set[now][u * a.words + w] : 0u);
      up[now ^ 1][i] = v;
      more |= v >= 0;
    }
    if (!__syncthreads_or(more)) {
      now ^= 1;
      break;
    }
  }
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    int size = 0;
    for (int w = 0; w < a.words; ++w) {
      const uint32_t x = set[now][i * a.words + w];
      size += __popc(x);
      a.ancestors[(size_t)(c0 + i) * a.words + w] = x;
    }
    a.positions[c0 + i] = L - n + size - 1;
  }
}

constexpr int TC_THREADS = 256;
constexpr int TC_BATCH = 8;      // 16-byte loads of a lane on their way

template <int D>
__global__ void __launch_bounds__(TC_THREADS) tree_commit_kernel(const __grid_constant__ TreeCommitArgs a) {
  constexpr int LPR = D / 8, RPP = 32 / LPR;   // lanes of a row, rows of a pass
  __shared__ long long moves[TC_THREADS / 32][32][2];   // source and destination rows (of head 0) of 32 places
  const int lane = threadIdx.x & 31;
  const long long gw = (long long)blockIdx.x * (TC_THREADS / 32) + (threadIdx.x >> 5);
  const int per = a.npools * a.slices;
  const int b = (int)(gw / per);
  if (b >= a.B) return;
  const int rest = (int)(gw - (long long)b * per);
  const int pool = rest / a.slices, h0 = (rest - pool * a.slices) * a.heads, nh = min(a.heads, a.Hkv - h0);
  const bool first = rest == 0;   // of the sequence: reports, and writes its length
  const int n = __ldg(a.cu_q + b + 1) - __ldg(a.cu_q + b), L = __ldg(a.seq_lens + b), len = __ldg(a.path_lens + b);
  if (n < 0 || n > L) {
    if (first && lane == 0) {
      record_error(a.err, n < 0 ? INK_DEVERR_BAD_ROWS : INK_DEVERR_QLEN_EXCEEDS_KV);
      if (a.seq_lens_out) a.seq_lens_out[b] = L;
    }
    return;
  }
  const int32_t* path = a.path + (size_t)b * a.max_path;
  const int m = tree_path(path, len, a.max_path, n, lane, a.err);
  const int H = L - n;
  if (first && lane == 0 && a.seq_lens_out) a.seq_lens_out[b] = H + m;
  // row of head 0 of a key (-1: not in the pool)
  auto row = [&](int key) -> long long {
    const int pi = key >> a.log2_page;
    const int page = pi < a.max_pages ? __ldg(a.block_table + (size_t)b * a.max_pages + min(pi, a.max_pages - 1)) : -1;
    if (page < 0 || page >= a.num_pages) return -1;
    return ((long long)page * a.Hkv << a.log2_page) + (key & ((1 << a.log2_page) - 1));
  };
  long long (*mv)[2] = moves[threadIdx.x >> 5];
  uint16_t* base = a.pool[pool];
  const int lr = lane % LPR, rip = lane / LPR;
  for (int j0 = 0; j0 < m; j0 += 32) {
    const int j = j0 + lane, i = j < m ? __ldg(path + min(j, m - 1)) : j;
    long long src = -1, dst = -1;
    if (i != j) {
      src = row(H + i);
      dst = row(H + j);
      if (src < 0 || dst < 0) record_error(a.err, INK_DEVERR_PAGE_OUT_OF_RANGE);
    }
    const bool go = src >= 0 && dst >= 0;
    const uint32_t who = __ballot_sync(0xffffffffu, go);
    __syncwarp();   // the list of the 32 places before is read
    if (go) {
      const int at = __popc(who & ((1u << lane) - 1u));
      mv[at][0] = src;
      mv[at][1] = dst;
    }
    __syncwarp();
    const int rows = __popc(who) * nh;   // in order of the path, its heads side by side
    for (int r0 = 0; r0 < rows; r0 += TC_BATCH * RPP) {
      uint4 x[TC_BATCH];
      long long to[TC_BATCH];
#pragma unroll
      for (int y = 0; y < TC_BATCH; ++y) {
        const int r = r0 + y * RPP + rip;
        to[y] = -1;
        if (r < rows) {
          const int at = r / nh, h = h0 + r - at * nh;
          x[y] = *reinterpret_cast<const uint4*>(base + ((mv[at][0] + ((long long)h << a.log2_page)) * D + lr * 8));
          to[y] = (mv[at][1] + ((long long)h << a.log2_page)) * D + lr * 8;
        }
      }
      __syncwarp();   // (a lane's stores come after every lane's loads of the batch)
#pragma unroll
      for (int y = 0; y < TC_BATCH; ++y)
        if (to[y] >= 0) *reinterpret_cast<uint4*>(base + to[y]) = x[y];
      __syncwarp();
    }
  }
}

}  // namespace

cudaError_t launch_tree_plan(const TreePlanArgs& a, cudaStream_t stream) {
  const int cap = 32 * a.words;
  const int smem = 2 * cap * (a.words + 1) * 4;
  if (smem > 48 * 1024) {
    static std::atomic<unsigned long long> opted{0};
    const cudaError_t e = smem_opt_in_once(tree_plan_kernel, 2 * 32 * TREE_MAX_WORDS * (TREE_MAX_WORDS + 1) * 4, opted);
    if (e != cudaSuccess) return e;
  }
  tree_plan_kernel<<<a.B, std::min(256, cap), smem, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_tree_commit(TreeCommitArgs& a, int head_dim, int num_sms, cudaStream_t stream) {
  // a warp takes as many heads as leave enough warps to hide their chains of loads
  const long long pairs = (long long)a.B * a.npools, want = (long long)num_sms * 16;
  a.slices = (int)std::max(1ll, std::min<long long>(a.Hkv, (want + pairs - 1) / pairs));
  a.heads = (a.Hkv + a.slices - 1) / a.slices;
  a.slices = (a.Hkv + a.heads - 1) / a.heads;
  const long long blocks = (pairs * a.slices + TC_THREADS / 32 - 1) / (TC_THREADS / 32);
  if (blocks >= (1ll << 31)) return cudaErrorInvalidConfiguration;
  if (head_dim == 128) tree_commit_kernel<128><<<(int)blocks, TC_THREADS, 0, stream>>>(a);
  else tree_commit_kernel<64><<<(int)blocks, TC_THREADS, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace ink
