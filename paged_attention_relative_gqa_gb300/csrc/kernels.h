// kernels.h -- argument blocks and launchers shared between the host API (api.cu)
// and the kernel translation units.
#pragma once

#include <atomic>
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/inkling_attn.h"

namespace ink {

// Keys per K/V tile: one TMA box is 64 rows of 128 bytes (64 bf16 of head_dim).
constexpr int TILE_KEYS = 64;

// Largest number of key splits a decode launch may use (bounds the merge scratch).
constexpr int MAX_DECODE_SPLITS = 64;

struct DecodeArgs {
  const void* q;              // bf16 [B, Hq, D]
  const int32_t* block_table; // [B, max_pages]
  const int32_t* seq_lens;    // [B]
  const float* rel;           // fp32 [B, Hq, E]
  void* out;                  // bf16 [B, Hq, D]
  float* part_o;              // fp32 [B, Hq, num_splits, D]
  float* part_ml;             // fp32 [B, Hq, num_splits, 2] (running max in log2 units, sum)
  int32_t* tickets;           // [B, Hkv * head_chunks]
  uint32_t* err;              // sticky error word
  int B, Hq, Hkv, G, head_chunks;
  int log2_page, max_pages, num_pages, E, W;
  float scale_log2;           // sm_scale * log2(e)
  int tiles_per_split, num_splits;
  unsigned long long wait_ns; // limit of one pipeline wait (the drain waits keep 2 s)
};

struct PrefillArgs {
  const void* q;              // bf16 [total_q, Hq, D]
  const int32_t* cu_q;        // [B+1]
  const int32_t* block_table; // [B, max_pages]
  const int32_t* seq_lens;    // [B]
  const void* rel;            // [total_q, Hq, E], fp32, or bf16 when bias_bf16
  void* out;                  // bf16 [total_q, Hq, D]
  uint32_t* err;
  int B, Hq, Hkv, G;
  int log2_page, max_pages, num_pages, E, W;
  float scale_log2;
  float sm_scale;             // multiplies q.k (the bias is added unscaled)
  int max_q_len, num_q_tiles;
  int bias_bulk;              // rows of rel are 16-byte aligned (E a multiple of 16 bytes, aligned base)
  int bias_bf16;              // rel holds bf16 values (always with bias_bulk)
  int bias_lowrank;           // bias from r and proj_t (rel unused)
  const void* lr_r;           // bf16 [total_q, Hq, d_rel]
  const void* lr_proj_t;      // bf16 [E, d_rel]
  int d_rel;                  // a multiple of 8 in [8, 64]
  unsigned long long wait_ns; // limit of one pipeline wait (the drain waits keep 2 s)
  int io32;                   // q and out 32-byte aligned: rows move in 256-bit loads and stores
};

// TMA descriptors of one decode call: K/V pools viewed as [num_pages*Hkv*P rows, D]
// with 64-row boxes (whole tiles) and 16-row boxes (tiles cut by the window start or
// the sequence end), and q viewed as [B*Hq rows, D] with 16-row boxes.
struct DecodeMaps {
  CUtensorMap k_seg, v_seg;   // 2-D, boxes of min(P, 16) rows x 64 columns (pages of 8 keys)
  CUtensorMap k_tile, v_tile; // 4-D group view, one box = 4 groups (a whole 64-key tile; P >= 64)
  CUtensorMap k_grp, v_grp;   // 4-D group view, one box = 1 group of 16 keys (P >= 16)
  CUtensorMap q3;             // 16 query rows, all column blocks in one box
};

// The current device's id and SM count, looked up once per device (host-only afterwards,
// so launches stay legal inside CUDA-graph stream capture).
int current_device_sms(int* dev_out);

// Opt a kernel into `bytes` of dynamic shared memory on the current device, once per
// device and kernel (the setting persists; repeating it inside stream capture is avoided).
template <typename Kernel>
inline cudaError_t smem_opt_in_once(Kernel kernel, int bytes, std::atomic<unsigned long long>& done) {
  int dev = 0;
  if (current_device_sms(&dev) <= 0 || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  const unsigned long long bit = 1ull << dev;
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_acq_rel);
  return e;
}

cudaError_t launch_decode(const DecodeMaps& maps, const DecodeArgs& a, int head_dim,
                          cudaStream_t stream);
// TMA descriptors of one prefill call: K/V pools as for decode (min(P, 64)-row boxes) and
// q viewed as [total_q rows, Hq*D] with 128-row boxes (rows past total_q read as zero).
// bias: rel_logits viewed as [E, Hq, total_q] fp32 (innermost first) with boxes of
// 84 buckets x 1 head x 16 tokens (only built when rows of rel are 16-byte aligned).
struct PrefillMaps {
  CUtensorMap k, v, bias;
  CUtensorMap lr_r;     // low-rank bias: r viewed as {64, Hq, total_q}, box {64, 1, 128} (MMA operand A)
  CUtensorMap lr_p;     // low-rank bias: proj_t viewed as {64, E}, box {64, LOWRANK_CHUNK} (MMA operand B)
  CUtensorMap k3, v3;   // whole 64-key tiles, all column blocks in one box (P >= 64 only)
  CUtensorMap q3;       // 128 query rows of one head, all column blocks in one box
};

constexpr int BIAS_BOX_COLS = 84;   // buckets per bias box row
constexpr int BIAS_BOX_ROWS = 16;   // tokens per bias box
constexpr int BIAS_BOX_COLS_BF16 = 88;   // buckets per bias box row, bf16 bias
constexpr int PREFILL_ROWS = 128;        // new tokens per prefill work item
constexpr int LOWRANK_CHUNK = 64;        // projection rows per TMA box (one key tile's new buckets)
constexpr int LOWRANK_MAX_D = 64;        // largest d_rel of the low-rank bias (the MMA's K: four K-steps of 16)

cudaError_t launch_prefill_tc(const PrefillMaps& maps, const PrefillArgs& a, int head_dim,
                              cudaStream_t stream);

// The head-pair prefill (prefill_pair.cu): bias given as rel_logits with 16-byte rows, read by
// 3-D TMA boxes of PAIR_BIAS_ROWS tokens x PAIR_BIAS_COLS_* buckets of one head.
constexpr int PAIR_BIAS_ROWS = 32;
constexpr int PAIR_BIAS_COLS_F32 = 100;
constexpr int PAIR_BIAS_COLS_BF16 = 104;
cudaError_t launch_prefill_pair(const PrefillMaps& maps, const PrefillArgs& a, int head_dim,
                                cudaStream_t stream);

// One call of the K/V short convolution and paged write (kv_conv.cu).  Rows of the
// step's K/V and of the carried state are Hkv*D bf16 (nvec 16-byte vectors).
struct KvConvArgs {
  const uint16_t* x[2];        // k_new, v_new: bf16 [T, Hkv, D]
  const float* w[2];           // taps: fp32 [Hkv, D, ks]
  const uint16_t* st_in[2];    // bf16 [B, ks-1, Hkv, D], oldest row first
  uint16_t* st_out[2];         // same layout, never overlapping st_in
  uint16_t* cache[2];          // bf16 [num_pages, Hkv, P, D]
  const int32_t* cu_q;         // [B+1]
  const int32_t* seq_lens;     // [B]
  const int32_t* block_table;  // [B, max_pages]
  uint32_t* err;
  int B, T, Hkv, D, log2_page, max_pages, num_pages;
  int nvec;                    // Hkv * D / 8
  int tok;                     // tokens per thread (1 or 8)
  int nchunks;                 // ceil(T / tok)
  long long conv_items;        // 2 * nchunks * nvec threads of convolution
  long long state_items;       // 2 * B * nvec threads of state copy (each all ks-1 rows)
  int tile_tokens;             // staged kernel: new rows per tile (<= 32)
  int stages;                  // staged kernel: ring depth (0: use the per-thread kernel)
  unsigned long long wait_ns;  // limit of one pipeline wait (the drain waits keep 2 s)
};

// Largest dynamic shared memory of the staged K/V kernel.
constexpr size_t KV_STAGED_SMEM_MAX = 216 * 1024;

int kv_conv_tokens_per_thread(long long total_q, int nvec, int num_sms);
size_t kv_staged_smem_bytes(int tile_tokens, int kernel_size, int nvec, int stages);
// Fill tile_tokens, stages, tok, nchunks and conv_items of `a` (T, nvec, B set).
void kv_conv_plan(KvConvArgs& a, int kernel_size, int num_sms);
cudaError_t launch_kv_conv(const KvConvArgs& a, int kernel_size, cudaStream_t stream);

// One call of the per-head norm, rotation and paged K/V write (qk_norm_rope.cu).
struct NormRopeArgs {
  const uint16_t* x[3];        // q, k, v rows: bf16, token stride x_stride[s] elements
  long long x_stride[3];
  uint16_t* q_out;             // bf16 [T, Hq, D]
  uint16_t* cache[2];          // K, V: bf16 [num_pages, Hkv, P, D]
  const float* w[2];           // norm weights of q, k: fp32 [D] or null
  const float* inv_freq;       // fp32 [rot_dim / 2]
  const int32_t* cu_q;         // [B+1]
  const int32_t* seq_lens;     // [B]
  const int32_t* block_table;  // [B, max_pages]
  uint32_t* err;
  int B, T, H[3], log2_page, max_pages, num_pages;
  int rot_dim;
  const int32_t* positions;    // [T] positions of the rotation, or null: the slot's
  float eps, rot_scale;
  int passes;                  // passes of a warp over one token's rows: ceil(Hq / rows) + 2 ceil(Hkv / rows)
  int chunk, nchunks;          // passes per warp, warps per token
};

cudaError_t launch_qk_norm_rope(NormRopeArgs& a, int head_dim, bool interleaved, int num_sms, cudaStream_t stream);

constexpr int NEAR_TERMS = 4, MID_TERMS = 6;   // of the capped score's polynomials

// One call of the masked attention (no bias tensor; a visible key range per token).
struct MaskedArgs {
  const void* q;               // bf16 [total_q, Hq, D]
  const int32_t* cu_q;         // [B+1] (null: decode, row b is sequence b)
  const int32_t* block_table;  // [B, max_pages]
  const int32_t* seq_lens;     // [B]
  const int32_t* key_begin;    // [total_q] or null
  const int32_t* key_end;      // [total_q] or null
  const float* slopes;         // [Hq] or null
  const void* k;               // bf16 [num_pages, Hkv, P, D]
  const void* v;
  void* out;                   // bf16 [total_q, Hq, D]
  float* lse;                  // fp32 [total_q, Hq] or null
  uint32_t* err;
  int B, T, Hq, Hkv, G, log2_page, max_pages, num_pages, W;
  float sm_scale, softcap;
  float scale_log2;            // sm_scale * log2(e)
  float cap_k1;                // 2 * sm_scale * log2(e) / softcap
  float cap_log2;              // softcap * log2(e)
  float cap_inv;               // sm_scale / softcap
  // prefill: for |x| = |<q, K[k]>| <= cap_near the capped score is x (near[0] + near[1] x^2 + ...), up to
  // cap_mid x (mid[0] + mid[1] x^2 + ...)
  float cap_near, near[NEAR_TERMS], cap_mid, mid[MID_TERMS];
  unsigned long long wait_ns;  // limit of one pipeline wait (the drain waits keep 2 s)
  // prefill: a row tile holds tok_per_tile tokens x heads_per_tile query heads of one KV head
  int head_chunks, heads_per_tile, tok_per_tile;
  int io32;                    // out 32-byte aligned: its rows are stored 32 bytes at a time
  uint32_t* stale;             // nonzero after a timeout of a prefill, until the workspace is initialised again
  uint32_t* counters;          // [0] items handed out, [1] CTAs done; zero between calls
  // decode: partials of cut groups, two places per CTA of `rows` heads (8 or 16), and a ticket per
  // CTA, for the group cut at its end; zero between calls
  float* part_o;               // [2 * CTAs, rows, D]; prefill: [pieces, 2, D / 4, 128 rows] float4
  float* part_ml;              // [2 * CTAs, rows, 2] (running max in log2 units, sum); prefill: [pieces, 2, 128 rows] float4
  int32_t* tickets;            // prefill: [pieces, 2]
};

constexpr int MASKED_PIECES = 480;        // most pieces of cut items in one masked prefill

constexpr int MASKED_DECODE_CTAS = 320;   // most CTAs of a masked decode (bounds its partials)

constexpr int MASKED_ROWS = 128;   // rows of a tile

// TMA descriptors: the pools with boxes of min(P, 128) rows, q as {D, Hq, T} with boxes of
// 64 channels x heads_per_tile x tok_per_tile.
struct MaskedMaps {
  CUtensorMap k, v, q;
};

cudaError_t launch_prefill_masked(const MaskedMaps& m, const MaskedArgs& a, int head_dim, cudaStream_t stream);
cudaError_t launch_decode_masked(const DecodeMaps& m, const MaskedArgs& a, int head_dim, cudaStream_t stream);

// Rows of a tree of drafted tokens: plan and commit (tree_plan.cu).
constexpr int TREE_MAX_WORDS = 16;   // words of a token's ancestor bits: 512 drafted tokens a sequence

struct TreePlanArgs {
  const int32_t* cu_q;         // [B+1]
  const int32_t* seq_lens;     // [B]
  const int32_t* parents;      // [T]
  int32_t* positions;          // [T]
  uint32_t* ancestors;         // [T, words]
  uint32_t* err;
  int B, T, words;
};

cudaError_t launch_tree_plan(const TreePlanArgs& a, cudaStream_t stream);

struct TreeCommitArgs {
  uint16_t* pool[2 * INK_TREE_MAX_POOLS];   // K and V of each layer: bf16 [num_pages, Hkv, P, D]
  const int32_t* cu_q;         // [B+1]
  const int32_t* seq_lens;     // [B]
  const int32_t* block_table;  // [B, max_pages]
  const int32_t* path;         // [B, max_path]
  const int32_t* path_lens;    // [B]
  int32_t* seq_lens_out;       // [B] or null
  uint32_t* err;
  int npools;                  // K and V counted
  int B, Hkv, log2_page, max_pages, num_pages, max_path;
  int heads, slices;           // heads of a warp, warps per sequence and pool
};

cudaError_t launch_tree_commit(TreeCommitArgs& a, int head_dim, int num_sms, cudaStream_t stream);

// The K/V short convolution along the paths of a tree, and its state behind an accepted path (kv_conv_tree.cu).
struct TreeConvArgs {
  const uint16_t* x[2];        // k_new, v_new: bf16 [T, Hkv, D]
  const float* w[2];           // taps: fp32 [Hkv, D, ks]
  const uint16_t* st_in[2];    // bf16 [B, ks-1, Hkv, D], oldest row first
  uint16_t* st_out[2];
  uint16_t* cache[2];          // bf16 [num_pages, Hkv, P, D]
  const int32_t* cu_q;         // [B+1]
  const int32_t* seq_lens;     // [B]
  const int32_t* block_table;  // [B, max_pages]
  const int32_t* parents;      // [T]
  const int32_t* path;         // [B, max_path]
  const int32_t* path_lens;    // [B]
  uint32_t* err;
  int B, T, D, log2_page, max_pages, num_pages, max_path;
  int nvec;                    // Hkv * D / 8
};

cudaError_t launch_kv_conv_tree(const TreeConvArgs& a, int kernel_size, int num_sms, cudaStream_t stream);
cudaError_t launch_kv_conv_state_tree(const TreeConvArgs& a, int kernel_size, cudaStream_t stream);

// One call of the attention over a tree of drafted tokens (tree.cu).
struct TreeArgs {
  const void* q;               // bf16 [T, Hq, D]
  const int32_t* cu_q;         // [B+1]
  const int32_t* block_table;  // [B, max_pages]
  const int32_t* seq_lens;     // [B]
  const int32_t* positions;    // [T]
  const uint32_t* ancestors;   // [T, words]
  const float* slopes;         // [Hq] or null
  const void* rel;             // [T, Hq, E] fp32 or bf16, or null
  const void* k;               // bf16 [num_pages, Hkv, P, D]
  const void* v;
  void* out;                   // bf16 [T, Hq, D]
  float* lse;                  // fp32 [T, Hq] or null
  uint32_t* err;
  int B, T, Hq, Hkv, G, log2_page, max_pages, num_pages, W, E, words;
  int rel_bf16;
  int rel_rows;                // rows of rel begin on 16-byte boundaries: boxes of a token's heads can be copied
  int bias_stride;             // bytes from one token's box to the next in shared memory
  float sm_scale, softcap;
  float scale_log2;            // sm_scale * log2(e)
  float cap_k1, cap_log2, cap_inv, cap_near, near[NEAR_TERMS], cap_mid, mid[MID_TERMS];   // as in MaskedArgs
  unsigned long long wait_ns;  // limit of one pipeline wait (the drain waits keep 2 s)
  int head_chunks, heads_per_tile, tok_per_tile;   // as in MaskedArgs
  // partials of cut items, two places of two row tiles per CTA, and the item that each CTA begins and does not end
  float* part_o;               // [2 CTAs, 2, D / 4, 128 rows] float4
  float* part_ml;              // [2 CTAs, 2, 128 rows] (maximum in log2 units, sum)
  struct TreeCut* cuts;        // [CTAs]
};

struct TreeCut {
  int parts;                   // pieces (at most one: no such item)
  int t0, ntok, h0, gh;        // first row, tokens; first query head, heads
};

constexpr int TREE_ROWS = 128;       // rows of a row tile
constexpr int TREE_MAX_CTAS = 160;   // most CTAs (bounds the partials)
constexpr int TREE_BIAS_BYTES = 40960;   // a chain's bias in shared memory

// Columns of a bias box: a tile's values from a 16-byte boundary on.
__host__ __device__ constexpr int tree_bias_cols(bool bf16) { return TILE_KEYS + (bf16 ? 8 : 4); }

cudaError_t launch_tree(const MaskedMaps& m, const CUtensorMap& bias, const TreeArgs& a, int head_dim, cudaStream_t stream);

}  // namespace ink
