// api.cu -- the C ABI of libinkling_attn.so (declared in include/inkling_attn.h):
// argument validation, workspace layout, TMA tensor-map encoding and kernel launch.
// Host code here touches only scalars and pointer values; it never synchronises,
// allocates or copies (except inkling_attn_read_device_error, which is documented to).
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <cstring>
#include <functional>
#include <mutex>

#include "../../include/inkling_attn.h"
#include "kernels.h"

namespace {

using ink::DecodeArgs;
using ink::PrefillArgs;

constexpr size_t kHeaderBytes = 256;  // error word lives at offset 0

// Limit of one pipeline wait inside the kernels launched from now on (default 2 s).
std::atomic<unsigned long long> g_wait_limit_ns{2000000000ull};

size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

bool is_pow2(int x) { return x > 0 && (x & (x - 1)) == 0; }

int ilog2(int x) {
  int r = 0;
  while ((1 << r) < x) ++r;
  return r;
}

ink_status_t validate(const ink_attn_params_t* p) {
  if (!p) return INK_ERR_NULL_PTR;
  if (p->num_seqs < 0 || p->num_q_heads < 1 || p->num_kv_heads < 1 || p->rel_extent < 1 ||
      p->max_pages_per_seq < 1 || p->num_pages < 1)
    return INK_ERR_BAD_SHAPE;
  if (p->num_q_heads % p->num_kv_heads != 0) return INK_ERR_BAD_SHAPE;
  if (p->head_dim != 64 && p->head_dim != 128) return INK_ERR_BAD_SHAPE;
  if (!is_pow2(p->page_size) || p->page_size < 8 || p->page_size > (1 << 20))
    return INK_ERR_BAD_PAGE_SIZE;
  // TMA row coordinates and in-kernel row arithmetic are 32-bit
  const long long rows = (long long)p->num_pages * p->num_kv_heads * p->page_size;
  if (rows >= (1ll << 31)) return INK_ERR_TOO_LARGE;
  if ((long long)p->max_pages_per_seq * p->page_size >= (1ll << 31)) return INK_ERR_TOO_LARGE;
  if (!(p->sm_scale == p->sm_scale)) return INK_ERR_BAD_SHAPE;  // NaN scale
  return INK_OK;
}

struct DecodePlan {
  int head_chunks, tiles_per_split, num_splits;
};

// Split-K plan for decode.  Visible keys of one sequence span at most `max_tiles`
// 64-key tiles (window-limited on sliding-window layers).  The persistent decode kernel
// runs one CTA per SM over work units (split, sequence, KV head, head chunk); the tiles
// of a sequence are cut into splits so that there are about kTargetUnits units in the
// worst case, enough for an even spread over the SMs, while each split keeps at least
// two tiles.
constexpr long long kTargetUnits = 608;  // 4 units per SM on a 152-SM GB300

DecodePlan plan_decode(const ink_attn_params_t* p) {
  DecodePlan d;
  const int G = p->num_q_heads / p->num_kv_heads;
  d.head_chunks = (G + 15) / 16;
  const long long max_keys = (long long)p->max_pages_per_seq * p->page_size;
  long long max_tiles = (max_keys + ink::TILE_KEYS - 1) / ink::TILE_KEYS;
  if (p->window > 0) {
    const long long wt = (p->window + ink::TILE_KEYS - 1) / ink::TILE_KEYS + 1;
    if (wt < max_tiles) max_tiles = wt;
  }
  if (max_tiles < 1) max_tiles = 1;
  const long long units = (long long)(p->num_seqs > 0 ? p->num_seqs : 1) * p->num_kv_heads * d.head_chunks;
  long long tps = (units * max_tiles + kTargetUnits - 1) / kTargetUnits;
  if (tps < 2) tps = 2;
  if (tps > 64) tps = 64;
  long long splits = (max_tiles + tps - 1) / tps;
  if (splits > ink::MAX_DECODE_SPLITS) splits = ink::MAX_DECODE_SPLITS;
  tps = (max_tiles + splits - 1) / splits;  // rebalance
  splits = (max_tiles + tps - 1) / tps;
  d.tiles_per_split = (int)tps;
  d.num_splits = (int)splits;
  return d;
}

struct DecodeLayout {
  size_t tickets_off, part_o_off, part_ml_off, total;
};

DecodeLayout decode_layout(const ink_attn_params_t* p, const DecodePlan& d) {
  DecodeLayout l;
  const size_t B = (size_t)(p->num_seqs > 0 ? p->num_seqs : 1);
  const size_t nt = B * p->num_kv_heads * d.head_chunks;
  l.tickets_off = kHeaderBytes;
  l.part_o_off = align_up(l.tickets_off + nt * sizeof(int32_t), 256);
  const size_t rows = B * p->num_q_heads * (size_t)d.num_splits;
  l.part_ml_off = align_up(l.part_o_off + rows * p->head_dim * sizeof(float), 256);
  l.total = align_up(l.part_ml_off + rows * 2 * sizeof(float), 256);
  return l;
}

// ---- TMA tensor maps over a K or V pool viewed as [num_pages*Hkv*P rows, D] bf16

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  });
  return fn;
}

// A bf16 matrix [rows, cols] (row pitch cols*2 bytes) with boxes of 64 columns x box_rows
// rows, 128-byte swizzle.
bool make_rows_map(CUtensorMap* map, const void* base, uint64_t rows, int cols, int box_rows) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)cols * 2};
  cuuint32_t box[2] = {64, (cuuint32_t)box_rows};
  cuuint32_t estr[2] = {1, 1};
  CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides,
                  box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// The same bf16 rows as a 3-D tensor {64 columns, rows, column blocks} (row pitch
// `pitch` elements, blocks 128 bytes apart): one box of box_rows rows x `blocks` column
// blocks lands in shared memory as the 128-byte-swizzled sub-tiles [block][row][64] that
// separate 2-D boxes would give, block stride box_rows * 128 bytes.
bool make_rows_map3(CUtensorMap* map, const void* base, uint64_t rows, uint64_t pitch, int blocks, int box_rows) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {64, (cuuint64_t)rows, (cuuint64_t)(pitch / 64)};
  cuuint64_t strides[2] = {(cuuint64_t)pitch * 2, 128};
  cuuint32_t box[3] = {64, (cuuint32_t)box_rows, (cuuint32_t)blocks};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// A K or V pool of `rows` rows (a multiple of 16) as a 4-D tensor {64 columns, 16 rows,
// column blocks, 16-row groups}: one box of `groups` groups lands in shared memory as
// [group][block][16 rows][64], 2 KB blocks with the 128-byte swizzle.
bool make_group_map(CUtensorMap* map, const void* base, uint64_t rows, int D, int groups) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[4] = {64, 16, (cuuint64_t)(D / 64), (cuuint64_t)(rows / 16)};
  cuuint64_t strides[3] = {(cuuint64_t)D * 2, 128, (cuuint64_t)D * 2 * 16};
  cuuint32_t box[4] = {64, 16, (cuuint32_t)(D / 64), (cuuint32_t)groups};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

uint64_t pool_rows(const ink_attn_params_t* p) {
  return (uint64_t)p->num_pages * p->num_kv_heads * p->page_size;
}

// K or V pool as [num_pages*Hkv*P rows, D], boxes of min(P, box_cap) rows.
bool make_pool_map(CUtensorMap* map, const void* base, const ink_attn_params_t* p, int box_cap) {
  const int box_rows = p->page_size < box_cap ? p->page_size : box_cap;
  return make_rows_map(map, base, pool_rows(p), p->head_dim, box_rows);
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// rel_logits [total_q, Hq, E] (fp32 or bf16) as a 3-D tensor {E, Hq, total_q}; boxes of
// box_cols buckets x box_heads heads x box_rows tokens, out-of-range elements read as 0.
bool make_bias_map(CUtensorMap* map, const void* rel, bool bf16, const ink_attn_params_t* p, int total_q,
                   int box_cols, int box_rows, int box_heads = 1) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t es = bf16 ? 2 : 4;
  cuuint64_t dims[3] = {(cuuint64_t)p->rel_extent, (cuuint64_t)p->num_q_heads, (cuuint64_t)total_q};
  cuuint64_t strides[2] = {(cuuint64_t)p->rel_extent * es, (cuuint64_t)p->rel_extent * es * p->num_q_heads};
  cuuint32_t box[3] = {(cuuint32_t)box_cols, (cuuint32_t)box_heads, (cuuint32_t)box_rows};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3,
                  const_cast<void*>(rel), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// Low-rank bias operands: r [total_q, Hq, d_rel] as {d_rel, Hq, total_q} with boxes of 64
// columns x 128 tokens of one head, and proj_t [E, d_rel] as {d_rel, E} with boxes of 64
// columns x LOWRANK_CHUNK buckets; 128-byte rows with the 128-byte swizzle, as the bias MMA's
// K-major operands (K = 64) want them.  Columns past d_rel, tokens past total_q and buckets
// outside [0, E) read as zeros, so a smaller d_rel adds zero products.
bool make_lowrank_maps(ink::PrefillMaps* m, const void* r, const void* proj_t, const ink_attn_params_t* p,
                       int total_q, int d_rel) {
  auto fn = encode_fn();
  if (!fn) return false;
  const CUtensorMapSwizzle sw = CU_TENSOR_MAP_SWIZZLE_128B;
  cuuint64_t dims_r[3] = {(cuuint64_t)d_rel, (cuuint64_t)p->num_q_heads, (cuuint64_t)total_q};
  cuuint64_t str_r[2] = {(cuuint64_t)d_rel * 2, (cuuint64_t)d_rel * 2 * p->num_q_heads};
  cuuint32_t box_r[3] = {(cuuint32_t)ink::LOWRANK_MAX_D, 1, (cuuint32_t)ink::PREFILL_ROWS};
  cuuint32_t e3[3] = {1, 1, 1};
  CUresult e = fn(&m->lr_r, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(r), dims_r, str_r, box_r, e3,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (e != CUDA_SUCCESS) return false;
  cuuint64_t dims_p[2] = {(cuuint64_t)d_rel, (cuuint64_t)p->rel_extent};
  cuuint64_t str_p[1] = {(cuuint64_t)d_rel * 2};
  cuuint32_t box_p[2] = {(cuuint32_t)ink::LOWRANK_MAX_D, (cuuint32_t)ink::LOWRANK_CHUNK};
  cuuint32_t e2[2] = {1, 1};
  e = fn(&m->lr_p, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(proj_t), dims_p, str_p, box_p, e2,
         CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return e == CUDA_SUCCESS;
}

bool make_decode_maps(ink::DecodeMaps* m, const void* q, const void* k_cache, const void* v_cache,
                      const ink_attn_params_t* params) {
  const int D = params->head_dim;
  std::memset(m, 0, sizeof *m);
  if (!make_rows_map3(&m->q3, q, (uint64_t)params->num_seqs * params->num_q_heads, D, D / 64, 16)) return false;
  if (params->page_size < 16)   // the only page size whose tiles come in 8-key boxes
    return make_pool_map(&m->k_seg, k_cache, params, 16) && make_pool_map(&m->v_seg, v_cache, params, 16);
  if (!make_group_map(&m->k_grp, k_cache, pool_rows(params), D, 1) ||
      !make_group_map(&m->v_grp, v_cache, pool_rows(params), D, 1))
    return false;
  return params->page_size < ink::TILE_KEYS ||
         (make_group_map(&m->k_tile, k_cache, pool_rows(params), D, ink::TILE_KEYS / 16) &&
          make_group_map(&m->v_tile, v_cache, pool_rows(params), D, ink::TILE_KEYS / 16));
}

}  // namespace

extern "C" {

int32_t inkling_attn_version(void) { return 100; }

void inkling_attn_set_wait_limit_ns(uint64_t limit_ns) {
  g_wait_limit_ns.store(limit_ns > 2000000000ull ? 2000000000ull : limit_ns, std::memory_order_relaxed);
}

const char* inkling_attn_status_string(ink_status_t s) {
  switch (s) {
    case INK_OK: return "ok";
    case INK_ERR_NULL_PTR: return "null pointer argument";
    case INK_ERR_BAD_SHAPE: return "bad shape (heads not divisible, head_dim not 64/128, or non-positive size)";
    case INK_ERR_BAD_PAGE_SIZE: return "page_size must be a power of two >= 8";
    case INK_ERR_WORKSPACE: return "workspace too small";
    case INK_ERR_ALIGNMENT: return "misaligned pointer (16 bytes for q/k/v/out, 4 for index and bias arrays)";
    case INK_ERR_CUDA: return "CUDA runtime error";
    case INK_ERR_TOO_LARGE: return "sizes overflow 32-bit coordinates";
  }
  return "unknown status";
}

size_t inkling_attn_workspace_bytes(const ink_attn_params_t* params, int is_decode) {
  if (validate(params) != INK_OK) return 0;
  if (!is_decode) return kHeaderBytes;
  return decode_layout(params, plan_decode(params)).total;
}

ink_status_t inkling_attn_workspace_init(void* workspace, size_t workspace_bytes, void* stream) {
  if (!workspace) return INK_ERR_NULL_PTR;
  if (workspace_bytes < kHeaderBytes) return INK_ERR_WORKSPACE;
  if (cudaMemsetAsync(workspace, 0, workspace_bytes, (cudaStream_t)stream) != cudaSuccess)
    return INK_ERR_CUDA;
  return INK_OK;
}

ink_status_t inkling_attn_read_device_error(void* workspace, size_t workspace_bytes, void* stream,
                                            uint32_t* err_out, int clear) {
  if (!workspace || !err_out) return INK_ERR_NULL_PTR;
  if (workspace_bytes < kHeaderBytes) return INK_ERR_WORKSPACE;
  cudaStream_t st = (cudaStream_t)stream;
  uint32_t v = 0;
  if (cudaMemcpyAsync(&v, workspace, sizeof v, cudaMemcpyDeviceToHost, st) != cudaSuccess)
    return INK_ERR_CUDA;
  if (cudaStreamSynchronize(st) != cudaSuccess) return INK_ERR_CUDA;
  *err_out = v;
  if (clear) {
    if (cudaMemsetAsync(workspace, 0, sizeof v, st) != cudaSuccess) return INK_ERR_CUDA;
    if (cudaStreamSynchronize(st) != cudaSuccess) return INK_ERR_CUDA;
  }
  return INK_OK;
}

ink_status_t inkling_attn_decode(const ink_attn_params_t* params, const void* q, const void* k_cache,
                                 const void* v_cache, const int32_t* block_table,
                                 const int32_t* seq_lens, const float* rel_logits, void* out,
                                 void* workspace, size_t workspace_bytes, void* stream) {
  ink_status_t st = validate(params);
  if (st != INK_OK) return st;
  if (!q || !k_cache || !v_cache || !block_table || !seq_lens || !rel_logits || !out || !workspace)
    return INK_ERR_NULL_PTR;
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) ||
      !aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(rel_logits, 4) ||
      !aligned(workspace, 256))
    return INK_ERR_ALIGNMENT;
  const DecodePlan plan = plan_decode(params);
  const DecodeLayout lay = decode_layout(params, plan);
  if (workspace_bytes < lay.total) return INK_ERR_WORKSPACE;
  if (params->num_seqs == 0) return INK_OK;
  ink::DecodeMaps maps;
  if (!make_decode_maps(&maps, q, k_cache, v_cache, params)) return INK_ERR_CUDA;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  DecodeArgs a;
  a.q = q;
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.rel = rel_logits;
  a.out = out;
  a.part_o = reinterpret_cast<float*>(ws + lay.part_o_off);
  a.part_ml = reinterpret_cast<float*>(ws + lay.part_ml_off);
  a.tickets = reinterpret_cast<int32_t*>(ws + lay.tickets_off);
  a.err = reinterpret_cast<uint32_t*>(ws);
  a.B = params->num_seqs;
  a.Hq = params->num_q_heads;
  a.Hkv = params->num_kv_heads;
  a.G = params->num_q_heads / params->num_kv_heads;
  a.head_chunks = plan.head_chunks;
  a.log2_page = ilog2(params->page_size);
  a.max_pages = params->max_pages_per_seq;
  a.num_pages = params->num_pages;
  a.E = params->rel_extent;
  a.W = params->window;
  a.scale_log2 = params->sm_scale * 1.4426950408889634f;
  a.tiles_per_split = plan.tiles_per_split;
  a.num_splits = plan.num_splits;
  a.wait_ns = g_wait_limit_ns.load(std::memory_order_relaxed);
  if (ink::launch_decode(maps, a, params->head_dim, (cudaStream_t)stream) != cudaSuccess)
    return INK_ERR_CUDA;
  return INK_OK;
}

}  // extern "C"

namespace {

// The bias of a prefill call: rel_logits in fp32 or bf16, or its low-rank factors.
enum class BiasIn { F32, BF16, LOWRANK };

// Shared by the fp32-bias, bf16-bias and low-rank-bias prefill entry points.
ink_status_t prefill_impl(const ink_attn_params_t* params, const void* q, const int32_t* cu_q_lens,
                          int32_t max_q_len, int32_t total_q, const void* k_cache, const void* v_cache,
                          const int32_t* block_table, const int32_t* seq_lens, const void* rel_logits,
                          BiasIn bias_in, const void* lr_r, const void* lr_proj_t, int32_t d_rel, void* out,
                          void* workspace, size_t workspace_bytes, void* stream) {
  ink_status_t st = validate(params);
  if (st != INK_OK) return st;
  const bool bias_bf16 = bias_in == BiasIn::BF16, lowrank = bias_in == BiasIn::LOWRANK;
  if (!q || !cu_q_lens || !k_cache || !v_cache || !block_table || !seq_lens || !out || !workspace)
    return INK_ERR_NULL_PTR;
  if (lowrank ? (!lr_r || !lr_proj_t) : !rel_logits) return INK_ERR_NULL_PTR;
  if (max_q_len < 0 || total_q < 0) return INK_ERR_BAD_SHAPE;
  if (lowrank && (d_rel < 8 || d_rel > ink::LOWRANK_MAX_D || d_rel % 8 != 0)) return INK_ERR_BAD_SHAPE;
  if ((long long)total_q * params->num_q_heads >= (1ll << 31)) return INK_ERR_TOO_LARGE;
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) ||
      !aligned(cu_q_lens, 4) || !aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(workspace, 256))
    return INK_ERR_ALIGNMENT;
  if (lowrank ? (!aligned(lr_r, 16) || !aligned(lr_proj_t, 16)) : !aligned(rel_logits, bias_bf16 ? 16 : 4))
    return INK_ERR_ALIGNMENT;
  if (bias_bf16 && params->rel_extent % 8 != 0) return INK_ERR_BAD_SHAPE;   // 16-byte bias rows
  if (workspace_bytes < kHeaderBytes) return INK_ERR_WORKSPACE;
  if (params->num_seqs == 0 || max_q_len == 0 || total_q == 0) return INK_OK;
  const int num_q_tiles = (max_q_len + ink::PREFILL_ROWS - 1) / ink::PREFILL_ROWS;
  if (num_q_tiles > 65535 || params->num_seqs > 65535) return INK_ERR_TOO_LARGE;
  ink::PrefillMaps maps;
  const int cblocks = params->head_dim / 64;
  std::memset(&maps.k3, 0, sizeof maps.k3);
  std::memset(&maps.v3, 0, sizeof maps.v3);
  if (params->page_size >= ink::TILE_KEYS &&
      (!make_rows_map3(&maps.k3, k_cache, pool_rows(params), params->head_dim, cblocks, ink::TILE_KEYS) ||
       !make_rows_map3(&maps.v3, v_cache, pool_rows(params), params->head_dim, cblocks, ink::TILE_KEYS)))
    return INK_ERR_CUDA;
  if (!make_pool_map(&maps.k, k_cache, params, ink::TILE_KEYS) ||
      !make_pool_map(&maps.v, v_cache, params, ink::TILE_KEYS) ||
      !make_rows_map3(&maps.q3, q, (uint64_t)total_q, (uint64_t)params->num_q_heads * params->head_dim, cblocks, 128))
    return INK_ERR_CUDA;
  PrefillArgs a;
  a.q = q;
  a.cu_q = cu_q_lens;
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.rel = rel_logits;
  a.out = out;
  a.err = reinterpret_cast<uint32_t*>(workspace);
  a.B = params->num_seqs;
  a.Hq = params->num_q_heads;
  a.Hkv = params->num_kv_heads;
  a.G = params->num_q_heads / params->num_kv_heads;
  a.log2_page = ilog2(params->page_size);
  a.max_pages = params->max_pages_per_seq;
  a.num_pages = params->num_pages;
  a.E = params->rel_extent;
  a.W = params->window;
  a.scale_log2 = params->sm_scale * 1.4426950408889634f;
  a.sm_scale = params->sm_scale;
  a.max_q_len = max_q_len;
  a.num_q_tiles = num_q_tiles;
  a.bias_bf16 = bias_bf16 ? 1 : 0;
  a.bias_lowrank = lowrank ? 1 : 0;
  a.lr_r = lr_r;
  a.lr_proj_t = lr_proj_t;
  a.d_rel = d_rel;
  a.bias_bulk = !lowrank && (bias_bf16 || ((params->rel_extent % 4 == 0) && aligned(rel_logits, 16)));
  a.wait_ns = g_wait_limit_ns.load(std::memory_order_relaxed);
  a.io32 = aligned(q, 32) && aligned(out, 32) ? 1 : 0;
  std::memset(&maps.bias, 0, sizeof maps.bias);
  std::memset(&maps.lr_r, 0, sizeof maps.lr_r);
  std::memset(&maps.lr_p, 0, sizeof maps.lr_p);
  if (lowrank && !make_lowrank_maps(&maps, lr_r, lr_proj_t, params, total_q, d_rel)) return INK_ERR_CUDA;
  if (a.bias_bulk) {
    // the head-pair kernel: 32-token bias boxes
    if (!make_bias_map(&maps.bias, rel_logits, bias_bf16, params, total_q,
                       bias_bf16 ? ink::PAIR_BIAS_COLS_BF16 : ink::PAIR_BIAS_COLS_F32, ink::PAIR_BIAS_ROWS))
      return INK_ERR_CUDA;
    if (ink::launch_prefill_pair(maps, a, params->head_dim, (cudaStream_t)stream) != cudaSuccess)
      return INK_ERR_CUDA;
    return INK_OK;
  }
  if (ink::launch_prefill_tc(maps, a, params->head_dim, (cudaStream_t)stream) != cudaSuccess)
    return INK_ERR_CUDA;
  return INK_OK;
}

}  // namespace

extern "C" {

ink_status_t inkling_attn_prefill(const ink_attn_params_t* params, const void* q,
                                  const int32_t* cu_q_lens, int32_t max_q_len, int32_t total_q,
                                  const void* k_cache,
                                  const void* v_cache, const int32_t* block_table,
                                  const int32_t* seq_lens, const float* rel_logits, void* out,
                                  void* workspace, size_t workspace_bytes, void* stream) {
  return prefill_impl(params, q, cu_q_lens, max_q_len, total_q, k_cache, v_cache, block_table, seq_lens,
                      rel_logits, BiasIn::F32, nullptr, nullptr, 0, out, workspace, workspace_bytes, stream);
}

ink_status_t inkling_attn_prefill_bf16bias(const ink_attn_params_t* params, const void* q,
                                           const int32_t* cu_q_lens, int32_t max_q_len, int32_t total_q,
                                           const void* k_cache, const void* v_cache,
                                           const int32_t* block_table, const int32_t* seq_lens,
                                           const void* rel_logits_bf16, void* out, void* workspace,
                                           size_t workspace_bytes, void* stream) {
  return prefill_impl(params, q, cu_q_lens, max_q_len, total_q, k_cache, v_cache, block_table, seq_lens,
                      rel_logits_bf16, BiasIn::BF16, nullptr, nullptr, 0, out, workspace, workspace_bytes, stream);
}

ink_status_t inkling_attn_prefill_lowrank_bias(const ink_attn_params_t* params, const void* q,
                                               const int32_t* cu_q_lens, int32_t max_q_len, int32_t total_q,
                                               const void* k_cache, const void* v_cache,
                                               const int32_t* block_table, const int32_t* seq_lens,
                                               const void* r, const void* rel_proj_t, int32_t d_rel, void* out,
                                               void* workspace, size_t workspace_bytes, void* stream) {
  return prefill_impl(params, q, cu_q_lens, max_q_len, total_q, k_cache, v_cache, block_table, seq_lens,
                      nullptr, BiasIn::LOWRANK, r, rel_proj_t, d_rel, out, workspace, workspace_bytes, stream);
}

ink_status_t inkling_attn_kv_conv_write(const ink_attn_params_t* params, const void* k_new,
                                        const void* v_new, const int32_t* cu_q_lens, int32_t total_q,
                                        const int32_t* seq_lens, const int32_t* block_table,
                                        const float* w_k, const float* w_v, int32_t kernel_size,
                                        const void* state_k_in, const void* state_v_in,
                                        void* state_k_out, void* state_v_out, void* k_cache,
                                        void* v_cache, void* workspace, size_t workspace_bytes,
                                        void* stream) {
  ink_status_t st = validate(params);
  if (st != INK_OK) return st;
  if (kernel_size < 1 || kernel_size > 8 || total_q < 0) return INK_ERR_BAD_SHAPE;
  const bool has_state = kernel_size > 1;
  if (!k_new || !v_new || !cu_q_lens || !seq_lens || !block_table || !w_k || !w_v || !k_cache ||
      !v_cache || !workspace)
    return INK_ERR_NULL_PTR;
  if (has_state && (!state_k_in || !state_v_in || !state_k_out || !state_v_out)) return INK_ERR_NULL_PTR;
  if (!aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
      !aligned(w_k, 16) || !aligned(w_v, 16) || !aligned(cu_q_lens, 4) || !aligned(seq_lens, 4) ||
      !aligned(block_table, 4) || !aligned(workspace, 256))
    return INK_ERR_ALIGNMENT;
  if (has_state && (!aligned(state_k_in, 16) || !aligned(state_v_in, 16) || !aligned(state_k_out, 16) ||
                    !aligned(state_v_out, 16)))
    return INK_ERR_ALIGNMENT;
  if (workspace_bytes < kHeaderBytes) return INK_ERR_WORKSPACE;
  const int nvec = params->num_kv_heads * params->head_dim / 8;
  if ((long long)total_q * nvec * 8 >= (1ll << 40)) return INK_ERR_TOO_LARGE;
  ink::KvConvArgs a;
  a.x[0] = static_cast<const uint16_t*>(k_new);
  a.x[1] = static_cast<const uint16_t*>(v_new);
  a.w[0] = w_k;
  a.w[1] = w_v;
  a.st_in[0] = static_cast<const uint16_t*>(state_k_in);
  a.st_in[1] = static_cast<const uint16_t*>(state_v_in);
  a.st_out[0] = static_cast<uint16_t*>(state_k_out);
  a.st_out[1] = static_cast<uint16_t*>(state_v_out);
  a.cache[0] = static_cast<uint16_t*>(k_cache);
  a.cache[1] = static_cast<uint16_t*>(v_cache);
  a.cu_q = cu_q_lens;
  a.seq_lens = seq_lens;
  a.block_table = block_table;
  a.err = reinterpret_cast<uint32_t*>(workspace);
  a.B = params->num_seqs;
  a.T = total_q;
  a.Hkv = params->num_kv_heads;
  a.D = params->head_dim;
  a.log2_page = ilog2(params->page_size);
  a.max_pages = params->max_pages_per_seq;
  a.num_pages = params->num_pages;
  a.nvec = nvec;
  a.wait_ns = g_wait_limit_ns.load(std::memory_order_relaxed);
  if (total_q == 0 && (params->num_seqs == 0 || !has_state)) return INK_OK;   // nothing to write
  int dev = 0;
  const int sms = ink::current_device_sms(&dev);
  if (sms <= 0) return INK_ERR_CUDA;
  ink::kv_conv_plan(a, kernel_size, sms);
  a.state_items = has_state ? 2ll * a.B * nvec : 0;   // each copies all ks - 1 rows of a vector
  if ((a.conv_items + a.state_items + 255) / 256 >= (1ll << 31)) return INK_ERR_TOO_LARGE;
  if (ink::launch_kv_conv(a, kernel_size, (cudaStream_t)stream) != cudaSuccess) return INK_ERR_CUDA;
  return INK_OK;
}

}  // extern "C"

namespace {

struct MaskedLayout {
  size_t prefill_tickets, decode_tickets, part_o_off, part_ml_off, total;
};

// Header, the tickets of both kinds (what has to be zero between calls, at the same place for every
// shape), then partials, which carry nothing from one call to the next: one workspace serves prefills
// and decodes of any sizes in turn.
MaskedLayout masked_layout(const ink_attn_params_t* p, bool decode) {
  MaskedLayout l;
  const size_t G = (size_t)(p->num_q_heads / p->num_kv_heads);
  const size_t rows = decode ? 2 * (size_t)ink::MASKED_DECODE_CTAS * (G <= 8 ? 8 : 16)
                             : 2 * (size_t)ink::MASKED_PIECES * ink::MASKED_ROWS;
  l.prefill_tickets = kHeaderBytes;
  l.decode_tickets = l.prefill_tickets + 2 * ink::MASKED_PIECES * sizeof(int32_t);
  l.part_o_off = align_up(l.decode_tickets + ink::MASKED_DECODE_CTAS * sizeof(int32_t), 256);
  l.part_ml_off = l.part_o_off + rows * p->head_dim * sizeof(float);
  l.total = align_up(l.part_ml_off + rows * (decode ? 2 : 4) * sizeof(float), 256);
  return l;
}

// q [total_q, Hq, D] as {D, Hq, total_q}, boxes of 64 channels x heads x tokens with the 128-byte
// swizzle: the rows of an MMA operand, tokens outermost.  Rows outside the tensor read as zeros.
bool make_token_map(CUtensorMap* map, const void* q, const ink_attn_params_t* p, int total_q, int heads, int tokens) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t row = (cuuint64_t)p->head_dim * 2;
  cuuint64_t dims[3] = {(cuuint64_t)p->head_dim, (cuuint64_t)p->num_q_heads, (cuuint64_t)total_q};
  cuuint64_t strides[2] = {row, row * p->num_q_heads};
  cuuint32_t box[3] = {64, (cuuint32_t)heads, (cuuint32_t)tokens};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(q), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Span {
  const void* at;   // (null: absent)
  size_t bytes;
};

// Does one of the first `written` of n spans share bytes with another one?
bool overlap(const Span* s, int written, int n) {
  for (int w = 0; w < written; ++w)
    for (int x = w + 1; x < n; ++x) {
      const uintptr_t a = reinterpret_cast<uintptr_t>(s[w].at), b = reinterpret_cast<uintptr_t>(s[x].at);
      if (a && b && a < b + s[x].bytes && b < a + s[w].bytes) return true;
    }
  return false;
}

struct TreeLayout {
  size_t cuts, part_ml_off, part_o_off, total;
};

// Header, then what a call writes before it reads it: nothing is kept between calls.
TreeLayout tree_layout(const ink_attn_params_t* p) {
  const size_t rows = 4 * (size_t)ink::TREE_MAX_CTAS * ink::TREE_ROWS;   // two places of two row tiles a CTA
  TreeLayout l;
  l.cuts = kHeaderBytes;
  l.part_ml_off = align_up(l.cuts + ink::TREE_MAX_CTAS * sizeof(ink::TreeCut), 256);
  l.part_o_off = l.part_ml_off + rows * 2 * sizeof(float);
  l.total = l.part_o_off + rows * p->head_dim * sizeof(float);
  return l;
}

size_t pool_bytes(const ink_attn_params_t* p) { return pool_rows(p) * p->head_dim * 2; }

size_t table_bytes(const ink_attn_params_t* p) { return (size_t)p->num_seqs * p->max_pages_per_seq * 4; }

// Scale and cap of the scores, for the masked and the tree kernels.
template <class Args>
void fill_scores(Args& a, float sm_scale, float softcap) {
  a.sm_scale = sm_scale;
  a.softcap = softcap;
  a.scale_log2 = sm_scale * 1.4426950408889634f;
  a.cap_log2 = softcap * 1.4426950408889634f;
  a.cap_k1 = softcap > 0.f ? (float)(2.0 * 1.4426950408889634 * sm_scale / softcap) : 0.f;
  a.cap_inv = softcap > 0.f ? sm_scale / softcap : 0.f;
  // tanh(y) / y as polynomials in y^2 of the least relative error, in terms of the raw product: for
  // |y| <= 0.45 (2^-22) and for |y| <= 1 (2^-20.7, of the score itself: a 64th of a bf16 weight's
  // rounding for scores to 20).  Left out where the coefficients would leave fp32's range: a negative
  // reach, or the near one in the other's place.
  static const double kNear[ink::NEAR_TERMS] = {0.9999997567401877, -0.3332946719023333, 0.13236369052154567,
                                                -0.04602819379882759};
  static const double kMid[ink::MID_TERMS] = {0.99999941361031, -0.3332904245054663, 0.1328143441522219,
                                              -0.05160568907876395, 0.01674313284460914, -0.003067067657993291};
  const double inv = softcap > 0.f ? (double)sm_scale / softcap : 0.0, ainv = inv < 0 ? -inv : inv;
  a.cap_near = ainv >= 1e-5 && ainv <= 1e3 ? (float)(0.45 / ainv) : -1.f;
  a.cap_mid = ainv > 0 ? (float)(1.0 / ainv) : -1.f;
  double c = 1.4426950408889634 * sm_scale;
  for (int i = 0; i < ink::MID_TERMS; ++i, c *= inv * inv) {
    if (i < ink::NEAR_TERMS) a.near[i] = a.cap_near > 0.f ? (float)(c * kNear[i]) : 0.f;
    const double m = c * kMid[i], am = m < 0 ? -m : m;
    a.mid[i] = (float)m;
    if (!(am >= 1e-36 && am <= 1e36)) a.cap_mid = -1.f;
  }
  if (a.cap_mid < 0.f) {
    a.cap_mid = a.cap_near;
    for (int i = 0; i < ink::MID_TERMS; ++i) a.mid[i] = i < ink::NEAR_TERMS ? a.near[i] : 0.f;
  }
}

// A row tile: the heads of a KV head (in equal chunks when there are more than 128) times as many tokens as fit.
template <class Args>
void fill_rows(Args& a) {
  a.head_chunks = (a.G + ink::MASKED_ROWS - 1) / ink::MASKED_ROWS;
  a.heads_per_tile = (a.G + a.head_chunks - 1) / a.head_chunks;
  a.tok_per_tile = ink::MASKED_ROWS / a.heads_per_tile;
}

ink_status_t masked_impl(const ink_attn_params_t* params, const ink_attn_mask_t* mask, const void* q,
                         const int32_t* cu_q_lens, int32_t total_q, const void* k_cache, const void* v_cache,
                         const int32_t* block_table, const int32_t* seq_lens, void* out, float* lse,
                         void* workspace, size_t workspace_bytes, void* stream, bool decode) {
  ink_status_t st = validate(params);
  if (st != INK_OK) return st;
  static const ink_attn_mask_t kNone = {0.f, nullptr, nullptr, nullptr};
  const ink_attn_mask_t& mk = mask ? *mask : kNone;
  if (!q || !k_cache || !v_cache || !block_table || !seq_lens || !out || !workspace || (!decode && !cu_q_lens))
    return INK_ERR_NULL_PTR;
  if (total_q < 0 || !(mk.softcap == 0.f || (mk.softcap >= 1e-6f && mk.softcap <= 1e6f))) return INK_ERR_BAD_SHAPE;
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) ||
      !aligned(cu_q_lens, 4) || !aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(lse, 4) ||
      !aligned(mk.key_begin, 4) || !aligned(mk.key_end, 4) || !aligned(mk.slopes, 4) || !aligned(workspace, 256))
    return INK_ERR_ALIGNMENT;
  if ((long long)total_q * params->num_q_heads >= (1ll << 31)) return INK_ERR_TOO_LARGE;
  const MaskedLayout lay = masked_layout(params, decode);
  if (workspace_bytes < lay.total) return INK_ERR_WORKSPACE;
  if (params->num_seqs == 0 || total_q == 0) return INK_OK;
  const size_t rows = (size_t)total_q * params->num_q_heads, seqs = (size_t)params->num_seqs * 4;
  const Span spans[] = {{out, rows * params->head_dim * 2}, {lse, rows * 4}, {workspace, lay.total},
                        {q, rows * params->head_dim * 2}, {k_cache, pool_bytes(params)}, {v_cache, pool_bytes(params)},
                        {block_table, table_bytes(params)}, {seq_lens, seqs}, {decode ? nullptr : cu_q_lens, seqs + 4},
                        {mk.key_begin, (size_t)total_q * 4}, {mk.key_end, (size_t)total_q * 4},
                        {mk.slopes, (size_t)params->num_q_heads * 4}};
  if (overlap(spans, 3, sizeof spans / sizeof *spans)) return INK_ERR_BAD_SHAPE;
  ink::MaskedArgs a;
  a.q = q;
  a.cu_q = decode ? nullptr : cu_q_lens;
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.key_begin = mk.key_begin;
  a.key_end = mk.key_end;
  a.slopes = mk.slopes;
  a.k = k_cache;
  a.v = v_cache;
  a.out = out;
  a.lse = lse;
  a.err = reinterpret_cast<uint32_t*>(workspace);
  a.B = params->num_seqs;
  a.T = total_q;
  a.Hq = params->num_q_heads;
  a.Hkv = params->num_kv_heads;
  a.G = params->num_q_heads / params->num_kv_heads;
  a.log2_page = ilog2(params->page_size);
  a.max_pages = params->max_pages_per_seq;
  a.num_pages = params->num_pages;
  a.W = params->window;
  a.wait_ns = g_wait_limit_ns.load(std::memory_order_relaxed);
  fill_scores(a, params->sm_scale, mk.softcap);
  fill_rows(a);
  a.stale = reinterpret_cast<uint32_t*>(workspace) + 15;   // these three inside the header
  a.counters = reinterpret_cast<uint32_t*>(workspace) + 16;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.tickets = reinterpret_cast<int32_t*>(ws + (decode ? lay.decode_tickets : lay.prefill_tickets));
  a.part_o = reinterpret_cast<float*>(ws + lay.part_o_off);
  a.part_ml = reinterpret_cast<float*>(ws + lay.part_ml_off);
  a.io32 = aligned(out, 32) ? 1 : 0;
  if (decode) {
    a.head_chunks = (a.G + 15) / 16;
    ink::DecodeMaps maps;
    if (!make_decode_maps(&maps, q, k_cache, v_cache, params)) return INK_ERR_CUDA;
    if (ink::launch_decode_masked(maps, a, params->head_dim, (cudaStream_t)stream) != cudaSuccess) return INK_ERR_CUDA;
    return INK_OK;
  }
  ink::MaskedMaps maps;
  if (!make_pool_map(&maps.k, k_cache, params, 128) || !make_pool_map(&maps.v, v_cache, params, 128) ||
      !make_token_map(&maps.q, q, params, total_q, a.heads_per_tile, a.tok_per_tile))
    return INK_ERR_CUDA;
  if (ink::launch_prefill_masked(maps, a, params->head_dim, (cudaStream_t)stream) != cudaSuccess)
    return INK_ERR_CUDA;
  return INK_OK;
}

}  // namespace

extern "C" {

size_t inkling_attn_masked_workspace_bytes(const ink_attn_params_t* params, int is_decode) {
  if (validate(params) != INK_OK) return 0;
  return masked_layout(params, is_decode != 0).total;
}

ink_status_t inkling_attn_prefill_masked(const ink_attn_params_t* params, const ink_attn_mask_t* mask,
                                         const void* q, const int32_t* cu_q_lens, int32_t total_q,
                                         const void* k_cache, const void* v_cache,
                                         const int32_t* block_table, const int32_t* seq_lens,
                                         void* out, float* lse, void* workspace,
                                         size_t workspace_bytes, void* stream) {
  return masked_impl(params, mask, q, cu_q_lens, total_q, k_cache, v_cache, block_table, seq_lens, out, lse,
                     workspace, workspace_bytes, stream, false);
}

ink_status_t inkling_attn_decode_masked(const ink_attn_params_t* params, const ink_attn_mask_t* mask,
                                        const void* q, const void* k_cache, const void* v_cache,
                                        const int32_t* block_table, const int32_t* seq_lens, void* out,
                                        float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  return masked_impl(params, mask, q, nullptr, params ? params->num_seqs : 0, k_cache, v_cache, block_table,
                     seq_lens, out, lse, workspace, workspace_bytes, stream, true);
}

}  // extern "C"

namespace {

ink_status_t norm_rope_impl(const ink_attn_params_t* params, const ink_norm_rope_t* rope, const int32_t* positions,
                            const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                            const void* v, int64_t v_stride, const int32_t* cu_q_lens,
                            int32_t total_q, const int32_t* seq_lens, const int32_t* block_table,
                            void* q_out, void* k_cache, void* v_cache, void* workspace,
                            size_t workspace_bytes, void* stream) {
  ink_status_t st = validate(params);
  if (st != INK_OK) return st;
  if (!rope || !q || !k || !v || !cu_q_lens || !seq_lens || !block_table || !q_out || !k_cache || !v_cache ||
      !workspace)
    return INK_ERR_NULL_PTR;
  const int D = params->head_dim, Hq = params->num_q_heads, Hkv = params->num_kv_heads;
  if (rope->rot_dim < 0 || rope->rot_dim > D || rope->rot_dim % 16 != 0) return INK_ERR_BAD_SHAPE;
  if (rope->rot_dim > 0 && !rope->inv_freq) return INK_ERR_NULL_PTR;
  if (rope->layout != INK_ROPE_HALF && rope->layout != INK_ROPE_INTERLEAVED) return INK_ERR_BAD_SHAPE;
  if (!(rope->eps >= 0.f) || !(rope->rot_scale == rope->rot_scale) || total_q < 0) return INK_ERR_BAD_SHAPE;
  if (q_stride < (int64_t)Hq * D || k_stride < (int64_t)Hkv * D || v_stride < (int64_t)Hkv * D)
    return INK_ERR_BAD_SHAPE;
  if (q_stride % 8 != 0 || k_stride % 8 != 0 || v_stride % 8 != 0 || !aligned(q, 16) || !aligned(k, 16) ||
      !aligned(v, 16) || !aligned(q_out, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
      !aligned(rope->w_q, 16) || !aligned(rope->w_k, 16) || !aligned(rope->inv_freq, 4) || !aligned(cu_q_lens, 4) ||
      !aligned(seq_lens, 4) || !aligned(block_table, 4) || !aligned(positions, 4) || !aligned(workspace, 256))
    return INK_ERR_ALIGNMENT;
  if (q_out == q && q_stride != (int64_t)Hq * D) return INK_ERR_BAD_SHAPE;
  if (workspace_bytes < kHeaderBytes) return INK_ERR_WORKSPACE;
  if (params->num_seqs == 0 || total_q == 0) return INK_OK;
  // what is written overlaps neither what is read (but for q in place) nor what else is written
  auto span = [&](int64_t stride, int n) { return 2 * ((size_t)(total_q - 1) * (size_t)stride + (size_t)n * D); };
  const Span spans[] = {{q_out, span((int64_t)Hq * D, Hq)}, {k_cache, pool_bytes(params)}, {v_cache, pool_bytes(params)},
                        {workspace, kHeaderBytes}, {q_out == q ? nullptr : q, span(q_stride, Hq)},
                        {k, span(k_stride, Hkv)}, {v, span(v_stride, Hkv)}, {block_table, table_bytes(params)},
                        {seq_lens, (size_t)params->num_seqs * 4}, {cu_q_lens, (size_t)params->num_seqs * 4 + 4},
                        {rope->w_q, (size_t)D * 4}, {rope->w_k, (size_t)D * 4},
                        {rope->rot_dim > 0 ? rope->inv_freq : nullptr, (size_t)rope->rot_dim * 2},
                        {positions, (size_t)total_q * 4}};
  if (overlap(spans, 4, sizeof spans / sizeof *spans)) return INK_ERR_BAD_SHAPE;
  ink::NormRopeArgs a;
  a.x[0] = static_cast<const uint16_t*>(q);
  a.x[1] = static_cast<const uint16_t*>(k);
  a.x[2] = static_cast<const uint16_t*>(v);
  a.x_stride[0] = q_stride;
  a.x_stride[1] = k_stride;
  a.x_stride[2] = v_stride;
  a.q_out = static_cast<uint16_t*>(q_out);
  a.cache[0] = static_cast<uint16_t*>(k_cache);
  a.cache[1] = static_cast<uint16_t*>(v_cache);
  a.w[0] = rope->w_q;
  a.w[1] = rope->w_k;
  a.inv_freq = rope->inv_freq;
  a.cu_q = cu_q_lens;
  a.seq_lens = seq_lens;
  a.block_table = block_table;
  a.err = reinterpret_cast<uint32_t*>(workspace);
  a.B = params->num_seqs;
  a.T = total_q;
  a.H[0] = Hq;
  a.H[1] = a.H[2] = Hkv;
  a.log2_page = ilog2(params->page_size);
  a.max_pages = params->max_pages_per_seq;
  a.num_pages = params->num_pages;
  a.rot_dim = rope->rot_dim;
  a.positions = positions;
  a.eps = rope->eps;
  a.rot_scale = rope->rot_scale;
  int dev = 0;
  const int sms = ink::current_device_sms(&dev);
  if (sms <= 0) return INK_ERR_CUDA;
  if (ink::launch_qk_norm_rope(a, D, rope->layout == INK_ROPE_INTERLEAVED, sms, (cudaStream_t)stream) != cudaSuccess)
    return INK_ERR_CUDA;
  return INK_OK;
}

}  // namespace

extern "C" {

ink_status_t inkling_attn_qk_norm_rope_write(const ink_attn_params_t* params, const ink_norm_rope_t* rope,
                                             const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                                             const void* v, int64_t v_stride, const int32_t* cu_q_lens,
                                             int32_t total_q, const int32_t* seq_lens, const int32_t* block_table,
                                             void* q_out, void* k_cache, void* v_cache, void* workspace,
                                             size_t workspace_bytes, void* stream) {
  return norm_rope_impl(params, rope, nullptr, q, q_stride, k, k_stride, v, v_stride, cu_q_lens, total_q, seq_lens,
                        block_table, q_out, k_cache, v_cache, workspace, workspace_bytes, stream);
}

ink_status_t inkling_attn_qk_norm_rope_write_at(const ink_attn_params_t* params, const ink_norm_rope_t* rope,
                                                const int32_t* positions, const void* q, int64_t q_stride,
                                                const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                                                const int32_t* cu_q_lens, int32_t total_q, const int32_t* seq_lens,
                                                const int32_t* block_table, void* q_out, void* k_cache, void* v_cache,
                                                void* workspace, size_t workspace_bytes, void* stream) {
  if (params && !positions) return INK_ERR_NULL_PTR;
  return norm_rope_impl(params, rope, positions, q, q_stride, k, k_stride, v, v_stride, cu_q_lens, total_q, seq_lens,
                        block_table, q_out, k_cache, v_cache, workspace, workspace_bytes, stream);
}

ink_status_t inkling_attn_tree_plan(const ink_attn_params_t* params, const int32_t* cu_q_lens, int32_t total_q,
                                    const int32_t* seq_lens, const int32_t* parents, int32_t words,
                                    int32_t* positions, uint32_t* ancestors, void* workspace,
                                    size_t workspace_bytes, void* stream) {
  ink_status_t st = validate(params);
  if (st != INK_OK) return st;
  if (!cu_q_lens || !seq_lens || !parents || !positions || !ancestors || !workspace) return INK_ERR_NULL_PTR;
  if (total_q < 0 || words < 1 || words > ink::TREE_MAX_WORDS) return INK_ERR_BAD_SHAPE;
  if (!aligned(cu_q_lens, 4) || !aligned(seq_lens, 4) || !aligned(parents, 4) || !aligned(positions, 4) ||
      !aligned(ancestors, 4) || !aligned(workspace, 256))
    return INK_ERR_ALIGNMENT;
  if (workspace_bytes < kHeaderBytes) return INK_ERR_WORKSPACE;
  if (params->num_seqs == 0 || total_q == 0) return INK_OK;
  const size_t seqs = (size_t)params->num_seqs * 4, rows = (size_t)total_q * 4;
  const Span spans[] = {{positions, rows}, {ancestors, rows * words}, {workspace, kHeaderBytes}, {cu_q_lens, seqs + 4},
                        {seq_lens, seqs}, {parents, rows}};
  if (overlap(spans, 3, sizeof spans / sizeof *spans)) return INK_ERR_BAD_SHAPE;
  ink::TreePlanArgs a;
  a.cu_q = cu_q_lens;
  a.seq_lens = seq_lens;
  a.parents = parents;
  a.positions = positions;
  a.ancestors = ancestors;
  a.err = reinterpret_cast<uint32_t*>(workspace);
  a.B = params->num_seqs;
  a.T = total_q;
  a.words = words;
  return ink::launch_tree_plan(a, (cudaStream_t)stream) == cudaSuccess ? INK_OK : INK_ERR_CUDA;
}

size_t inkling_attn_tree_workspace_bytes(const ink_attn_params_t* params) {
  if (validate(params) != INK_OK) return 0;
  return tree_layout(params).total;
}

ink_status_t inkling_attn_tree(const ink_attn_params_t* params, const ink_attn_tree_t* tree,
                               const ink_attn_tree_options_t* options, const void* q, const int32_t* cu_q_lens,
                               int32_t total_q, const void* k_cache, const void* v_cache,
                               const int32_t* block_table, const int32_t* seq_lens, void* out, float* lse,
                               void* workspace, size_t workspace_bytes, void* stream) {
  ink_status_t st = validate(params);
  if (st != INK_OK) return st;
  static const ink_attn_tree_options_t kNone = {0.f, nullptr, nullptr, 0};
  const ink_attn_tree_options_t& o = options ? *options : kNone;
  if (!tree || !tree->positions || !tree->ancestors || !q || !cu_q_lens || !k_cache || !v_cache || !block_table ||
      !seq_lens || !out || !workspace)
    return INK_ERR_NULL_PTR;
  if (total_q < 0 || tree->words < 1 || tree->words > ink::TREE_MAX_WORDS) return INK_ERR_BAD_SHAPE;
  if (!(o.softcap == 0.f || (o.softcap >= 1e-6f && o.softcap <= 1e6f))) return INK_ERR_BAD_SHAPE;
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) ||
      !aligned(cu_q_lens, 4) || !aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(lse, 4) ||
      !aligned(tree->positions, 4) || !aligned(tree->ancestors, 4) || !aligned(o.slopes, 4) ||
      !aligned(o.rel_logits, o.rel_is_bf16 ? 2 : 4) || !aligned(workspace, 256))
    return INK_ERR_ALIGNMENT;
  if ((long long)total_q * params->num_q_heads >= (1ll << 31)) return INK_ERR_TOO_LARGE;
  const TreeLayout lay = tree_layout(params);
  if (workspace_bytes < lay.total) return INK_ERR_WORKSPACE;
  if (params->num_seqs == 0 || total_q == 0) return INK_OK;
  const size_t rows = (size_t)total_q * params->num_q_heads, seqs = (size_t)params->num_seqs * 4;
  const Span spans[] = {{out, rows * params->head_dim * 2}, {lse, rows * 4}, {workspace, lay.total},
                        {q, rows * params->head_dim * 2}, {k_cache, pool_bytes(params)}, {v_cache, pool_bytes(params)},
                        {block_table, table_bytes(params)}, {seq_lens, seqs}, {cu_q_lens, seqs + 4},
                        {tree->positions, (size_t)total_q * 4}, {tree->ancestors, (size_t)total_q * tree->words * 4},
                        {o.slopes, (size_t)params->num_q_heads * 4},
                        {o.rel_logits, rows * params->rel_extent * (o.rel_is_bf16 ? 2 : 4)}};
  if (overlap(spans, 3, sizeof spans / sizeof *spans)) return INK_ERR_BAD_SHAPE;
  ink::TreeArgs a;
  a.q = q;
  a.cu_q = cu_q_lens;
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.positions = tree->positions;
  a.ancestors = tree->ancestors;
  a.words = tree->words;
  a.slopes = o.slopes;
  a.rel = o.rel_logits;
  a.rel_bf16 = o.rel_is_bf16 ? 1 : 0;
  a.k = k_cache;
  a.v = v_cache;
  a.out = out;
  a.lse = lse;
  a.err = reinterpret_cast<uint32_t*>(workspace);
  a.B = params->num_seqs;
  a.T = total_q;
  a.Hq = params->num_q_heads;
  a.Hkv = params->num_kv_heads;
  a.G = params->num_q_heads / params->num_kv_heads;
  a.log2_page = ilog2(params->page_size);
  a.max_pages = params->max_pages_per_seq;
  a.num_pages = params->num_pages;
  a.W = params->window;
  a.E = params->rel_extent;
  fill_scores(a, params->sm_scale, o.softcap);
  fill_rows(a);
  a.wait_ns = g_wait_limit_ns.load(std::memory_order_relaxed);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.cuts = reinterpret_cast<ink::TreeCut*>(ws + lay.cuts);
  a.part_ml = reinterpret_cast<float*>(ws + lay.part_ml_off);
  a.part_o = reinterpret_cast<float*>(ws + lay.part_o_off);
  // A token's bias box stands on 128 bytes; with few heads a tile holds as many tokens as there is room for.
  const size_t size = a.rel_bf16 ? 2 : 4, box = (size_t)a.heads_per_tile * ink::tree_bias_cols(a.rel_bf16) * size;
  a.rel_rows = a.rel && aligned(a.rel, 16) && params->rel_extent * size % 16 == 0;
  a.bias_stride = (int)align_up(box, 128);
  if (a.rel_rows && a.tok_per_tile > ink::TREE_BIAS_BYTES / a.bias_stride) a.tok_per_tile = ink::TREE_BIAS_BYTES / a.bias_stride;
  CUtensorMap bias;
  std::memset(&bias, 0, sizeof bias);
  if (a.rel_rows && !make_bias_map(&bias, a.rel, a.rel_bf16 != 0, params, total_q, ink::tree_bias_cols(a.rel_bf16), 1, a.heads_per_tile))
    return INK_ERR_CUDA;
  ink::MaskedMaps maps;
  // whole tiles by one box where they lie in one page, else boxes of a page and 64 channels
  auto pool_map = [&](CUtensorMap* m, const void* base) {
    return params->page_size >= ink::TILE_KEYS ? make_rows_map3(m, base, pool_rows(params), params->head_dim, params->head_dim / 64,
                                                                ink::TILE_KEYS)
                                               : make_pool_map(m, base, params, ink::TILE_KEYS);
  };
  if (!pool_map(&maps.k, k_cache) || !pool_map(&maps.v, v_cache) ||
      !make_token_map(&maps.q, q, params, total_q, a.heads_per_tile, a.tok_per_tile))
    return INK_ERR_CUDA;
  return ink::launch_tree(maps, bias, a, params->head_dim, (cudaStream_t)stream) == cudaSuccess ? INK_OK : INK_ERR_CUDA;
}

ink_status_t inkling_attn_kv_conv_write_tree(const ink_attn_params_t* params, const void* k_new, const void* v_new,
                                             const int32_t* cu_q_lens, int32_t total_q, const int32_t* seq_lens,
                                             const int32_t* block_table, const int32_t* parents, const float* w_k,
                                             const float* w_v, int32_t kernel_size, const void* state_k_in,
                                             const void* state_v_in, void* k_cache, void* v_cache, void* workspace,
                                             size_t workspace_bytes, void* stream) {
  ink_status_t st = validate(params);
  if (st != INK_OK) return st;
  if (kernel_size < 1 || kernel_size > 8 || total_q < 0) return INK_ERR_BAD_SHAPE;
  if (!k_new || !v_new || !cu_q_lens || !seq_lens || !block_table || !parents || !w_k || !w_v || !k_cache || !v_cache ||
      !workspace || (kernel_size > 1 && (!state_k_in || !state_v_in)))
    return INK_ERR_NULL_PTR;
  if (kernel_size == 1) state_k_in = state_v_in = nullptr;
  if (!aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(w_k, 16) ||
      !aligned(w_v, 16) || !aligned(state_k_in, 16) || !aligned(state_v_in, 16) || !aligned(cu_q_lens, 4) ||
      !aligned(seq_lens, 4) || !aligned(block_table, 4) || !aligned(parents, 4) || !aligned(workspace, 256))
    return INK_ERR_ALIGNMENT;
  if (workspace_bytes < kHeaderBytes) return INK_ERR_WORKSPACE;
  if ((long long)params->num_seqs * (kernel_size - 1) >= (1ll << 31)) return INK_ERR_TOO_LARGE;   // rows of the states
  if (params->num_seqs == 0 || total_q == 0) return INK_OK;
  const size_t row = (size_t)params->num_kv_heads * params->head_dim * 2, taps = row * 2 * kernel_size;
  const size_t state = (size_t)params->num_seqs * (kernel_size - 1) * row, seqs = (size_t)params->num_seqs * 4;
  const Span spans[] = {{k_cache, pool_bytes(params)}, {v_cache, pool_bytes(params)}, {workspace, kHeaderBytes},
                        {k_new, total_q * row}, {v_new, total_q * row}, {cu_q_lens, seqs + 4}, {seq_lens, seqs},
                        {block_table, table_bytes(params)}, {parents, (size_t)total_q * 4}, {w_k, taps}, {w_v, taps},
                        {state_k_in, state}, {state_v_in, state}};
  if (overlap(spans, 3, sizeof spans / sizeof *spans)) return INK_ERR_BAD_SHAPE;
  ink::TreeConvArgs a{};
  a.x[0] = static_cast<const uint16_t*>(k_new);
  a.x[1] = static_cast<const uint16_t*>(v_new);
  a.w[0] = w_k;
  a.w[1] = w_v;
  a.st_in[0] = static_cast<const uint16_t*>(state_k_in);
  a.st_in[1] = static_cast<const uint16_t*>(state_v_in);
  a.cache[0] = static_cast<uint16_t*>(k_cache);
  a.cache[1] = static_cast<uint16_t*>(v_cache);
  a.cu_q = cu_q_lens;
  a.seq_lens = seq_lens;
  a.block_table = block_table;
  a.parents = parents;
  a.err = reinterpret_cast<uint32_t*>(workspace);
  a.B = params->num_seqs;
  a.T = total_q;
  a.D = params->head_dim;
  a.log2_page = ilog2(params->page_size);
  a.max_pages = params->max_pages_per_seq;
  a.num_pages = params->num_pages;
  a.nvec = params->num_kv_heads * params->head_dim / 8;
  int dev = 0;
  const int sms = ink::current_device_sms(&dev);
  if (sms <= 0) return INK_ERR_CUDA;
  return ink::launch_kv_conv_tree(a, kernel_size, sms, (cudaStream_t)stream) == cudaSuccess ? INK_OK : INK_ERR_CUDA;
}

ink_status_t inkling_attn_kv_conv_state_tree(const ink_attn_params_t* params, const void* k_new, const void* v_new,
                                             const int32_t* cu_q_lens, int32_t total_q, const int32_t* path,
                                             const int32_t* path_lens, int32_t max_path, int32_t kernel_size,
                                             const void* state_k_in, const void* state_v_in, void* state_k_out,
                                             void* state_v_out, void* workspace, size_t workspace_bytes, void* stream) {
  ink_status_t st = validate(params);
  if (st != INK_OK) return st;
  if (kernel_size < 1 || kernel_size > 8 || total_q < 0 || max_path < 1) return INK_ERR_BAD_SHAPE;
  if (!cu_q_lens || !path || !path_lens || !workspace || (total_q > 0 && (!k_new || !v_new))) return INK_ERR_NULL_PTR;
  if (kernel_size > 1 && (!state_k_in || !state_v_in || !state_k_out || !state_v_out)) return INK_ERR_NULL_PTR;
  if (!aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(cu_q_lens, 4) || !aligned(path, 4) || !aligned(path_lens, 4) ||
      !aligned(workspace, 256))
    return INK_ERR_ALIGNMENT;
  if (kernel_size > 1 && (!aligned(state_k_in, 16) || !aligned(state_v_in, 16) || !aligned(state_k_out, 16) ||
                          !aligned(state_v_out, 16)))
    return INK_ERR_ALIGNMENT;
  if (workspace_bytes < kHeaderBytes) return INK_ERR_WORKSPACE;
  if ((long long)params->num_seqs * (kernel_size - 1) >= (1ll << 31)) return INK_ERR_TOO_LARGE;
  if (params->num_seqs == 0 || kernel_size == 1) return INK_OK;
  const size_t row = (size_t)params->num_kv_heads * params->head_dim * 2, seqs = (size_t)params->num_seqs * 4;
  const size_t state = (size_t)params->num_seqs * (kernel_size - 1) * row;
  const Span spans[] = {{state_k_out, state}, {state_v_out, state}, {workspace, kHeaderBytes}, {state_k_in, state},
                        {state_v_in, state}, {k_new, total_q * row}, {v_new, total_q * row}, {cu_q_lens, seqs + 4},
                        {path, seqs * max_path}, {path_lens, seqs}};
  if (overlap(spans, 3, sizeof spans / sizeof *spans)) return INK_ERR_BAD_SHAPE;
  ink::TreeConvArgs a{};
  a.x[0] = static_cast<const uint16_t*>(k_new);
  a.x[1] = static_cast<const uint16_t*>(v_new);
  a.st_in[0] = static_cast<const uint16_t*>(state_k_in);
  a.st_in[1] = static_cast<const uint16_t*>(state_v_in);
  a.st_out[0] = static_cast<uint16_t*>(state_k_out);
  a.st_out[1] = static_cast<uint16_t*>(state_v_out);
  a.cu_q = cu_q_lens;
  a.path = path;
  a.path_lens = path_lens;
  a.max_path = max_path;
  a.err = reinterpret_cast<uint32_t*>(workspace);
  a.B = params->num_seqs;
  a.T = total_q;
  a.D = params->head_dim;
  a.nvec = params->num_kv_heads * params->head_dim / 8;
  return ink::launch_kv_conv_state_tree(a, kernel_size, (cudaStream_t)stream) == cudaSuccess ? INK_OK : INK_ERR_CUDA;
}

ink_status_t inkling_attn_tree_commit(const ink_attn_params_t* params, const int32_t* cu_q_lens,
                                      const int32_t* seq_lens, const int32_t* block_table, const int32_t* path,
                                      const int32_t* path_lens, int32_t max_path, int32_t num_pools,
                                      void* const* k_caches, void* const* v_caches, int32_t* seq_lens_out,
                                      void* workspace, size_t workspace_bytes, void* stream) {
  ink_status_t st = validate(params);
  if (st != INK_OK) return st;
  if (!cu_q_lens || !seq_lens || !block_table || !path || !path_lens || !k_caches || !v_caches || !workspace)
    return INK_ERR_NULL_PTR;
  if (max_path < 1 || num_pools < 1 || num_pools > INK_TREE_MAX_POOLS) return INK_ERR_BAD_SHAPE;
  if (!aligned(cu_q_lens, 4) || !aligned(seq_lens, 4) || !aligned(block_table, 4) || !aligned(path, 4) ||
      !aligned(path_lens, 4) || !aligned(seq_lens_out, 4) || !aligned(workspace, 256))
    return INK_ERR_ALIGNMENT;
  ink::TreeCommitArgs a;
  a.npools = 2 * num_pools;
  for (int i = 0; i < num_pools; ++i) {
    a.pool[2 * i] = static_cast<uint16_t*>(k_caches[i]);
    a.pool[2 * i + 1] = static_cast<uint16_t*>(v_caches[i]);
  }
  for (int i = 0; i < a.npools; ++i) {
    if (!a.pool[i]) return INK_ERR_NULL_PTR;
    if (!aligned(a.pool[i], 16)) return INK_ERR_ALIGNMENT;
  }
  if (workspace_bytes < kHeaderBytes) return INK_ERR_WORKSPACE;
  if (params->num_seqs == 0) return INK_OK;
  const size_t seqs = (size_t)params->num_seqs * 4, pool = pool_bytes(params);
  Span spans[] = {{nullptr, pool}, {seq_lens_out, seqs}, {workspace, kHeaderBytes}, {cu_q_lens, seqs + 4}, {seq_lens, seqs},
                  {block_table, table_bytes(params)}, {path, seqs * max_path}, {path_lens, seqs}};
  constexpr int kSpans = sizeof spans / sizeof *spans;
  for (int i = 0; i < a.npools; ++i) {
    spans[0].at = a.pool[i];
    if (overlap(spans, i == 0 ? 3 : 1, kSpans)) return INK_ERR_BAD_SHAPE;
  }
  const uint16_t* sorted[2 * INK_TREE_MAX_POOLS];   // pools side by side: each ends before the next begins
  std::copy(a.pool, a.pool + a.npools, sorted);
  std::sort(sorted, sorted + a.npools, std::less<const uint16_t*>());
  for (int i = 0; i + 1 < a.npools; ++i)
    if (reinterpret_cast<uintptr_t>(sorted[i]) + pool > reinterpret_cast<uintptr_t>(sorted[i + 1])) return INK_ERR_BAD_SHAPE;
  a.cu_q = cu_q_lens;
  a.seq_lens = seq_lens;
  a.block_table = block_table;
  a.path = path;
  a.path_lens = path_lens;
  a.max_path = max_path;
  a.seq_lens_out = seq_lens_out;
  a.err = reinterpret_cast<uint32_t*>(workspace);
  a.B = params->num_seqs;
  a.Hkv = params->num_kv_heads;
  a.log2_page = ilog2(params->page_size);
  a.max_pages = params->max_pages_per_seq;
  a.num_pages = params->num_pages;
  int dev = 0;
  const int sms = ink::current_device_sms(&dev);
  if (sms <= 0) return INK_ERR_CUDA;
  return ink::launch_tree_commit(a, params->head_dim, sms, (cudaStream_t)stream) == cudaSuccess ? INK_OK : INK_ERR_CUDA;
}

}  // extern "C"
