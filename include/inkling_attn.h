/*
 * inkling_attn.h -- C ABI of libinkling_attn.so: paged prefill and decode attention
 * with a per-token relative-position bias, grouped-query heads, and sliding-window or
 * full-causal masking, for NVIDIA GB300 (sm_103a).
 *
 * The operation is the attention of the RoPE-free hybrid model described in
 * "Support Inkling-NVFP4 model" (TensorRT-LLM PR #17062):
 *   - section "Architecture": position enters only through a learned bias per
 *     (query token, head, relative distance) added to the scores before the softmax;
 *     local layers attend over a 512-key sliding window (16 KV heads), global layers
 *     are full causal (8 KV heads);
 *   - section "Implementation", row attention_backend/inkling_triton.py: paged prefill
 *     and decode kernels apply the bias as a score modifier; rel_logits has a static
 *     shape so decode can be captured in a CUDA graph;
 *   - review of _build_rel_logits: the bias tensor is [tokens, heads, rel_extent] fp32.
 * and in "Inkling attn backend cleanup fake registry" (TensorRT-LLM PR #17860):
 *   - commit on GQA input checks: query head h reads KV head h / (Hq / Hkv); a
 *     non-divisible head pair is an error;
 *   - commit moving attention into the backend: per-layer scalars sm_scale,
 *     rel_extent, window_left (-1 on global layers);
 *   - commits on borrowing the base page table: key k lives in page
 *     block_table[b][k / page_size] (a positional table), and k < seq_len bounds every
 *     access, so entries past a sequence's own blocks are never read.
 *
 * Definition (exact; the kernels compute it in fp32 with bf16 inputs):
 *   sequence b has L_b = seq_lens[b] keys; its n_b new query tokens are the last n_b
 *   positions, so new token i sits at p = L_b - n_b + i.
 *   visible keys:  0 <= k <= p, and p - k <= window - 1 when window > 0
 *   s_k = sm_scale * <q[t,h,:], K[k,h/G,:]> + rel_logits[t, h, min(p - k, E - 1)]
 *   out[t,h,:] = sum_k softmax(s)_k * V[k,h/G,:]          (bf16, round to nearest even)
 *
 * Conventions for every entry point:
 *   - Pointers named "device" must point to GPU memory of the current device; the
 *     caller owns every buffer.  Calls never allocate, free or synchronise: they enqueue
 *     kernels on `stream` (a cudaStream_t; NULL = legacy default stream) and return.
 *   - Host-side validation reads only the scalars and pointer values.  On failure the
 *     call returns an error code and launches nothing.
 *   - Device-side problems (a page id outside [0, num_pages) for a key that must be
 *     read, more new tokens than history, a bounded wait that ran out) never fault:
 *     the kernel skips the access, treats the affected keys as masked, and ORs a bit
 *     into the sticky error word in the workspace (INK_DEVERR_*), which
 *     inkling_attn_read_device_error() returns.
 *   - Keys that sit in a loaded page but are not visible get weight exactly 0 and
 *     their V rows are zeroed before use, so any bit pattern (NaN included) may sit
 *     there.  Pages that hold no visible key are never read.
 *   - A sequence with seq_lens[b] == 0 writes zeros to its output rows.
 */
#ifndef INKLING_ATTN_H
#define INKLING_ATTN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  INK_OK = 0,
  INK_ERR_NULL_PTR = 1,        /* a required pointer is NULL */
  INK_ERR_BAD_SHAPE = 2,       /* Hq % Hkv != 0, head_dim not 64/128, non-positive sizes */
  INK_ERR_BAD_PAGE_SIZE = 3,   /* page_size not a power of two in [8, 2^20] */
  INK_ERR_WORKSPACE = 4,       /* workspace smaller than inkling_attn_workspace_bytes() */
  INK_ERR_ALIGNMENT = 5,       /* q/k/v/out not 16-byte aligned, or index arrays not 4-byte */
  INK_ERR_CUDA = 6,            /* a CUDA runtime call failed (launch, attribute, ...) */
  INK_ERR_TOO_LARGE = 7        /* an index would overflow the 32-bit coordinates used */
} ink_status_t;

/* Sticky device error bits (see inkling_attn_read_device_error). */
#define INK_DEVERR_PAGE_OUT_OF_RANGE 0x1u  /* block_table entry outside [0, num_pages) */
#define INK_DEVERR_QLEN_EXCEEDS_KV   0x2u  /* cu_q_lens gives more new tokens than seq_lens */
#define INK_DEVERR_WAIT_TIMEOUT      0x4u  /* a bounded wait on a copy ran out */
#define INK_DEVERR_QLEN_EXCEEDS_MAX  0x8u  /* a sequence has more new tokens than max_q_len */
#define INK_DEVERR_BAD_ROWS          0x10u /* cu_q_lens names rows outside [0, total_q) */
#define INK_DEVERR_BAD_TREE          0x20u /* a parent or an accepted path that no tree of drafted tokens has */

/* Per-call shape and layer scalars.  All sizes are element counts. */
typedef struct {
  int32_t num_seqs;           /* B */
  int32_t num_q_heads;        /* Hq */
  int32_t num_kv_heads;       /* Hkv; Hq % Hkv == 0 */
  int32_t head_dim;           /* D: 64 or 128 */
  int32_t page_size;          /* P: power of two, >= 8 */
  int32_t max_pages_per_seq;  /* row stride of block_table */
  int32_t num_pages;          /* pages in each K/V pool */
  int32_t rel_extent;         /* E >= 1: distances >= E-1 use bucket E-1 */
  int32_t window;             /* > 0: keys at distances 0..window-1; <= 0: full causal */
  float sm_scale;             /* multiplies q.k only; the bias is added unscaled */
} ink_attn_params_t;

/*
 * Bytes of device workspace a call needs.  is_decode != 0 sizes it for
 * inkling_attn_decode (split-K partials and tickets), else for inkling_attn_prefill.
 * Returns 0 if the parameters are invalid.  A buffer sized for decode also serves
 * prefill with the same params.
 */
size_t inkling_attn_workspace_bytes(const ink_attn_params_t* params, int is_decode);

/*
 * Zero a workspace (error word and split-K tickets) on `stream`.  Must be called once
 * after allocating a workspace and before its first use; the kernels leave the tickets
 * at zero when they finish, so later calls need no re-initialisation.
 */
ink_status_t inkling_attn_workspace_init(void* workspace, size_t workspace_bytes, void* stream);

/*
 * Paged prefill (context phase), any number of new tokens per sequence.
 *   q          device, bf16 [total_q, Hq, D], rows packed by sequence
 *   cu_q_lens  device, int32 [B+1], cu_q_lens[0] = 0, non-decreasing; n_b = cu[b+1]-cu[b]
 *   max_q_len  host int >= every n_b (sizes the grid; larger n_b set INK_DEVERR_QLEN_EXCEEDS_MAX)
 *   total_q    host int = cu_q_lens[B], the number of rows of q, rel_logits and out (bounds
 *              the tensor-memory copies of q; rows past it are never read)
 *   k_cache, v_cache  device, bf16 [num_pages, Hkv, P, D]; the step's K/V must already
 *              be written (new tokens are the last n_b of seq_lens[b])
 *   block_table device, int32 [B, max_pages_per_seq], positional page ids
 *   seq_lens   device, int32 [B], KV length including the new tokens
 *   rel_logits device, fp32 [total_q, Hq, E]
 *   out        device, bf16 [total_q, Hq, D]
 *   workspace  device, >= inkling_attn_workspace_bytes(params, 0), initialised once
 * q and out must be 16-byte aligned; when both are 32-byte aligned the kernels move their
 * rows in 256-bit loads and stores (the same results, fewer memory requests).
 */
ink_status_t inkling_attn_prefill(const ink_attn_params_t* params, const void* q,
                                  const int32_t* cu_q_lens, int32_t max_q_len, int32_t total_q,
                                  const void* k_cache, const void* v_cache,
                                  const int32_t* block_table, const int32_t* seq_lens,
                                  const float* rel_logits, void* out, void* workspace,
                                  size_t workspace_bytes, void* stream);

/*
 * inkling_attn_prefill with the bias in bf16: rel_logits_bf16 is bf16 [total_q, Hq, E]
 * (same layout as rel_logits), every other argument and result as for
 * inkling_attn_prefill.  The review of _build_rel_logits in "Support Inkling-NVFP4 model"
 * (TensorRT-LLM PR #17062) suggests producing the bias in bf16 where the kernel can take
 * it: on long prompts the fp32 bias is the largest input of the call, and bf16 halves it.
 * The bias enters the scores as exactly the bf16 values given (widened to fp32); the
 * rest of the arithmetic is unchanged.
 *   Requirements beyond inkling_attn_prefill: E a multiple of 8 (else INK_ERR_BAD_SHAPE)
 *   and rel_logits_bf16 16-byte aligned (else INK_ERR_ALIGNMENT).
 */
ink_status_t inkling_attn_prefill_bf16bias(const ink_attn_params_t* params, const void* q,
                                           const int32_t* cu_q_lens, int32_t max_q_len, int32_t total_q,
                                           const void* k_cache, const void* v_cache,
                                           const int32_t* block_table, const int32_t* seq_lens,
                                           const void* rel_logits_bf16, void* out, void* workspace,
                                           size_t workspace_bytes, void* stream);

/*
 * inkling_attn_prefill with the bias given in low-rank form: the kernel computes each bias
 * tile itself, so the [total_q, Hq, E] bias tensor is never built or read.  "Support
 * Inkling-NVFP4 model" (TensorRT-LLM PR #17062), review of _build_rel_logits: a layer's
 * bias is the product over d_rel of a per-(token, head) vector r and the layer's
 * projection rel_logits_proj [d_rel, E]:
 *     rel[t, h, e] = sum_c r[t, h, c] * rel_logits_proj[c, e]
 *   r           device, bf16 [total_q, Hq, d_rel], 16-byte aligned
 *   rel_proj_t  device, bf16 [E, d_rel]: rel_logits_proj transposed (bucket-major, so each
 *               bucket's d_rel coefficients are contiguous), 16-byte aligned
 *   d_rel       a multiple of 8 in [8, 64] (else INK_ERR_BAD_SHAPE); the pages do not give it.
 *               The bias products run with K = 64; columns past d_rel are zeros.
 * The products are summed in fp32 from the bf16 operands (tensor-core MMA for the buckets
 * of a tile, a plain fp32 dot product for the clamped bucket E - 1) and the tile's bias
 * values are kept in fp16 until they are added to the fp32 scores (relative rounding
 * 2^-11); the rest of the arithmetic is that of inkling_attn_prefill.  Every other
 * argument and result as for inkling_attn_prefill.
 */
ink_status_t inkling_attn_prefill_lowrank_bias(const ink_attn_params_t* params, const void* q,
                                               const int32_t* cu_q_lens, int32_t max_q_len, int32_t total_q,
                                               const void* k_cache, const void* v_cache,
                                               const int32_t* block_table, const int32_t* seq_lens,
                                               const void* r, const void* rel_proj_t, int32_t d_rel, void* out,
                                               void* workspace, size_t workspace_bytes, void* stream);

/*
 * Paged decode: one new token per sequence (row b of q is sequence b, at p = L_b - 1).
 *   q          device, bf16 [B, Hq, D]
 *   rel_logits device, fp32 [B, Hq, E]
 *   out        device, bf16 [B, Hq, D]
 *   workspace  device, >= inkling_attn_workspace_bytes(params, 1), initialised once.
 *              Calls that share a workspace must not overlap on the GPU (the split-K
 *              partials and tickets live there).
 * Other arguments as for prefill.  Stream-ordered, no allocation, no host sync: the
 * call can be captured in a CUDA graph.
 */
ink_status_t inkling_attn_decode(const ink_attn_params_t* params, const void* q,
                                 const void* k_cache, const void* v_cache,
                                 const int32_t* block_table, const int32_t* seq_lens,
                                 const float* rel_logits, void* out, void* workspace,
                                 size_t workspace_bytes, void* stream);

/*
 * inkling_attn_decode without a workspace argument, for callers that cannot allocate
 * device memory: for example a plugin whose host framework owns every device buffer
 * and hands out only fixed-size tensors, or a serving loop that must not grow its
 * memory after start-up.  Such a caller has no way to create the workspace that
 * inkling_attn_decode needs.  The pages this library follows have no counterpart to
 * this entry point.
 *   - Scratch: a 64 MiB device array inside the library, held by every GPU that loads
 *     it until the process exits.  A call whose workspace need
 *     (inkling_attn_workspace_bytes(params, 1)) exceeds 64 MiB returns
 *     INK_ERR_WORKSPACE and launches nothing.
 *   - The call allocates nothing: no cudaMalloc, no cudaFree, no allocating library
 *     routine.  It clears the array's error word and split-K tickets on `stream`
 *     (cudaMemsetAsync), then runs the same kernel as inkling_attn_decode.
 *   - The first call on each device looks up the array's device address
 *     (cudaGetSymbolAddress) with that device current.  Make that first call before any
 *     stream capture.
 *   - All calls on a device share the array, which keeps the last call's contents.
 *     Calls that overlap on the GPU (different streams, no ordering between them) race
 *     on it and give wrong results.  Device-side error bits are kept in the array and
 *     not reported.
 * Other arguments and results as for inkling_attn_decode.
 */
ink_status_t inkling_attn_decode_noalloc(const ink_attn_params_t* params, const void* q,
                                         const void* k_cache, const void* v_cache,
                                         const int32_t* block_table, const int32_t* seq_lens,
                                         const float* rel_logits, void* out, void* stream);

/*
 * The step's K/V write: causal short convolution of the new K and V rows, written into
 * the paged caches, and the convolution state carried to the next step.
 * "Support Inkling-NVFP4 model" (TensorRT-LLM PR #17062), section "Architecture": every
 * attention layer runs a causal short convolution over K and over V, with per-request
 * state between steps.  "Inkling attn backend cleanup fake registry" (TensorRT-LLM PR
 * #17860): the state is a window of kernel_size - 1 past inputs per request, carried with
 * the request; the backend itself writes the step's K/V into the paged cache through the
 * block table.  Neither page gives the kernel size, a bias or an activation: the
 * convolution here is depthwise (one filter per channel), without bias or activation.
 * For request b with n_b = cu_q_lens[b+1] - cu_q_lens[b] new rows and L_b = seq_lens[b]
 * (history including them), new row i sits at position p = L_b - n_b + i, and for each
 * channel c = (g, d) of K (and likewise of V)
 *     y[p, c] = sum_{j=0}^{ks-1} w_k[g, d, j] * x[p - (ks-1) + j, c]
 * where x at the ks - 1 positions before the first new row is state_k_in[b] (oldest
 * first).  y is computed in fp32 and stored rounded to bf16 (nearest even) at
 * k_cache[block_table[b][p / P], g, p % P, :].  state_k_out[b] receives the last ks - 1
 * rows of (state_k_in[b], new rows of b), unconvolved.
 *   k_new, v_new          device, bf16 [total_q, Hkv, D], rows packed by request
 *   cu_q_lens             device, int32 [B+1], cu_q_lens[0] = 0, cu_q_lens[B] = total_q
 *   seq_lens, block_table device, as for inkling_attn_prefill
 *   w_k, w_v              device, fp32 [Hkv, D, kernel_size] (a depthwise Conv1d weight over
 *                         the Hkv*D channels), 16-byte aligned
 *   kernel_size           1..8 (else INK_ERR_BAD_SHAPE); 1 stores x * w unshifted
 *   state_*_in/out        device, bf16 [B, kernel_size - 1, Hkv, D]; unused (may be NULL)
 *                         when kernel_size == 1.  Outputs must not overlap inputs; a fresh
 *                         request passes zero rows.
 *   k_cache, v_cache      device, bf16 [num_pages, Hkv, P, D]; only the slots of the step's
 *                         positions are written
 *   workspace             device, >= inkling_attn_workspace_bytes(params, 0) (error word)
 * Only num_seqs, num_kv_heads, head_dim, page_size, max_pages_per_seq and num_pages of
 * params are used; the rest must still be valid.  Device-side checks: a request with
 * n_b > L_b (INK_DEVERR_QLEN_EXCEEDS_KV) or a page id outside [0, num_pages)
 * (INK_DEVERR_PAGE_OUT_OF_RANGE) has those rows skipped; rows named outside [0, total_q)
 * set INK_DEVERR_BAD_ROWS.  Stream-ordered, no allocation: capturable in a CUDA graph.
 */
ink_status_t inkling_attn_kv_conv_write(const ink_attn_params_t* params, const void* k_new,
                                        const void* v_new, const int32_t* cu_q_lens, int32_t total_q,
                                        const int32_t* seq_lens, const int32_t* block_table,
                                        const float* w_k, const float* w_v, int32_t kernel_size,
                                        const void* state_k_in, const void* state_v_in,
                                        void* state_k_out, void* state_v_out, void* k_cache,
                                        void* v_cache, void* workspace, size_t workspace_bytes,
                                        void* stream);

/*
 * Options of the masked attention entry points (a NULL pointer to this struct: none of them).
 * Query token t of sequence b sits at position p as above and sees the keys
 *     max(key_begin[t], p - window + 1 when window > 0, 0) <= k < min(key_end[t], L_b)
 * so one pair of numbers per token expresses packed documents (key_begin = the document's first
 * position), a bidirectional prefix or image block (key_end = its end), padding (an empty
 * range), and windows.  The window bounds the past only.  The score of a visible key is
 *     x   = sm_scale * <q[t,h,:], K[k,h/G,:]>
 *     s_k = (softcap > 0 ? softcap * tanh(x / softcap) : x) - slopes[h] * |p - k|
 */
typedef struct {
  float softcap;             /* in [1e-6, 1e6]: scores capped by a tanh; 0: not capped */
  const int32_t* key_begin;  /* device int32 [rows of q] first visible key, or NULL: 0 */
  const int32_t* key_end;    /* device int32 [rows of q] last visible key + 1, or NULL: p + 1 */
  const float* slopes;       /* device fp32 [Hq], or NULL: no distance bias */
} ink_attn_mask_t;

/*
 * Bytes of device workspace a masked attention call needs; initialise it once with
 * inkling_attn_workspace_init.  Returns 0 if the parameters are invalid.  It depends on the head
 * counts and head_dim only (about 65 MB for a prefill at D = 128, 3 to 6 MB for a decode), and one workspace
 * of the largest size serves masked prefills and decodes of any sizes, one after the other; the
 * other entry points' workspaces are laid out differently.  Calls that share a workspace must not
 * overlap on the GPU.  After INK_DEVERR_WAIT_TIMEOUT initialise it again: until then a prefill of
 * few rows against long histories does nothing but report the timeout.
 */
size_t inkling_attn_masked_workspace_bytes(const ink_attn_params_t* params, int is_decode);

/*
 * Paged prefill without a per-token bias tensor: capped scores, distance bias and a visible key
 * range per token (ink_attn_mask_t).  For models that take their positions from a rotation of q
 * and k (inkling_attn_qk_norm_rope_write) or from the distance bias.
 *   q, cu_q_lens, k_cache, v_cache, block_table, seq_lens, out: as for inkling_attn_prefill,
 *              except that there is no max_q_len; out, lse and the workspace must overlap neither
 *              one another nor anything that is read (INK_ERR_BAD_SHAPE)
 *   total_q    rows of q and out; rows from cu_q_lens[B] on belong to no sequence: they are not
 *              written, and what they hold changes nothing
 *   lse        device, fp32 [total_q, Hq], or NULL: log of the sum of exp(s_k) over the visible
 *              keys (natural units), with which outputs over parts of a history are joined
 *   workspace  device, >= inkling_attn_masked_workspace_bytes(params, 0), initialised once
 * A token that sees no key gets a zero output row and lse = -infinity; one that sees a single key gets
 * that key's V.  Softmax weights are rounded to bf16 before they multiply V and divided by the sum of
 * the unrounded ones, so an output may be off by 2^-8 of sum_k w_k |V_k| beside its own rounding.  Capped
 * scores are off by at most 2^-20 of themselves (beyond the cap, 2^-21 of the cap); which of three forms of
 * the tanh a row takes goes by the largest score of the 32 rows that are computed together, so within
 * these bounds its bits may change with how a prompt is cut into calls.  Sums are held in fp32 and divided
 * at the end: |V| up to 2^100 is safe (2^70 when scores are capped).  params.rel_extent is not used
 * (any valid value).  A sequence whose rows lie outside [0, total_q) is skipped
 * (INK_DEVERR_BAD_ROWS); one with more new tokens than history gets zero rows
 * (INK_DEVERR_QLEN_EXCEEDS_KV).
 */
ink_status_t inkling_attn_prefill_masked(const ink_attn_params_t* params, const ink_attn_mask_t* mask,
                                         const void* q, const int32_t* cu_q_lens, int32_t total_q,
                                         const void* k_cache, const void* v_cache,
                                         const int32_t* block_table, const int32_t* seq_lens,
                                         void* out, float* lse, void* workspace,
                                         size_t workspace_bytes, void* stream);

/*
 * Paged decode without a per-token bias tensor: row b of q is sequence b at p = L_b - 1; the
 * options, results and requirements are those of inkling_attn_prefill_masked
 * (workspace: inkling_attn_masked_workspace_bytes(params, 1)).  A sequence with
 * seq_lens[b] <= 0 gets a zero row and lse = -infinity.
 */
ink_status_t inkling_attn_decode_masked(const ink_attn_params_t* params, const ink_attn_mask_t* mask,
                                        const void* q, const void* k_cache, const void* v_cache,
                                        const int32_t* block_table, const int32_t* seq_lens, void* out,
                                        float* lse, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Pairing of the channels that are rotated together.
 */
typedef enum {
  INK_ROPE_HALF = 0,         /* channel i with channel i + rot_dim / 2 */
  INK_ROPE_INTERLEAVED = 1   /* channel 2 i with channel 2 i + 1 */
} ink_rope_layout_t;

/* Norm and rotation of inkling_attn_qk_norm_rope_write. */
typedef struct {
  const float* w_q;          /* device fp32 [D], 16-byte aligned: weight of the RMS norm of q, or NULL: no norm */
  const float* w_k;          /* the same for k */
  float eps;                 /* added to the mean square; >= 0 */
  const float* inv_freq;     /* device fp32 [rot_dim / 2]: angle per position of each pair (unused when rot_dim == 0) */
  int32_t rot_dim;           /* 0 (no rotation) or a multiple of 16, at most D: the first channels, rotated */
  int32_t layout;            /* ink_rope_layout_t */
  float rot_scale;           /* multiplies cos and sin (1, or the attention factor of a long-context scaling) */
} ink_norm_rope_t;

/*
 * The step's K/V write for models with normed or rotated heads: RMS norm of every query and key
 * head, rotation by the token's position, and K and V into the paged caches, in one pass.
 *   y = x * (mean(x^2) + eps)^(-1/2) * w          (fp32; without weights y = x)
 *   pair (a, b) of channels with frequency f at position p, in fp32:
 *     a' = rot_scale * (a cos(p f) - b sin(p f)),  b' = rot_scale * (b cos(p f) + a sin(p f))
 * rounded to bf16 once.  p f is reduced to a turn in integers, so that its error is below 2^-25 of a
 * turn at any position (f up to 50).  V is stored as it is.
 *   q, k, v       device, bf16; row t of q holds Hq heads of D contiguous channels at
 *                 q + t * q_stride elements (k, v: Hkv heads): parts of a fused projection's
 *                 rows pass without a copy.  Strides are multiples of 8, 16-byte aligned bases.
 *   cu_q_lens, seq_lens, block_table   as for inkling_attn_prefill: new row i of request b sits
 *                 at p = L_b - n_b + i
 *   q_out         device, bf16 [total_q, Hq, D]; may be q itself when q_stride == Hq * D
 *   k_cache, v_cache  device, bf16 [num_pages, Hkv, P, D]; only the slots of the step's
 *                 positions are written
 *                 What is written (the workspace's first 256 bytes among it) must overlap neither
 *                 what is read nor what else is written, but for q in place (INK_ERR_BAD_SHAPE).
 *   workspace     device, initialised, of any entry point's size; only its error word is used
 * Rows from cu_q_lens[B] on belong to no request and are left as they were.  A request whose rows
 * lie outside [0, total_q) (INK_DEVERR_BAD_ROWS) or with n_b > L_b (INK_DEVERR_QLEN_EXCEEDS_KV) has
 * its rows skipped, as the attention entry points skip them; a page id outside [0, num_pages)
 * (INK_DEVERR_PAGE_OUT_OF_RANGE) has the K/V rows of its keys skipped.  Two rows that name the
 * same slot (requests sharing a page they write to) race: each 16 bytes of the slot hold either row's.
 */
ink_status_t inkling_attn_qk_norm_rope_write(const ink_attn_params_t* params, const ink_norm_rope_t* rope,
                                             const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                                             const void* v, int64_t v_stride, const int32_t* cu_q_lens,
                                             int32_t total_q, const int32_t* seq_lens, const int32_t* block_table,
                                             void* q_out, void* k_cache, void* v_cache, void* workspace,
                                             size_t workspace_bytes, void* stream);

/*
 * ---- Trees of drafted tokens.
 *
 * A step that checks drafted tokens writes the n_b = cu_q_lens[b+1] - cu_q_lens[b] tokens of sequence b
 * behind its history of H_b = seq_lens[b] - n_b keys, parents before children: token i takes slot
 * H_b + i of the cache, whatever its position.  Its position is H_b plus its depth in the tree (siblings
 * share one), and it sees the history and the drafted tokens on its way to the root, itself among them.
 * The step's calls, in order:
 *     inkling_attn_tree_plan                once: positions and visible drafted tokens from the parents
 *     per layer: inkling_attn_qk_norm_rope_write_at or inkling_attn_kv_conv_write_tree, then
 *                inkling_attn_tree
 *     inkling_attn_tree_commit              once: the accepted path's K and V rows move to where a
 *                                           sequence without the other tokens would have them
 *     inkling_attn_kv_conv_state_tree       per layer with a convolution: its state behind that path
 *
 * Plan of a tree, from the parents.
 *   cu_q_lens, seq_lens   as for inkling_attn_prefill
 *   total_q    rows of parents, positions and ancestors; rows from cu_q_lens[B] on are left as they were
 *   parents    device, int32 [total_q]: the parent's place i in its sequence, -1 for a child of the last
 *              token of the history (a sequence may have several).  One that is not in [-1, own place)
 *              sets INK_DEVERR_BAD_TREE and counts as -1.
 *   words      32-bit words of a token's bits, 1..16: a sequence may draft up to 32 * words tokens; one with
 *              more sets INK_DEVERR_QLEN_EXCEEDS_MAX and is skipped
 *   positions  device, int32 [total_q]: H_b + depth, the depth of a child of the history being 0
 *   ancestors  device, uint32 [total_q, words]: bit j % 32 of word j / 32 is set for every drafted token j on
 *              the way from the token to the root and for the token itself
 *   workspace  device, initialised, of any entry point's size; only its error word is used
 * Outputs (the workspace's first 256 bytes among them) must overlap neither inputs nor one another
 * (INK_ERR_BAD_SHAPE).  Only num_seqs of params is used; the rest must still be valid.  A sequence whose
 * rows lie outside [0, total_q) (INK_DEVERR_BAD_ROWS) or with n_b > seq_lens[b]
 * (INK_DEVERR_QLEN_EXCEEDS_KV) is skipped.
 */
ink_status_t inkling_attn_tree_plan(const ink_attn_params_t* params, const int32_t* cu_q_lens, int32_t total_q,
                                    const int32_t* seq_lens, const int32_t* parents, int32_t words,
                                    int32_t* positions, uint32_t* ancestors, void* workspace,
                                    size_t workspace_bytes, void* stream);

/* The drafted tokens of a call, as inkling_attn_tree_plan lays them out (or the caller: any bits will do). */
typedef struct {
  const int32_t* positions;   /* device int32 [total_q]; one below H_b counts as H_b */
  const uint32_t* ancestors;  /* device uint32 [total_q, words]; bits from n_b on are not looked at */
  int32_t words;              /* 1..16 */
} ink_attn_tree_t;

/* Options of inkling_attn_tree (a NULL pointer to this struct: none of them). */
typedef struct {
  float softcap;              /* in [1e-6, 1e6]: scores capped by a tanh; 0: not capped */
  const float* slopes;        /* device fp32 [Hq], or NULL: no bias linear in the distance */
  const void* rel_logits;     /* device [total_q, Hq, rel_extent], 4-byte (bf16: 2-byte) aligned, or NULL: no
                                 bias tensor.  Rows that begin on 16 bytes (rel_extent a multiple of 4, bf16: of 8)
                                 are read up to four times as fast */
  int32_t rel_is_bf16;        /* rel_logits holds bf16 instead of fp32 */
} ink_attn_tree_options_t;

/* Bytes of device workspace inkling_attn_tree needs; initialise it once with inkling_attn_workspace_init.
 * Returns 0 if the parameters are invalid.  It depends on head_dim only (about 43 MB at D = 128), so one
 * workspace serves calls of any sizes, one after the other; calls that share a workspace must not overlap on the GPU. */
size_t inkling_attn_tree_workspace_bytes(const ink_attn_params_t* params);

/*
 * Attention of drafted tokens over the paged cache.  Token t at place i of sequence b has position
 * p = max(positions[t], H_b); key k < H_b has position k, drafted key H_b + j the position of token j.
 * Of the keys below seq_lens[b] the token sees
 *     k < H_b,  and  H_b + j when bit j of its ancestors is set,
 * both only at p - pos(k) <= window - 1 when window > 0.  The score of a visible key, d = |p - pos(k)|:
 *     x   = sm_scale * <q[t,h,:], K[k,h/G,:]>
 *     s_k = (softcap > 0 ? softcap * tanh(x / softcap) : x) - slopes[h] * d + rel_logits[t, h, min(d, E - 1)]
 *   q, cu_q_lens, total_q, k_cache, v_cache, block_table, seq_lens, out, lse: as for
 *              inkling_attn_prefill_masked; the step's K and V rows must already be written
 *   workspace  device, >= inkling_attn_tree_workspace_bytes(params), initialised once
 * One token per sequence with a bit of its own makes this a decode, so that a batch may mix sequences that
 * draft with sequences that do not.  What is written must overlap nothing else (INK_ERR_BAD_SHAPE).
 * Rounding, infinities and NaN, |V|: as for inkling_attn_prefill_masked.  Scores are held in fp32 whatever their size, so a row
 * whose keys all carry a bias of the type's lowest value (a mask written that way) is the mean over those that share its largest
 * score; a bias of -infinity takes a key's weight altogether.  A token that sees no key gets a zero row and
 * lse = -infinity; so do the tokens of a sequence with n_b > seq_lens[b] (INK_DEVERR_QLEN_EXCEEDS_KV) or
 * n_b > 32 * words (INK_DEVERR_QLEN_EXCEEDS_MAX).  A sequence whose rows lie outside [0, total_q) is skipped
 * (INK_DEVERR_BAD_ROWS).
 */
ink_status_t inkling_attn_tree(const ink_attn_params_t* params, const ink_attn_tree_t* tree,
                               const ink_attn_tree_options_t* options, const void* q, const int32_t* cu_q_lens,
                               int32_t total_q, const void* k_cache, const void* v_cache,
                               const int32_t* block_table, const int32_t* seq_lens, void* out, float* lse,
                               void* workspace, size_t workspace_bytes, void* stream);

/*
 * inkling_attn_qk_norm_rope_write with a position per row: row t is rotated by positions[t] (device int32
 * [total_q]; a negative one counts as 0) and still written to slot H_b + i.  Every other argument and result as there.
 */
ink_status_t inkling_attn_qk_norm_rope_write_at(const ink_attn_params_t* params, const ink_norm_rope_t* rope,
                                                const int32_t* positions, const void* q, int64_t q_stride,
                                                const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                                                const int32_t* cu_q_lens, int32_t total_q, const int32_t* seq_lens,
                                                const int32_t* block_table, void* q_out, void* k_cache, void* v_cache,
                                                void* workspace, size_t workspace_bytes, void* stream);

/*
 * inkling_attn_kv_conv_write for a tree of drafted tokens: the rows before a token are those of its ancestors,
 * and past the root those of the state,
 *     y_i = sum_{d=0}^{ks-1} w[g, d', ks-1-d] * x[ancestor of i at distance d]      (d = 0: the token itself)
 * with the state's newest row as the parent of a root.  y_i goes to slot H_b + i.  The state is not advanced: that takes the
 * accepted path (inkling_attn_kv_conv_state_tree).
 *   parents    device, int32 [total_q], as for inkling_attn_tree_plan (a bad one: INK_DEVERR_BAD_TREE, -1)
 * Every other argument as for inkling_attn_kv_conv_write.  What is written (the workspace's first 256 bytes
 * among it) must overlap nothing else (INK_ERR_BAD_SHAPE).  A request whose rows lie outside [0, total_q)
 * or with n_b > seq_lens[b] has its rows skipped and reported, a page id outside [0, num_pages) its row.
 */
ink_status_t inkling_attn_kv_conv_write_tree(const ink_attn_params_t* params, const void* k_new, const void* v_new,
                                             const int32_t* cu_q_lens, int32_t total_q, const int32_t* seq_lens,
                                             const int32_t* block_table, const int32_t* parents, const float* w_k,
                                             const float* w_v, int32_t kernel_size, const void* state_k_in,
                                             const void* state_v_in, void* k_cache, void* v_cache, void* workspace,
                                             size_t workspace_bytes, void* stream);

/*
 * The convolution state behind an accepted path: state_k_out[b] receives the last kernel_size - 1 rows of
 * (state_k_in[b], k_new of the path's tokens), and likewise V.
 *   path, path_lens, max_path   as for inkling_attn_tree_commit; a path that is refused there counts as
 *              empty (INK_DEVERR_BAD_TREE): the state is copied
 * Other arguments as for inkling_attn_kv_conv_write.  A request whose rows lie outside [0, total_q) has its
 * state copied (INK_DEVERR_BAD_ROWS).  With kernel_size 1 nothing is done.  What is written (the workspace's first 256
 * bytes among it) must overlap nothing else (INK_ERR_BAD_SHAPE).
 */
ink_status_t inkling_attn_kv_conv_state_tree(const ink_attn_params_t* params, const void* k_new, const void* v_new,
                                             const int32_t* cu_q_lens, int32_t total_q, const int32_t* path,
                                             const int32_t* path_lens, int32_t max_path, int32_t kernel_size,
                                             const void* state_k_in, const void* state_v_in, void* state_k_out,
                                             void* state_v_out, void* workspace, size_t workspace_bytes, void* stream);

/* Most pairs of pools in one inkling_attn_tree_commit. */
#define INK_TREE_MAX_POOLS 128

/*
 * Acceptance of a path: in every pool the K and V rows of token path[b][j] move from slot H_b + path[b][j] to slot
 * H_b + j, j < path_lens[b].  The rows behind them stay as they are.
 *   cu_q_lens, seq_lens, block_table   of the step (seq_lens with all drafted tokens)
 *   path       device, int32 [B, max_path]: places of the accepted tokens in their sequence, from the root on,
 *              so strictly increasing; entries from path_lens[b] on are not looked at.  That each is a child of
 *              the one before is the caller's to keep: the call has no parents to check it with, and K rows of
 *              another way would stay rotated for other positions than those they move to
 *   path_lens  device, int32 [B], 0..max_path
 *   k_caches, v_caches   host arrays of num_pools device pointers (1..INK_TREE_MAX_POOLS): pools of the layers that share
 *              block_table and the geometry of params
 *   seq_lens_out  device, int32 [B], or NULL: H_b + path_lens[b], the lengths without what was not accepted
 *   workspace  device, initialised, of any entry point's size; only its error word is used
 * Pools must not overlap one another, and what is written must overlap nothing that is read
 * (INK_ERR_BAD_SHAPE).  A path whose entries are not strictly increasing places of drafted tokens, or whose
 * length is not in [0, max_path], moves nothing and counts as empty (INK_DEVERR_BAD_TREE); a sequence with n_b > seq_lens[b]
 * (INK_DEVERR_QLEN_EXCEEDS_KV) or n_b < 0 (INK_DEVERR_BAD_ROWS) is skipped and keeps its length; a row
 * on a page outside [0, num_pages) is skipped (INK_DEVERR_PAGE_OUT_OF_RANGE).
 * Two sequences that share a page they move rows on race.
 */
ink_status_t inkling_attn_tree_commit(const ink_attn_params_t* params, const int32_t* cu_q_lens,
                                      const int32_t* seq_lens, const int32_t* block_table, const int32_t* path,
                                      const int32_t* path_lens, int32_t max_path, int32_t num_pools,
                                      void* const* k_caches, void* const* v_caches, int32_t* seq_lens_out,
                                      void* workspace, size_t workspace_bytes, void* stream);

/*
 * Synchronise `stream`, copy the sticky device error word (INK_DEVERR_* bits) to
 * *err_out, and clear it when `clear` is non-zero.  This is the only entry point that
 * blocks the host.
 */
ink_status_t inkling_attn_read_device_error(void* workspace, size_t workspace_bytes,
                                            void* stream, uint32_t* err_out, int clear);

/* Static, human-readable name of a status code. */
const char* inkling_attn_status_string(ink_status_t status);

/* ABI version of the library (major * 100 + minor). */
int32_t inkling_attn_version(void);

/*
 * Time limit, in nanoseconds, of one pipeline wait inside every kernel launched after this
 * call (process-wide; the default is 2 000 000 000, larger values are clamped to it).  A
 * wait that runs out sets INK_DEVERR_WAIT_TIMEOUT in the workspace error word; the kernel
 * then stops issuing work, waits (up to 2 s each) for the copies and tensor-core
 * operations it has already issued, and returns, leaving the device usable.  0 makes every
 * wait that finds its data not yet ready give up at once: a way for tests to drive the
 * timeout path without a fault.  Failure detection by status, not by fault, follows the
 * epoch-checked "ready" flag of "Inkling attn backend cleanup fake registry" (TensorRT-LLM
 * PR #17860), where stale decode metadata is detected rather than read.  Not for use in
 * production: launches in flight keep the limit they were launched with.
 */
void inkling_attn_set_wait_limit_ns(uint64_t limit_ns);

#ifdef __cplusplus
}
#endif

#endif /* INKLING_ATTN_H */
