// prefill_masked.cu -- paged prefill without a bias tensor on the 5th-generation tensor cores:
// scores capped by a tanh, a bias linear in the distance, and a visible key range per token.
//
//   x = sm_scale <q[t,h], K[k]>,  s = cap(x) - slope_h |p - k|,  out = softmax(s) V,  lse = log sum exp(s)
//   over keys max(begin_t, p - W + 1, 0) <= k < min(end_t, L)
//
// Work item: up to 256 rows of one sequence and KV head in two row tiles of 128 (the M of an
// MMA).  A row is a (token, query head) pair, tokens outermost, so that the heads of a group fill
// a tile together: 16 tokens x 8 heads, 128 tokens x 1 head, 25 tokens x 5 heads (125 rows used).
// Both tiles read the same K and V tiles of 128 keys, a short run of tokens keeps the masked part
// of the diagonal small, and a few new tokens still fill the rows.
//
// Tensor memory (512 columns for D = 128): S of both tiles (128 fp32 columns each), with P, the
// bf16 numerators, over the first 64 columns of its S once that is in registers, and O of both
// tiles (D columns each).  Q, K and V sit in shared memory (two Q tiles and a ring of K and V
// tiles, 224 KB of the 227 KB).
//
// Warps (384 threads; registers moved from the last warpgroup to the two that run the softmax):
//   0-3, 4-7  softmax of row tile 0 and 1, a thread per row: reads its 128 scores, caps, masks, keeps
//             the running maximum (moved only when it grows by more than 2^8) and sum, writes P;
//             at the end O / l and lse.
//   8   K and V producer: TMA boxes of whole pages or 128 rows, table entries 32 at a time in lanes.
//   9   MMA issue, in the order P_0 V(j), Q_0 K(j+1), P_1 V(j), Q_1 K(j+1): while one tile's softmax
//       runs, the tensor cores work for the other.
//   10  scheduler: hands out items (a counter in the workspace, longest first within a sequence),
//       finds their key ranges, publishes them in shared memory, and loads their Q tiles by TMA.
//   11  K and V check: in a V tile that not every row of the item sees whole, rows of V that nobody sees
//       are zeroed, and so is every infinity or NaN (0 * NaN would reach rows that do not
//       see the key); rows that do see one get it back in the epilogue.
// When there are fewer items than SMs (a chunk of a prompt or a few drafted tokens against a long
// history), the key tiles of an item are cut into pieces of one length, chosen on the device so that
// the rounds over the SMs are full ones; a piece leaves O, maximum and sum in the workspace, and the
// last one to finish (an atomic ticket, no waiting) joins them in order.
// Every wait is bounded; after a timeout the CTA records it, stops issuing, waits for what is in
// flight and exits.
//
// What bounds it: the softmax.  Two row tiles and 128 keys take 2048 clocks of the tensor cores at D = 128,
// but about 2650 pass: a row tile's chain (128 scores from tensor memory, 1200 clocks of softmax, P V and the
// next S, four hand-overs of about 100 clocks) is longer than half of that, and the exponentials of both
// tiles alone keep the special function units busy for 1024.  Measured with 64 query and 8 KV heads of
// 128, prompts of about 5,000 tokens, GPU time alone: 1.36 PFLOP/s causal, 1.43 on whole histories, 1.11
// capped, 1.01 with slopes (which cost 3 operations a score).  D = 64: 0.86 causal, 0.90 on whole histories;
// there the products of both tiles take 1024 clocks, no longer than their exponentials take the special
// function units, and the chain stays as long as at D = 128.  A window of 512 keys: 0.82, since an item is 5
// tiles long and its start, masks and output run in no tile's shadow.
// Tried without gain: P V in two halves, numerators against the last tile's maximum, P beside S, 64-key
// tiles with Q in tensor memory, a third Q tile, S read in halves, output rows staged in shared memory.
#include <algorithm>
#include <climits>

#include "masked_common.cuh"
#include "prefill_common.cuh"

namespace ink {
namespace {

using namespace pf;

constexpr int PM_THREADS = 384;
constexpr int PM_KEYS = 128;      // keys per K or V tile
constexpr int PM_ITEMS = 4;       // published items in flight
constexpr int PM_BAD = 8;         // tiles whose unreadable keys are remembered
// Barriers of K and V tiles go by tile, not by slot: at most 4 tiles of a kind are in the ring, and
// every waiter waits for every tile of a kind in order, so a barrier is never a phase off.  (By slot,
// whose fills alternate between K and V and may land out of order, one who waits for V alone would
// at times see the phase before.)
constexpr int PM_TILES = 4;
constexpr int PM_REGS_SOFTMAX = 208, PM_REGS_REST = 88;   // registers a thread after the split
// Least tiles of a piece of a cut item (64 tokens of 32 + 2 x 8 heads of 128 against 2 K keys: 30.3 us with 8,
// 27.9 with 6; with 4 already 1 K keys are cut, 21.5 -> 23.9).
constexpr int PM_PIECE_TILES = 6;
constexpr float RESCALE_LOG2 = 8.f;
constexpr float CALM_LOG2 = 40.f;

template <int D>
struct PMShape {
  static constexpr int CB = D / 64;
  static constexpr int SUB = PM_KEYS * 128;        // one 64-channel block of a tile
  static constexpr int TILE = CB * SUB;            // K, V and Q tiles alike
  static constexpr int NS = D == 128 ? 5 : 8;      // ring slots, K and V tiles in turn
  static constexpr uint32_t TO = 256;              // S_h at 128 h, O_h at TO + D h
};

struct PMItem {
  int b, kvh, h0, gh;        // sequence, KV head, first query head, heads of the item
  int t0, ntok, pos0, L;     // first packed row, tokens, position of the first, length
  int lo_min, hi_max;        // keys any row sees lie in [lo_min, hi_max)
  int lo_max, hi_min;        // keys in [lo_max, hi_min) are seen by every row (ends of tiles are not added up:
                             // the last tile before 2^31 ends past the integers)
  int kt0, nt, nh, bad_len;  // first key tile, tiles (-1: no more items), row tiles
  int slot, np, one;         // of a cut item: its first place in the partials, its pieces, this one
};

enum Stretch { General, Calm, Mild, Plain };   // loops over an item's tiles

template <int D>
struct PMSmem {
  using S = PMShape<D>;
  static constexpr size_t q = 0;
  static constexpr size_t ring = 2 * (size_t)S::TILE;
  static constexpr size_t bars = ring + (size_t)S::NS * S::TILE;
  // k_full[TILES], v_full[TILES], v_ok[TILES], k_ok[TILES], empty[NS], s_full[2], p_full[2], o_full[2], q_full[2], q_empty[2],
  // item_full[ITEMS], item_empty[ITEMS], stored[2], ticket[2], drain
  static constexpr int NBAR = S::NS + 4 * PM_TILES + 14 + 2 * PM_ITEMS + 1;
  static constexpr size_t items = bars + (NBAR * 8 + 15) / 16 * 16;
  static constexpr size_t kbad = items + PM_ITEMS * sizeof(PMItem);
  static constexpr size_t poison = kbad + PM_BAD * 16;
  static constexpr size_t misc = poison + PM_ITEMS * 8;
  static constexpr size_t total = misc + 32;
  static constexpr size_t alloc = total + 1024;
  static_assert(alloc <= 227 * 1024, "shared memory budget");
};

// Bounded wait of a whole warp (inline: a call would keep the registers from being split).
__device__ __forceinline__ bool pm_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, const MaskedArgs& a) {
  bool ok = mbar_probe(bar, parity, a.wait_ns);
  if (!ok && !*abort_flag) {
    ok = mbar_wait_limit(bar, parity, a.wait_ns);
    if (!ok) {
      record_error(a.err, INK_DEVERR_WAIT_TIMEOUT);
      *a.stale = 1;   // tickets of cut items may be left over
      *abort_flag = 1;
    }
  }
  return __all_sync(0xffffffffu, ok);
}

__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// CAP: capped scores.  Models keep most scores well inside the cap: while no score of a warp's tile
// passes 0.45 of it, tanh is an odd polynomial of four terms in the raw product (relative error
// 2^-21.8; five packed operations for two scores and no special function), up to the cap one of six
// terms (2^-20.7, seven operations), else score_log2.  The choice is a warp's: its 32 rows (of one sequence) go
// one way, so the bits of a token's output can change with the tokens that share its row tile.
// SPLIT: items may be cut into pieces (a kernel of its own: the joining code would cost the others
// registers).
template <int D, bool CAP, bool SPLIT>
__global__ void __launch_bounds__(PM_THREADS, 1)
prefill_masked_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                      const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ MaskedArgs a) {
  using S = PMShape<D>;
  using L_ = PMSmem<D>;
  constexpr int NS = S::NS;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_align1024(smem_raw);
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + L_::bars);
  uint64_t* v_full = k_full + PM_TILES;
  uint64_t* v_ok = v_full + PM_TILES;   // V tile checked
  uint64_t* k_ok = v_ok + PM_TILES;     // K tile checked (capped scores)
  uint64_t* empty = k_ok + PM_TILES;
  uint64_t* s_full = empty + NS;        // [2] S_h in TMEM, every earlier product of h done
  uint64_t* p_full = s_full + 2;        // [2] P_h written
  uint64_t* o_full = p_full + 2;        // [2] the item's last O_h product done
  uint64_t* q_full = o_full + 2;        // [2]
  uint64_t* q_empty = q_full + 2;       // [2] the item's last S_h product done
  uint64_t* item_full = q_empty + 2;    // [ITEMS]
  uint64_t* item_empty = item_full + PM_ITEMS;
  uint64_t* stored = item_empty + PM_ITEMS;   // [2] a piece's part of row tile h is in the workspace
  uint64_t* ticket = stored + 2;        // [2] and its ticket is drawn
  uint64_t* drain = ticket + 2;
  PMItem* items = reinterpret_cast<PMItem*>(smem + L_::items);
  uint32_t* kbad = reinterpret_cast<uint32_t*>(smem + L_::kbad);      // [BAD][4] bit per unreadable key
  int* poison = reinterpret_cast<int*>(smem + L_::poison);   // [ITEMS][2] first and last tile of V with an infinity or NaN
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L_::misc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L_::misc + 4);
  volatile int* joins = reinterpret_cast<volatile int*>(smem + L_::misc + 8);   // [2] this piece joins its item

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int P = 1 << a.log2_page;

  if (tid == 0) {
    for (int x = 0; x < NS; ++x) mbar_init(&empty[x], 1);
    for (int x = 0; x < PM_TILES; ++x) {
      mbar_init(&k_full[x], 1);
      mbar_init(&v_full[x], 1);
      mbar_init(&v_ok[x], 1);
      mbar_init(&k_ok[x], 1);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&s_full[x], 1);
      mbar_init(&p_full[x], 4);
      mbar_init(&o_full[x], 1);
      mbar_init(&q_full[x], 1);
      mbar_init(&q_empty[x], 1);
      mbar_init(&stored[x], 4);
      mbar_init(&ticket[x], 1);
    }
    for (int x = 0; x < PM_ITEMS; ++x) {
      mbar_init(&item_full[x], 1);
      mbar_init(&item_empty[x], 11);   // producer, MMA, V check, 8 softmax warps
    }
    mbar_init(drain, 1);
    fence_mbar_init();
    *abort_flag = 0;
  }
  // rows of a Q tile past the last (token, head) pair stay zero
  for (int x = tid; x < 2 * S::TILE / 16; x += PM_THREADS)
    *reinterpret_cast<uint4*>(smem + L_::q + (size_t)x * 16) = make_uint4(0u, 0u, 0u, 0u);
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "n"(512));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // The k-th item of this CTA into `it`; false when there is none (or after a timeout).
  auto next_item = [&](int k, PMItem& it) -> bool {
    if (!pm_wait(&item_full[k % PM_ITEMS], (uint32_t)(k / PM_ITEMS) & 1u, abort_flag, a)) return false;
    it = items[k % PM_ITEMS];
    return it.nt >= 0;
  };
  auto done_item = [&](int k) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&item_empty[k % PM_ITEMS]);
  };

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(PM_REGS_REST));
    if (warp == 8) {
      // ---------------------------------------------------------------- K and V producer
      if (lane == 0) {
        prefetch_tensormap(&tmK);
        prefetch_tensormap(&tmV);
      }
      const int seg = min(P, PM_KEYS), nseg = PM_KEYS / seg;
      int chunk_base = 0, chunk_val = -1;   // table entries chunk_base + lane
      int f = 0;                            // fills issued
      bool go = true;
      PMItem it;
      for (int k = 0; go && next_item(k, it); ++k) {
        done_item(k);
        for (int j = 0; j < it.nt && go; ++j) {
          const int k0 = (it.kt0 + j) * PM_KEYS;
          const int last_idx = (it.hi_max - 1) >> a.log2_page;
          const int pfirst = k0 >> a.log2_page, plast = (k0 + PM_KEYS - 1) >> a.log2_page;
          if (j == 0 || plast >= chunk_base + 32) {
            chunk_base = pfirst;   // entries past the item's last key are not read
            chunk_val = __ldg(a.block_table + (size_t)it.b * a.max_pages + min(chunk_base + lane, last_idx));
          }
          const int ks = k0 + lane * seg;                 // lane < nseg takes one segment
          const bool want = lane < nseg && ks < it.hi_max && ks + seg > it.lo_min;
          const int page = __shfl_sync(0xffffffffu, chunk_val, min(max((ks >> a.log2_page) - chunk_base, 0), 31));
          const bool bad_seg = want && (page < 0 || page >= a.num_pages);
          const bool load = want && !bad_seg;
          const uint32_t nload = __popc(__ballot_sync(0xffffffffu, load));
          const uint32_t bmask = __ballot_sync(0xffffffffu, bad_seg);
          const int row = load ? ((page * a.Hkv + it.kvh) << a.log2_page) + (ks & (P - 1)) : 0;
#pragma unroll 1
          for (int kv = 0; kv < 2; ++kv, ++f) {
            const int st = f % NS;
            if (f >= NS && !pm_wait(&empty[st], (uint32_t)((f / NS) - 1) & 1u, abort_flag, a)) {
              go = false;
              break;
            }
            if (kv == 0 && lane < 4) {   // keys of this tile whose page is outside the pool
              uint32_t bad = 0;
              for (uint32_t mm = bmask; mm; mm &= mm - 1) {
                const int x0 = (__ffs(mm) - 1) * seg - 32 * lane, x1 = x0 + seg;   // bits [x0, x1) of this word
                const int y0 = max(x0, 0), y1 = min(x1, 32);
                if (y1 > y0) bad |= (0xffffffffu >> (32 - (y1 - y0))) << y0;
              }
              kbad[((f >> 1) % PM_BAD) * 4 + lane] = bad;
              if (bmask && lane == 0) record_error(a.err, INK_DEVERR_PAGE_OUT_OF_RANGE);
            }
            uint64_t* full = (kv ? v_full : k_full) + (f >> 1) % PM_TILES;
            __syncwarp();
            if (lane == 0) mbar_arrive_expect_tx(full, nload * (uint32_t)(seg * D * 2));
            __syncwarp();
            if (load) {
              uint8_t* dst = smem + L_::ring + (size_t)st * S::TILE + lane * seg * 128;
#pragma unroll
              for (int cb = 0; cb < S::CB; ++cb)
                tma_load_2d(dst + cb * S::SUB, kv ? &tmV : &tmK, cb * 64, row, full);
            }
          }
        }
      }
      if (lane == 0) {
        pp_drain_ring(k_full, PM_TILES, (f + 1) >> 1, a.err);
        pp_drain_ring(v_full, PM_TILES, f >> 1, a.err);
      }
    } else if (warp == 9) {
      // ---------------------------------------------------------------- MMA issue
      constexpr uint32_t IDESC_S = umma_idesc_bf16(128, PM_KEYS, false, false);
      constexpr uint32_t IDESC_PV = umma_idesc_bf16(128, D, false, true);
      const uint32_t qaddr = smem_u32(smem + L_::q), raddr = smem_u32(smem + L_::ring);
      int g = 0;                       // tiles walked: K of tile g is fill 2 g, V fill 2 g + 1
      uint32_t qn0 = 0, qn1 = 0, pn0 = 0, pn1 = 0;
      bool go = true;
      auto slot = [&](int f) { return f % NS; };
      auto wait_tile = [&](uint64_t* bars, int tile) {
        return pm_wait(&bars[tile % PM_TILES], (uint32_t)(tile / PM_TILES) & 1u, abort_flag, a);
      };
      auto issue_s = [&](int h, int f) {
        const uint64_t ad = umma_desc_sw128(qaddr + h * S::TILE, 16, 1024);
        const uint64_t bd = umma_desc_sw128(raddr + slot(f) * S::TILE, 16, 1024);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint64_t off = (uint64_t)(((kk >> 2) * S::SUB + (kk & 3) * 32) >> 4);
          umma_ss_warp(tmem + 128u * h, ad + off, bd + off, IDESC_S, kk > 0 ? 1u : 0u);
        }
      };
      auto issue_pv = [&](int h, int f, bool acc) {
        const uint64_t bd = umma_desc_sw128(raddr + slot(f) * S::TILE, S::SUB, 1024);
#pragma unroll
        for (int ks = 0; ks < PM_KEYS / 16; ++ks)
          umma_ts_warp(tmem + S::TO + (uint32_t)(D * h), tmem + 128u * h + ks * 8, bd + (uint64_t)((ks * 16 * 128) >> 4),
                       IDESC_PV, (acc || ks > 0) ? 1u : 0u);
      };
      PMItem it;
      for (int k = 0; go && next_item(k, it); ++k) {
        done_item(k);
        if (it.nt <= 0) continue;
        go = wait_tile(k_full, g) && (!CAP || wait_tile(k_ok, g));
        for (int h = 0; h < it.nh && go; ++h) {
          uint32_t& qn = h ? qn1 : qn0;
          go = pm_wait(&q_full[h], qn & 1u, abort_flag, a);
          ++qn;
          if (!go) break;
          tc_fence_after();
          issue_s(h, 2 * g);
          umma_commit_warp(&s_full[h]);
          if (it.nt == 1) umma_commit_warp(&q_empty[h]);
          __syncwarp();
        }
        if (!go) break;
        umma_commit_warp(&empty[slot(2 * g)]);
        for (int j = 0; j < it.nt && go; ++j, ++g) {
          const int vf = 2 * g + 1, kf = 2 * g + 2;
          const bool more = j + 1 < it.nt;
          go = wait_tile(v_full, g) && wait_tile(v_ok, g);
          for (int h = 0; h < it.nh && go; ++h) {
            uint32_t& pn = h ? pn1 : pn0;
            go = pm_wait(&p_full[h], pn & 1u, abort_flag, a);
            ++pn;
            if (!go) break;
            tc_fence_after();
            issue_pv(h, vf, j > 0);
            if (more) {
              if (h == 0) go = wait_tile(k_full, g + 1) && (!CAP || wait_tile(k_ok, g + 1));
              if (!go) break;
              issue_s(h, kf);
              umma_commit_warp(&s_full[h]);
              if (j + 2 == it.nt) umma_commit_warp(&q_empty[h]);
            } else {
              umma_commit_warp(&o_full[h]);
            }
            __syncwarp();
          }
          if (!go) break;
          umma_commit_warp(&empty[slot(vf)]);
          if (more) umma_commit_warp(&empty[slot(kf)]);
          __syncwarp();
        }
      }
      umma_commit_warp(drain);
      __syncwarp();
      if (!mbar_wait_bounded(drain, 0)) record_error(a.err, INK_DEVERR_WAIT_TIMEOUT);
    } else if (warp == 10) {
      // ---------------------------------------------------------------- scheduler and Q loads
      if (lane == 0) prefetch_tensormap(&tmQ);
      const int per = a.Hkv * a.head_chunks, tpi = 2 * a.tok_per_tile;
      int cb = 0, base = 0, cnt = 0, incl = 0, total = 0;
      int my_c0 = 0, my_n = 0, my_len = 0;   // of this lane's sequence
      int piece_tiles = INT_MAX, my_np = 1;  // tiles of a piece, pieces of an item of this lane's sequence
      // most tiles of an item of a sequence of length len
      auto tiles_of = [&](int len) {
        const long long keys = min(max((long long)len, 1ll), (long long)a.max_pages << a.log2_page);
        int t = (int)((keys + PM_KEYS - 1) / PM_KEYS);
        if (a.W > 0 && !a.key_end) t = min(t, (int)(((uint32_t)a.W + tpi) / PM_KEYS) + 2);
        return t;
      };
      auto load_chunk = [&]() {   // pieces of sequences cb + lane
        const int b = cb + lane;
        cnt = my_len = 0;
        if (b < a.B) {
          const int c0 = __ldg(a.cu_q + b), c1 = __ldg(a.cu_q + b + 1);
          my_len = __ldg(a.seq_lens + b);
          my_c0 = c0;
          my_n = c1 - c0;
          if (c0 < 0 || c1 > a.T || c1 < c0) {
            if (blockIdx.x == 0) record_error(a.err, INK_DEVERR_BAD_ROWS);
          } else {
            cnt = (c1 - c0 + tpi - 1) / tpi * per;
            if constexpr (SPLIT) {
              my_np = piece_tiles == INT_MAX ? 1 : (tiles_of(my_len) + piece_tiles - 1) / piece_tiles;
              cnt *= my_np;
            }
          }
        }
        incl = cnt;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int v = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += v;
        }
        total = __shfl_sync(0xffffffffu, incl, 31);
      };
      load_chunk();
      if constexpr (SPLIT) {
        // Lane i tries pieces of 1 / (i + 1) and 2 / (2 i + 3) of the longest item.  The cost in eighths of a
        // tile, with 5 tiles for a piece's partials: the longest piece, or the rounds over the SMs (with a
        // sixteenth to spare: CTAs that join are late for their next piece) times the mean one; and the last
        // join, 1.2 tiles per piece of an item.
        const uint32_t stale = *reinterpret_cast<volatile uint32_t*>(a.stale);
        int longest = 0;
        for (int c = 0;;) {
          longest = max(longest, cnt > 0 ? tiles_of(my_len) : 0);
          c += 32;
          if (c >= a.B) break;
          cb = c;
          load_chunk();
        }
        longest = __reduce_max_sync(0xffffffffu, longest);
        int mine[2], pieces[2] = {0, 0}, top[2] = {0, 0};
        for (int y = 0; y < 2; ++y) mine[y] = max(PM_PIECE_TILES, (2 * longest - 1) / (2 * lane + 2 + y) + 1);
        long long tiles = 0;
        for (int c = 0; c < a.B; c += 32) {
          if (cb != c) {
            cb = c;
            load_chunk();
          }
          const int t = tiles_of(my_len);
          for (int x = 0; x < min(32, a.B - c); ++x) {
            const int n = __shfl_sync(0xffffffffu, cnt, x), tx = __shfl_sync(0xffffffffu, t, x);
            if (n == 0) continue;
            for (int y = 0; y < 2; ++y) {
              const int np = (tx + mine[y] - 1) / mine[y];
              pieces[y] += n * np;
              top[y] = max(top[y], (tx + np - 1) / np);
            }
            tiles += (long long)n * tx;
          }
        }
        const int sms = (int)gridDim.x;
        uint32_t cost = 0xffffffffu;
        for (int y = 0; y < 2; ++y) {
          const int rounds = pieces[y] <= sms ? 1 : (pieces[y] + pieces[y] / 16 + sms - 1) / sms;
          const long long c8 = max((long long)8 * top[y] + 40, rounds * (8 * tiles / max(pieces[y], 1) + 40)) +
                               10 * (longest / mine[y]);
          if (pieces[y] <= MASKED_PIECES) cost = min(cost, (uint32_t)min(c8, 0x1ffffffll) << 6 | (uint32_t)(2 * lane + y));
        }
        const uint32_t best = __reduce_min_sync(0xffffffffu, cost);
        const int won = __shfl_sync(0xffffffffu, best & 1 ? mine[1] : mine[0], (int)((best & 63u) >> 1));
        if (best != 0xffffffffu) piece_tiles = won;
        cb = stale ? a.B : 0;
        if (cb < a.B) load_chunk();
        if (stale && lane == 0) record_error(a.err, INK_DEVERR_WAIT_TIMEOUT);   // left unusable by a timeout
      }
      int idx = blockIdx.x, qn0 = 0, qn1 = 0;
      for (int k = 0;;) {
        int next = 0;
        if (lane == 0) next = (int)atomicAdd(a.counters, 1u) + (int)gridDim.x;
        while (cb < a.B && idx >= base + total) {
          base += total;
          cb += 32;
          if (cb < a.B) load_chunk();
        }
        const int sl = k % PM_ITEMS;
        if (k >= PM_ITEMS && !pm_wait(&item_empty[sl], (uint32_t)((k / PM_ITEMS) - 1) & 1u, abort_flag, a)) break;
        if (cb >= a.B) {
          if (lane == 0) {
            items[sl].nt = -1;
            mbar_arrive(&item_full[sl]);
          }
          break;
        }
        const int src = __ffs(__ballot_sync(0xffffffffu, idx < base + incl)) - 1;
        int li = idx - base - __shfl_sync(0xffffffffu, incl - cnt, src);   // piece, then item of the sequence
        int nq = __shfl_sync(0xffffffffu, cnt, src) / per, one = 0;
        if constexpr (SPLIT) {
          const int np = __shfl_sync(0xffffffffu, my_np, src);
          one = li % np;
          li /= np;
          nq /= np;
        }
        PMItem it;
        it.b = cb + src;
        const int qrev = li / per, r = li - qrev * per;
        const int qt = nq - 1 - qrev;
        it.kvh = r / a.head_chunks;
        const int hc = r - it.kvh * a.head_chunks;
        it.h0 = it.kvh * a.G + hc * a.heads_per_tile;
        it.gh = min(a.heads_per_tile, a.G - hc * a.heads_per_tile);
        const int c0 = __shfl_sync(0xffffffffu, my_c0, src), n = __shfl_sync(0xffffffffu, my_n, src);
        it.L = __shfl_sync(0xffffffffu, my_len, src);
        it.t0 = c0 + qt * tpi;
        it.ntok = min(tpi, n - qt * tpi);
        it.pos0 = it.L - n + qt * tpi;
        it.nh = it.ntok > a.tok_per_tile ? 2 : 1;
        it.bad_len = n > it.L;
        it.lo_min = INT_MAX;
        it.hi_max = 0;
        it.lo_max = 0;
        it.hi_min = INT_MAX;
        if (!it.bad_len) {
          for (int i = lane; i < it.ntok; i += 32) {
            int lo, hi;
            token_keys(a, it.t0 + i, it.pos0 + i, it.L, lo, hi);
            if (lo < hi) {
              it.lo_min = min(it.lo_min, lo);
              it.hi_max = max(it.hi_max, hi);
              it.lo_max = max(it.lo_max, lo);
              it.hi_min = min(it.hi_min, hi);
            } else {
              it.lo_max = INT_MAX;
            }
          }
          it.lo_min = __reduce_min_sync(0xffffffffu, it.lo_min);
          it.hi_max = __reduce_max_sync(0xffffffffu, it.hi_max);
          it.lo_max = __reduce_max_sync(0xffffffffu, it.lo_max);
          it.hi_min = __reduce_min_sync(0xffffffffu, it.hi_min);
        }
        it.kt0 = it.lo_min / PM_KEYS;
        it.nt = it.hi_max > it.lo_min ? (it.hi_max - 1) / PM_KEYS - it.kt0 + 1 : 0;
        it.np = 1;
        if constexpr (SPLIT) {
          it.np = max(1, (it.nt - 1) / piece_tiles + 1);
          const int len = (it.nt + it.np - 1) / it.np;
          it.slot = idx - one;
          it.one = one;
          if (it.np > 1) {
            it.kt0 += one * len;
            it.nt = min(len, it.nt - one * len);
          }
          if (one >= it.np) {   // no such piece
            idx = __shfl_sync(0xffffffffu, next, 0);
            continue;
          }
        }
        if (lane == 0) {
          if (it.bad_len) record_error(a.err, INK_DEVERR_QLEN_EXCEEDS_KV);
          else if ((long long)it.L > ((long long)a.max_pages << a.log2_page)) record_error(a.err, INK_DEVERR_PAGE_OUT_OF_RANGE);
          items[sl] = it;
          reinterpret_cast<volatile int*>(poison)[2 * sl] = INT_MAX;
          reinterpret_cast<volatile int*>(poison)[2 * sl + 1] = -1;
          mbar_arrive(&item_full[sl]);
        }
        __syncwarp();
        bool go = true;
        for (int h = 0; h < it.nh && it.nt > 0 && go; ++h) {
          int& qn = h ? qn1 : qn0;
          if (qn > 0) go = pm_wait(&q_empty[h], (uint32_t)(qn - 1) & 1u, abort_flag, a);
          if (!go) break;
          ++qn;
          if (lane == 0) {
            mbar_arrive_expect_tx(&q_full[h], (uint32_t)(S::CB * a.heads_per_tile * a.tok_per_tile * 128));
#pragma unroll
            for (int c = 0; c < S::CB; ++c)
              tma_load_3d(smem + L_::q + h * S::TILE + c * S::SUB, &tmQ, c * 64, it.h0, it.t0 + h * a.tok_per_tile,
                          &q_full[h]);
          }
          __syncwarp();
        }
        if (!go) break;
        idx = __shfl_sync(0xffffffffu, next, 0);
        ++k;
      }
      if (lane == 0) {
        for (int h = 0; h < 2; ++h) {
          const int n = h ? qn1 : qn0;
          if (n > 0 && !mbar_wait_bounded(&q_full[h], (uint32_t)(n - 1) & 1u)) record_error(a.err, INK_DEVERR_WAIT_TIMEOUT);
        }
        // the last CTA to stop taking items leaves the counters at zero for the next call
        __threadfence();
        if (atomicAdd(a.counters + 1, 1u) == gridDim.x - 1) {
          a.counters[0] = 0u;
          a.counters[1] = 0u;
        }
      }
    } else {
      // ---------------------------------------------------------------- V check
      int g = 0;
      bool go = true;
      PMItem it;
      for (int k = 0; go && next_item(k, it); ++k) {
        for (int j = 0; j < it.nt; ++j, ++g) {
          const int st = (2 * g + 1) % NS;
          if constexpr (CAP) {
            // Rows of K that nobody sees are zeroed: how scores are capped goes by the largest score of a
            // tile, which must not hang on what lies in a slot or a page by chance.
            go = pm_wait(&k_full[g % PM_TILES], (uint32_t)(g / PM_TILES) & 1u, abort_flag, a);
            if (!go) break;
            const int kb = (it.kt0 + j) * PM_KEYS;
            const uint4 kw = *reinterpret_cast<const uint4*>(kbad + (g % PM_BAD) * 4);
            if (kb < it.lo_min || it.hi_max - kb < PM_KEYS || (kw.x | kw.y | kw.z | kw.w)) {
              const uint32_t kbw[4] = {kw.x, kw.y, kw.z, kw.w};
              uint8_t* kt = smem + L_::ring + (size_t)((2 * g) % NS) * S::TILE;
#pragma unroll 1
              for (int x = 0; x < 4; ++x) {
                const int kk = kb + 32 * x + lane;
                if (kk >= it.lo_min && kk < it.hi_max && !((kbw[x] >> lane) & 1u)) continue;
                uint4* row = reinterpret_cast<uint4*>(kt + (32 * x + lane) * 128);
#pragma unroll
                for (int c = 0; c < S::CB; ++c)
#pragma unroll
                  for (int y = 0; y < 8; ++y) row[c * (S::SUB / 16) + (y ^ (lane & 7))] = make_uint4(0u, 0u, 0u, 0u);
              }
              asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&k_ok[g % PM_TILES]);
          }
          go = pm_wait(&v_full[g % PM_TILES], (uint32_t)(g / PM_TILES) & 1u, abort_flag, a);
          if (!go) break;
          const int k0 = (it.kt0 + j) * PM_KEYS;
          const uint4 bad = *reinterpret_cast<const uint4*>(kbad + (g % PM_BAD) * 4);
          if (k0 < it.lo_max || it.hi_min - k0 < PM_KEYS || (bad.x | bad.y | bad.z | bad.w)) {
            const uint32_t badw[4] = {bad.x, bad.y, bad.z, bad.w};
            uint8_t* vt = smem + L_::ring + (size_t)st * S::TILE;
            bool found = false;
#pragma unroll 1
            for (int x = 0; x < 4; ++x) {
              const int kk = k0 + 32 * x + lane;
              uint4* row = reinterpret_cast<uint4*>(vt + (32 * x + lane) * 128);
              const bool zero = kk < it.lo_min || kk >= it.hi_max || ((badw[x] >> lane) & 1u);
              if (!zero) {   // exponents all ones carry into the sign places
                uint32_t odd = 0;
#pragma unroll
                for (int c = 0; c < S::CB; ++c)
#pragma unroll
                  for (int y = 0; y < 8; ++y) {
                    const uint4 w = row[c * (S::SUB / 16) + (y ^ (lane & 7))];
                    odd |= ((w.x & 0x7F807F80u) + 0x00800080u) | ((w.y & 0x7F807F80u) + 0x00800080u) |
                           ((w.z & 0x7F807F80u) + 0x00800080u) | ((w.w & 0x7F807F80u) + 0x00800080u);
                  }
                if (odd & 0x80008000u) {
                  found = true;
                  auto finite = [](uint32_t w) {   // infinities and NaN to zero, the other half as it is
                    return w & ~(((((w & 0x7F807F80u) + 0x00800080u) >> 15) & 0x00010001u) * 0xFFFFu);
                  };
#pragma unroll 1
                  for (int y = 0; y < 8 * S::CB; ++y) {
                    uint4& w = row[(y >> 3) * (S::SUB / 16) + ((y & 7) ^ (lane & 7))];
                    w = make_uint4(finite(w.x), finite(w.y), finite(w.z), finite(w.w));
                  }
                }
              } else {
#pragma unroll
                for (int c = 0; c < S::CB; ++c)
#pragma unroll
                  for (int y = 0; y < 8; ++y) row[c * (S::SUB / 16) + (y ^ (lane & 7))] = make_uint4(0u, 0u, 0u, 0u);
              }
            }
            if (found) {
              atomicMin(poison + 2 * (k % PM_ITEMS), it.kt0 + j);
              atomicMax(poison + 2 * (k % PM_ITEMS) + 1, it.kt0 + j);
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&v_ok[g % PM_TILES]);
        }
        done_item(k);
      }
    }
  } else {
    // ------------------------------------------------------------------ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(PM_REGS_SOFTMAX));
    const int h = warp >> 2, r = tid & 127;
    const uint32_t tlane = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t tm_s = tlane + 128u * h, tm_o = tlane + S::TO + (uint32_t)(D * h);
    const int my_i = r / a.heads_per_tile, my_g = r - my_i * a.heads_per_tile;
    __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(a.out);
    const bool scaled = CAP || a.slopes != nullptr || !(a.scale_log2 > 0.f);
    const float mul = scaled ? 1.f : a.scale_log2;
    // The largest magnitude of a tile, which decides how its scores are capped, bounds them from above
    // and below.  As long as it is small (|s| <= 40 in log2 units) in every row of a warp, no maximum is looked
    // for: the numerators are taken against 0 and lie within [2^-40, 2^40], far inside bf16's range (sums
    // of 2^17 of them times V overflow past |V| = 2^70).  2 sequences of 5,000 tokens, 64 + 2 x 8 heads of
    // 128, cap 50: 886 us with every tile's maximum, 760 without.  A tile with larger scores goes the general
    // way, whose maximum leaves 0 only when it has to.  Not with slopes, whose scores have no lower bound,
    // nor for an item of one tile, whose rows see few keys: against its maximum a row's largest numerator
    // is 1, which bf16 holds exactly.  (Against 0 it is rounded; a row of one key divides by what was
    // rounded.)
    const float reach = CAP && a.slopes == nullptr ? fminf(a.cap_mid, CALM_LOG2 / fabsf(a.scale_log2)) : -1.f;
    uint32_t sn = 0, on = 0, jn = 0;
    int g = 0;
    bool go = true;
    for (int k = 0; go; ++k) {
      // (read where it is needed, from shared memory: the tile loop has no registers to spare)
      const PMItem& it = items[k % PM_ITEMS];
      if (!pm_wait(&item_full[k % PM_ITEMS], (uint32_t)(k / PM_ITEMS) & 1u, abort_flag, a) || it.nt < 0) break;
      const int nt = it.nt, kt0 = it.kt0, lo_max = it.lo_max, hi_min = it.hi_min;
      if (h >= it.nh) {
        g += nt;
        done_item(k);
        continue;
      }
      const int ti = h * a.tok_per_tile + my_i;
      const bool rv = my_i < a.tok_per_tile && ti < it.ntok && my_g < it.gh;
      const int t = it.t0 + (rv ? ti : 0), head = it.h0 + (rv ? my_g : 0), p = it.pos0 + ti;
      int lo = 0, hi = 0;
      if (rv && !it.bad_len) token_keys(a, t, p, it.L, lo, hi);
      const size_t orow = (size_t)t * a.Hq + head;
      if (nt == 0) {   // no row sees a key
        if (rv) {
          uint4* o = reinterpret_cast<uint4*>(out + orow * D);
#pragma unroll
          for (int c = 0; c < D / 8; ++c) o[c] = make_uint4(0u, 0u, 0u, 0u);
          if (a.lse) a.lse[orow] = -INFINITY;
        }
        done_item(k);
        continue;
      }
      const float slope2 = a.slopes ? __ldg(a.slopes + head) * LOG2E : 0.f;
      // the largest magnitudes that need no maximum, for the short polynomial and for the longer one
      const float mild = nt > 1 ? reach : -1.f, calm = fminf(mild, a.cap_near);
      float m = mild >= 0.f ? 0.f : -INFINITY, l = 0.f;
      int j = 0;
      bool waited = false;   // for S of tile j
      // From tile j on: in a calm or mild stretch until a tile that is none (its scores are read again), in a
      // mild one to a calm tile; one tile between two such stretches; else to the end.
      // Scores that are neither capped nor shifted have a loop of their own at D = 128 (window of 512 keys,
      // 7,949 tokens: 159 -> 155 us, whole history: 778 -> 763); at D = 64 two loops are slower than one (494 ->
      // 507 us).
      auto tiles = [&](auto stretch) {
        constexpr Stretch ST = decltype(stretch)::value;
        constexpr bool CALM = ST == Calm || ST == Mild, PLAIN = ST == Plain;
        for (; j < nt; ++j, ++g) {
          const int k0 = (kt0 + j) * PM_KEYS;
          if (!waited) {
            go = pm_wait(&s_full[h], sn & 1u, abort_flag, a);
            if (!go) return;
            ++sn;
            tc_fence_after();
          }
          waited = false;
          uint32_t sr[128];
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32(tm_s + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(&sr[32 * c]));
          tmem_wait_ld();
          const uint4 bad = *reinterpret_cast<const uint4*>(kbad + (g % PM_BAD) * 4);
          bool over = false;   // a mild stretch has come to a calm tile
          // ---- scores
          if constexpr (CAP) {
            float fv[4] = {0.f, 0.f, 0.f, 0.f};   // largest |<q, K[k]>| of the tile
#pragma unroll
            for (int c = 0; c < 128; c += 2)
              fv[(c >> 1) & 3] = fmax3(fv[(c >> 1) & 3], fabsf(__uint_as_float(sr[c])), fabsf(__uint_as_float(sr[c + 1])));
            // (rows of other sequences have no say)
            const float far = rv ? fmaxf(fmax3(fv[0], fv[1], fv[2]), fv[3]) : 0.f;
            auto polynomial = [&](auto terms) {
              constexpr int TERMS = decltype(terms)::value;
              uint64_t co[TERMS];
#pragma unroll
              for (int i = 0; i < TERMS; ++i) {
                const float f = TERMS == NEAR_TERMS ? a.near[i] : a.mid[i];
                co[i] = f2_pack(f, f);
              }
#pragma unroll
              for (int c = 0; c < 128; c += 2) {
                const uint64_t x = f2_pack(__uint_as_float(sr[c]), __uint_as_float(sr[c + 1]));
                const uint64_t u = f2_mul(x, x);
                uint64_t t = co[TERMS - 1];
#pragma unroll
                for (int i = TERMS - 2; i >= 0; --i) t = f2_fma(t, u, co[i]);
                float s0, s1;
                f2_unpack(f2_mul(t, x), s0, s1);
                sr[c] = __float_as_uint(s0);
                sr[c + 1] = __float_as_uint(s1);
              }
            };
            auto within = [&](float reach) { return __all_sync(0xffffffffu, far <= reach); };
            if constexpr (CALM) {
              if (!within(ST == Calm ? calm : mild)) {
                waited = true;
                return;
              }
              over = ST == Mild && within(calm);
              polynomial(std::integral_constant<int, ST == Calm ? NEAR_TERMS : MID_TERMS>{});
            } else if (within(a.cap_near)) {
              polynomial(std::integral_constant<int, NEAR_TERMS>{});
            } else if (within(a.cap_mid)) {
              polynomial(std::integral_constant<int, MID_TERMS>{});
            } else {
#pragma unroll
              for (int c = 0; c < 128; ++c) sr[c] = __float_as_uint(score_log2<true>(a, __uint_as_float(sr[c])));
            }
          } else if (!PLAIN && scaled) {
#pragma unroll
            for (int c = 0; c < 128; ++c) sr[c] = __float_as_uint(__uint_as_float(sr[c]) * a.scale_log2);
          }
          if (!CALM && !PLAIN && a.slopes) {
            const float d0 = (float)(p - k0);
#pragma unroll
            for (int c = 0; c < 128; ++c)
              sr[c] = __float_as_uint(fmaf(-slope2, fabsf(d0 - (float)c), __uint_as_float(sr[c])));
          }
          // ---- keys that this row does not see
          if (k0 < lo_max || hi_min - k0 < PM_KEYS || (bad.x | bad.y | bad.z | bad.w)) {
            const uint32_t badw[4] = {bad.x, bad.y, bad.z, bad.w};
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const int x0 = max(lo - k0 - 32 * w, 0), x1 = min(hi - k0 - 32 * w, 32);   // visible bits [x0, x1)
              uint32_t vis = x1 > x0 ? (0xffffffffu >> (32 - (x1 - x0))) << x0 : 0u;
              vis &= ~badw[w];
#pragma unroll
              for (int c = 0; c < 32; ++c)
                if (!((vis >> c) & 1u)) sr[32 * w + c] = 0xff800000u;   // -infinity
            }
          }
          // ---- running maximum
          if constexpr (!CALM) {
            float mxv[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int c = 0; c < 128; c += 2)
              mxv[(c >> 1) & 3] = fmax3(mxv[(c >> 1) & 3], __uint_as_float(sr[c]), __uint_as_float(sr[c + 1]));
            const float mx = fmaxf(fmaxf(mxv[0], mxv[1]), fmaxf(mxv[2], mxv[3])) * mul;
            const bool mine = mx > m + (mild >= 0.f ? CALM_LOG2 : RESCALE_LOG2);
            const float to = mild >= 0.f && fabsf(mx) <= CALM_LOG2 ? 0.f : mx;   // (back to 0 where that will do)
            if (__any_sync(0xffffffffu, mine)) {
              if (j > 0) {   // every earlier product into O_h is done: s_full came after it
                const float fr = mine ? fast_exp2(m - to) : 1.f;
#pragma unroll 1
                for (int c2 = 0; c2 < D / 16; ++c2) {
                  uint32_t ov[16];
                  tmem_ld16(tm_o + c2 * 16, ov);
                  tmem_wait_ld();
#pragma unroll
                  for (int x = 0; x < 16; ++x) ov[x] = __float_as_uint(__uint_as_float(ov[x]) * fr);
                  tmem_st16(tm_o + c2 * 16, ov);
                }
                l *= fr;
              }
              if (mine) m = to;
            }
          }
          // ---- numerators
          const float nm = m == -INFINITY ? 0.f : -m;
          const uint64_t mul2 = f2_pack(mul, mul), nm2 = f2_pack(nm, nm);
          uint64_t ls2[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
          for (int quarter = 0; quarter < 4; ++quarter) {
            uint32_t pk[16];
#pragma unroll
            for (int c = 0; c < 16; ++c) {
              const int e = 32 * quarter + 2 * c;
              float t0 = __uint_as_float(sr[e]), t1 = __uint_as_float(sr[e + 1]);
              if constexpr (!CALM) f2_unpack(f2_fma(f2_pack(t0, t1), mul2, nm2), t0, t1);
              const float p0 = fast_exp2(t0), p1 = fast_exp2(t1);
              ls2[c & 3] = f2_add(ls2[c & 3], f2_pack(p0, p1));
              pk[c] = pack_bf16(p0, p1);
            }
            tmem_st16(tm_s + 16 * quarter, pk);
          }
          {
            float x0, x1, y0, y1;
            f2_unpack(f2_add(ls2[0], ls2[1]), x0, x1);
            f2_unpack(f2_add(ls2[2], ls2[3]), y0, y1);
            l += (x0 + y0) + (x1 + y1);
          }
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[h]);
          if (over || (CAP && !CALM && mild >= 0.f)) {
            ++j, ++g;
            return;
          }
        }
      };
      if (CAP) {
        bool rough = false;   // the tile before was neither calm nor mild
        while (go && j < nt) {
          if (mild >= 0.f && __all_sync(0xffffffffu, m == 0.f || l == 0.f)) {
            m = 0.f;
            if (!rough) tiles(std::integral_constant<Stretch, Calm>{});
            if (go && j < nt) tiles(std::integral_constant<Stretch, Mild>{});
            rough = waited;
            if (!rough) continue;
            if (l == 0.f) m = -INFINITY;   // no key seen yet: any maximum will do
          }
          if (go && j < nt) tiles(std::integral_constant<Stretch, General>{});
        }
      } else if (D == 64 || scaled) {
        tiles(std::integral_constant<Stretch, General>{});
      } else {
        tiles(std::integral_constant<Stretch, Plain>{});
      }
      if (!go) break;
      // ---- epilogue
      go = pm_wait(&o_full[h], on & 1u, abort_flag, a);
      if (!go) break;
      ++on;
      tc_fence_after();
      int pfirst = reinterpret_cast<volatile int*>(poison)[2 * (k % PM_ITEMS)];
      int plast = reinterpret_cast<volatile int*>(poison)[2 * (k % PM_ITEMS) + 1];
      // a piece of a cut item: its part into the workspace; who is last goes on with the joined row
      float4* part_o = reinterpret_cast<float4*>(a.part_o) + (size_t)(it.slot * 2 + h) * (D / 4) * MASKED_ROWS + r;
      float4* part_ml = reinterpret_cast<float4*>(a.part_ml) + (size_t)(it.slot * 2 + h) * MASKED_ROWS + r;
      constexpr size_t PART = (size_t)2 * (D / 4) * MASKED_ROWS;   // from one piece to the next
      // the row that this thread finishes, and its blocks of 32 channels
      bool wv = rv;
      size_t wrow = orow;
      int wlo = lo, whi = hi, cfirst = 0, cstep = 1;
      if (SPLIT && it.np > 1) {
#pragma unroll 1
        for (int c2 = 0; c2 < D / 32; ++c2) {
          uint32_t ov[32];
          tmem_ld32(tm_o + c2 * 32, ov);
          tmem_wait_ld();
#pragma unroll
          for (int x = 0; x < 8 && rv; ++x)
            __stcg(part_o + it.one * PART + (size_t)(c2 * 8 + x) * MASKED_ROWS,
                   make_float4(__uint_as_float(ov[4 * x]), __uint_as_float(ov[4 * x + 1]), __uint_as_float(ov[4 * x + 2]),
                               __uint_as_float(ov[4 * x + 3])));
        }
        __stcg(part_ml + (size_t)it.one * 2 * MASKED_ROWS, make_float4(l == 0.f ? -INFINITY : m, l, __int_as_float(pfirst), __int_as_float(plast)));
        tc_fence_before();
        // Every thread's stores come before its warp's arrival, the ticket's add releases them and acquires
        // the other pieces'.  (Barriers whose waits are bounded: after a timeout a warp may be gone.)
        __syncwarp();
        if (lane == 0) mbar_arrive(&stored[h]);
        if ((warp & 3) == 0) {
          go = pm_wait(&stored[h], jn & 1u, abort_flag, a);
          if (!go) break;
          if (lane == 0) {
            int prev;
            asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;"
                         : "=r"(prev)
                         : "l"(a.tickets + 2 * it.slot + h)
                         : "memory");
            joins[h] = prev == it.np - 1;
            if (prev == it.np - 1) a.tickets[2 * it.slot + h] = 0;   // ready for the next call
            mbar_arrive(&ticket[h]);
          }
          __syncwarp();
        }
        go = pm_wait(&ticket[h], jn & 1u, abort_flag, a);
        if (!go) break;
        ++jn;
        if (!joins[h]) {
          done_item(k);
          continue;
        }
        // rows past the last token are idle: the rest of the threads take other blocks of the rows there are
        const int rows = min(a.tok_per_tile, it.ntok - h * a.tok_per_tile) * a.heads_per_tile;
        cstep = min(MASKED_ROWS / rows, D / 32);
        cfirst = r / rows;
        const int row = r - cfirst * rows, wi = row / a.heads_per_tile, wg = row - wi * a.heads_per_tile;
        const int wt = h * a.tok_per_tile + wi;
        wv = cfirst < cstep && wg < it.gh;
        wrow = (size_t)(it.t0 + wt) * a.Hq + it.h0 + wg;
        if (wv) token_keys(a, it.t0 + wt, it.pos0 + wt, it.L, wlo, whi);
        part_o += row - r;
        part_ml += row - r;
        m = -INFINITY;
#pragma unroll 4
        for (int x = 0; x < it.np; ++x) m = fmaxf(m, __ldcg(part_ml + (size_t)x * 2 * MASKED_ROWS).x);
        l = 0.f;
#pragma unroll 4
        for (int x = 0; x < it.np; ++x) {
          const float4 ml = __ldcg(part_ml + (size_t)x * 2 * MASKED_ROWS);
          l += ml.y * (ml.x == -INFINITY ? 0.f : fast_exp2(ml.x - m));
          pfirst = min(pfirst, __float_as_int(ml.z));
          plast = max(plast, __float_as_int(ml.w));
        }
      }
      // (a row of one key: the numerator that V was multiplied by was rounded, so that it drops out)
      const float inv = l > 0.f ? 1.f / (whi - wlo == 1 ? __bfloat162float(__float2bfloat16(l)) : l) : 0.f;
      const bool nothing = l == 0.f;
#pragma unroll 1
      for (int c2 = cfirst; c2 < D / 32; c2 += cstep) {
        uint32_t ov[32];
        if (SPLIT && it.np > 1) {
          float acc[32];
#pragma unroll
          for (int x = 0; x < 32; ++x) acc[x] = 0.f;
          // (four pieces at a time: 36 loads in flight a thread)
#pragma unroll 4
          for (int y = 0; y < (wv ? it.np : 0); ++y) {
            const float my = __ldcg(part_ml + (size_t)y * 2 * MASKED_ROWS).x;
            float4 vv[8];
#pragma unroll
            for (int x = 0; x < 8; ++x) vv[x] = __ldcg(part_o + y * PART + (size_t)(c2 * 8 + x) * MASKED_ROWS);
            const float w = my == -INFINITY ? 0.f : fast_exp2(my - m);
#pragma unroll
            for (int x = 0; x < 8; ++x) {
              const float4 v = vv[x];
              acc[4 * x] = fmaf(w, v.x, acc[4 * x]);
              acc[4 * x + 1] = fmaf(w, v.y, acc[4 * x + 1]);
              acc[4 * x + 2] = fmaf(w, v.z, acc[4 * x + 2]);
              acc[4 * x + 3] = fmaf(w, v.w, acc[4 * x + 3]);
            }
          }
#pragma unroll
          for (int x = 0; x < 32; ++x) ov[x] = __float_as_uint(acc[x]);
        } else {
          tmem_ld32(tm_o + c2 * 32, ov);
          tmem_wait_ld();
        }
#pragma unroll
        for (int x = 0; x < 32; ++x) ov[x] = nothing ? 0u : __float_as_uint(__uint_as_float(ov[x]) * (l == l ? inv : l));
        if (plast >= 0 && wv) {
          // infinities and NaN of the keys this row sees (key by key, but from the first tile to the last that
          // holds one: over a whole history of a million keys that took as long as a wait may)
          const int kend = min(whi - 1, plast * PM_KEYS + PM_KEYS - 1);
#pragma unroll 1
          for (int kk = max(wlo, pfirst * PM_KEYS); kk <= kend; ++kk) {
            const int page = __ldg(a.block_table + (size_t)it.b * a.max_pages + (kk >> a.log2_page));
            if (page < 0 || page >= a.num_pages) continue;
            const size_t vrow = ((((size_t)page * a.Hkv + it.kvh) << a.log2_page) + (kk & (P - 1))) * D + c2 * 32;
            const uint16_t* vp = static_cast<const uint16_t*>(a.v) + vrow;
#pragma unroll
            for (int x = 0; x < 32; ++x) {
              const uint32_t w = (uint32_t)__ldg(vp + x) << 16;
              if ((w & 0x7F800000u) == 0x7F800000u) ov[x] = __float_as_uint(__uint_as_float(ov[x]) + __uint_as_float(w));
            }
          }
        }
        if (wv) {
          uint4* o = reinterpret_cast<uint4*>(out + wrow * D) + c2 * 4;
#pragma unroll
          for (int q8 = 0; q8 < 2; ++q8) {
            uint32_t w[8];
#pragma unroll
            for (int x = 0; x < 8; ++x)
              w[x] = pack_bf16(__uint_as_float(ov[16 * q8 + 2 * x]), __uint_as_float(ov[16 * q8 + 2 * x + 1]));
            if (a.io32) {
              asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(o + 2 * q8), "r"(w[0]), "r"(w[1]),
                           "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                           : "memory");
            } else {
              o[2 * q8] = make_uint4(w[0], w[1], w[2], w[3]);
              o[2 * q8 + 1] = make_uint4(w[4], w[5], w[6], w[7]);
            }
          }
        }
      }
      if (wv && cfirst == 0 && a.lse) a.lse[wrow] = nothing ? -INFINITY : (m == -INFINITY ? 0.f : m) * LN2 + logf(l);
      tc_fence_before();
      done_item(k);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(512));
  }
}

template <int D, bool CAP, bool SPLIT>
cudaError_t launch_t(const MaskedMaps& m, const MaskedArgs& a, int grid, cudaStream_t stream) {
  static std::atomic<unsigned long long> opted{0};
  cudaError_t e = smem_opt_in_once(prefill_masked_kernel<D, CAP, SPLIT>, (int)PMSmem<D>::alloc, opted);
  if (e != cudaSuccess) return e;
  // The softmax warps' extra registers come out of what the block is launched with: a build with
  // fewer would wait for them without end.
  static const bool enough = [] {
    cudaFuncAttributes at;
    return cudaFuncGetAttributes(&at, prefill_masked_kernel<D, CAP, SPLIT>) == cudaSuccess &&
           at.numRegs * PM_THREADS >= 128 * (2 * PM_REGS_SOFTMAX + PM_REGS_REST);
  }();
  if (!enough) return cudaErrorInvalidConfiguration;
  prefill_masked_kernel<D, CAP, SPLIT><<<grid, PM_THREADS, PMSmem<D>::alloc, stream>>>(m.k, m.v, m.q, a);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_d(const MaskedMaps& m, const MaskedArgs& a, int grid, bool split, cudaStream_t stream) {
  if (a.softcap == 0.f) return split ? launch_t<D, false, true>(m, a, grid, stream) : launch_t<D, false, false>(m, a, grid, stream);
  return split ? launch_t<D, true, true>(m, a, grid, stream) : launch_t<D, true, false>(m, a, grid, stream);
}

}  // namespace

cudaError_t launch_prefill_masked(const MaskedMaps& m, const MaskedArgs& a, int head_dim, cudaStream_t stream) {
  int dev = 0;
  const int sms = current_device_sms(&dev);
  if (sms <= 0) return cudaErrorInvalidDevice;
  // Every sequence adds at most one unfilled item per KV head.  Cutting pays when the items cannot fill
  // the SMs and an item can have two pieces' tiles (50 + 41 + 65 tokens against 25 to 33 K keys: 433 us
  // whole, 177 us cut; a prompt that fills the SMs loses 3 % to the joining code's registers).
  const long long tpi = 2ll * a.tok_per_tile, per = (long long)a.Hkv * a.head_chunks;
  const long long items = (a.T / tpi + a.B) * per;
  long long reach = (long long)a.max_pages << a.log2_page;
  if (a.W > 0 && !a.key_end) reach = std::min<long long>(reach, a.W + tpi + PM_KEYS);
  const long long pieces = reach / (PM_KEYS * PM_PIECE_TILES);
  const bool split = items < sms && pieces >= 2;
  const int grid = (int)std::max(1ll, std::min<long long>(split ? items * (pieces + 1) : items, sms));
  return head_dim == 128 ? launch_d<128>(m, a, grid, split, stream) : launch_d<64>(m, a, grid, split, stream);
}

}  // namespace ink
