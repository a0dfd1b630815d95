// tree.cu -- attention of drafted tokens over the paged cache on the 5th-generation tensor cores: every token sees its
// sequence's history and the drafted tokens on its way to the root.
//
//   x = sm_scale <q[t,h], K[k]>,  d = |p - pos(k)|,  s = cap(x) - slope_h d + rel[t,h,min(d, E - 1)]
//   out = softmax(s) V,  lse = log sum exp(s)
//
// A few tokens against a long history: the bytes of K and V, and of the bias rows where there is a bias tensor, bound
// it, so they have to flow evenly over the SMs whatever the lengths are.  The rows of a tile of 128 (the M of an MMA) are (token,
// query head) pairs of one sequence and KV head, tokens outermost; an item is up to two row tiles.  All key tiles of all items
// stand in one row, tiles of an item side by side, and every CTA takes an equal run of them, found on
// the device from the lengths (a graph replays with other ones).  A run cuts two items at most; pieces of
// a cut item leave O, maximum and sum in fp32, two places a CTA, and a second kernel joins them in order, spread over
// all SMs (one CTA that joined the 20 pieces of an item of a single long sequence would take as long as six key tiles).
//
// Tensor memory: two chains, each S (KT fp32 columns, with P, the bf16 numerators, over its first half once S is in
// registers) and O (D columns).  An item of two row tiles gives a chain to each; an item of one (up to 16 tokens of 8 heads)
// gives the even key tiles to one chain and the odd ones to the other, with maxima and sums of
// their own that are joined at the end: one row tile's serial chain (scores to registers, softmax, P V, the next S,
// four hand-overs: about 2650 clocks for 128 keys) is as long as the bytes of its tiles take to arrive.
//
// Warps:
//   0-3, 4-7  softmax of chain 0 and 1, a thread per row
//   8   K and V producer: TMA boxes of whole pages or tiles, table entries 32 at a time in lanes
//   9   MMA issue
//   10  scheduler: cuts the run into pieces, publishes them in shared memory, loads their Q tiles by TMA
//   11  V check: in tiles that not every row sees whole, rows of V that nobody sees are zeroed and so is
//       every infinity or NaN (0 * NaN would reach rows that do not see the key); rows that do see one get it back at the end
//   12-15 (with a bias) bias, see below
// The bias of a row has no alignment: it starts at the row's distance from the tile.  Within the history it is KT values side
// by side, which one bulk copy a row brings from the 16-byte boundary before them; the softmax reads its row 16 bytes at a time (a
// pitch of KT + 4 words keeps 8 rows in different banks) and shifts the values into place with two selects each.  Tiles whose
// distances are all E - 1 or more take one value a row.  Behind the history distances have no order, and a bias warp brings them element
// by element, a lane a key.  With a bias tiles have 64 keys: two buffers of 128 rows take 70 KB of shared memory.
// Every wait is bounded; after a timeout the CTA records it, stops issuing, waits for what is in flight and exits.
#include <algorithm>
#include <climits>

#include "masked_common.cuh"
#include "prefill_common.cuh"

namespace ink {
namespace {

using namespace pf;

constexpr int TR_ITEMS = 3;       // published items in flight
constexpr int TR_BAD = 8;         // tiles whose unreadable keys are remembered
constexpr int TR_TILES = 4;       // barriers of K and V tiles go by tile (at most 4 of a kind are in the ring)
constexpr int TR_MIN_TILES = 2;   // least run of a CTA
constexpr int TR_DUAL_SLACK = 4;  // most tiles that two pieces may differ in to run side by side
constexpr int TR_REGS_SOFTMAX = 208, TR_REGS_REST = 88;   // registers a thread after the split (without a bias)
constexpr float TR_RESCALE_LOG2 = 8.f;

template <int D, bool BIAS>
struct TRShape {
  static constexpr int KT = BIAS ? 64 : 128;       // keys of a tile
  static constexpr int THREADS = BIAS ? 512 : 384;
  static constexpr int CB = D / 64;
  static constexpr int SUB = KT * 128;             // one 64-channel block of a K or V tile
  static constexpr int TILE = CB * SUB;
  static constexpr int QSUB = TREE_ROWS * 128;
  static constexpr int QTILE = CB * QSUB;
  static constexpr int NS = D == 128 ? 5 : 8;      // ring slots, K and V tiles in turn
  static constexpr int PITCH = KT + 4;             // words of a bias row: KT values from a 16-byte boundary on
  static constexpr int ELEMENTS = KT + 1;          // the same of one filled element by element
  static constexpr uint32_t TO = 256;              // S_h at 128 h, O_h at TO + D h
};

// A run of key tiles of one or two row tiles.
struct TRPart {
  int b, kvh, h0, gh;        // sequence, KV head, first query head, heads
  int t0, ntok, c0, n;       // first packed row, tokens; the sequence's first row and tokens
  int H, lo, hi, lo_max;     // history; keys any row sees lie in [lo, hi), every row sees [lo_max, min(H, hi))
  int kt0, nt;               // first key tile, tiles
  int place, parts;          // of a cut item (parts > 1): where this piece leaves its partials
};

// What the two chains do: two row tiles over the same key tiles; the even and the odd tiles of one piece (part 1 is part 0 with
// other tiles); a piece each.
enum TRMode { End = -1, Pair, Split, Dual };

struct TRItem {
  TRPart part[2];
  int mode, qs;              // (qs: the Q slot of Split; part or row tile h has slot h otherwise)

  __device__ __forceinline__ const TRPart& of(int h) const { return part[mode == Pair ? 0 : h]; }
  __device__ __forceinline__ int step() const { return mode == Split ? 2 : 1; }
  // Place of chain h's tile j among the item's tiles, which take turns: j + min(j + h, beside(h)).
  __device__ __forceinline__ int beside(int h) const { return mode == Pair ? 0 : part[h ^ 1].nt; }
  __device__ __forceinline__ int tiles() const { return part[0].nt + (mode == Pair ? 0 : part[1].nt); }
  __device__ __forceinline__ int longest() const { return mode == Pair ? part[0].nt : max(part[0].nt, part[1].nt); }
};

template <int D, bool BIAS>
struct TRSmem {
  using S = TRShape<D, BIAS>;
  static constexpr size_t q = 0;
  static constexpr size_t ring = 2 * (size_t)S::QTILE;
  static constexpr size_t bias = ring + (size_t)S::NS * S::TILE;
  static constexpr size_t bars = bias + (BIAS ? 2 * (size_t)TREE_ROWS * S::PITCH * 4 : 0);
  // k_full[TILES], v_full[TILES], v_ok[TILES], empty[NS], s_full[2], p_full[2], o_full[2], q_full[2], q_empty[2],
  // bias_full[2], bias_empty[2], item_full[ITEMS], item_empty[ITEMS], o_free, ml, drain
  static constexpr int NBAR = S::NS + 3 * TR_TILES + 14 + 2 * TR_ITEMS + 3;
  static constexpr size_t items = bars + (NBAR * 8 + 15) / 16 * 16;
  static constexpr size_t kbad = items + TR_ITEMS * sizeof(TRItem);
  static constexpr size_t poison = kbad + TR_BAD * 16;
  static constexpr size_t ml = poison + TR_ITEMS * 16;           // [2 chains][128 rows] float2
  static constexpr size_t misc = ml + 2 * TREE_ROWS * 8;
  static constexpr size_t alloc = misc + 16;   // (no room to align within: the array itself has to be)
  static_assert(alloc <= 227 * 1024, "shared memory budget");
};

// Bounded wait of a whole warp, with one answer for all its lanes (inline: a call would keep the registers
// from being split).
__device__ __forceinline__ bool tr_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, const TreeArgs& a) {
  bool ok = mbar_probe(bar, parity, a.wait_ns);
  if (!ok && !*abort_flag) {
    ok = mbar_wait_limit(bar, parity, a.wait_ns);
    if (!ok) {
      record_error(a.err, INK_DEVERR_WAIT_TIMEOUT);
      *abort_flag = 1;
    }
  }
  return __all_sync(0xffffffffu, ok);
}

// A sequence's rows and keys; tiles == 0: none of its rows sees a key (or it has none).
struct TRSeq {
  int c0, n, L, lo, hi, tiles;
  uint32_t bad;   // error bits; BAD_ROWS: its rows are not touched

  __device__ __forceinline__ void load(const TreeArgs& a, int b, int kt) {
    c0 = __ldg(a.cu_q + b);
    const int c1 = __ldg(a.cu_q + b + 1);
    L = __ldg(a.seq_lens + b);
    n = c1 - c0;
    lo = hi = tiles = 0;
    bad = 0;
    if (c0 < 0 || c1 > a.T || c1 < c0) {
      bad = INK_DEVERR_BAD_ROWS;
      n = 0;
    } else if (n == 0) {
      bad = 0;
    } else if (n > L) {
      bad = INK_DEVERR_QLEN_EXCEEDS_KV;
    } else if (n > 32 * a.words) {
      bad = INK_DEVERR_QLEN_EXCEEDS_MAX;
    } else {
      const long long cap = (long long)a.max_pages << a.log2_page;
      if (L > cap) bad = INK_DEVERR_PAGE_OUT_OF_RANGE;
      hi = (int)min((long long)L, cap);
      lo = a.W > 0 ? max(0, L - n - a.W + 1) : 0;
      if (lo < hi) tiles = (hi - 1) / kt - lo / kt + 1;
    }
  }
};

// The row of tiles, walked by a whole warp: 32 sequences at a time in the lanes.  Divisions, which take as long as a load, are
// made once per run: later pieces begin with their item.
struct TRWalk {
  long long base, incl, chunk, total;   // tiles before sequence cb; up to and with this lane's; of a run; of the 32
  long long pos, end;                   // of this CTA's run
  int cb, per, items, kt, cta;
  int src, groups, left;                // the sequence's lane; its items; of these not begun
  int kvh, hc, item;                    // the next one
  TRSeq s;

  __device__ __forceinline__ void load(const TreeArgs& a, int lane) {
    const int b = cb + lane;
    s.tiles = s.n = 0;
    if (b < a.B) s.load(a, b, kt);
    items = (s.n + 2 * a.tok_per_tile - 1) / (2 * a.tok_per_tile);
    incl = (long long)s.tiles * items * per;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    total = __shfl_sync(0xffffffffu, incl, 31);
  }

  __device__ __forceinline__ void begin(const TreeArgs& a, int lane, int tile_keys) {
    kt = tile_keys;
    per = a.Hkv * a.head_chunks;
    cta = (int)blockIdx.x;
    long long all = 0;
    for (cb = ((a.B - 1) >> 5) << 5; cb >= 0; cb -= 32) {
      load(a, lane);
      all += total;
    }
    cb = 0;
    base = 0;
    left = 0;
    chunk = max((all + gridDim.x - 1) / (long long)gridDim.x, (long long)TR_MIN_TILES);
    pos = min(cta * chunk, all);
    end = min(pos + chunk, all);
  }

  // The next piece of the run; first: the CTA where its item begins.
  __device__ __forceinline__ TRPart next(const TreeArgs& a, int lane, int& first) {
    int x0 = 0;
    first = cta;
    if (left == 0) {   // of another sequence than the one before
      while (pos >= base + total) {
        base += total;
        cb += 32;
        load(a, lane);
      }
      src = __ffs(__ballot_sync(0xffffffffu, pos < base + incl)) - 1;
      const int ni = __shfl_sync(0xffffffffu, items, src), tiles = __shfl_sync(0xffffffffu, s.tiles, src);
      groups = ni * per;
      const long long off = pos - (base + __shfl_sync(0xffffffffu, incl - (long long)s.tiles * items * per, src));
      int gi = 0;
      if (off > 0) {   // the run begins within a sequence
        gi = (int)(off / tiles);
        x0 = (int)(off - (long long)gi * tiles);
        first = (int)((pos - x0) / chunk);
      }
      left = groups - gi;
      const int hk = gi / ni;
      item = gi - hk * ni;
      kvh = hk / a.head_chunks;
      hc = hk - kvh * a.head_chunks;
    }
    const int ni = __shfl_sync(0xffffffffu, items, src), tiles = __shfl_sync(0xffffffffu, s.tiles, src);
    TRPart w;
    w.b = cb + src;
    w.c0 = __shfl_sync(0xffffffffu, s.c0, src);
    w.n = __shfl_sync(0xffffffffu, s.n, src);
    w.lo = __shfl_sync(0xffffffffu, s.lo, src);
    w.hi = __shfl_sync(0xffffffffu, s.hi, src);
    w.H = __shfl_sync(0xffffffffu, s.L, src) - w.n;
    w.kvh = kvh;
    w.h0 = kvh * a.G + hc * a.heads_per_tile;
    w.gh = min(a.heads_per_tile, a.G - hc * a.heads_per_tile);
    w.t0 = w.c0 + item * 2 * a.tok_per_tile;
    w.ntok = min(2 * a.tok_per_tile, w.n - item * 2 * a.tok_per_tile);
    w.kt0 = w.lo / kt + x0;
    w.nt = (int)min((long long)(tiles - x0), end - pos);
    const long long g1 = pos - x0 + tiles;
    w.parts = (g1 <= end ? cta : (int)((g1 - 1) / chunk)) - first + 1;
    w.place = 2 * cta + (cta == first ? 1 : 0);
    pos += w.nt;
    --left;
    if (++item == ni) {
      item = 0;
      if (++hc == a.head_chunks) {
        hc = 0;
        ++kvh;
      }
    }
    return w;
  }
};

// Bit c: does the row see key base + c?  History [lo, hist) and, behind H, the row's bits.
struct TRRow {
  const uint32_t* bits;
  uint32_t w0;                    // bits[0]
  int p, lo, hist, H, nlim, c0;   // hist: readable end of the history; nlim: drafted keys that can be read
  bool cut;                       // the window may hide an ancestor

  __device__ __forceinline__ uint32_t word(const TreeArgs& a, int i) const {
    return i == 0 ? w0 : i > 0 && i < a.words ? __ldg(bits + i) : 0u;
  }
  __device__ __forceinline__ uint32_t sees(const TreeArgs& a, int base) const {
    const int x0 = max(lo - base, 0), x1 = min(hist - base, 32);
    uint32_t vis = x1 > x0 ? (0xffffffffu >> (32 - (x1 - x0))) << x0 : 0u;
    const int j0 = base - H;
    if (j0 > -32 && j0 < nlim) {
      uint32_t t = __funnelshift_r(word(a, j0 >> 5), word(a, (j0 >> 5) + 1), j0 & 31);
      if (nlim - j0 < 32) t &= (1u << (nlim - j0)) - 1u;
      if (cut)
        for (uint32_t x = t; x; x &= x - 1) {
          const int c = __ffs(x) - 1;
          if (p - max(__ldg(a.positions + c0 + j0 + c), H) >= a.W) t &= ~(1u << c);
        }
      vis |= t;
    }
    return vis;
  }
};

// Row t at position p, w0 its first bits.
__device__ __forceinline__ TRRow tr_row(const TreeArgs& a, const TRPart& it, int t, int p, uint32_t w0, bool valid) {
  TRRow r;
  r.bits = a.ancestors + (size_t)t * a.words;
  r.w0 = w0;
  r.p = p;
  r.H = it.H;
  r.c0 = it.c0;
  r.hist = valid ? min(it.H, it.hi) : 0;
  r.nlim = valid ? min(it.n, it.hi - it.H) : 0;
  r.lo = a.W > 0 ? max(0, p - a.W + 1) : 0;
  r.cut = a.W > 0 && p - it.H >= a.W;
  return r;
}

// How the bias of a tile comes to the softmax.  Behind the history distances have no order.  Before it a row's are KT values
// side by side, one copy a row where 16-byte boundaries can be kept inside the tensor; all of them at E - 1 or more are one value.
enum TRBias { NoLoad, RowCopies, Elements };

__device__ __forceinline__ TRBias tr_bias(const TreeArgs& a, const TRPart& it, int k0, int kt) {
  if (min(it.H, it.hi) - k0 < kt) return Elements;
  if (!a.rel || it.H - (k0 + kt - 1) >= a.E - 1) return NoLoad;
  return a.rel_rows ? RowCopies : Elements;
}

__device__ __forceinline__ uint64_t tr_mul(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// An infinity or NaN of a part stays one, whatever the part's weight.
__device__ __forceinline__ float tr_weigh(float w, float x) { return fabsf(x) <= 3.4028235e38f ? w * x : x; }

// CAP: capped scores, by a polynomial where all scores of a warp's tile allow it (as in the masked prefill).
template <int D, bool CAP, bool BIAS>
__global__ void __launch_bounds__(TRShape<D, BIAS>::THREADS, 1)
tree_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
            const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ TreeArgs a) {
  using S = TRShape<D, BIAS>;
  using L_ = TRSmem<D, BIAS>;
  constexpr int NS = S::NS, KT = S::KT, KW = KT / 32;

  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + L_::bars);
  uint64_t* v_full = k_full + TR_TILES;
  uint64_t* v_ok = v_full + TR_TILES;   // V tile checked
  uint64_t* empty = v_ok + TR_TILES;
  uint64_t* s_full = empty + NS;        // [2] S_h in TMEM, every earlier product of h done
  uint64_t* p_full = s_full + 2;        // [2] P_h written
  uint64_t* o_full = p_full + 2;        // [2] the piece's last O_h product done
  uint64_t* q_full = o_full + 2;        // [2]
  uint64_t* q_empty = q_full + 2;       // [2] the piece's last product with a Q tile done
  uint64_t* bias_full = q_empty + 2;    // [2]
  uint64_t* bias_empty = bias_full + 2; // [2]
  uint64_t* item_full = bias_empty + 2; // [ITEMS]
  uint64_t* item_empty = item_full + TR_ITEMS;
  uint64_t* o_free = item_empty + TR_ITEMS;   // both O of a Split item read
  uint64_t* ml_bar = o_free + 1;        // maxima and sums of both chains written
  uint64_t* drain = ml_bar + 1;
  TRItem* items = reinterpret_cast<TRItem*>(smem + L_::items);
  uint32_t* kbad = reinterpret_cast<uint32_t*>(smem + L_::kbad);   // [BAD][4] bit per unreadable key
  int* poison = reinterpret_cast<int*>(smem + L_::poison);   // [ITEMS][2 chains][2] first and last tile of V with an infinity or NaN
  float2* ml = reinterpret_cast<float2*>(smem + L_::ml);
  float* bias = reinterpret_cast<float*>(smem + L_::bias);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L_::misc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L_::misc + 4);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int P = 1 << a.log2_page;

  if (smem_u32(smem) & 1023u) {   // (swizzled tiles would lie elsewhere than they are looked for)
    if (tid == 0) {
      record_error(a.err, INK_DEVERR_WAIT_TIMEOUT);
      a.cuts[blockIdx.x].parts = 0;
    }
    return;
  }
  if (tid == 0) {
    for (int x = 0; x < NS; ++x) mbar_init(&empty[x], 1);
    for (int x = 0; x < TR_TILES; ++x) {
      mbar_init(&k_full[x], 1);
      mbar_init(&v_full[x], 1);
      mbar_init(&v_ok[x], 1);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&s_full[x], 1);
      mbar_init(&p_full[x], 4);
      mbar_init(&o_full[x], 1);
      mbar_init(&q_full[x], 1);
      mbar_init(&q_empty[x], 1);
      mbar_init(&bias_full[x], 64);   // every lane of two warps
      mbar_init(&bias_empty[x], 4);
    }
    for (int x = 0; x < TR_ITEMS; ++x) {
      mbar_init(&item_full[x], 1);
      mbar_init(&item_empty[x], 11 + (BIAS ? 4 : 0));   // producer, MMA, V check, 8 softmax warps, bias warps
    }
    mbar_init(o_free, 8);
    mbar_init(ml_bar, 8);
    mbar_init(drain, 1);
    fence_mbar_init();
    *abort_flag = 0;
  }
  TRWalk walk;
  if (warp == 10) walk.begin(a, lane, KT);   // (its loads are on their way while the rest is set up)
  // rows of a Q tile past the last (token, head) pair stay zero
  for (int x = tid; x < 2 * S::QTILE / 16; x += S::THREADS)
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

  // The k-th item of this CTA is in its slot; false when there is none (or after a timeout).
  auto next_item = [&](int k) -> bool {
    return tr_wait(&item_full[k % TR_ITEMS], (uint32_t)(k / TR_ITEMS) & 1u, abort_flag, a) && items[k % TR_ITEMS].mode != End;
  };
  auto done_item = [&](int k) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&item_empty[k % TR_ITEMS]);
  };

  if (warp >= 8) {
    if constexpr (!BIAS) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(TR_REGS_REST));
    if (warp == 8) {
      // ---------------------------------------------------------------- K and V producer
      if (lane == 0) {
        prefetch_tensormap(&tmK);
        prefetch_tensormap(&tmV);
      }
      const int seg = min(P, KT), nseg = KT / seg;
      int f = 0;                            // fills issued
      bool go = true;
      for (int k = 0; go && next_item(k); ++k) {
        const TRItem& item = items[k % TR_ITEMS];
        int chunk_base[2] = {0, 0}, chunk_val[2] = {-1, -1};   // table entries chunk_base + lane, of each chain's part
        for (int j = 0; j < item.longest() && go; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const TRPart& it = item.part[h];
          if (!go || (h == 1 && item.mode == Pair) || j >= it.nt) continue;
          const int k0 = (it.kt0 + j * item.step()) * KT;
          const int last_idx = (it.hi - 1) >> a.log2_page;
          const int pfirst = k0 >> a.log2_page, plast = (k0 + KT - 1) >> a.log2_page;
          if (j == 0 || plast >= chunk_base[h] + 32) {
            chunk_base[h] = pfirst;   // entries past the sequence's last key are not read
            chunk_val[h] = __ldg(a.block_table + (size_t)it.b * a.max_pages + min(chunk_base[h] + lane, last_idx));
          }
          const int ks = k0 + lane * seg;                 // lane < nseg takes one segment
          const bool want = lane < nseg && ks < it.hi && ks + seg > it.lo;
          const int page = __shfl_sync(0xffffffffu, chunk_val[h], min(max((ks >> a.log2_page) - chunk_base[h], 0), 31));
          const bool bad_seg = want && (page < 0 || page >= a.num_pages);
          const bool load = want && !bad_seg;
          const uint32_t nload = __popc(__ballot_sync(0xffffffffu, load));
          const uint32_t bmask = __ballot_sync(0xffffffffu, bad_seg);
          const int row = load ? ((page * a.Hkv + it.kvh) << a.log2_page) + (ks & (P - 1)) : 0;
#pragma unroll 1
          for (int kv = 0; kv < 2; ++kv, ++f) {
            const int st = f % NS;
            if (f >= NS && !tr_wait(&empty[st], (uint32_t)((f / NS) - 1) & 1u, abort_flag, a)) {
              go = false;
              break;
            }
            if (kv == 0 && lane < KW) {   // keys of this tile whose page is outside the pool
              uint32_t bad = 0;
              for (uint32_t mm = bmask; mm; mm &= mm - 1) {
                const int x0 = (__ffs(mm) - 1) * seg - 32 * lane, x1 = x0 + seg;   // bits [x0, x1) of this word
                const int y0 = max(x0, 0), y1 = min(x1, 32);
                if (y1 > y0) bad |= (0xffffffffu >> (32 - (y1 - y0))) << y0;
              }
              kbad[((f >> 1) % TR_BAD) * 4 + lane] = bad;
              if (bmask && lane == 0) record_error(a.err, INK_DEVERR_PAGE_OUT_OF_RANGE);
            }
            uint64_t* full = (kv ? v_full : k_full) + (f >> 1) % TR_TILES;
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
        done_item(k);
      }
      if (lane == 0) {
        pp_drain_ring(k_full, TR_TILES, (f + 1) >> 1, a.err);
        pp_drain_ring(v_full, TR_TILES, f >> 1, a.err);
      }
    } else if (warp == 9) {
      // ---------------------------------------------------------------- MMA issue
      constexpr uint32_t IDESC_S = umma_idesc_bf16(128, KT, false, false);
      constexpr uint32_t IDESC_PV = umma_idesc_bf16(128, D, false, true);
      const uint32_t qaddr = smem_u32(smem + L_::q), raddr = smem_u32(smem + L_::ring);
      // S and P V products each walk the tiles in their order: K of tile g is fill 2 g, V fill 2 g + 1
      int gk = 0, gv = 0, k_slot = 0, v_slot = 1;
      uint32_t qn = 0, pn = 0;         // a parity bit per Q tile and per chain
      bool go = true;
      auto wait_tile = [&](uint64_t* bars, int tile) {
        return tr_wait(&bars[tile % TR_TILES], (uint32_t)(tile / TR_TILES) & 1u, abort_flag, a);
      };
      auto wait_q = [&](int s) {
        const bool ok = tr_wait(&q_full[s], (qn >> s) & 1u, abort_flag, a);
        qn ^= 1u << s;
        return ok;
      };
      // S_h of tile gk with Q tile qs; the tile's last product frees its slot, a Q tile's last one that
      auto issue_s = [&](int h, int qs, bool frees_k, bool frees_q) {
        const uint64_t ad = umma_desc_sw128(qaddr + qs * S::QTILE, 16, 1024);
        const uint64_t bd = umma_desc_sw128(raddr + k_slot * S::TILE, 16, 1024);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          umma_ss_warp(tmem + 128u * h, ad + (uint64_t)(((kk >> 2) * S::QSUB + (kk & 3) * 32) >> 4),
                       bd + (uint64_t)(((kk >> 2) * S::SUB + (kk & 3) * 32) >> 4), IDESC_S, kk > 0 ? 1u : 0u);
        umma_commit_warp(&s_full[h]);
        if (frees_k) {
          umma_commit_warp(&empty[k_slot]);
          ++gk;
          k_slot = k_slot + 2 < NS ? k_slot + 2 : k_slot + 2 - NS;
        }
        if (frees_q) umma_commit_warp(&q_empty[qs]);
        __syncwarp();
      };
      auto issue_pv = [&](int h, bool acc, bool frees_v) {
        const uint64_t bd = umma_desc_sw128(raddr + v_slot * S::TILE, S::SUB, 1024);
#pragma unroll
        for (int ks = 0; ks < KT / 16; ++ks)
          umma_ts_warp(tmem + S::TO + (uint32_t)(D * h), tmem + 128u * h + ks * 8, bd + (uint64_t)((ks * 16 * 128) >> 4),
                       IDESC_PV, (acc || ks > 0) ? 1u : 0u);
        if (frees_v) {
          umma_commit_warp(&empty[v_slot]);
          ++gv;
          v_slot = v_slot + 2 < NS ? v_slot + 2 : v_slot + 2 - NS;
        }
      };
      uint32_t merges = 0;             // Split items so far
      bool merged = false;             // the item before was one
      for (int k = 0; go && next_item(k); ++k) {
        const TRItem& it = items[k % TR_ITEMS];
        const int mode = it.mode, qs1 = mode == Split ? it.qs : 1, qs0 = mode == Split ? it.qs : 0;
        const int n0 = it.part[0].nt, n1 = mode == Pair ? n0 : it.part[1].nt, last = gk + n0 + n1 - 1;
        const bool pair = mode == Pair;
        // the last S with a Q tile: of the chain, of the piece in Split
        auto last_s = [&](int j, int h) { return mode == Split ? gk == last : j == (h ? n1 : n0) - 1; };
        for (int h = 0; h < 2 && go; ++h) {
          if (h == 1 && n1 == 0) continue;
          if (mode != Split || h == 0) go = wait_q(h ? qs1 : qs0);
          if (go && (!pair || h == 0)) go = wait_tile(k_full, gk);
          if (!go) break;
          tc_fence_after();
          issue_s(h, h ? qs1 : qs0, !pair || h == 1, last_s(0, h));
        }
        // both O of a Split item have been read
        if (go && merged) go = tr_wait(o_free, (merges - 1) & 1u, abort_flag, a);
        merged = mode == Split;
        merges += merged;
        for (int j = 0; j < max(n0, n1) && go; ++j)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int nh = h ? n1 : n0;
            if (!go || j >= nh) continue;
            // (v_ok comes after v_full)
            if (!pair || h == 0) go = wait_tile(v_ok, gv);
            if (go) go = tr_wait(&p_full[h], (pn >> h) & 1u, abort_flag, a);
            if (!go) continue;
            pn ^= 1u << h;
            tc_fence_after();
            issue_pv(h, j > 0, !pair || h == 1);
            if (j + 1 < nh) {
              if (!pair || h == 0) go = wait_tile(k_full, gk);
              if (!go) continue;
              issue_s(h, h ? qs1 : qs0, !pair || h == 1, last_s(j + 1, h));
            } else {
              umma_commit_warp(&o_full[h]);
              __syncwarp();
            }
          }
        done_item(k);
      }
      umma_commit_warp(drain);
      __syncwarp();
      if (!mbar_wait_bounded(drain, 0)) record_error(a.err, INK_DEVERR_WAIT_TIMEOUT);
    } else if (warp == 10) {
      // ---------------------------------------------------------------- scheduler and Q loads
      if (lane == 0) prefetch_tensormap(&tmQ);
      TreeCut cut;                       // the item that this run begins and does not end
      cut.parts = 0;
      uint32_t qn = 0, loaded = 0;       // bits per Q tile: loads so far, odd or even; any
      int qs = 1;
      auto piece = [&]() {               // the next one of the run
        int first;
        TRPart w = walk.next(a, lane, first);
        if (w.parts > 1 && first == (int)blockIdx.x) cut = {w.parts, w.t0, w.ntok, w.h0, w.gh};
        // all rows see the keys from the largest first one on
        w.lo_max = 0;
        if (a.W > 0) {
          for (int i = lane; i < w.ntok; i += 32) w.lo_max = max(w.lo_max, max(__ldg(a.positions + w.t0 + i), w.H) - a.W + 1);
          w.lo_max = __reduce_max_sync(0xffffffffu, w.lo_max);
        }
        return w;
      };
      TRPart next;
      bool have = false;                 // next was looked at, and is an item of its own
      for (int k = 0;; ++k) {
        const int sl = k % TR_ITEMS;
        TRItem it;
        it.mode = End;
        it.qs = 0;
        if (have || walk.pos < walk.end) {
          it.part[0] = have ? next : piece();
          have = false;
          if (it.part[0].ntok > a.tok_per_tile) {
            it.mode = Pair;
          } else {
            it.mode = Split;
            if (walk.pos < walk.end) {
              next = piece();
              have = next.ntok > a.tok_per_tile || abs(it.part[0].nt - next.nt) > TR_DUAL_SLACK;
              if (!have) it.mode = Dual;
            }
          }
        }
        if (k >= TR_ITEMS && !tr_wait(&item_empty[sl], (uint32_t)((k / TR_ITEMS) - 1) & 1u, abort_flag, a)) break;
        if (it.mode == End) {
          if (lane == 0) {
            items[sl].mode = End;
            mbar_arrive(&item_full[sl]);
          }
          break;
        }
        qs = it.mode == Split ? qs ^ 1 : 1;
        it.qs = qs;
        if (it.mode == Dual) {
          it.part[1] = next;
        } else {
          it.part[1] = it.part[0];
          if (it.mode == Split) {
            it.part[0].nt = (it.part[0].nt + 1) >> 1;
            it.part[1].nt >>= 1;
            ++it.part[1].kt0;
          }
        }
        if (lane == 0) {
          items[sl] = it;
          volatile int* p = poison + 4 * sl;
          p[0] = p[2] = INT_MAX;
          p[1] = p[3] = -1;
          mbar_arrive(&item_full[sl]);
        }
        __syncwarp();
        bool go = true;
        for (int x = 0; x < (it.mode == Split ? 1 : 2) && go; ++x) {
          const int s = it.mode == Split ? qs : x;
          if ((loaded >> s) & 1u) go = tr_wait(&q_empty[s], ((qn >> s) & 1u) ^ 1u, abort_flag, a);
          if (!go) break;
          qn ^= 1u << s;
          loaded |= 1u << s;
          if (lane == 0) {
            const TRPart& w = it.part[x];
            const int t0 = w.t0 + (it.mode == Pair ? x * a.tok_per_tile : 0);
            mbar_arrive_expect_tx(&q_full[s], (uint32_t)(S::CB * a.heads_per_tile * a.tok_per_tile * 128));
#pragma unroll
            for (int c = 0; c < S::CB; ++c)
              tma_load_3d(smem + L_::q + s * S::QTILE + c * S::QSUB, &tmQ, c * 64, w.h0, t0, &q_full[s]);
          }
          __syncwarp();
        }
        if (!go) break;
      }
      if (lane == 0) {
        a.cuts[blockIdx.x] = cut;
        for (int s = 0; s < 2; ++s)
          if (((loaded >> s) & 1u) && !mbar_wait_bounded(&q_full[s], ((qn >> s) & 1u) ^ 1u)) record_error(a.err, INK_DEVERR_WAIT_TIMEOUT);
      }
    } else if (warp == 11) {
      // ---------------------------------------------------------------- V check
      int g = 0;
      bool go = true;
      for (int k = 0; go && next_item(k); ++k) {
        const TRItem& item = items[k % TR_ITEMS];
        for (int j = 0; j < item.longest() && go; ++j)
        for (int h = 0; h < (item.mode == Pair ? 1 : 2); ++h) {
          const TRPart& it = item.part[h];
          if (j >= it.nt) continue;
          const int hist = min(it.H, it.hi), kt = it.kt0 + j * item.step();
          const int st = (2 * g + 1) % NS;
          go = tr_wait(&v_full[g % TR_TILES], (uint32_t)(g / TR_TILES) & 1u, abort_flag, a);
          if (!go) break;
          const int k0 = kt * KT;
          const uint32_t* badw = kbad + (g % TR_BAD) * 4;
          uint32_t any = 0;
#pragma unroll
          for (int x = 0; x < KW; ++x) any |= badw[x];
          if (k0 < it.lo_max || hist - k0 < KT || any) {
            uint8_t* vt = smem + L_::ring + (size_t)st * S::TILE;
            bool found = false;
#pragma unroll 1
            for (int x = 0; x < KW; ++x) {
              const int kk = k0 + 32 * x + lane;
              uint4* row = reinterpret_cast<uint4*>(vt + (32 * x + lane) * 128);
              const bool zero = kk < it.lo || kk >= it.hi || ((badw[x] >> lane) & 1u);
              if (!zero && kk >= it.lo_max && kk < hist) continue;   // every row sees it
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
              atomicMin(poison + 4 * (k % TR_ITEMS) + 2 * h, kt);
              atomicMax(poison + 4 * (k % TR_ITEMS) + 2 * h + 1, kt);
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&v_ok[g % TR_TILES]);
          ++g;
        }
        done_item(k);
      }
    } else if constexpr (BIAS) {
      // ---------------------------------------------------------------- bias loads: two warps a chain, 64 rows each
      const int h = (warp - 12) >> 1, r0 = ((warp - 12) & 1) * 64;
      float* buf = bias + (size_t)h * TREE_ROWS * S::PITCH;
      const int last = a.E - 1, size = a.rel_bf16 ? 2 : 4;
      uint32_t fills = 0;
      bool go = true;
      for (int k = 0; go && next_item(k); ++k) {
        const TRItem& item = items[k % TR_ITEMS];
        const TRPart& it = item.of(h);
        const int tok0 = item.mode == Pair ? h * a.tok_per_tile : 0;
        const int rows = min(a.tok_per_tile, it.ntok - tok0) * a.heads_per_tile;
        const int i0 = r0 / a.heads_per_tile;
        // this lane's rows r0 + lane and 32 more: position and elements before the row; tokens of the warp's rows
        int pr[2], pt[2];
        size_t at[2];
        bool live[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int r = r0 + 32 * x + lane, i = r / a.heads_per_tile, hd = r - i * a.heads_per_tile;
          live[x] = r < rows && hd < it.gh;
          const int t = it.t0 + tok0 + (live[x] ? i : 0);
          pr[x] = max(__ldg(a.positions + t), it.H);
          at[x] = ((size_t)t * a.Hq + it.h0 + hd) * a.E;
          const int ti = min(i0 + 32 * x + lane, it.ntok - tok0 - 1);
          pt[x] = max(__ldg(a.positions + it.t0 + tok0 + ti), it.H);
        }
        for (int j = 0; j < it.nt && go; ++j) {
          const int k0 = (it.kt0 + j * item.step()) * KT;
          const TRBias how = tr_bias(a, it, k0, KT);
          if (how == NoLoad) continue;
          if (fills > 0) go = tr_wait(&bias_empty[h], (fills - 1) & 1u, abort_flag, a);
          if (!go) break;
          ++fills;
          if (how == RowCopies) {
            // distances [s, e) of a row, from the 16 bytes that hold the first to those that hold the last
            uint32_t bytes[2];
            uintptr_t from[2];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const int s = pr[x] - (k0 + KT - 1), e = min(pr[x] - k0, last) + 1;
              const uintptr_t base = reinterpret_cast<uintptr_t>(a.rel) + at[x] * size;
              from[x] = (base + (size_t)s * size) & ~(uintptr_t)15;
              bytes[x] = live[x] && s < e ? (uint32_t)(((base + (size_t)e * size + 15) & ~(uintptr_t)15) - from[x]) : 0u;
            }
            mbar_arrive_expect_tx(&bias_full[h], bytes[0] + bytes[1]);
#pragma unroll
            for (int x = 0; x < 2; ++x)
              if (bytes[x])
                bulk_copy_g2s(smem_u32(buf + (r0 + 32 * x + lane) * S::PITCH), reinterpret_cast<const void*>(from[x]), bytes[x],
                              &bias_full[h]);
            __syncwarp();
            continue;
          }
          // element by element: a lane has two keys and goes over the rows
          int pk[2];
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int kk = k0 + 32 * x + lane;
            pk[x] = kk >= it.H && kk < it.hi ? max(__ldg(a.positions + it.c0 + kk - it.H), it.H) : kk;
          }
          // (all loads of a batch first, from rows that are there: what is not seen is masked)
          auto fill = [&](auto load) {
            int i = i0, hd = r0 - i0 * a.heads_per_tile;
#pragma unroll 1
            for (int r = r0; r < min(r0 + 64, rows); r += 16) {
              float v[16][2], far[16][2], slope[16];
#pragma unroll
              for (int y = 0; y < 16; ++y) {
                const int off = min(i - i0, 63);
                const int p0 = __shfl_sync(0xffffffffu, pt[0], off & 31), p1 = __shfl_sync(0xffffffffu, pt[1], off & 31);
                const int p = off < 32 ? p0 : p1;
                const int head = it.h0 + min(hd, it.gh - 1);
                const size_t row = ((size_t)(it.t0 + min(tok0 + i, it.ntok - 1)) * a.Hq + head) * a.E;
                slope[y] = a.slopes ? __ldg(a.slopes + head) : 0.f;
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                  const int d = abs(p - pk[x]);
                  far[y][x] = (float)d;
                  v[y][x] = load(row + min(d, last));
                }
                if (++hd == a.heads_per_tile) {
                  hd = 0;
                  ++i;
                }
              }
#pragma unroll
              for (int y = 0; y < 16; ++y) {
                buf[(r + y) * S::ELEMENTS + lane] = fmaf(-slope[y], far[y][0], v[y][0]);
                buf[(r + y) * S::ELEMENTS + 32 + lane] = fmaf(-slope[y], far[y][1], v[y][1]);
              }
            }
          };
          if (!a.rel) fill([](size_t) { return 0.f; });
          else if (a.rel_bf16) fill([&](size_t x) { return __uint_as_float((uint32_t)__ldg(static_cast<const uint16_t*>(a.rel) + x) << 16); });
          else fill([&](size_t x) { return __ldg(static_cast<const float*>(a.rel) + x); });
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // (copies may write here next)
          mbar_arrive(&bias_full[h]);
          __syncwarp();
        }
        done_item(k);
      }
      if (lane == 0 && fills > 0 && !mbar_wait_bounded(&bias_full[h], (fills - 1) & 1u)) record_error(a.err, INK_DEVERR_WAIT_TIMEOUT);
    }
  } else {
    // ------------------------------------------------------------------ softmax
    if constexpr (!BIAS) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(TR_REGS_SOFTMAX));
    const int h = warp >> 2, r = tid & 127;
    const uint32_t tlane = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t tm_s = tlane + 128u * h, tm_o = tlane + S::TO;
    const int my_i = r / a.heads_per_tile, my_g = r - my_i * a.heads_per_tile;
    __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(a.out);

    // sequences that see no key: zero rows, shared out over the CTAs; what is wrong with a sequence is told here
    for (int b = (int)blockIdx.x; b < a.B; b += (int)gridDim.x) {
      TRSeq s;
      s.load(a, b, KT);
      if (tid == 0 && s.bad) record_error(a.err, s.bad);
      if (s.tiles > 0 || s.n <= 0) continue;
      for (long long x = tid; x < (long long)s.n * a.Hq * (D / 8); x += 256)
        reinterpret_cast<uint4*>(out + (size_t)s.c0 * a.Hq * D)[x] = make_uint4(0u, 0u, 0u, 0u);
      if (a.lse)
        for (long long x = tid; x < (long long)s.n * a.Hq; x += 256) a.lse[(size_t)s.c0 * a.Hq + x] = -INFINITY;
    }

    const bool scaled = CAP || BIAS || !(a.scale_log2 > 0.f);
    const float mul = scaled ? 1.f : a.scale_log2;
    uint32_t sn = 0, on = 0, bn = 0, mn = 0;   // (on: a parity bit per chain)
    int g = 0;
    bool go = true;
    for (int k = 0; go && next_item(k); ++k) {
      // (read where it is needed, from shared memory: the tile loop has no registers to spare)
      const TRItem& item = items[k % TR_ITEMS];
      const TRPart& it = item.of(h);
      const int nt = it.nt;
      const bool pair = item.mode == Pair, merge = item.mode == Split;
      const int ti = (pair ? h * a.tok_per_tile : 0) + my_i;
      const bool rv = my_i < a.tok_per_tile && ti < it.ntok && my_g < it.gh;
      const int t = it.t0 + (rv ? ti : 0), head = it.h0 + (rv ? my_g : 0);
      // (position and bits come from L1 where they are needed; without a bias there are no registers for them)
      prefetch_l1(a.positions + t);
      prefetch_l1(a.ancestors + (size_t)t * a.words);
      int p = 0;
      if constexpr (BIAS) p = max(__ldg(a.positions + t), it.H);
      auto my_row = [&]() {
        return tr_row(a, it, t, BIAS ? p : max(__ldg(a.positions + t), it.H), __ldg(a.ancestors + (size_t)t * a.words), rv);
      };
      float rc = 0.f;   // the row's last value
      if constexpr (BIAS) {
        if (a.rel) {
          const size_t x = ((size_t)t * a.Hq + head + 1) * a.E - 1;
          rc = a.rel_bf16 ? __uint_as_float((uint32_t)__ldg(static_cast<const uint16_t*>(a.rel) + x) << 16)
                          : __ldg(static_cast<const float*>(a.rel) + x);
        }
      }
      const int beside = item.beside(h), kstep = item.step() * KT, lo_max = it.lo_max, hist = min(it.H, it.hi);
      int k0 = it.kt0 * KT;
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < nt; ++j, k0 += kstep) {
        const int tile = g + j + min(j + h, beside);
        go = tr_wait(&s_full[h], sn & 1u, abort_flag, a);
        if (!go) break;
        ++sn;
        tc_fence_after();
        uint32_t sr[KT];
#pragma unroll
        for (int c = 0; c < KW; ++c) tmem_ld32(tm_s + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(&sr[32 * c]));
        tmem_wait_ld();
        uint32_t badw[KW], any = 0;
#pragma unroll
        for (int x = 0; x < KW; ++x) any |= badw[x] = kbad[(tile % TR_BAD) * 4 + x];
        const bool part = k0 < lo_max || hist - k0 < KT || any;   // not every row sees all of it
        if (CAP && part) {   // (what nobody may see has no say in how scores are capped)
          const TRRow row = my_row();
#pragma unroll
          for (int w = 0; w < KW; ++w) {
            const uint32_t vis = row.sees(a, k0 + 32 * w) & ~badw[w];
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (!((vis >> c) & 1u)) sr[32 * w + c] = 0u;
          }
        }
        // ---- scores
        if constexpr (CAP) {
          float fv[4] = {0.f, 0.f, 0.f, 0.f};   // largest |<q, K[k]>| of the tile
#pragma unroll
          for (int c = 0; c < KT; c += 2)
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
            for (int c = 0; c < KT; c += 2) {
              const uint64_t x = f2_pack(__uint_as_float(sr[c]), __uint_as_float(sr[c + 1]));
              const uint64_t u = tr_mul(x, x);
              uint64_t y = co[TERMS - 1];
#pragma unroll
              for (int i = TERMS - 2; i >= 0; --i) y = f2_fma(y, u, co[i]);
              float s0, s1;
              f2_unpack(tr_mul(y, x), s0, s1);
              sr[c] = __float_as_uint(s0);
              sr[c + 1] = __float_as_uint(s1);
            }
          };
          auto within = [&](float reach) { return __all_sync(0xffffffffu, far <= reach); };
          if (within(a.cap_near)) {
            polynomial(std::integral_constant<int, NEAR_TERMS>{});
          } else if (within(a.cap_mid)) {
            polynomial(std::integral_constant<int, MID_TERMS>{});
          } else {
#pragma unroll
            for (int c = 0; c < KT; ++c) sr[c] = __float_as_uint(score_log2<true>(a, __uint_as_float(sr[c])));
          }
        } else if (scaled) {
#pragma unroll
          for (int c = 0; c < KT; ++c) sr[c] = __float_as_uint(__uint_as_float(sr[c]) * a.scale_log2);
        }
        if constexpr (BIAS) {
          const TRBias how = tr_bias(a, it, k0, KT);
          const float* br = bias + (size_t)h * TREE_ROWS * S::PITCH;
          if (how != NoLoad) {
            go = tr_wait(&bias_full[h], bn & 1u, abort_flag, a);
            if (!go) break;
            ++bn;
          }
          if (how == Elements) {
            br += r * S::ELEMENTS;
#pragma unroll
            for (int c = 0; c < KT; ++c) sr[c] = __float_as_uint(fmaf(br[c], LOG2E, __uint_as_float(sr[c])));
          } else {
            if (how == RowCopies) {
              // element e of the tile's distances, s = p - (k0 + KT - 1) up: key KT - 1 - e
              const int d0 = p - k0;   // of key 0
              const uintptr_t src = reinterpret_cast<uintptr_t>(a.rel) + (((size_t)t * a.Hq + head) * a.E + (size_t)(d0 - KT + 1)) * (a.rel_bf16 ? 2 : 4);
              const bool beyond = __any_sync(0xffffffffu, d0 >= a.E - 1);
              const int c_last = d0 - (a.E - 1);   // keys up to this one are at a distance of E - 1 or more
              const uint4* row = reinterpret_cast<const uint4*>(br + r * S::PITCH);
              uint4 cur = row[0];
              if (a.rel_bf16) {
                const bool o1 = src & 2, o2 = src & 4, o4 = src & 8;
#pragma unroll
                for (int q = 0; q < KT / 8; ++q) {
                  const uint4 nxt = row[q + 1];
                  const uint32_t w[8] = {cur.x, cur.y, cur.z, cur.w, nxt.x, nxt.y, nxt.z, nxt.w};
                  cur = nxt;
                  uint32_t u[6], v[4];
                  uint32_t o[7];
#pragma unroll
                  for (int i = 0; i < 7; ++i) o[i] = o1 ? __funnelshift_r(w[i], w[i + 1], 16) : w[i];
#pragma unroll
                  for (int i = 0; i < 6; ++i) u[i] = o2 ? o[i + 1] : o[i];
#pragma unroll
                  for (int i = 0; i < 4; ++i) v[i] = o4 ? u[i + 2] : u[i];
#pragma unroll
                  for (int i = 0; i < 8; ++i) {
                    const int c = KT - 1 - (8 * q + i);
                    float x = __uint_as_float(i & 1 ? v[i >> 1] & 0xFFFF0000u : v[i >> 1] << 16);
                    if (beyond) x = c <= c_last ? rc : x;
                    sr[c] = __float_as_uint(fmaf(x, LOG2E, __uint_as_float(sr[c])));
                  }
                }
              } else {
                const bool o1 = src & 4, o2 = src & 8;
#pragma unroll
                for (int q = 0; q < KT / 4; ++q) {
                  const uint4 nxt = row[q + 1];
                  const uint32_t w[7] = {cur.x, cur.y, cur.z, cur.w, nxt.x, nxt.y, nxt.z};
                  cur = nxt;
                  uint32_t u[6];
#pragma unroll
                  for (int i = 0; i < 6; ++i) u[i] = o1 ? w[i + 1] : w[i];
#pragma unroll
                  for (int i = 0; i < 4; ++i) {
                    const int c = KT - 1 - (4 * q + i);
                    float x = __uint_as_float(o2 ? u[i + 2] : u[i]);
                    if (beyond) x = c <= c_last ? rc : x;
                    sr[c] = __float_as_uint(fmaf(x, LOG2E, __uint_as_float(sr[c])));
                  }
                }
              }
            } else if (a.rel) {   // all at E - 1 or beyond
              const float x = rc * LOG2E;
#pragma unroll
              for (int c = 0; c < KT; ++c) sr[c] = __float_as_uint(__uint_as_float(sr[c]) + x);
            }
            if (a.slopes) {
              const float slope2 = __ldg(a.slopes + head) * LOG2E, d0 = (float)(p - k0);
#pragma unroll
              for (int c = 0; c < KT; ++c) sr[c] = __float_as_uint(fmaf(-slope2, d0 - (float)c, __uint_as_float(sr[c])));
            }
          }
          if (how != NoLoad) {
            __syncwarp();
            if (lane == 0) mbar_arrive(&bias_empty[h]);
          }
        }
        // ---- keys that this row does not see
        if (part) {
          const TRRow row = my_row();
#pragma unroll
          for (int w = 0; w < KW; ++w) {
            const uint32_t vis = row.sees(a, k0 + 32 * w) & ~badw[w];
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (!((vis >> c) & 1u)) sr[32 * w + c] = 0xff800000u;   // -infinity
          }
        }
        // ---- running maximum, moved only when it grows by more than 2^8
        float mxv[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < KT; c += 2)
          mxv[(c >> 1) & 3] = fmax3(mxv[(c >> 1) & 3], __uint_as_float(sr[c]), __uint_as_float(sr[c + 1]));
        const float mx = fmaxf(fmaxf(mxv[0], mxv[1]), fmaxf(mxv[2], mxv[3])) * mul;
        const bool mine = mx > m + TR_RESCALE_LOG2;
        if (__any_sync(0xffffffffu, mine)) {
          if (j > 0) {   // every earlier product into O_h is done: s_full came after it
            const float fr = mine ? fast_exp2(m - mx) : 1.f;
#pragma unroll 1
            for (int c2 = 0; c2 < D / 16; ++c2) {
              uint32_t ov[16];
              tmem_ld16(tm_o + D * h + c2 * 16, ov);
              tmem_wait_ld();
#pragma unroll
              for (int x = 0; x < 16; ++x) ov[x] = __float_as_uint(__uint_as_float(ov[x]) * fr);
              tmem_st16(tm_o + D * h + c2 * 16, ov);
            }
            l *= fr;
          }
          if (mine) m = mx;
        }
        // ---- numerators
        const float nm = m == -INFINITY ? 0.f : -m;
        const uint64_t mul2 = f2_pack(mul, mul), nm2 = f2_pack(nm, nm);
        uint64_t ls2[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
        for (int quarter = 0; quarter < KW; ++quarter) {
          uint32_t pk[16];
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            const int e = 32 * quarter + 2 * c;
            float t0, t1;
            f2_unpack(f2_fma(f2_pack(__uint_as_float(sr[e]), __uint_as_float(sr[e + 1])), mul2, nm2), t0, t1);
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
      }
      if (!go) break;
      g += item.tiles();
      // ---- epilogue
      if (nt > 0) {
        go = tr_wait(&o_full[h], (on >> h) & 1u, abort_flag, a);
        if (!go) break;
      }
      const bool both = merge && item.part[1].nt > 0;   // both chains hold a part of this row
      float M = l == 0.f ? -INFINITY : m, f0 = 1.f, f1 = 0.f;   // weights of O_h, or of O_0 and O_1
      if (merge) {
        // (The next item's are written once its own O is there, which waits for o_free.  A chain without a tile has nothing to say.)
        if (nt > 0) ml[h * TREE_ROWS + r] = make_float2(M, l);
        __syncwarp();
        if (lane == 0) mbar_arrive(ml_bar);
        go = tr_wait(ml_bar, mn & 1u, abort_flag, a);
        if (!go) break;
        ++mn;
        if (h == 1 || both) go = tr_wait(&o_full[h ^ 1], (on >> (h ^ 1)) & 1u, abort_flag, a);   // (its warps have waited for it)
        if (!go) break;
        const float2 x0 = ml[r], x1 = both ? ml[TREE_ROWS + r] : make_float2(-INFINITY, 0.f);
        M = fmaxf(x0.x, x1.x);
        f0 = x0.x == -INFINITY ? 0.f : fast_exp2(x0.x - M);
        f1 = x1.x == -INFINITY ? 0.f : fast_exp2(x1.x - M);
        l = (x0.y == 0.f ? 0.f : x0.y * f0) + (x1.y == 0.f ? 0.f : x1.y * f1);
      }
      on ^= merge && !both ? 1u : 3u;
      tc_fence_after();
      const volatile int* ps = poison + 4 * (k % TR_ITEMS) + (merge || pair ? 0 : 2 * h);
      const int pfirst = both ? min(ps[0], ps[2]) : ps[0], plast = both ? max(ps[1], ps[3]) : ps[1];
      const bool whole = it.parts <= 1, nothing = l == 0.f;
      const float inv = whole ? (nothing ? 0.f : 1.f / l) : 1.f;   // (a NaN stays one)
      const float g0 = nothing ? 0.f : f0 * inv, g1 = nothing ? 0.f : f1 * inv;
      const uint32_t o0 = tm_o + (merge ? 0 : D * h);
      const size_t orow = (size_t)t * a.Hq + head;
      const int rt = pair ? h : 0;   // row tile
      float4* part_o = reinterpret_cast<float4*>(a.part_o) + ((size_t)it.place * 2 + rt) * (D / 4) * TREE_ROWS + r;
      // after a merge each of the two threads of a row has half of its channels
      const int c_first = merge ? h * (D / 64) : 0, c_end = merge ? c_first + D / 64 : D / 32;
#pragma unroll 1
      for (int c2 = c_first; c2 < c_end; ++c2) {
        uint32_t ov[32];
        tmem_ld32(o0 + c2 * 32, ov);
        float odd = 0.f;   // NaN if there is an infinity or NaN
        if (both) {
          uint32_t ow[32];
          tmem_ld32(tm_o + D + c2 * 32, ow);
          tmem_wait_ld();
#pragma unroll
          for (int x = 0; x < 32; ++x) {
            const float y = fmaf(g1, __uint_as_float(ow[x]), g0 * __uint_as_float(ov[x]));
            odd = fmaf(y, 0.f, odd);
            ov[x] = __float_as_uint(y);
          }
          if (__any_sync(0xffffffffu, odd != odd)) {   // (an infinity must not meet a weight of 0)
            tmem_ld32(o0 + c2 * 32, ov);
            tmem_wait_ld();
#pragma unroll
            for (int x = 0; x < 32; ++x)
              ov[x] = nothing ? 0u : __float_as_uint(tr_weigh(g0, __uint_as_float(ov[x])) + tr_weigh(g1, __uint_as_float(ow[x])));
          }
        } else {
          tmem_wait_ld();
#pragma unroll
          for (int x = 0; x < 32; ++x) ov[x] = nothing ? 0u : __float_as_uint(__uint_as_float(ov[x]) * g0);
        }
        if (plast >= 0 && rv) {
          const TRRow row = my_row();
          // infinities and NaN of the keys this row sees, from the first tile to the last that holds one
#pragma unroll 1
          for (int tile = pfirst; tile <= plast; ++tile)
#pragma unroll 1
            for (int w = 0; w < KW; ++w)
#pragma unroll 1
              for (uint32_t vis = row.sees(a, tile * KT + 32 * w); vis; vis &= vis - 1) {
                const int kk = tile * KT + 32 * w + __ffs(vis) - 1;
                const int page = __ldg(a.block_table + (size_t)it.b * a.max_pages + (kk >> a.log2_page));
                if (page < 0 || page >= a.num_pages) continue;
                const uint16_t* vp = static_cast<const uint16_t*>(a.v) +
                                     ((((size_t)page * a.Hkv + it.kvh) << a.log2_page) + (kk & (P - 1))) * D + c2 * 32;
#pragma unroll
                for (int x = 0; x < 32; ++x) {
                  const uint32_t v = (uint32_t)__ldg(vp + x) << 16;
                  if ((v & 0x7F800000u) == 0x7F800000u) ov[x] = __float_as_uint(__uint_as_float(ov[x]) + __uint_as_float(v));
                }
              }
        }
        if (!whole) {
#pragma unroll
          for (int x = 0; x < 8 && rv; ++x)
            __stcg(part_o + (size_t)(c2 * 8 + x) * TREE_ROWS,
                   make_float4(__uint_as_float(ov[4 * x]), __uint_as_float(ov[4 * x + 1]), __uint_as_float(ov[4 * x + 2]),
                               __uint_as_float(ov[4 * x + 3])));
        } else if (rv) {
          uint4* o = reinterpret_cast<uint4*>(out + orow * D) + c2 * 4;
#pragma unroll
          for (int x = 0; x < 4; ++x)
            o[x] = make_uint4(pack_bf16(__uint_as_float(ov[8 * x]), __uint_as_float(ov[8 * x + 1])),
                              pack_bf16(__uint_as_float(ov[8 * x + 2]), __uint_as_float(ov[8 * x + 3])),
                              pack_bf16(__uint_as_float(ov[8 * x + 4]), __uint_as_float(ov[8 * x + 5])),
                              pack_bf16(__uint_as_float(ov[8 * x + 6]), __uint_as_float(ov[8 * x + 7])));
        }
      }
      if (!merge || h == 0) {
        if (!whole) __stcg(reinterpret_cast<float2*>(a.part_ml) + ((size_t)it.place * 2 + rt) * TREE_ROWS + r, make_float2(M, l));
        else if (rv && a.lse) a.lse[orow] = nothing ? -INFINITY : M * LN2 + logf(l);
      }
      tc_fence_before();
      __syncwarp();
      if (merge && lane == 0) mbar_arrive(o_free);
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

// Items that a run begins and does not end: block x takes the one that CTA x of the attention began, block y a row tile and 16
// channels, a thread a row.  Pieces are added in order, so results do not depend on who finishes when.
template <int D>
__global__ void __launch_bounds__(TREE_ROWS) tree_join_kernel(const TreeArgs a) {
  const TreeCut cut = a.cuts[blockIdx.x];
  const int rt = blockIdx.y / (D / 16), c = blockIdx.y - rt * (D / 16);
  if (cut.parts <= 1 || rt * a.tok_per_tile >= cut.ntok) return;
  const int r = threadIdx.x, i = r / a.heads_per_tile, gq = r - i * a.heads_per_tile, ti = rt * a.tok_per_tile + i;
  if (i >= a.tok_per_tile || ti >= cut.ntok || gq >= cut.gh) return;
  // piece x of the item is at place 2 (first + x), the first at 2 first + 1
  auto place = [&](int x) { return (size_t)(2 * ((int)blockIdx.x + x) + (x == 0 ? 1 : 0)) * 2 + rt; };
  const float2* ml = reinterpret_cast<const float2*>(a.part_ml) + r;
  const float4* po = reinterpret_cast<const float4*>(a.part_o) + (size_t)c * 4 * TREE_ROWS + r;
  float M = -INFINITY;
#pragma unroll 8
  for (int x = 0; x < cut.parts; ++x) M = fmaxf(M, __ldcg(ml + place(x) * TREE_ROWS).x);
  float l = 0.f, acc[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) acc[e] = 0.f;
#pragma unroll 4
  for (int x = 0; x < cut.parts; ++x) {
    const float2 p = __ldcg(ml + place(x) * TREE_ROWS);
    float4 v[4];
#pragma unroll
    for (int y = 0; y < 4; ++y) v[y] = __ldcg(po + (place(x) * (D / 4) + y) * TREE_ROWS);
    const float w = p.x == -INFINITY ? 0.f : fast_exp2(p.x - M);
    if (p.y != 0.f) l = fmaf(p.y, w, l);
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      acc[4 * y] += tr_weigh(w, v[y].x);
      acc[4 * y + 1] += tr_weigh(w, v[y].y);
      acc[4 * y + 2] += tr_weigh(w, v[y].z);
      acc[4 * y + 3] += tr_weigh(w, v[y].w);
    }
  }
  const bool nothing = l == 0.f;
  const float inv = nothing ? 0.f : 1.f / l;
  uint32_t o[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) o[e] = nothing ? 0u : pack_bf16(acc[2 * e] * inv, acc[2 * e + 1] * inv);
  const size_t row = (size_t)(cut.t0 + ti) * a.Hq + cut.h0 + gq;
  uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + row * D + c * 16);
  dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
  dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
  if (c == 0 && a.lse) a.lse[row] = nothing ? -INFINITY : M * LN2 + logf(l);
}

template <int D, bool CAP, bool BIAS>
cudaError_t launch_t(const MaskedMaps& m, const TreeArgs& a, int grid, cudaStream_t stream) {
  using S = TRShape<D, BIAS>;
  static std::atomic<unsigned long long> opted{0};
  cudaError_t e = smem_opt_in_once(tree_kernel<D, CAP, BIAS>, (int)TRSmem<D, BIAS>::alloc, opted);
  if (e != cudaSuccess) return e;
  // The softmax warps' extra registers come out of what the block is launched with: a build with
  // fewer would wait for them without end.
  static const bool enough = [] {
    cudaFuncAttributes at;
    return BIAS || (cudaFuncGetAttributes(&at, tree_kernel<D, CAP, BIAS>) == cudaSuccess &&
                    at.numRegs * S::THREADS >= 128 * (2 * TR_REGS_SOFTMAX + TR_REGS_REST));
  }();
  if (!enough) return cudaErrorInvalidConfiguration;
  tree_kernel<D, CAP, BIAS><<<grid, S::THREADS, TRSmem<D, BIAS>::alloc, stream>>>(m.k, m.v, m.q, a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  tree_join_kernel<D><<<dim3(grid, 2 * (D / 16)), TREE_ROWS, 0, stream>>>(a);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_d(const MaskedMaps& m, const TreeArgs& a, int grid, cudaStream_t stream) {
  const bool cap = a.softcap != 0.f;
  if (a.rel || a.slopes) return cap ? launch_t<D, true, true>(m, a, grid, stream) : launch_t<D, false, true>(m, a, grid, stream);
  return cap ? launch_t<D, true, false>(m, a, grid, stream) : launch_t<D, false, false>(m, a, grid, stream);
}

}  // namespace

int tree_tile_keys(bool bias) { return bias ? TRShape<128, true>::KT : TRShape<128, false>::KT; }

cudaError_t launch_tree(const MaskedMaps& m, const TreeArgs& a, int head_dim, cudaStream_t stream) {
  int dev = 0;
  const int sms = current_device_sms(&dev);
  if (sms <= 0) return cudaErrorInvalidDevice;
  const long long items = (a.T / (2ll * a.tok_per_tile) + a.B) * a.Hkv * a.head_chunks;
  const long long tiles = ((long long)a.max_pages << a.log2_page) / tree_tile_keys(a.rel || a.slopes) + 1;
  const int grid = (int)std::min<long long>(std::min(sms, TREE_MAX_CTAS), items * tiles);
  return head_dim == 128 ? launch_d<128>(m, a, grid, stream) : launch_d<64>(m, a, grid, stream);
}

}  // namespace ink
