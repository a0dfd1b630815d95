// tree.cu -- attention of drafted tokens over the paged cache on the 5th-generation tensor cores: every token sees its
// sequence's history and the drafted tokens on its way to the root.
//
//   x = sm_scale <q[t,h], K[k]>,  d = |p - pos(k)|,  s = cap(x) - slope_h d + rel[t,h,min(d, E - 1)]
//   out = softmax(s) V,  lse = log sum exp(s)
//
// A few tokens against a long history: the bytes of K and V, and of the bias rows where there is a bias tensor, bound
// it, so they have to flow evenly over the SMs whatever the lengths are.  The rows of a tile of 128 (the M of an MMA) are (token,
// query head) pairs of one sequence and KV head, tokens outermost; an item is up to two row tiles.  All tiles of 64 keys of all
// items stand in one row, tiles of an item side by side, and every CTA takes a run of them that takes as long as the others', found
// on the device from the lengths (a graph replays with other ones).  A run cuts two items at most; pieces of
// a cut item leave O, maximum and sum in fp32, two places a CTA, and a second kernel joins them in order, spread over
// all SMs (one CTA that joined the 20 pieces of an item of a single long sequence would take as long as six key tiles).
//
// Two chains a CTA, each S (64 fp32 columns of tensor memory, with P, the bf16 numerators, over its first half once S is in
// registers) and O (D columns).  An item of two row tiles gives a chain to each; two pieces of one row tile (up to 16 tokens of 8
// heads) run side by side; a piece alone gives its even key tiles to one chain and the odd ones to the other, with maxima and sums
// of their own that are joined at the end.  One row tile's serial chain (scores to registers, softmax, P V, the next S and the
// hand-overs between) takes as long as the bytes of its tiles take to arrive, so one chain alone would starve the memory.
// Without a bias a chain has two S, so that the tensor cores never wait for a softmax to hand the next tile out; 128 keys a tile
// with one S took 5 % longer, and 35 % with the scores read twice.  With a bias the second S is Q's place, and shared memory holds
// the bias instead of Q.
//
// Warps:
//   0-3, 4-7  softmax of chain 0 and 1, a thread per row
//   8         K producer: TMA boxes of whole pages or tiles, table entries 32 at a time in lanes
//   9, 12     MMA issue of chain 0 and 1 (one warp for both had each chain wait for the other's barriers)
//   10        scheduler: cuts the run into pieces, publishes them in shared memory, loads their Q tiles by TMA
//   11        V check: in tiles that not every row sees whole, rows of V that nobody sees are zeroed and so is
//             every infinity or NaN (0 * NaN would reach rows that do not see the key); rows that do see one get it back at the end
//   13        V producer; with a bias 13 and 14 bring the bias of chain 0 and 1, and 15 V
// The bias of a row has no alignment: it starts at the row's distance from the tile.  Within the history it is 64 values side by
// side, and all heads of a token start at the same distance: one TMA box a token brings them from the 16-byte boundary before
// them (128 rows by a bulk copy each: 5,000 clocks of issue).  Tiles whose distances are all E - 1 or more take one value a row,
// which changes no order among a row's scores: they stay as the tensor cores left them, and the value joins the exponent.
// Behind the history distances have no order, and a bias warp brings them element by element, a lane a key.
// Every wait is bounded; after a timeout the CTA records it, stops issuing, waits for what is in flight and exits.
//
// Measured (GPU time alone; 64 query heads, D = 128): 32 trees of up to 16 tokens against up to 16 K keys, 8 KV heads, 255 us
// (6.4 TB/s), capped 273, with slopes 444, D = 64 206; 4 of up to 16 against 64 K 137 us (6.0 TB/s); 4 of up to 61 (two items that
// read K and V each for themselves) 255 us, 0.99 PFLOP/s: 64 keys of both chains take 2,000 clocks, of which their softmax warps
// are busy 1,850 and the tensor cores 1,050; 16 of up to 16 against 16 K with 4,096 fp32 distances 211 us (147 at the rate of a
// copy), with 4,095, whose rows do not begin on 16 bytes, 829; 64 of up to 8 in a window of 512 with 512 distances 143 us (49),
// without 77 (42): items of nine tiles, whose start, masks, last tile and output run code that the instruction cache does not hold
// from one item to the next (20 % of its requests miss, against 2 % on long histories).  How the code happens to lie moves the two
// last by 5 to 8 % and D = 64 by 4 %.
#include <algorithm>
#include <climits>

#include "masked_common.cuh"
#include "prefill_common.cuh"

namespace ink {
namespace {

using namespace pf;

constexpr int TR_ITEMS = 2;       // published items in flight
constexpr int TR_BAD = 16;        // tiles whose unreadable keys are remembered (K is up to 8 ahead of a softmax)
// Barriers of K and V tiles go by tile.  A chain waits for its own tiles only, so a barrier must not be two of its phases behind
// one who waits: next to a chain's last tile its next is at most TR_DUAL_SLACK + 1 behind it (the other chain's longer
// piece, or two items of one tile, whose Q tiles a chain without tiles waits for).  Nor may it be two phases ahead of one who waits.  A
// chain frees a tile's slots after its own waits, but S, which frees K's, runs up to three tiles ahead of the one that the V check is
// at: with 8 K slots (D = 64) K of the tile 11 further on may come before the check of the next ones.  So the V check frees K's
// slots too, once it has seen K, and there are no more slots than barriers.
constexpr int TR_TILES = 8;
// What a tile takes, in units: for two row tiles (2,000 clocks; bound by its softmax), for one (1,150 to 1,500, by the softmax or by
// memory); one whose bias rows have to be read takes twice as much.  TR_ENDS tiles more for an item's start, its last tile and its
// output, TR_ENDS_BIAS with a bias tensor (10,000 clocks).  Runs of as many tiles each, against these: 4 trees of up to 61 tokens
// against 64 K keys 281 -> 255 us (some CTAs had one row tile a tile, and were done after 330 of 560 thousand clocks), 16 of up to
// 40 against 16 K with 2,048 distances 445 -> 375, of up to 16 with 4,096 221 -> 211, windows of 512 with a bias 137 -> 140.  With
// 4 for both, windows with a bias take 149; with 15 for both, 16 trees of up to 40 without one 200 instead of 193.  Two row tiles at
// 3 against 2 serve the other forms too: 4 trees of up to 61 tokens with D = 64 256 instead of 274, capped 369 (414), with slopes
// 635 (713); slopes with 15 for the ends 500 instead of 474 (16 of up to 40).
constexpr int TR_PAIR = 3, TR_ONE = 2, TR_ENDS = 4, TR_ENDS_BIAS = 15;
constexpr int TR_MIN_RUN = 4 * TR_ONE;   // least run of a CTA; no tile but an item's last takes more
constexpr int TR_DUAL_SLACK = 4;  // most tiles that two pieces may differ in to run side by side
constexpr float TR_RESCALE_LOG2 = 8.f;
// With a bias a row's scores may all be as low as its type goes (a mask written that way), where a factor of log2(e) overflows and the
// rounding of score times factor is more than an exponent holds.  Scores of TR_BIG and beyond are 16 apart or equal: of such rows only
// the keys that share the maximum weigh anything, and 2^(s - max) says so.  Maxima are kept in units of which the exponent takes two,
// s log2(e) / 2, and beyond TR_BIG as they are: one order, no overflow.
constexpr float TR_BIG = 134217728.f;

constexpr int KT = TILE_KEYS, KW = KT / 32;   // keys of a tile, words of 32
constexpr int TR_ELEMENTS = KT + 1;           // words of a bias row that is filled element by element

template <int D, bool CAP, bool BIAS>
struct TRShape {
  static constexpr int CB = D / 64;
  static constexpr int SUB = KT * 128;             // one 64-channel block of a K or V tile
  static constexpr int TILE = CB * SUB;
  static constexpr int QSUB = TREE_ROWS * 128;
  static constexpr int QTILE = CB * QSUB;
  // Ring slots, K and V tiles in turn: each kind has slots, and a producer, of its own.
  static constexpr int NS = D == 64 ? 16 : BIAS ? 8 : 10;
  static_assert(NS / 2 <= TR_TILES, "a tile's barriers are used again before all who wait have seen it");
  static constexpr int V_WARP = BIAS ? 15 : 13;    // the producer of V
  static constexpr int THREADS = (V_WARP + 1) * 32;
  // S that a chain has at a time: the second one waits for no softmax.  A bias takes the room of Q in shared memory, and Q that of
  // the second S in tensor memory.
  static constexpr int AHEAD = BIAS ? 1 : 2;
  // Scores 32 at a time, through tensor memory between their maximum and their exponentials, where there is more to do for a
  // score: straight-line code for all 64 is then longer than what the warps' instructions come from at once (two in three issue
  // slots went by without one).
  static constexpr bool ROLL = CAP || BIAS;
  static constexpr uint32_t TQ = 128;              // with a bias: S_h at 64 h, Q_h at TQ + 64 h
  static constexpr uint32_t TO = 256;              // without: S_h at 128 h, two of them; O_h at TO + D h
  static constexpr uint32_t TS = BIAS ? 64 : 128;
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

template <int D, bool CAP, bool BIAS>
struct TRSmem {
  using S = TRShape<D, CAP, BIAS>;
  static constexpr size_t q = 0;
  static constexpr size_t ring = BIAS ? 0 : 2 * (size_t)S::QTILE;
  static constexpr size_t bias = ring + (size_t)S::NS * S::TILE;
  static constexpr size_t bars = bias + (BIAS ? 2 * (size_t)TREE_BIAS_BYTES : 0);
  // k_full[TILES], v_full[TILES], v_ok[TILES], empty[NS], s_full[2][2], p_full[2][2], o_done[2][2], q_full[2], q_empty[2],
  // item_full[ITEMS], item_empty[ITEMS], o_free, ml, drain[2], bias_full[2], bias_empty[2]
  static constexpr int NBAR = S::NS + 3 * TR_TILES + 16 + 2 * TR_ITEMS + 4 + (BIAS ? 4 : 0);
  static constexpr size_t items = bars + (NBAR * 8 + 15) / 16 * 16;
  static constexpr size_t kbad = items + TR_ITEMS * sizeof(TRItem);
  static constexpr size_t poison = kbad + TR_BAD * KW * 4;
  static constexpr size_t ml = poison + TR_ITEMS * 16;           // [2 chains][128 rows] float2
  static constexpr size_t tokens = ml + 2 * TREE_ROWS * 8;       // [2 chains][128] positions (with a bias)
  static constexpr size_t misc = tokens + (BIAS ? 2 * TREE_ROWS * 4 : 0);
  static constexpr size_t alloc = misc + 16;   // (no room to align within: the array itself has to be)
  static_assert(alloc <= 227 * 1024, "shared memory budget");
};

// What runs once in a while is kept out of line: the kernel's code is longer than the caches its instructions come from.

__device__ __noinline__ bool tr_wait_slow(uint64_t* bar, uint32_t parity, volatile int* abort_flag, uint32_t* err,
                                          unsigned long long wait_ns) {
  if (*abort_flag) return false;
  if (mbar_wait_limit(bar, parity, wait_ns)) return true;
  record_error(err, INK_DEVERR_WAIT_TIMEOUT);
  *abort_flag = 1;
  return false;
}

// Bounded wait of a whole warp, with one answer for all its lanes.
__device__ __forceinline__ bool tr_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, const TreeArgs& a) {
  return __all_sync(0xffffffffu, mbar_test_wait(bar, parity) || tr_wait_slow(bar, parity, abort_flag, a.err, a.wait_ns));
}

// a / b of numbers that are not negative: tiles are fewer than 2^32 in all but the longest calls, and a 64-bit division takes ten
// times as long as one of 32 bits.
__device__ __forceinline__ long long tr_div(long long a, long long b) {
  if (((unsigned long long)(a | b) >> 32) == 0) return (uint32_t)a / (uint32_t)b;
  return a / b;
}

// A sequence's rows and keys; tiles == 0: none of its rows sees a key (or it has none).
struct TRSeq {
  int c0, n, L, lo, hi, tiles;
  int plain;      // tiles, the first ones, of which no row needs more of its bias than the last value
  uint32_t bad;   // error bits; BAD_ROWS: its rows are not touched

  __device__ __forceinline__ void load(const TreeArgs& a, int b) {
    c0 = __ldg(a.cu_q + b);
    const int c1 = __ldg(a.cu_q + b + 1);
    L = __ldg(a.seq_lens + b);
    n = c1 - c0;
    lo = hi = tiles = plain = 0;
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
      if (lo < hi) tiles = (hi - 1) / KT - lo / KT + 1;
      plain = tiles;
      if (a.rel) {   // (as tr_bias finds it)
        const long long far = (long long)L - n - (KT - 1) - (a.E - 1);   // the last first key of such a tile
        plain = far < 0 ? 0 : min(max((int)(far / KT) + 1 - lo / KT, 0), tiles);
      }
    }
  }
};

// The row of tiles, walked by a whole warp: 32 sequences at a time in the lanes.  It is measured in units; a tile belongs to the run
// in which it begins.  Divisions are made once per run: later pieces begin with their item.
struct TRWalk {
  long long base, incl, chunk, total;   // units before sequence cb; up to and with this lane's; of a run; of the 32
  long long pos, end;                   // of this CTA's run
  long long units;                      // of all items of this lane's sequence for one head chunk
  int items, last;                      // their number; units of a tile of the last one
  int cb, per, cta, ends;
  int src, left;                        // the sequence's lane; its items not begun
  int kvh, hc, item;                    // the next one
  TRSeq s;

  __device__ __forceinline__ void load(const TreeArgs& a, int lane) {
    const int b = cb + lane;
    s.tiles = s.plain = s.n = 0;
    if (b < a.B) s.load(a, b);
    items = (s.n + 2 * a.tok_per_tile - 1) / (2 * a.tok_per_tile);
    last = s.n - (items - 1) * 2 * a.tok_per_tile > a.tok_per_tile ? TR_PAIR : TR_ONE;
    units = s.tiles > 0 ? (long long)(2 * s.tiles - s.plain + ends) * (TR_PAIR * (items - 1) + last) : 0;
    incl = units * per;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    total = __shfl_sync(0xffffffffu, incl, 31);
  }

  __device__ __forceinline__ void begin(const TreeArgs& a, int lane) {
    per = a.Hkv * a.head_chunks;
    ends = a.rel ? TR_ENDS_BIAS : TR_ENDS;
    cta = (int)blockIdx.x;
    long long all = 0;
#pragma unroll 1
    for (cb = ((a.B - 1) >> 5) << 5; cb >= 0; cb -= 32) {
      load(a, lane);
      all += total;
    }
    cb = 0;
    base = 0;
    left = 0;
    chunk = max(tr_div(all + gridDim.x - 1, gridDim.x), (long long)TR_MIN_RUN);
    pos = min(cta * chunk, all);
    end = min(pos + chunk, all);
  }

  // The next piece of the run (pos < end), with no tile if there is none; first: the CTA where its item begins.
  __device__ __forceinline__ TRPart next(const TreeArgs& a, int lane, int& first) {
    TRPart w;
    int x0 = 0, ni, tiles, plain, weight;
    first = cta;
    for (;;) {
      long long off = 0;
      if (left == 0) {   // of another sequence than the one before
#pragma unroll 1
        while (pos >= base + total) {
          base += total;
          cb += 32;
          load(a, lane);
        }
        src = __ffs(__ballot_sync(0xffffffffu, pos < base + incl)) - 1;
        off = pos - (base + __shfl_sync(0xffffffffu, incl - units * per, src));
      }
      w.n = __shfl_sync(0xffffffffu, s.n, src);
      tiles = __shfl_sync(0xffffffffu, s.tiles, src);
      plain = __shfl_sync(0xffffffffu, s.plain, src);
      ni = __shfl_sync(0xffffffffu, items, src);
      const int wl = __shfl_sync(0xffffffffu, last, src), size = 2 * tiles - plain + ends;
      if (left == 0) {
        int hk = 0;
        item = 0;
        if (off > 0) {   // the run begins within a sequence
          const long long one = (long long)size * (TR_PAIR * (ni - 1) + wl);
          hk = (int)tr_div(off, one);
          off -= hk * one;
          item = min((int)tr_div(off, (long long)size * TR_PAIR), ni - 1);
          off -= (long long)item * size * TR_PAIR;
        }
        left = per * ni - (hk * ni + item);
        kvh = hk / a.head_chunks;
        hc = hk - kvh * a.head_chunks;
      }
      weight = item == ni - 1 ? wl : TR_PAIR;
      if (off > 0) {       // and within an item
        const int y = weight == TR_PAIR ? ((int)off + TR_PAIR - 1) / TR_PAIR : ((int)off + TR_ONE - 1) / TR_ONE;
        first = (int)tr_div(pos - off, chunk);
        x0 = y <= plain ? y : plain + (y - plain + 1) / 2;
        pos += (long long)weight * (x0 >= tiles ? size : x0 <= plain ? x0 : 2 * x0 - plain) - off;
        if (x0 >= tiles) { // in its last tile: the run begins with the next one
          x0 = 0;
          first = cta;
          left = 0;
          w.nt = 0;
          if (pos >= end) return w;
          continue;
        }
      }
      break;
    }
    const long long start = pos - (long long)weight * (x0 <= plain ? x0 : 2 * x0 - plain);   // of the item
    w.b = cb + src;
    w.c0 = __shfl_sync(0xffffffffu, s.c0, src);
    w.lo = __shfl_sync(0xffffffffu, s.lo, src);
    w.hi = __shfl_sync(0xffffffffu, s.hi, src);
    w.H = __shfl_sync(0xffffffffu, s.L, src) - w.n;
    w.kvh = kvh;
    w.h0 = kvh * a.G + hc * a.heads_per_tile;
    w.gh = min(a.heads_per_tile, a.G - hc * a.heads_per_tile);
    w.t0 = w.c0 + item * 2 * a.tok_per_tile;
    w.ntok = min(2 * a.tok_per_tile, w.n - item * 2 * a.tok_per_tile);
    w.kt0 = w.lo / KT + x0;
    // the tiles that begin before the run's end
    const long long room = end - start;
    int x1 = tiles;
    if (room < (long long)weight * (2 * tiles - plain + ends)) {
      const int y = weight == TR_PAIR ? ((int)room + TR_PAIR - 1) / TR_PAIR : ((int)room + TR_ONE - 1) / TR_ONE;
      x1 = min(y <= plain ? y : plain + (y - plain + 1) / 2, tiles);
    }
    w.nt = x1 - x0;
    const long long last_tile = start + (long long)weight * (tiles - 1 <= plain ? tiles - 1 : 2 * (tiles - 1) - plain);
    w.parts = (last_tile < end ? cta : (int)tr_div(last_tile, chunk)) - first + 1;
    w.place = 2 * cta + (cta == first ? 1 : 0);
    pos = start + (long long)weight * (x1 == tiles ? 2 * tiles - plain + ends : x1 <= plain ? x1 : 2 * x1 - plain);
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
    // (a load behind a select may be issued whatever the select says: every such address is one that is there)
    return i == 0 ? w0 : i > 0 && i < a.words ? __ldg(bits + min(max(i, 0), a.words - 1)) : 0u;
  }
  __device__ __forceinline__ uint32_t sees(const TreeArgs& a, int base) const {
    const int x0 = max(lo - base, 0), x1 = min(hist - base, 32);
    uint32_t vis = x1 > x0 ? (0xffffffffu >> (32 - (x1 - x0))) << x0 : 0u;
    const int j0 = base - H;
    if (j0 > -32 && j0 < nlim) {
      uint32_t t = __funnelshift_r(word(a, j0 >> 5), word(a, (j0 >> 5) + 1), j0 & 31);
      if (nlim - j0 < 32) t &= (1u << (nlim - j0)) - 1u;
      if (cut)
#pragma unroll 1
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
// side by side, brought by a box a token where rows of the tensor begin on 16 bytes, else element by element (four times as long on
// long histories); all of them at E - 1 or more are one value.
enum TRBias { NoLoad, Boxes, Elements };

__device__ __forceinline__ TRBias tr_bias(const TreeArgs& a, const TRPart& it, int k0) {
  if (min(it.H, it.hi) - k0 < KT) return Elements;
  if (!a.rel || it.H - (k0 + KT - 1) >= a.E - 1) return NoLoad;
  return a.rel_rows ? Boxes : Elements;
}

// Infinities and NaN of the keys that this row sees, in tiles first to last, into channels [c0, c1) of what it has stored: its
// output, or its partial (channel c at float 4 (c / 4) rows + c % 4).  Tiles between the windows' beginnings and the history's
// end are seen by every row and were left as they are: nothing of them is missing, and they are passed over (a look at each of
// 300 K keys, channel by channel, took longer than 20 ms, the time of hundreds of calls).  A warp that shares the work among its lanes
// needs registers that cost windows 6 %, called or not.
__device__ __noinline__ void tr_infinite(const TreeArgs& a, const TRPart& it, const TRRow& row, int first, int last, int c0, int c1,
                                         __nv_bfloat16* out, float* part, int D) {
#pragma unroll 1
  for (int w = first * KW; w < (last + 1) * KW; ++w) {
    if (w * 32 >= it.lo_max && min(it.H, it.hi) - w * 32 >= KT) w = min(it.H, it.hi) / KT * KW;
    if (w >= (last + 1) * KW) break;
    const int base = w * 32;
#pragma unroll 1
    for (uint32_t vis = row.sees(a, base); vis; vis &= vis - 1) {
      const int kk = base + __ffs(vis) - 1;
      const int page = __ldg(a.block_table + (size_t)it.b * a.max_pages + (kk >> a.log2_page));
      if (page < 0 || page >= a.num_pages) continue;
      const uint16_t* v = static_cast<const uint16_t*>(a.v) +
                          ((((size_t)page * a.Hkv + it.kvh) << a.log2_page) + (kk & ((1 << a.log2_page) - 1))) * D;
#pragma unroll 1
      for (int c = c0; c < c1; ++c) {
        if ((c & 7) == 0) {
          const uint4 x = __ldg(reinterpret_cast<const uint4*>(v + c));
          if (!((((x.x & 0x7F807F80u) + 0x00800080u) | ((x.y & 0x7F807F80u) + 0x00800080u) | ((x.z & 0x7F807F80u) + 0x00800080u) |
                 ((x.w & 0x7F807F80u) + 0x00800080u)) & 0x80008000u)) {
            c += 7;
            continue;
          }
        }
        const uint32_t x = (uint32_t)__ldg(v + c) << 16;
        if ((x & 0x7F800000u) != 0x7F800000u) continue;
        if (out) {
          out[c] = __float2bfloat16(__bfloat162float(out[c]) + __uint_as_float(x));
        } else {
          float* y = part + (size_t)(c >> 2) * 4 * TREE_ROWS + (c & 3);
          __stcg(y, __ldcg(y) + __uint_as_float(x));
        }
      }
    }
  }
}

__device__ __forceinline__ uint64_t tr_mul(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// An infinity or NaN of a part stays one, whatever the part's weight.
__device__ __forceinline__ float tr_weigh(float w, float x) { return fabsf(x) <= 3.4028235e38f ? w * x : x; }

// A maximum in natural units.
__device__ __forceinline__ float tr_natural(float m, bool bias) {
  return bias && fabsf(m) >= TR_BIG ? m : m * (bias ? 2.f * LN2 : LN2);
}

// CAP: capped scores, by a polynomial where all scores of a warp's tile allow it (as in the masked prefill).
template <int D, bool CAP, bool BIAS>
__global__ void __launch_bounds__(TRShape<D, CAP, BIAS>::THREADS, 1)
tree_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
            const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmB,
            const __grid_constant__ TreeArgs a) {
  using S = TRShape<D, CAP, BIAS>;
  using L_ = TRSmem<D, CAP, BIAS>;
  constexpr int NS = S::NS;

  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + L_::bars);
  uint64_t* v_full = k_full + TR_TILES;
  uint64_t* v_ok = v_full + TR_TILES;   // V tile checked
  uint64_t* empty = v_ok + TR_TILES;
  uint64_t* s_full = empty + NS;        // [2 chains][2] S in TMEM, every product before it done
  uint64_t* p_full = s_full + 4;        // [2 chains][2] P written
  uint64_t* o_done = p_full + 4;        // [2 chains][2] product of that P done
  uint64_t* q_full = o_done + 4;        // [2]
  uint64_t* q_empty = q_full + 2;       // [2] the piece's last product with a Q tile done, and all waits for it
  uint64_t* item_full = q_empty + 2;    // [ITEMS]
  uint64_t* item_empty = item_full + TR_ITEMS;
  uint64_t* o_free = item_empty + TR_ITEMS;   // both O of a Split item read
  uint64_t* ml_bar = o_free + 1;        // maxima and sums of both chains written
  uint64_t* drain = ml_bar + 1;         // [2]
  uint64_t* bias_full = drain + 2;      // [2]
  uint64_t* bias_empty = bias_full + 2; // [2]
  TRItem* items = reinterpret_cast<TRItem*>(smem + L_::items);
  uint32_t* kbad = reinterpret_cast<uint32_t*>(smem + L_::kbad);   // [BAD][KW] bit per unreadable key
  int* poison = reinterpret_cast<int*>(smem + L_::poison);   // [ITEMS][2 chains][2] first and last tile of V with an infinity or NaN
  float2* ml = reinterpret_cast<float2*>(smem + L_::ml);
  uint8_t* bias = smem + L_::bias;
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
    for (int x = 0; x < NS; ++x) mbar_init(&empty[x], x & 1 ? 2 : 3);   // two products; K's wait for the V check too
    for (int x = 0; x < TR_TILES; ++x) {
      mbar_init(&k_full[x], 1);
      mbar_init(&v_full[x], 1);
      mbar_init(&v_ok[x], 1);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&s_full[2 * x], 1);
      mbar_init(&s_full[2 * x + 1], 1);
      mbar_init(&p_full[2 * x], 4);
      mbar_init(&p_full[2 * x + 1], 4);
      mbar_init(&o_done[2 * x], 1);
      mbar_init(&o_done[2 * x + 1], 1);
      mbar_init(&q_full[x], BIAS ? 4 : 1);
      mbar_init(&q_empty[x], 3);   // last products, and a chain that has no part in them (Split: the first) is past its wait
      mbar_init(&drain[x], 1);
      if constexpr (BIAS) {
        mbar_init(&bias_full[x], 32);   // every lane of a warp
        mbar_init(&bias_empty[x], 4);
      }
    }
    for (int x = 0; x < TR_ITEMS; ++x) {
      mbar_init(&item_full[x], 1);
      mbar_init(&item_empty[x], 13 + (BIAS ? 2 : 0));   // producers, 2 MMA, V check, 8 softmax warps, bias warps
    }
    mbar_init(o_free, 8);
    mbar_init(ml_bar, 8);
    fence_mbar_init();
    *abort_flag = 0;
  }
  TRWalk walk;
  if (warp == 10) walk.begin(a, lane);   // (its loads are on their way while the rest is set up)
  // rows of a Q tile past the last (token, head) pair stay zero
  if constexpr (!BIAS) {
    for (int x = tid; x < 2 * S::QTILE / 16; x += S::THREADS)
      *reinterpret_cast<uint4*>(smem + L_::q + (size_t)x * 16) = make_uint4(0u, 0u, 0u, 0u);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
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
    if (warp == 8 || warp == S::V_WARP) {
      // ---------------------------------------------------------------- K and V producer
      if (lane == 0) {
        prefetch_tensormap(&tmK);
        prefetch_tensormap(&tmV);
      }
      const int seg = min(P, KT), nseg = KT / seg;
      const bool wide = P >= KT;            // a tile lies in one page: one box a tensor
      const int kv = warp != 8;             // K or V
      int x = 0, st = kv;                   // tiles issued, slot of the next one
      uint32_t round = 0;                   // times the slots have been gone through
      bool go = true;
      for (int k = 0; go && next_item(k); ++k) {
        const TRItem& item = items[k % TR_ITEMS];
        const int parts = item.mode == Pair ? 1 : 2, longest = item.longest(), kstep = item.step() * KT;
        const int32_t* bt[2];
        int kvh[2], lo[2], hi[2], nt[2], k0[2], chunk_base[2], chunk_val[2];   // table entries chunk_base + lane, of each chain's part
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const TRPart& it = item.part[h];
          bt[h] = a.block_table + (size_t)it.b * a.max_pages;
          kvh[h] = it.kvh;
          lo[h] = it.lo;
          hi[h] = it.hi;
          nt[h] = h < parts ? it.nt : 0;
          k0[h] = it.kt0 * KT;
          chunk_base[h] = k0[h] >> a.log2_page;   // entries past the sequence's last key are not read
          chunk_val[h] = __ldg(bt[h] + min(chunk_base[h] + lane, (hi[h] - 1) >> a.log2_page));
        }
        done_item(k);
        for (int j = 0; j < longest && go; ++j) {   // (the chains' tiles take turns)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (!go || j >= nt[h]) continue;
            if (((k0[h] + KT - 1) >> a.log2_page) >= chunk_base[h] + 32) {
              chunk_base[h] = k0[h] >> a.log2_page;
              chunk_val[h] = __ldg(bt[h] + min(chunk_base[h] + lane, (hi[h] - 1) >> a.log2_page));
            }
            const int ks = k0[h] + (wide ? 0 : lane * seg);   // lane < nseg takes one segment
            const bool want = lane < nseg && ks < hi[h] && ks + seg > lo[h];
            const int page = __shfl_sync(0xffffffffu, chunk_val[h], min(max((ks >> a.log2_page) - chunk_base[h], 0), 31));
            const bool bad_seg = want && (page < 0 || page >= a.num_pages);
            const bool load = want && !bad_seg;
            const uint32_t bmask = __ballot_sync(0xffffffffu, bad_seg);
            const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, load)) * (uint32_t)(seg * D * 2);
            const int row = load ? ((page * a.Hkv + kvh[h]) << a.log2_page) + (ks & (P - 1)) : 0;
            if (round > 0) go = tr_wait(&empty[st], (round - 1) & 1u, abort_flag, a);
            if (!go) continue;
            uint64_t* full = (kv ? v_full : k_full) + x % TR_TILES;
            uint8_t* dst = smem + L_::ring + (size_t)st * S::TILE + (wide ? 0 : lane * seg * 128);
            if (lane == 0) {
              if (kv == 0) {   // keys of this tile whose page is outside the pool
                uint64_t bad = 0;
#pragma unroll 1
                for (uint32_t mm = bmask; mm; mm &= mm - 1) bad |= (~0ull >> (64 - seg)) << ((__ffs(mm) - 1) * seg);
                *reinterpret_cast<uint64_t*>(kbad + x % TR_BAD * KW) = bad;
                if (bmask) record_error(a.err, INK_DEVERR_PAGE_OUT_OF_RANGE);
              }
              mbar_arrive_expect_tx(full, bytes);
              if (wide && load) tma_load_3d(dst, kv ? &tmV : &tmK, 0, row, 0, full);
            }
            if (!wide && load) {
#pragma unroll
              for (int cb = 0; cb < S::CB; ++cb)
                tma_load_2d(dst + cb * S::SUB, kv ? &tmV : &tmK, cb * 64, row, full);
            }
            st += 2;
            if (st >= NS) {
              st = kv;
              ++round;
            }
            ++x;
            k0[h] += kstep;
          }
        }
      }
      if (lane == 0) pp_drain_ring(kv ? v_full : k_full, TR_TILES, x, a.err);
    } else if (warp == 9 || warp == 12) {
      // ---------------------------------------------------------------- MMA issue of one chain
      constexpr uint32_t IDESC_S = umma_idesc_bf16(128, KT, false, false);
      constexpr uint32_t IDESC_PV = umma_idesc_bf16(128, D, false, true);
      const int h = warp == 12;
      const uint32_t qaddr = smem_u32(smem + L_::q), raddr = smem_u32(smem + L_::ring);
      const uint32_t tm_s = tmem + S::TS * h, tm_o = tmem + S::TO + (uint32_t)(D * h), tm_q = tmem + S::TQ + 64u * h;
      int g = 0;                       // tiles of earlier items: K of tile x is fill 2 x, V fill 2 x + 1
      uint32_t qn = 0;                 // a parity bit per Q tile (with a bias, of the only one)
      uint32_t sc = 0, pc = 0;         // S and P V products so far: the two S take turns
      bool go = true;
      auto wait_tile = [&](uint64_t* bars, int x) {
        return tr_wait(&bars[x % TR_TILES], (uint32_t)(x / TR_TILES) & 1u, abort_flag, a);
      };
      // What both chains may read is free after two arrivals: one of each, or both of the only one.
      auto free_slot = [&](uint64_t* bar, bool shared) {
        if (!shared && lane == 0) mbar_arrive(bar);
        umma_commit_warp(bar);
      };
      uint32_t merges = 0;             // Split items so far
      bool merged = false;             // the item before was one
      for (int k = 0; go && next_item(k); ++k) {
        const TRItem& it = items[k % TR_ITEMS];
        const bool pair = it.mode == Pair, split = it.mode == Split;
        const int qs = split ? it.qs : h, beside = it.beside(h), nt = it.of(h).nt, all = it.tiles();
        const uint64_t qd = umma_desc_sw128(qaddr + qs * S::QTILE, 16, 1024);
        auto issue_s = [&](int j) {
          const int x = g + j + min(j + h, beside);
          go = wait_tile(k_full, x);
          if (!go) return;
          tc_fence_after();
          const int st = 2 * x % NS, last = j + 1 == nt;
          const uint64_t kd = umma_desc_sw128(raddr + st * S::TILE, 16, 1024);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            if constexpr (BIAS)
              umma_ts_warp(tm_s, tm_q + kk * 8, kd + (uint64_t)(((kk >> 2) * S::SUB + (kk & 3) * 32) >> 4), IDESC_S,
                           kk > 0 ? 1u : 0u);
            else
              umma_ss_warp(tm_s + KT * (sc & 1u), qd + (uint64_t)(((kk >> 2) * S::QSUB + (kk & 3) * 32) >> 4),
                           kd + (uint64_t)(((kk >> 2) * S::SUB + (kk & 3) * 32) >> 4), IDESC_S, kk > 0 ? 1u : 0u);
          umma_commit_warp(&s_full[2 * h + (sc & 1u)]);
          ++sc;
          free_slot(&empty[st], pair);
          if (!BIAS && last) free_slot(&q_empty[qs], split);
          __syncwarp();
        };
        if constexpr (BIAS) {
          if (nt > 0) {                // (its warps have brought the rows)
            go = tr_wait(&q_full[h], qn, abort_flag, a);
            qn ^= 1u;
          }
        } else {
          // (Every phase is waited for, of the other chain's Q tile and by a chain without a tile too: a parity tells a phase from
          // its neighbours only.  A Q tile goes back when both chains are past that wait: each tells so at its item's end.)
          go = tr_wait(&q_full[qs], (qn >> qs) & 1u, abort_flag, a);
          if (go && !split) go = tr_wait(&q_full[h ^ 1], (qn >> (h ^ 1)) & 1u, abort_flag, a);
          qn ^= split ? 1u << qs : 3u;
        }
        if (!go) break;
        if (nt > 0) {
          tc_fence_after();
#pragma unroll 1
          for (int j = 0; j < S::AHEAD && j < nt && go; ++j) issue_s(j);
        } else if (!BIAS) {            // (the only tile of a Split item is the other chain's)
          if (lane == 0) mbar_arrive(&q_empty[qs]);
          __syncwarp();
        }
        // both O of a Split item have been read (a chain without a tile does not wait: the item may be over before it looks, and the
        // one after would have the parity of the one before)
        if (go && merged && nt > 0) go = tr_wait(o_free, (merges - 1) & 1u, abort_flag, a);
        for (int j = 0; j < nt && go; ++j) {
          const int x = g + j + min(j + h, beside);
          // (v_ok comes after v_full)
          go = wait_tile(v_ok, x) && tr_wait(&p_full[2 * h + (pc & 1u)], (pc >> 1) & 1u, abort_flag, a);
          if (!go) break;
          tc_fence_after();
          const int st = (2 * x + 1) % NS;
          const uint64_t vd = umma_desc_sw128(raddr + st * S::TILE, S::SUB, 1024);
#pragma unroll
          for (int ks = 0; ks < KT / 16; ++ks)
            umma_ts_warp(tm_o, tm_s + (BIAS ? 0 : KT * (pc & 1u)) + ks * 8, vd + (uint64_t)((ks * 16 * 128) >> 4), IDESC_PV, (j > 0 || ks > 0) ? 1u : 0u);
          umma_commit_warp(&o_done[2 * h + (pc & 1u)]);
          ++pc;
          free_slot(&empty[st], pair);
          __syncwarp();
          if (j + S::AHEAD < nt) issue_s(j + S::AHEAD);   // (with two: over the P just read)
        }
        // (the other chain's Q tile, seen above; at the wait itself it cost short items 5 to 10 %)
        if (!BIAS && go && lane == 0 && (!split || h == 0)) mbar_arrive(&q_empty[split ? qs : h ^ 1]);
        merged = split;
        merges += split;
        g += all;
        done_item(k);
      }
      umma_commit_warp(&drain[h]);
      __syncwarp();
      if (!mbar_wait_bounded(&drain[h], 0)) record_error(a.err, INK_DEVERR_WAIT_TIMEOUT);
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
        if (w.nt == 0) return w;
        if (w.parts > 1 && first == (int)blockIdx.x) cut = {w.parts, w.t0, w.ntok, w.h0, w.gh};
        // all rows see the keys from the largest first one on
        w.lo_max = 0;
        if (a.W > 0) {
#pragma unroll 1
          for (int i = lane; i < w.ntok; i += 32) w.lo_max = max(w.lo_max, max(__ldg(a.positions + w.t0 + i), w.H) - a.W + 1);
          w.lo_max = __reduce_max_sync(0xffffffffu, w.lo_max);
        }
        return w;
      };
      TRPart next;
      bool have = false;                 // next was looked at, and did not go beside the one before
      for (int k = 0;; ++k) {
        const int sl = k % TR_ITEMS;
        TRItem it;
        it.mode = End;
        it.qs = 0;
#pragma unroll 1
        for (int x = 0; x < 2; ++x) {
          if (!have) {
            if (walk.pos >= walk.end) break;
            next = piece();
            if (next.nt == 0) break;
            have = true;
          }
          if (x == 0) {
            it.part[0] = it.part[1] = next;
            it.mode = next.ntok > a.tok_per_tile ? Pair : Split;
            have = false;
            if (it.mode == Pair) break;
          } else if (next.ntok <= a.tok_per_tile && abs(it.part[0].nt - next.nt) <= TR_DUAL_SLACK) {
            it.part[1] = next;
            it.mode = Dual;
            have = false;
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
        if (it.mode == Split) {
          it.part[0].nt = (it.part[0].nt + 1) >> 1;
          it.part[1].nt >>= 1;
          if (it.part[1].nt > 0) ++it.part[1].kt0;   // (a part without a tile keeps a tile that is there: its table entries are read)
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
        for (int x = 0; !BIAS && x < (it.mode == Split ? 1 : 2) && go; ++x) {
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
#pragma unroll 1
        for (int s = 0; s < 2; ++s)
          if (((loaded >> s) & 1u) && !mbar_wait_bounded(&q_full[s], ((qn >> s) & 1u) ^ 1u)) record_error(a.err, INK_DEVERR_WAIT_TIMEOUT);
      }
    } else if (warp == 11) {
      // ---------------------------------------------------------------- V check
      int g = 0;
      bool go = true;
      for (int k = 0; go && next_item(k); ++k) {
        const TRItem& item = items[k % TR_ITEMS];
        const int longest = item.longest(), step = item.step();
        for (int j = 0; j < longest && go; ++j) {
          for (int h = 0; h < (item.mode == Pair ? 1 : 2); ++h) {
            const TRPart& it = item.part[h];
            if (j >= it.nt) continue;
            const int hist = min(it.H, it.hi), kt = it.kt0 + j * step;
            const int st = (2 * g + 1) % NS;
            // (what cannot be read comes with K)
            go = tr_wait(&k_full[g % TR_TILES], (uint32_t)(g / TR_TILES) & 1u, abort_flag, a);
            if (!go) break;
            if (lane == 0) mbar_arrive(&empty[2 * g % NS]);
            go = tr_wait(&v_full[g % TR_TILES], (uint32_t)(g / TR_TILES) & 1u, abort_flag, a);
            if (!go) break;
            const int k0 = kt * KT;
            const uint32_t* badw = kbad + (g % TR_BAD) * KW;
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
        }
        done_item(k);
      }
    } else if constexpr (BIAS) {
      // ---------------------------------------------------------------- bias loads of one chain
      const int h = warp - 13;
      uint8_t* boxes = bias + h * TREE_BIAS_BYTES;
      float* buf = reinterpret_cast<float*>(boxes);
      const int size = a.rel_bf16 ? 2 : 4;
      // without a tensor the first position is loaded instead, and not used
      const void* rel = a.rel ? a.rel : a.positions;
      const int pitch = a.rel ? a.E : 0, last = a.rel ? a.E - 1 : 0;
      const float per_head = 1.f / a.heads_per_tile;   // (rows are few: no rounding shows)
      int* at_s = reinterpret_cast<int*>(smem + L_::tokens) + h * TREE_ROWS;   // positions of the part's tokens
      if (lane == 0 && a.rel_rows) prefetch_tensormap(&tmB);
      uint32_t fills = 0;
      bool go = true;
      for (int k = 0; go && next_item(k); ++k) {
        const TRItem& item = items[k % TR_ITEMS];
        const TRPart& it = item.of(h);
        const int tok0 = item.mode == Pair ? h * a.tok_per_tile : 0;
        const int rows = min(a.tok_per_tile, it.ntok - tok0) * a.heads_per_tile;
        const int tokens = min(a.tok_per_tile, it.ntok - tok0), first_t = it.t0 + tok0;
        int pt[4];                         // positions of this lane's tokens lane, lane + 32, ...
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          pt[x] = max(__ldg(a.positions + it.t0 + tok0 + min(32 * x + lane, tokens - 1)), it.H);
          at_s[32 * x + lane] = pt[x];
        }
        __syncwarp();
        for (int j = 0; j < it.nt && go; ++j) {
          const int k0 = (it.kt0 + j * item.step()) * KT;
          const TRBias how = tr_bias(a, it, k0);
          if (how == NoLoad) continue;
          if (fills > 0) go = tr_wait(&bias_empty[h], (fills - 1) & 1u, abort_flag, a);
          if (!go) break;
          ++fills;
          if (how == Boxes) {
            // a token's rows from the 16 bytes that hold their first distance in the tile (those at E - 1 or beyond alone: none)
            int at[4], n = 0;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const int s = pt[x] - (k0 + KT - 1);
              at[x] = 32 * x + lane < tokens && s < a.E ? s & ~(16 / size - 1) : -1;
              n += at[x] >= 0;
            }
            mbar_arrive_expect_tx(&bias_full[h], (uint32_t)(n * a.heads_per_tile * tree_bias_cols(a.rel_bf16) * size));
#pragma unroll
            for (int x = 0; x < 4; ++x)
              if (at[x] >= 0)
                tma_load_3d(boxes + (32 * x + lane) * a.bias_stride, &tmB, at[x], it.h0, it.t0 + tok0 + 32 * x + lane, &bias_full[h]);
            __syncwarp();
            continue;
          }
          // element by element: a lane has two keys and goes over the rows
          int pk[2];
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int kk = k0 + 32 * x + lane;
            pk[x] = kk >= it.H && kk < it.hi ? max(__ldg(a.positions + it.c0 + min(max(kk - it.H, 0), it.n - 1)), it.H) : kk;
          }
          // (all loads of a batch first, from rows that are there: what is not seen is masked)
          auto fill = [&](auto load) {
#pragma unroll 1
            for (int r = 0; r < rows; r += 8) {
              float v[8][2];
#pragma unroll
              for (int y = 0; y < 8; ++y) {
                const int rr = min(r + y, rows - 1), i = (int)(((float)rr + 0.5f) * per_head), hd = min(rr - i * a.heads_per_tile, it.gh - 1);
                const int t = first_t + i, p = at_s[i];
                const float slope = a.slopes ? __ldg(a.slopes + it.h0 + hd) : 0.f;
                const size_t row = ((size_t)t * a.Hq + it.h0 + hd) * pitch;
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                  const int d = abs(p - pk[x]);
                  v[y][x] = fmaf(-slope, (float)d, load(row + min(d, last)));
                }
              }
#pragma unroll
              for (int y = 0; y < 8; ++y) {
                buf[(r + y) * TR_ELEMENTS + KT - 1 - lane] = v[y][0];
                buf[(r + y) * TR_ELEMENTS + KT - 33 - lane] = v[y][1];
              }
            }
          };
          if (a.rel_bf16) fill([&](size_t x) { return __uint_as_float((uint32_t)__ldg(static_cast<const uint16_t*>(a.rel) + x) << 16); });
          else fill([&](size_t x) {
            const float v = __ldg(static_cast<const float*>(rel) + x);
            return a.rel ? v : 0.f;
          });
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
    const int h = warp >> 2, r = tid & 127;
    const uint32_t tlane = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t tm_chain = tlane + S::TS * h, tm_o = tlane + S::TO;
    const int my_i = r / a.heads_per_tile, my_g = r - my_i * a.heads_per_tile;
    __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(a.out);

    // sequences that see no key: zero rows, shared out over the CTAs; what is wrong with a sequence is told here
#pragma unroll 1
    for (int b = (int)blockIdx.x; b < a.B; b += (int)gridDim.x) {
      TRSeq s;
      s.load(a, b);
      if (tid == 0 && s.bad) record_error(a.err, s.bad);
      if (s.tiles > 0 || s.n <= 0) continue;
#pragma unroll 1
      for (long long x = tid; x < (long long)s.n * a.Hq * (D / 8); x += 256)
        reinterpret_cast<uint4*>(out + (size_t)s.c0 * a.Hq * D)[x] = make_uint4(0u, 0u, 0u, 0u);
      if (a.lse)
#pragma unroll 1
        for (long long x = tid; x < (long long)s.n * a.Hq; x += 256) a.lse[(size_t)s.c0 * a.Hq + x] = -INFINITY;
    }

    const bool scaled = CAP || BIAS || !(a.scale_log2 > 0.f);
    // With a bias scores are kept in natural units until the exponent: what is added needs no factor.
    const float mul_ = BIAS ? LOG2E : scaled ? 1.f : a.scale_log2;
    constexpr float UNIT = BIAS ? 2.f : 1.f;    // of a maximum, in the exponent
    const float pre = CAP ? LN2 : a.sm_scale;   // of the score to which a bias is added
    uint32_t c = 0, c_other = 0, bn = 0, mn = 0;   // tiles of this chain and of the other one so far
    int g = 0;
    bool go = true;
    for (int k = 0; go && next_item(k); ++k) {
      const TRItem& item = items[k % TR_ITEMS];
      const TRPart& it = item.of(h);
      const int nt = it.nt;
      const bool pair = item.mode == Pair, merge = item.mode == Split;
      const int ti = (pair ? h * a.tok_per_tile : 0) + my_i;
      const bool rv = my_i < a.tok_per_tile && ti < it.ntok && my_g < it.gh;
      const int t = it.t0 + (rv ? ti : 0), head = it.h0 + (rv ? my_g : 0);
      const int p = max(__ldg(a.positions + t), it.H);
      const uint32_t w0 = __ldg(a.ancestors + (size_t)t * a.words);
      auto my_row = [&]() { return tr_row(a, it, t, p, w0, rv); };
      float rc = 0.f, slope = 0.f;   // the row's last value and its slope
      if constexpr (BIAS) {
        if (a.slopes) slope = __ldg(a.slopes + head);
        if (a.rel) {
          const size_t x = ((size_t)t * a.Hq + head + 1) * a.E - 1;
          const void* here = a.positions;   // (for the load of the other type)
          const uint32_t two = __ldg(a.rel_bf16 ? static_cast<const uint16_t*>(a.rel) + x : static_cast<const uint16_t*>(here));
          const float one = __ldg(a.rel_bf16 ? static_cast<const float*>(here) : static_cast<const float*>(a.rel) + x);
          rc = a.rel_bf16 ? __uint_as_float(two << 16) : one;
        }
      }
      const bool near0 = BIAS && __all_sync(0xffffffffu, fabsf(rc) < TR_BIG);   // (beyond, a score's own bits are lost beside it)
      const size_t orow = (size_t)t * a.Hq + head;
      if (BIAS && nt > 0) {   // Q straight into tensor memory, a row a thread (every product with the one before is done)
#pragma unroll 1
        for (int c2 = 0; c2 < D / 64; ++c2) {
          const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) + orow * D) + 8 * c2;
          uint32_t qv[32];
#pragma unroll
          for (int x = 0; x < 8; ++x) {
            const uint4 v = rv ? __ldg(src + x) : make_uint4(0u, 0u, 0u, 0u);
            qv[4 * x] = v.x; qv[4 * x + 1] = v.y; qv[4 * x + 2] = v.z; qv[4 * x + 3] = v.w;
          }
          tmem_st32(tlane + S::TQ + 64u * h + 32 * c2, qv);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_full[h]);
      }
      const int beside = item.beside(h), kstep = item.step() * KT, lo_max = it.lo_max, hist = min(it.H, it.hi);
      int k0 = it.kt0 * KT;
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < nt; ++j, k0 += kstep) {
        const int tile = g + j + min(j + h, beside);
        const uint32_t buf = c & 1u, tm_s = tm_chain + (BIAS ? 0 : KT * buf);
        go = tr_wait(&s_full[2 * h + buf], (c >> 1) & 1u, abort_flag, a);
        if (!go) break;
        ++c;
        tc_fence_after();
        uint32_t any = 0;
#pragma unroll
        for (int x = 0; x < KW; ++x) any |= kbad[(tile % TR_BAD) * KW + x];
        const bool part = k0 < lo_max || hist - k0 < KT || any;   // not every row sees all of it
        TRBias how = NoLoad;
        if constexpr (BIAS) {
          how = tr_bias(a, it, k0);
          if (how != NoLoad) {
            go = tr_wait(&bias_full[h], bn & 1u, abort_flag, a);
            if (!go) break;
            ++bn;
          }
        }
        // this row's values, and how many of the tile's keys lie at E - 1 or beyond (the copy of a row ends there; within a window that
        // is no longer than the row they are not seen)
        const uint8_t* b_row = nullptr;
        if constexpr (BIAS) {
          if (how == Boxes) {
            const int size = a.rel_bf16 ? 2 : 4, d0 = p - k0;   // of key 0
            uint8_t* row = bias + h * TREE_BIAS_BYTES;   // (a row without a token reads the first one's: its own would lie outside)
            if (rv) row += my_i * a.bias_stride + my_g * (tree_bias_cols(a.rel_bf16) * size);
            row += ((d0 - KT + 1) & (16 / size - 1)) * size;
            b_row = row;
            const int n = min(d0 - (a.E - 1), KT);
            if (!(a.W > 0 && a.W <= a.E) && rv && n > 0) {
#pragma unroll 1
              for (int c = 0; c < n; ++c) {
                if (a.rel_bf16) reinterpret_cast<uint16_t*>(row)[KT - 1 - c] = (uint16_t)(__float_as_uint(rc) >> 16);
                else reinterpret_cast<float*>(row)[KT - 1 - c] = rc;
              }
              asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // (a copy may write here next)
            }
          } else {
            b_row = bias + h * TREE_BIAS_BYTES + r * TR_ELEMENTS * 4;
          }
        }
        // ---- scores and their maximum
        float mx = -INFINITY;
        auto score = [&](int w, uint32_t (&sr)[32]) {   // of keys 32 w and on
          uint32_t vis = 0xffffffffu;
          if (part) vis = my_row().sees(a, k0 + 32 * w) & ~kbad[(tile % TR_BAD) * KW + w];
          if constexpr (CAP) {
            if (part) {   // (what nobody may see has no say in how scores are capped)
#pragma unroll
              for (int c = 0; c < 32; ++c)
                if (!((vis >> c) & 1u)) sr[c] = 0u;
            }
            float fv[4] = {0.f, 0.f, 0.f, 0.f};   // largest |<q, K[k]>|
#pragma unroll
            for (int c = 0; c < 32; c += 2)
              fv[(c >> 1) & 3] = fmax3(fv[(c >> 1) & 3], fabsf(__uint_as_float(sr[c])), fabsf(__uint_as_float(sr[c + 1])));
            // (rows of other sequences have no say)
            const float far = rv ? fmaxf(fmax3(fv[0], fv[1], fv[2]), fv[3]) : 0.f;
            if (__all_sync(0xffffffffu, far <= a.cap_near)) {
              uint64_t co[NEAR_TERMS];
#pragma unroll
              for (int i = 0; i < NEAR_TERMS; ++i) co[i] = f2_pack(a.near[i], a.near[i]);
#pragma unroll
              for (int c = 0; c < 32; c += 2) {
                const uint64_t x = f2_pack(__uint_as_float(sr[c]), __uint_as_float(sr[c + 1]));
                const uint64_t u = tr_mul(x, x);
                uint64_t y = co[NEAR_TERMS - 1];
#pragma unroll
                for (int i = NEAR_TERMS - 2; i >= 0; --i) y = f2_fma(y, u, co[i]);
                float s0, s1;
                f2_unpack(tr_mul(y, x), s0, s1);
                sr[c] = __float_as_uint(s0);
                sr[c + 1] = __float_as_uint(s1);
              }
            } else {
#pragma unroll
              for (int c = 0; c < 32; ++c) sr[c] = __float_as_uint(score_log2<true>(a, __uint_as_float(sr[c])));
            }
          } else if (!BIAS && scaled) {
#pragma unroll
            for (int c = 0; c < 32; ++c) sr[c] = __float_as_uint(__uint_as_float(sr[c]) * a.scale_log2);
          }
          if constexpr (BIAS) {
            if (how != NoLoad) {
              // value of key c at place KT - 1 - c, distances rising
              if (how == Boxes && a.rel_bf16) {
                const uint16_t* br = reinterpret_cast<const uint16_t*>(b_row) + KT - 1 - 32 * w;
#pragma unroll
                for (int c = 0; c < 32; ++c)
                  sr[c] = __float_as_uint(fmaf(__uint_as_float(sr[c]), pre, __uint_as_float((uint32_t)br[-c] << 16)));
              } else {
                const float* br = reinterpret_cast<const float*>(b_row) + KT - 1 - 32 * w;
#pragma unroll
                for (int c = 0; c < 32; ++c) sr[c] = __float_as_uint(fmaf(__uint_as_float(sr[c]), pre, br[-c]));
              }
            } else {
              const float x = rc;   // (0 without a tensor)
#pragma unroll
              for (int c = 0; c < 32; ++c) sr[c] = __float_as_uint(fmaf(__uint_as_float(sr[c]), pre, x));
            }
            if (a.slopes && how != Elements) {
              const float d0 = (float)(p - k0 - 32 * w);
#pragma unroll
              for (int c = 0; c < 32; ++c) sr[c] = __float_as_uint(fmaf(-slope, d0 - (float)c, __uint_as_float(sr[c])));
            }
          }
          if (part) {   // keys that this row does not see
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (!((vis >> c) & 1u)) sr[c] = 0xff800000u;   // -infinity
          }
        };
        uint32_t all[S::ROLL ? 32 : KT];
        float mul = mul_, off = 0.f;      // a score's factor in the exponent, and what is added to it
        // One value for a whole row changes no order: such scores stay as they are.
        const bool lean = BIAS && !CAP && how == NoLoad && !part && !a.slopes && pre > 0.f && near0;
        if (lean) {
          mul = a.scale_log2;
          off = rc * LOG2E;
        }
        auto largest = [&](uint32_t (&sr)[32]) {
          float mv[2] = {mx, -INFINITY};
#pragma unroll
          for (int c = 0; c < 32; c += 2)
            mv[(c >> 1) & 1] = fmax3(mv[(c >> 1) & 1], __uint_as_float(sr[c]), __uint_as_float(sr[c + 1]));
          mx = fmaxf(mv[0], mv[1]);
        };
        if constexpr (S::ROLL) {
#pragma unroll 1
          for (int w = 0; w < KW; ++w) {
            tmem_ld32(tm_s + 32 * w, all);
            tmem_wait_ld();
            if (lean) {
              largest(all);
            } else {
              score(w, all);
              largest(all);
              tmem_st32(tm_s + 32 * w, all);
            }
          }
          if (!lean) tmem_wait_st();
        } else {
#pragma unroll
          for (int w = 0; w < KW; ++w) tmem_ld32(tm_s + 32 * w, *reinterpret_cast<uint32_t(*)[32]>(&all[32 * w]));
          tmem_wait_ld();
#pragma unroll
          for (int w = 0; w < KW; ++w) {
            uint32_t (&sr)[32] = *reinterpret_cast<uint32_t(*)[32]>(&all[32 * w]);
            if (!lean) score(w, sr);
            largest(sr);
          }
        }
        if constexpr (BIAS) {
          if (how != NoLoad) {
            __syncwarp();
            if (lane == 0) mbar_arrive(&bias_empty[h]);
          }
        }
        // ---- running maximum, moved only when it grows by more than 2^8
        if constexpr (BIAS) {
          const float s = lean ? fmaf(mx, pre, rc) : mx;
          mx = fabsf(s) < TR_BIG ? 0.5f * fmaf(mx, mul, off) : s;
        } else {
          mx = fmaf(mx, mul, off);
        }
        const bool mine = mx > m + TR_RESCALE_LOG2 / UNIT;
        if (__any_sync(0xffffffffu, mine)) {
          if (j > 0) {   // (s_full came after all products into O_h but the last one)
            go = tr_wait(&o_done[2 * h + (buf ^ 1u)], ((c - 2) >> 1) & 1u, abort_flag, a);
            if (!go) break;
            tc_fence_after();
            const float fr = mine ? fast_exp2(UNIT * (m - mx)) : 1.f;
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
        // ---- numerators, rounded to bf16 (an operand of the product has V's type: off by 2^-8 of a weight; the sum is of unrounded ones)
        float nm = off - (m == -INFINITY ? 0.f : UNIT * m);
        if constexpr (BIAS) {
          if (fabsf(m) >= TR_BIG && m != -INFINITY) {
            mul = lean ? pre : 1.f;
            nm = (lean ? rc : 0.f) - m;
          }
        }
        const uint64_t mul2 = f2_pack(mul, mul), nm2 = f2_pack(nm, nm);
        uint64_t ls2[4] = {0ull, 0ull, 0ull, 0ull};
        auto numerators = [&](int w, uint32_t (&sr)[32]) {
          uint32_t pk[16];
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            float t0, t1;
            f2_unpack(f2_fma(f2_pack(__uint_as_float(sr[2 * c]), __uint_as_float(sr[2 * c + 1])), mul2, nm2), t0, t1);
            const float p0 = fast_exp2(t0), p1 = fast_exp2(t1);
            ls2[c & 3] = f2_add(ls2[c & 3], f2_pack(p0, p1));
            pk[c] = pack_bf16(p0, p1);
          }
          tmem_st16(tm_s + 16 * w, pk);
        };
        if constexpr (S::ROLL) {
#pragma unroll 1
          for (int w = 0; w < KW; ++w) {
            tmem_ld32(tm_s + 32 * w, all);
            tmem_wait_ld();
            numerators(w, all);
          }
        } else {
#pragma unroll
          for (int w = 0; w < KW; ++w) numerators(w, *reinterpret_cast<uint32_t(*)[32]>(&all[32 * w]));
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
        if (lane == 0) mbar_arrive(&p_full[2 * h + buf]);
      }
      if (!go) break;
      g += item.tiles();
      c_other += pair ? nt : item.part[h ^ 1].nt;
      // ---- epilogue
      if (nt > 0) {
        go = tr_wait(&o_done[2 * h + ((c - 1) & 1u)], ((c - 1) >> 1) & 1u, abort_flag, a);
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
        if (h == 1 || both) go = tr_wait(&o_done[2 * (h ^ 1) + ((c_other - 1) & 1u)], ((c_other - 1) >> 1) & 1u, abort_flag, a);   // (its warps have waited for it)
        if (!go) break;
        const float2 x0 = ml[r], x1 = both ? ml[TREE_ROWS + r] : make_float2(-INFINITY, 0.f);
        M = fmaxf(x0.x, x1.x);
        f0 = x0.x == -INFINITY ? 0.f : fast_exp2(UNIT * (x0.x - M));
        f1 = x1.x == -INFINITY ? 0.f : fast_exp2(UNIT * (x1.x - M));
        l = (x0.y == 0.f ? 0.f : x0.y * f0) + (x1.y == 0.f ? 0.f : x1.y * f1);
      }
      tc_fence_after();
      const volatile int* ps = poison + 4 * (k % TR_ITEMS) + (merge || pair ? 0 : 2 * h);
      const int pfirst = both ? min(ps[0], ps[2]) : ps[0], plast = both ? max(ps[1], ps[3]) : ps[1];
      const bool whole = it.parts <= 1, nothing = l == 0.f;
      const float inv = whole ? (nothing ? 0.f : 1.f / l) : 1.f;   // (a NaN stays one)
      const float g0 = nothing ? 0.f : f0 * inv, g1 = nothing ? 0.f : f1 * inv;
      const uint32_t o0 = tm_o + (merge ? 0 : D * h);
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
      if (plast >= 0 && rv)
        tr_infinite(a, it, my_row(), pfirst, plast, 32 * c_first, 32 * c_end, whole ? out + orow * D : nullptr,
                    reinterpret_cast<float*>(part_o), D);
      if (!merge || h == 0) {
        if (!whole) __stcg(reinterpret_cast<float2*>(a.part_ml) + ((size_t)it.place * 2 + rt) * TREE_ROWS + r, make_float2(M, l));
        else if (rv && a.lse) a.lse[orow] = nothing ? -INFINITY : tr_natural(M, BIAS) + logf(l);
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
  const bool bias = a.rel || a.slopes;
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
    const float w = p.x == -INFINITY ? 0.f : fast_exp2((bias ? 2.f : 1.f) * (p.x - M));
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
  if (c == 0 && a.lse) a.lse[row] = nothing ? -INFINITY : tr_natural(M, bias) + logf(l);
}

template <int D, bool CAP, bool BIAS>
cudaError_t launch_t(const MaskedMaps& m, const CUtensorMap& bias, const TreeArgs& a, int grid, cudaStream_t stream) {
  using S = TRShape<D, CAP, BIAS>;
  static std::atomic<unsigned long long> opted{0};
  cudaError_t e = smem_opt_in_once(tree_kernel<D, CAP, BIAS>, (int)TRSmem<D, CAP, BIAS>::alloc, opted);
  if (e != cudaSuccess) return e;
  tree_kernel<D, CAP, BIAS><<<grid, S::THREADS, TRSmem<D, CAP, BIAS>::alloc, stream>>>(m.k, m.v, m.q, bias, a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  tree_join_kernel<D><<<dim3(grid, 2 * (D / 16)), TREE_ROWS, 0, stream>>>(a);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_d(const MaskedMaps& m, const CUtensorMap& bias, const TreeArgs& a, int grid, cudaStream_t stream) {
  const bool cap = a.softcap != 0.f;
  if (a.rel || a.slopes) return cap ? launch_t<D, true, true>(m, bias, a, grid, stream) : launch_t<D, false, true>(m, bias, a, grid, stream);
  return cap ? launch_t<D, true, false>(m, bias, a, grid, stream) : launch_t<D, false, false>(m, bias, a, grid, stream);
}

}  // namespace

cudaError_t launch_tree(const MaskedMaps& m, const CUtensorMap& bias, const TreeArgs& a, int head_dim, cudaStream_t stream) {
  int dev = 0;
  const int sms = current_device_sms(&dev);
  if (sms <= 0) return cudaErrorInvalidDevice;
  const long long items = (a.T / (2ll * a.tok_per_tile) + a.B) * a.Hkv * a.head_chunks;
  const long long tiles = ((long long)a.max_pages << a.log2_page) / KT + 1;
  const int grid = (int)std::min<long long>(std::min(sms, TREE_MAX_CTAS), items * tiles);
  return head_dim == 128 ? launch_d<128>(m, bias, a, grid, stream) : launch_d<64>(m, bias, a, grid, stream);
}

}  // namespace ink
