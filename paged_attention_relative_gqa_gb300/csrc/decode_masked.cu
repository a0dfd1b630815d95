// decode_masked.cu -- paged decode without a bias tensor: one token per sequence, capped scores, a
// bias linear in the distance, a visible key range per sequence.
//
//   x = sm_scale <q[b,h], K[k]>,  s = cap(x) - slope_h |p - k|,  out = softmax(s) V,  lse = log sum exp(s)
//
// The bytes of the visible K and V bound it, so they have to flow evenly over the SMs whatever the
// lengths are.  All 64-key tiles of all (sequence, KV head, chunk of query heads) groups stand in
// one row, tiles of a group side by side, and every CTA takes an equal run of them, computed on the
// device from the lengths and ranges (a graph replays with new ones).  A run cuts at most two
// groups; the pieces of a cut group leave fp32 partials, and the last CTA to finish one of them
// (an atomic ticket, no waiting) joins all of them in order, so results do not depend on who
// arrives when.  Partials need two places per CTA, not one per split and sequence.
//
// A CTA has four warps for the products and one that loads; two CTAs share an SM when at most 8
// query heads share a KV head.  Tiles come by TMA as [16-key group][64-channel block][16 rows], and
// warp w takes the 16 keys of group w: S^T = K Q^T and O^T = V^T P^T with mma.sync, so that no MMA
// row is padding when few heads share a KV head (a product this thin is bound by its bytes: the
// fifth-generation tensor cores' 128-row tiles would hold 8 useful rows).
//
// Measured (GPU time alone), 64 + 2 x 8 heads of 128: 32 sequences of up to 32 K keys (3.1 GB) 438 us, 7.1 TB/s, as
// fast as a copy; one sequence of 114 K keys 80 us, 5.8 TB/s; 128 of 2 K keys 125 us, 6.4 TB/s; windows of 512 keys, 16
// KV heads, 64 sequences 51 us, 5.3 TB/s: below 100 us the start (2.5 us), the first tiles' latency and the joins show.
// One short sequence 10 us, a chain of dependent latencies: lengths, table, tiles, products, partials, ticket, join.  Three stages with half the O buffer (445 -> 464 us), and the next piece's table
// entries and first tile ahead (no change), are not kept.
#include <algorithm>

#include "masked_common.cuh"

namespace ink {
namespace {

constexpr int DM_WARPS = 4;
constexpr int DM_THREADS = (DM_WARPS + 1) * 32;
constexpr int DM_QROWS = 16;     // query rows of a TMA box
constexpr int DM_MIN_TILES = 2;  // least run of a CTA

template <int D>
struct DMShape {
  static constexpr int CB = D / 64;
  static constexpr int BLOCK = 16 * 128;                 // 16 rows of 64 channels
  static constexpr int GROUP = CB * BLOCK;
  static constexpr int TILE = (TILE_KEYS / 16) * GROUP;
  static constexpr int STAGE = 2 * TILE;                 // K and V
  static constexpr int QSUB = DM_QROWS * 128;
  static constexpr int QSLOT = CB * QSUB;
  static constexpr int OPITCH = D + 4;
};

template <int D, int NSTAGE, int HB>
struct DMSmem {
  using S = DMShape<D>;
  static constexpr size_t q = (size_t)NSTAGE * S::STAGE;
  static constexpr size_t obuf = q + 2 * S::QSLOT;
  static constexpr size_t red = obuf + (size_t)DM_WARPS * HB * S::OPITCH * 4;
  static constexpr size_t bars = red + (2 * DM_WARPS * 16 + 2 * 16) * 4;
  static constexpr size_t bad = bars + (2 * NSTAGE + 2) * 8;
  static constexpr size_t flags = bad + NSTAGE * 8;
  static constexpr size_t total = flags + 16;
  static constexpr size_t alloc = total + 1024;
};

// A run of tiles of one group.
struct Piece {
  int b, kvh, h0, nh, L, lo, hi;
  int tile, n;            // first tile (absolute), tiles
  int c0, parts;          // first CTA of the group, CTAs
};

// The row of tiles, walked by a whole warp: 32 sequences at a time in the lanes.
struct Walk {
  long long base, incl, chunk;   // tiles before sequence cb; up to and with this lane's; tiles per CTA
  int cb, cnt, lo, hi, L;        // this lane's sequence cb + lane: tiles of one group, keys, length
  long long total;               // tiles of the 32
  int per;

  __device__ __forceinline__ void load(const MaskedArgs& a, int lane) {
    const int b = cb + lane;
    cnt = lo = hi = L = 0;
    if (b < a.B) {
      L = __ldg(a.seq_lens + b);
      if (L > 0) {
        token_keys(a, b, L - 1, L, lo, hi);
        if (lo < hi) cnt = (hi - 1) / TILE_KEYS - lo / TILE_KEYS + 1;
      }
    }
    incl = (long long)cnt * per;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    total = __shfl_sync(0xffffffffu, incl, 31);
  }

  // All tiles of the call; leaves the walk at its start.
  __device__ __forceinline__ long long begin(const MaskedArgs& a, int lane) {
    per = a.Hkv * a.head_chunks;
    long long all = 0;
    for (cb = ((a.B - 1) >> 5) << 5; cb >= 0; cb -= 32) {
      load(a, lane);
      all += total;
    }
    cb = 0;
    base = 0;
    return all;
  }

  // The piece that starts at tile `pos` of a run that ends at `end`.
  __device__ __forceinline__ Piece at(const MaskedArgs& a, int lane, long long pos, long long end) {
    while (pos >= base + total) {
      base += total;
      cb += 32;
      load(a, lane);
    }
    const int src = __ffs(__ballot_sync(0xffffffffu, pos < base + incl)) - 1;
    Piece w;
    const int T = __shfl_sync(0xffffffffu, cnt, src);
    const long long start = base + __shfl_sync(0xffffffffu, incl - (long long)cnt * per, src);
    w.b = cb + src;
    w.L = __shfl_sync(0xffffffffu, L, src);
    w.lo = __shfl_sync(0xffffffffu, lo, src);
    w.hi = __shfl_sync(0xffffffffu, hi, src);
    const int gi = (int)((pos - start) / T);
    const int x0 = (int)(pos - start - (long long)gi * T);
    w.tile = w.lo / TILE_KEYS + x0;
    w.n = (int)min((long long)(T - x0), end - pos);
    w.kvh = gi / a.head_chunks;
    const int c = gi - w.kvh * a.head_chunks;
    w.h0 = w.kvh * a.G + c * DM_QROWS;
    w.nh = min(DM_QROWS, a.G - c * DM_QROWS);
    const long long g0 = pos - x0;
    w.c0 = (int)(g0 / chunk);
    w.parts = (int)((g0 + T - 1) / chunk) - w.c0 + 1;
    return w;
  }
};

// Bounded wait of a whole warp, with one answer for all its lanes: each reads the flag, the barrier
// and the clock for itself, and what follows (matrix products, shuffles, branches around them) takes
// the warp whole.
__device__ __forceinline__ bool dm_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, const MaskedArgs& a) {
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

// The piece's partial is in the workspace: take the group's ticket (a CTA's run is the start of one cut
// group at most, so it goes by the first CTA); the last of its pieces joins all of them, in order, and
// resets the ticket.  Every thread's partial stores come before the
// barrier, the ticket's add releases them and acquires the others'.
template <int D, int HB>
__device__ __noinline__ void join_pieces(const float* part_o, const float* part_ml, int32_t* ticket, __nv_bfloat16* out,
                                         float* lse, int nh, int c0, int parts, int tid, int* flags, float* head_ml) {
  named_barrier_sync(1, DM_WARPS * 32);
  if (tid == 0) {
    int prev;
    asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;" : "=r"(prev) : "l"(ticket) : "memory");
    flags[0] = prev == parts - 1;
  }
  named_barrier_sync(1, DM_WARPS * 32);
  if (!flags[0]) return;
  // piece i of the group is at place 2 (c0 + i), the first at 2 c0 + 1
  auto place = [&](int i) { return (size_t)(2 * (c0 + i) + (i == 0 ? 1 : 0)); };
  const int warp = tid >> 5, lane = tid & 31;
  for (int r = warp; r < nh; r += DM_WARPS) {
    float M = -INFINITY;
    for (int i = lane; i < parts; i += 32) M = fmaxf(M, __ldcg(part_ml + (place(i) * HB + r) * 2));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    const float Mu = M == -INFINITY ? 0.f : M;
    float Lt = 0.f;
    for (int i = lane; i < parts; i += 32) {
      const float2 ml = __ldcg(reinterpret_cast<const float2*>(part_ml) + place(i) * HB + r);
      Lt += ml.y * fast_exp2(ml.x - Mu);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) Lt += __shfl_xor_sync(0xffffffffu, Lt, o);
    if (lane == 0) {
      head_ml[2 * r] = Mu;
      head_ml[2 * r + 1] = Lt == 0.f ? 0.f : 1.f / Lt;
      if (lse) lse[r] = Lt == 0.f ? -INFINITY : Mu * LN2 + logf(Lt);
    }
  }
  named_barrier_sync(1, DM_WARPS * 32);
  for (int idx = tid; idx < nh * (D / 4); idx += DM_WARPS * 32) {
    const int r = idx / (D / 4), d = (idx % (D / 4)) * 4;
    const float Mu = head_ml[2 * r], inv = head_ml[2 * r + 1];
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int i = 0; i < parts; ++i) {
      const size_t at = place(i) * HB + r;
      const float wt = fast_exp2(__ldcg(part_ml + at * 2) - Mu) * inv;
      const float4 v = __ldcg(reinterpret_cast<const float4*>(part_o + at * D + d));
      acc.x += wt * v.x;
      acc.y += wt * v.y;
      acc.z += wt * v.z;
      acc.w += wt * v.w;
    }
    *reinterpret_cast<uint2*>(out + (size_t)r * D + d) = make_uint2(pack_bf16(acc.x, acc.y), pack_bf16(acc.z, acc.w));
  }
  if (tid == 0) *ticket = 0;   // ready for the next call
}

template <int D, int NSTAGE, int HB, bool CAP>
__global__ void __launch_bounds__(DM_THREADS, HB == 8 ? 2 : 1)
decode_masked_kernel(const __grid_constant__ DecodeMaps maps, const __grid_constant__ MaskedArgs a) {
  using S = DMShape<D>;
  using L_ = DMSmem<D, NSTAGE, HB>;
  constexpr int KSTEPS = D / 16, NB = HB / 8;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_align1024(smem_raw);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L_::bars);
  uint64_t* empty = full + NSTAGE;
  uint64_t* qempty = empty + NSTAGE;   // [2]
  uint64_t* badmask = reinterpret_cast<uint64_t*>(smem + L_::bad);
  int* flags = reinterpret_cast<int*>(smem + L_::flags);   // [0] ticket winner, [1] abort
  float* red_m = reinterpret_cast<float*>(smem + L_::red);
  float* red_l = red_m + DM_WARPS * 16;
  float* head_ml = red_l + DM_WARPS * 16;                  // [16][2]
  float* obuf = reinterpret_cast<float*>(smem + L_::obuf);
  volatile int* abort_flag = flags + 1;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int P = 1 << a.log2_page;
  __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(a.out);

  if (tid == 0) {
    for (int s = 0; s < NSTAGE; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], DM_WARPS);
    }
    mbar_init(&qempty[0], DM_WARPS);
    mbar_init(&qempty[1], DM_WARPS);
    fence_mbar_init();
    flags[0] = 0;
    flags[1] = 0;
  }
  Walk walk;
  const long long all = walk.begin(a, lane);
  walk.chunk = max((all + gridDim.x - 1) / (long long)gridDim.x, (long long)DM_MIN_TILES);
  const long long run0 = min((long long)blockIdx.x * walk.chunk, all), run1 = min(run0 + walk.chunk, all);
  __syncthreads();

  if (warp == DM_WARPS) {
    // ------------------------------------------------------------------ loads
    if (lane == 0) {
      prefetch_tensormap(&maps.q3);
      if (P >= TILE_KEYS) {
        prefetch_tensormap(&maps.k_tile);
        prefetch_tensormap(&maps.v_tile);
      }
      prefetch_tensormap(P >= 16 ? &maps.k_grp : &maps.k_seg);
      prefetch_tensormap(P >= 16 ? &maps.v_grp : &maps.v_seg);
    }
    const int hkvp = a.Hkv << a.log2_page;
    const int seg = min(P, 16), nseg = TILE_KEYS / seg;
    int n = 0, uc = 0;
    bool go = true;
    for (long long pos = run0; pos < run1 && go;) {
      const Piece w = walk.at(a, lane, pos, run1);
      pos += w.n;
      const int slot = uc & 1;
      const int32_t* bt = a.block_table + (size_t)w.b * a.max_pages;
      const int last = (w.hi - 1) >> a.log2_page;    // the table is not read past here
      // table entries cbase + lane and the 32 after them; a tile's entries never straddle two chunks
      int cbase = ((w.tile * TILE_KEYS) >> a.log2_page) & ~7;
      int cur = __ldg(bt + min(cbase + lane, last)), nxt = __ldg(bt + min(cbase + 32 + lane, last));
      if (uc >= 2) {
        go = __all_sync(0xffffffffu, dm_wait(&qempty[slot], (uint32_t)((uc >> 1) - 1) & 1u, abort_flag, a) && !*abort_flag);
        if (!go) break;
      }
      for (int i = 0; i < w.n; ++i, ++n) {
        const int st = n % NSTAGE;
        const int k0 = (w.tile + i) * TILE_KEYS;
        if ((k0 >> a.log2_page) >= cbase + 32) {
          cbase += 32;
          cur = nxt;
          nxt = __ldg(bt + min(cbase + 32 + lane, last));
        }
        // lane < nseg takes one segment; a whole tile on one page is one box a tensor
        const int ks = k0 + lane * seg;
        const bool want = lane < nseg && ks < w.hi && ks + seg > w.lo;
        const int page = __shfl_sync(0xffffffffu, cur, min(max((ks >> a.log2_page) - cbase, 0), 31));
        const bool bad_seg = want && (page < 0 || page >= a.num_pages);
        const bool load = want && !bad_seg;
        const uint32_t lmask = __ballot_sync(0xffffffffu, load), bmask = __ballot_sync(0xffffffffu, bad_seg);
        const bool whole = P >= TILE_KEYS && lmask == (1u << nseg) - 1u;
        const int row = load ? page * hkvp + (w.kvh << a.log2_page) + (ks & (P - 1)) : 0;
        if (n >= NSTAGE) {
          go = __all_sync(0xffffffffu, dm_wait(&empty[st], (uint32_t)((n / NSTAGE) - 1) & 1u, abort_flag, a) && !*abort_flag);
          if (!go) break;
        }
        uint8_t* kdst = smem + (size_t)st * S::STAGE;
        uint8_t* vdst = kdst + S::TILE;
        if (lane == 0) {
          uint64_t bad = 0;
          for (uint32_t mm = bmask; mm; mm &= mm - 1) bad |= ((1ull << seg) - 1) << ((__ffs(mm) - 1) * seg);
          badmask[st] = bad;
          if (bmask) record_error(a.err, INK_DEVERR_PAGE_OUT_OF_RANGE);
          mbar_arrive_expect_tx(&full[st], (uint32_t)__popc(lmask) * (uint32_t)(2 * seg * D * 2) +
                                               (i == 0 ? (uint32_t)(S::CB * DM_QROWS * 128) : 0u));
          if (i == 0) tma_load_3d(smem + L_::q + slot * S::QSLOT, &maps.q3, 0, w.b * a.Hq + w.h0, 0, &full[st]);
        }
        __syncwarp();
        if (whole) {
          if (lane == 0) {
            tma_load_4d(kdst, &maps.k_tile, 0, 0, 0, row >> 4, &full[st]);
            tma_load_4d(vdst, &maps.v_tile, 0, 0, 0, row >> 4, &full[st]);
          }
        } else if (load) {
          const int off = ((ks - k0) >> 4) * S::GROUP;
          if (seg == 16) {
            tma_load_4d(kdst + off, &maps.k_grp, 0, 0, 0, row >> 4, &full[st]);
            tma_load_4d(vdst + off, &maps.v_grp, 0, 0, 0, row >> 4, &full[st]);
          } else {
            const int r8 = ((ks - k0) & 15) * 128;
#pragma unroll
            for (int cb = 0; cb < S::CB; ++cb) {
              tma_load_2d(kdst + off + cb * S::BLOCK + r8, &maps.k_seg, cb * 64, row, &full[st]);
              tma_load_2d(vdst + off + cb * S::BLOCK + r8, &maps.v_seg, cb * 64, row, &full[st]);
            }
          }
        }
        // the next tile towards L2, ahead of its stage
        if (P >= TILE_KEYS && i + 1 < w.n) {
          const int kn = k0 + TILE_KEYS;
          const int pi = (kn >> a.log2_page) - cbase;
          const int pn = __shfl_sync(0xffffffffu, pi < 32 ? cur : nxt, pi & 31);
          if (lane == 0 && kn >= w.lo && kn + TILE_KEYS <= w.hi && pn >= 0 && pn < a.num_pages) {
            const int rn = pn * hkvp + (w.kvh << a.log2_page) + (kn & (P - 1));
            tma_prefetch_l2_4d(&maps.k_tile, 0, 0, 0, rn >> 4);
            tma_prefetch_l2_4d(&maps.v_tile, 0, 0, 0, rn >> 4);
          }
        }
      }
      ++uc;
    }
    // the last load into each stage lands before the CTA exits
    if (lane == 0)
      for (int k = max(0, n - NSTAGE); k < n; ++k)
        if (!mbar_wait_bounded(&full[k % NSTAGE], (uint32_t)(k / NSTAGE) & 1u)) record_error(a.err, INK_DEVERR_WAIT_TIMEOUT);
    return;
  }

  // -------------------------------------------------------------------- products
  // sequences that see no key: zero rows, shared out over the CTAs
  for (int b = (int)blockIdx.x; b < a.B; b += (int)gridDim.x) {
    const int L = __ldg(a.seq_lens + b);
    int lo = 0, hi = 0;
    if (L > 0) token_keys(a, b, L - 1, L, lo, hi);
    if (tid == 0 && (long long)L > ((long long)a.max_pages << a.log2_page)) record_error(a.err, INK_DEVERR_PAGE_OUT_OF_RANGE);
    if (lo < hi) continue;
    for (int x = tid; x < a.Hq * D / 8; x += DM_WARPS * 32)
      reinterpret_cast<uint4*>(out + (size_t)b * a.Hq * D)[x] = make_uint4(0u, 0u, 0u, 0u);
    if (a.lse)
      for (int h = tid; h < a.Hq; h += DM_WARPS * 32) a.lse[(size_t)b * a.Hq + h] = -INFINITY;
  }

  // S^T has the warp's 16 keys as MMA rows and the heads as columns (NB blocks of 8).  A thread
  // owns keys (gq, gq + 8) and heads (8 j + 2 cq, + 1), the same heads in S^T and in O^T.
  const int gq = lane >> 2, cq = lane & 3, mi = lane >> 3;
  int n = 0, uc = 0;
  for (long long pos = run0; pos < run1;) {
    const Piece w = walk.at(a, lane, pos, run1);
    pos += w.n;
    uint32_t qb[NB][KSTEPS][2];
    float m_r[NB][2], l_r[NB][2], slope2[NB][2];
    float o[D / 16][NB][4];
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m_r[j][e] = -INFINITY;
        l_r[j][e] = 0.f;
        const int hh = 8 * j + 2 * cq + e;
        slope2[j][e] = a.slopes && hh < w.nh ? __ldg(a.slopes + w.h0 + hh) * LOG2E : 0.f;
      }
#pragma unroll
    for (int dn = 0; dn < D / 16; ++dn)
#pragma unroll
      for (int j = 0; j < NB; ++j) o[dn][j][0] = o[dn][j][1] = o[dn][j][2] = o[dn][j][3] = 0.f;

    for (int i = 0; i < w.n; ++i, ++n) {
      const int st = n % NSTAGE;
      const bool ok = dm_wait(&full[st], (uint32_t)(n / NSTAGE) & 1u, abort_flag, a);
      // The copies of a tile whose wait ran out may be in flight: its stage and Q slot are not handed
      // back (its barrier would be armed a second time, and the loader's last waits would not know which
      // copies they wait for).  The rest of the run is left out.
      if (!ok) {
        n += w.n - i;
        break;
      }
      if (i == 0) {
        const uint32_t qbase = smem_u32(smem + L_::q + (uc & 1) * S::QSLOT);
#pragma unroll
        for (int j = 0; j < NB; ++j) {
          const bool hv = 8 * j + gq < w.nh;
#pragma unroll
          for (int kk = 0; kk < KSTEPS; kk += 2) {
            const int chunk = 2 * kk + mi;
            uint32_t r0, r1, r2, r3;
            ldmatrix_x4(qbase + (chunk >> 3) * S::QSUB + swz128(8 * j + (lane & 7), chunk & 7), r0, r1, r2, r3);
            qb[j][kk][0] = hv ? r0 : 0u;
            qb[j][kk][1] = hv ? r1 : 0u;
            qb[j][kk + 1][0] = hv ? r2 : 0u;
            qb[j][kk + 1][1] = hv ? r3 : 0u;
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&qempty[uc & 1]);
      }
      const int kw = (w.tile + i) * TILE_KEYS + 16 * warp;
      const uint64_t bad = badmask[st];
      const int jlo = max(w.lo - kw, 0), jhi = min(w.hi - 1 - kw, 15);
      uint32_t valid = jhi >= jlo ? ((0xFFFFu >> (15 - jhi)) & (0xFFFFu << jlo)) : 0u;
      valid &= ~(uint32_t)(bad >> (16 * warp)) & 0xFFFFu;
      if (valid == 0) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[st]);
        continue;
      }
      const uint32_t kbase = smem_u32(smem + (size_t)st * S::STAGE) + warp * S::GROUP;
      float acc[NB][4];
#pragma unroll
      for (int j = 0; j < NB; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;
#pragma unroll
      for (int kk = 0; kk < KSTEPS; ++kk) {
        const int chunk = 2 * kk + (mi >> 1);
        uint32_t ka[4];
        ldmatrix_x4(kbase + (chunk >> 3) * S::BLOCK + swz128((mi & 1) * 8 + (lane & 7), chunk & 7), ka[0], ka[1], ka[2], ka[3]);
#pragma unroll
        for (int j = 0; j < NB; ++j) mma_bf16_16816(acc[j], ka, qb[j][kk][0], qb[j][kk][1]);
      }
      // V in registers, rows of keys not seen zeroed (0 * NaN); the stage is free after this
      const uint32_t mlo = pair_mask((valid >> (2 * cq)) & 1u, (valid >> (2 * cq + 1)) & 1u);
      const uint32_t mhi = pair_mask((valid >> (8 + 2 * cq)) & 1u, (valid >> (9 + 2 * cq)) & 1u);
      uint32_t va[D / 16][4];
#pragma unroll
      for (int dn = 0; dn < D / 16; ++dn) {
        const int chunk = 2 * dn + (mi & 1);
        ldmatrix_x4_trans(kbase + S::TILE + (chunk >> 3) * S::BLOCK + swz128((mi >> 1) * 8 + (lane & 7), chunk & 7),
                          va[dn][0], va[dn][1], va[dn][2], va[dn][3]);
        if (valid != 0xFFFFu) { va[dn][0] &= mlo; va[dn][1] &= mlo; va[dn][2] &= mhi; va[dn][3] &= mhi; }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[st]);
      const bool v0 = (valid >> gq) & 1u, v1 = (valid >> (gq + 8)) & 1u;
      const float d0 = fabsf((float)(w.L - 1 - kw - gq)), d1 = fabsf((float)(w.L - 1 - kw - gq - 8));
      uint32_t pb0[NB], pb1[NB];
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        // the maximum moves only when a score passes it by more than 8 (p < 2^8): most tiles skip
        // the cross-lane maximum and the rescale of O
        float sv[2][2];
        bool up = false;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          sv[e][0] = v0 ? fmaf(-slope2[j][e], d0, score_log2<CAP>(a, acc[j][e])) : -INFINITY;
          sv[e][1] = v1 ? fmaf(-slope2[j][e], d1, score_log2<CAP>(a, acc[j][2 + e])) : -INFINITY;
          up |= fmaxf(sv[e][0], sv[e][1]) > m_r[j][e] + 8.f;
        }
        if (__any_sync(0xffffffffu, up)) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float mx = fmaxf(sv[e][0], sv[e][1]);
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
            const float mn = fmaxf(m_r[j][e], mx);
            if (mn > m_r[j][e]) {
              const float al = fast_exp2(m_r[j][e] - mn);
              m_r[j][e] = mn;
              l_r[j][e] *= al;
#pragma unroll
              for (int dn = 0; dn < D / 16; ++dn) {
                o[dn][j][e] *= al;
                o[dn][j][2 + e] *= al;
              }
            }
          }
        }
        float pr[4];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float mu = m_r[j][e] == -INFINITY ? 0.f : m_r[j][e];
          pr[e] = fast_exp2(sv[e][0] - mu);
          pr[2 + e] = fast_exp2(sv[e][1] - mu);
          l_r[j][e] += pr[e] + pr[2 + e];
        }
        // P^T as B fragment: thread (g, c) needs keys 2c, 2c + 1 (and + 8) of head g
        const uint32_t X = pack_bf16(pr[0], pr[1]), Y = pack_bf16(pr[2], pr[3]);
        const int src0 = 8 * cq + (gq >> 1), src1 = src0 + 4;
        const uint32_t x0 = __shfl_sync(0xffffffffu, X, src0), x1 = __shfl_sync(0xffffffffu, X, src1);
        const uint32_t y0 = __shfl_sync(0xffffffffu, Y, src0), y1 = __shfl_sync(0xffffffffu, Y, src1);
        const uint32_t sel = (gq & 1) ? 0x7632u : 0x5410u;
        pb0[j] = __byte_perm(x0, x1, sel);
        pb1[j] = __byte_perm(y0, y1, sel);
      }
#pragma unroll
      for (int dn = 0; dn < D / 16; ++dn)
#pragma unroll
        for (int j = 0; j < NB; ++j) mma_bf16_16816(o[dn][j], va[dn], pb0[j], pb1[j]);
    }
    ++uc;

    // ---- the four warps' parts of the piece
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float l = l_r[j][e];
        l += __shfl_xor_sync(0xffffffffu, l, 4);
        l += __shfl_xor_sync(0xffffffffu, l, 8);
        l += __shfl_xor_sync(0xffffffffu, l, 16);
        if (gq == 0) {
          red_m[warp * 16 + 8 * j + 2 * cq + e] = m_r[j][e];
          red_l[warp * 16 + 8 * j + 2 * cq + e] = l;
        }
      }
    named_barrier_sync(1, DM_WARPS * 32);
    const bool single = w.parts == 1;
    const size_t rowbase = (size_t)w.b * a.Hq + w.h0;
    const size_t place = (size_t)2 * blockIdx.x + ((int)blockIdx.x == w.c0 ? 1 : 0);
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int h = 8 * j + 2 * cq + e;
        if (h >= w.nh) continue;
        float M = -INFINITY;
#pragma unroll
        for (int x = 0; x < DM_WARPS; ++x) M = fmaxf(M, red_m[x * 16 + h]);
        const float Mu = M == -INFINITY ? 0.f : M;
        float Lt = 0.f;
#pragma unroll
        for (int x = 0; x < DM_WARPS; ++x) Lt += red_l[x * 16 + h] * fast_exp2(red_m[x * 16 + h] - Mu);
        float f = fast_exp2(m_r[j][e] - Mu);
        if (single) f *= Lt == 0.f ? 0.f : 1.f / Lt;
        if (warp == 0 && gq == 0) {
          if (single) {
            if (a.lse) a.lse[rowbase + h] = Lt == 0.f ? -INFINITY : Mu * LN2 + logf(Lt);
          } else {
            a.part_ml[(place * HB + h) * 2] = M;
            a.part_ml[(place * HB + h) * 2 + 1] = Lt;
          }
        }
        float* row = obuf + (warp * HB + h) * S::OPITCH;
#pragma unroll
        for (int dn = 0; dn < D / 16; ++dn) {
          row[16 * dn + gq] = o[dn][j][e] * f;
          row[16 * dn + gq + 8] = o[dn][j][2 + e] * f;
        }
      }
    named_barrier_sync(1, DM_WARPS * 32);
    for (int idx = tid; idx < w.nh * (D / 4); idx += DM_WARPS * 32) {
      const int r = idx / (D / 4), d = (idx % (D / 4)) * 4;
      float4 acc = *reinterpret_cast<const float4*>(obuf + r * S::OPITCH + d);
#pragma unroll
      for (int x = 1; x < DM_WARPS; ++x) {
        const float4 v = *reinterpret_cast<const float4*>(obuf + (x * HB + r) * S::OPITCH + d);
        acc.x += v.x;
        acc.y += v.y;
        acc.z += v.z;
        acc.w += v.w;
      }
      if (single)
        *reinterpret_cast<uint2*>(out + (rowbase + r) * D + d) = make_uint2(pack_bf16(acc.x, acc.y), pack_bf16(acc.z, acc.w));
      else
        *reinterpret_cast<float4*>(a.part_o + (place * HB + r) * D + d) = acc;
    }
    if (!single)
      join_pieces<D, HB>(a.part_o, a.part_ml, a.tickets + w.c0, out + rowbase * D, a.lse ? a.lse + rowbase : nullptr,
                         w.nh, w.c0, w.parts, tid, flags, head_ml);
    named_barrier_sync(1, DM_WARPS * 32);   // red, obuf, head_ml and flags are reused
  }
}

template <int D, int NSTAGE, int HB, bool CAP>
cudaError_t launch_t(const DecodeMaps& m, const MaskedArgs& a, int sms, cudaStream_t stream) {
  constexpr size_t smem = DMSmem<D, NSTAGE, HB>::alloc;
  constexpr int ctas = HB == 8 ? 2 : 1;
  static_assert(smem * ctas <= 228 * 1024 - ctas * 1024, "shared memory budget");
  static std::atomic<unsigned long long> opted{0};
  cudaError_t e = smem_opt_in_once(decode_masked_kernel<D, NSTAGE, HB, CAP>, (int)smem, opted);
  if (e != cudaSuccess) return e;
  long long keys = (long long)a.max_pages << a.log2_page;
  if (a.W > 0 && !a.key_end) keys = std::min(keys, (long long)a.W + TILE_KEYS);
  const long long most = ((keys + TILE_KEYS - 1) / TILE_KEYS + 1) * a.B * a.Hkv * a.head_chunks;
  const int grid = (int)std::min<long long>(std::min<long long>(ctas * sms, MASKED_DECODE_CTAS), most);
  decode_masked_kernel<D, NSTAGE, HB, CAP><<<grid, DM_THREADS, smem, stream>>>(m, a);
  return cudaGetLastError();
}

template <int D, int NSTAGE, int HB>
cudaError_t launch_cap(const DecodeMaps& m, const MaskedArgs& a, int sms, cudaStream_t stream) {
  return a.softcap == 0.f ? launch_t<D, NSTAGE, HB, false>(m, a, sms, stream)
                          : launch_t<D, NSTAGE, HB, true>(m, a, sms, stream);
}

}  // namespace

cudaError_t launch_decode_masked(const DecodeMaps& m, const MaskedArgs& a, int head_dim, cudaStream_t stream) {
  int dev = 0;
  const int sms = current_device_sms(&dev);
  if (sms <= 0) return cudaErrorInvalidDevice;
  const bool narrow = a.G <= 8;   // one block of 8 heads: half the registers, two CTAs an SM
  if (head_dim == 128)
    return narrow ? launch_cap<128, 2, 8>(m, a, sms, stream) : launch_cap<128, 4, 16>(m, a, sms, stream);
  return narrow ? launch_cap<64, 4, 8>(m, a, sms, stream) : launch_cap<64, 8, 16>(m, a, sms, stream);
}

}  // namespace ink
