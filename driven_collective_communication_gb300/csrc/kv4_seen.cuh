// kv4_seen.cuh -- attention of many query rows over the 4-bit paged cache, for rows
// with sets of seen keys of their own: trees of drafted tokens, and windows whose
// first tokens stay visible.
//
// The steps and roles are the prompt kernel's (kv4_prompt.cuh: 256 rows of one
// sequence, rank and kv head, 128 keys a step; S = Q K^T, P = 2^(c S - ref) and O +=
// P V on tcgen05, one warp that loads, one that issues, four that unpack, eight
// that make P).  What differs:
//
// Which keys a row sees.  A step whose keys some row of a warp does not see first
// takes the rows' 128 bits -- a run of keys, the sinks, and of a tree the mask's
// words shifted into place -- and puts -infinity over the hidden scores in tensor
// memory.  What follows is one form for all steps.  A tree has a few such steps a
// tile (the drafted tokens lie at the end), a window two or three.
//
// Work split.  Verifying a tree, a segment has one or a few row tiles and thousands
// of keys, and there may be one sequence: tiles alone would leave the SMs idle.
// So all steps of all tiles form one line, cut evenly over the SMs; a CTA goes from
// piece to piece with its barriers' phases running on, the loading warp finds the
// pieces ahead, and the next piece's Q comes before this one's results are
// written.  A tile that is cut leaves its reference, sum and O in fp32, and a second
// kernel joins them in order: results do not depend on timing.
//
// Bound by neither the tensor pipe (37 %) nor the issue slots (47 %): the chain of
// hand-overs between the roles, as in the prompt kernel.  Measured on GB300, 128
// channels, 8 heads per kv head: 152 segments of 4096 keys x 32 drafted tokens fp16
// 91 us, bf16 109 (2.4 and 2.8 us a step, and 15 for start and end); 32 requests of
// up to 4096 keys, 8 ranks, bf16 149 us (0.37 PFLOP/s: a third is start, the ends of
// pieces and the join); one of 131,109 keys x 63 tokens, 16 kv heads of 4 heads, fp16
// 276 us (1.0 PFLOP/s).
//
// Code size decided most: each role's code has to stay in the instruction cache.
// A masked and an unmasked form of the steps, and Q and the results in unrolled
// loops, had taken 120 us instead of 91 (182 instead of 127 with a window).  Tried
// without gain: a warp for each row tile's MMAs (110 us: in one thread's order the
// tiles' chains stay half a step apart), eight unpacking warps with the registers
// split by roles (96 us), pages asked into L2 ahead (no change), the waits' loop as
// a function (96 us), Q's loads a step earlier (no change).
//
// The code stands apart from the prompt kernel's: as one template, that one's time
// moved by up to 7 % either way.
//
// What it rounds: as the prompt kernel, each of K, V and P to fp16; with 64 channels
// and fp16 output K is two numbers (kSeenExactK).
#pragma once
#include "kv4_prompt.cuh"

namespace dcc {

// What a CTA works on: up to 256 rows of one (sequence, rank, kv head) and some of
// the steps over their keys -- all of them, or what its share of them holds.
struct PromptPiece {
  int seq, rank, head, begin, pos0, news;  // (begin .. news: the sequence's rows, DecSeq)
  int row_lo, row_hi;
  int page0, kept, pages;                  // the tile's pages, as in DecSeq
  int len;                                 // keys from here on are seen by no row
  int j0, j1;                              // steps j0 .. j1 - 1
  int slot;                                // where its partial goes; -1: it is whole
  int parts;                               // the CTAs that hold a part of the tile, where this is the first of several
};

// ---- an even split.  The steps of all tiles (of 256 rows; by sequence, rank,
// kv head) form one line, of which every CTA takes an equal run; a tile that is
// cut leaves partials (reference, l, O), joined by a second kernel.  Each tile
// of a sequence counts the same number of steps: exact in a tree, where all rows
// see the whole context, and at most one too many with a window, unless the
// sequence is shorter than that.
__device__ __forceinline__ int seen_tile_steps(const AttnArgs& a, const DecSeq& q) {
  long long pages = q.pages;
  if (!a.mask) {
    const long long keys = (long long)a.window + (kPromptRows - 2 + a.share) / a.share;  // from the first row's first one
    const long long most = (keys + kKv4Page - 2) / kKv4Page + 1 + (a.sinks + kKv4Page - 1) / kKv4Page;
    if (most < pages) pages = most;
  }
  return (int)((pages + 1) / 2);
}
struct SeenWalk {
  long long u, end;  // the next step of the line, and the end of the CTA's run
  long long units;   // of the line
  int ctas;
  int s, seg, j;     // the sequence, its tile (rank and head slowest), the step within
  bool over;         // that was the sequence's last tile
};
// The next piece of a run, whose sequence has tiles from w.seg on (one thread).
__device__ __forceinline__ bool seen_next(const Kv4Dev& kv, const AttnArgs& a, SeenWalk& w, PromptPiece& p) {
  if (w.u >= w.end) return false;
  const DecSeq q = dec_seq<true>(kv, a, w.s, kPromptRows);
  const int rh = w.seg / q.tiles, tile = w.seg - rh * q.tiles, steps = seen_tile_steps(a, q);
  p.seq = w.s;
  p.rank = rh / kv.heads;
  p.head = rh - p.rank * kv.heads;
  p.begin = q.begin;
  p.pos0 = q.pos0;
  p.news = q.news;
  p.row_lo = tile * kPromptRows;
  p.row_hi = min(q.rows, p.row_lo + kPromptRows);
  p.page0 = q.page0;
  p.kept = q.kept;
  p.pages = q.empty ? 0 : q.pages;
  p.len = kv.len[w.s];
  if (!a.mask) {
    const int pos_lo = q.pos0 + p.row_lo / a.share, pos_hi = q.pos0 + (p.row_hi - 1) / a.share;
    p.page0 = max(0, pos_lo - a.window + 1) / kKv4Page;
    p.kept = min((a.sinks + kKv4Page - 1) / kKv4Page, p.page0);
    if (p.kept == p.page0) p.kept = 0, p.page0 = 0;
    p.page0 -= p.kept;
    p.pages = pos_hi < 0 ? 0 : min(pos_hi / kKv4Page, kv.max_pages) - p.page0 + 1;
    p.len = min(p.len, pos_hi + 1);
  }
  const int take = (int)min((long long)(steps - w.j), w.end - w.u), real = (p.pages + 1) / 2;
  p.j0 = min(w.j, real);
  p.j1 = min(w.j + take, real);
  p.slot = take == steps ? -1 : w.j > 0 ? 0 : 1;
  p.parts = 0;
  if (p.slot == 1)  // the CTA with the tile's last step
    p.parts = (int)(((w.u + steps) * w.ctas - 1) / w.units) - (int)(((w.u + 1) * w.ctas - 1) / w.units) + 1;
  w.u += take;
  w.j = 0;
  ++w.seg;
  w.over = w.seg >= kv.n * kv.heads * q.tiles;
  return true;
}
// what a call's workspace holds after the streaming kernel's counters
struct SeenJoin {
  int parts, rank, head, row_lo, row_hi, begin, pad[2];
};
constexpr int kSeenRing = 4;  // pieces known at a time
constexpr int kSeenJoinBytes = kDecMaxCtas * (int)sizeof(SeenJoin);
// floats of a partial: reference and l of each row, then O, four channels of all rows
// after the other (a warp holds 32 rows and writes whole lines)
__host__ __device__ constexpr size_t seen_part(int dim) { return (size_t)kPromptRows * (dim + 2); }
__host__ __device__ constexpr size_t seen_ws_bytes(int dim) {
  return 1024 + kSeenJoinBytes + 2 * kDecMaxCtas * seen_part(dim) * 4;
}
__device__ __forceinline__ SeenJoin* seen_joins(const AttnArgs& a) { return reinterpret_cast<SeenJoin*>(a.ws + 1024); }
__device__ __forceinline__ float* seen_parts(const AttnArgs& a, int dim, int cta, int slot) {
  return reinterpret_cast<float*>(a.ws + 1024 + kSeenJoinBytes) + (2 * (size_t)cta + slot) * seen_part(dim);
}

// fp16 output of 64-wide heads: K in two numbers.  Rounded to fp16, K, V and P
// together put an output that sees a few hundred keys 3.5e-4 off where its own
// rounding is 2.1e-4, and K is the largest of the three; the second number has room
// in shared memory at 64 channels only.
template <typename T, int D>
constexpr bool kSeenExactK = std::is_same<T, __half>::value && D == 64;
template <typename T, int D, int G>
constexpr size_t kSeenSmem = PromptShape<D, G>::smem + (kSeenExactK<T, D> ? 2 * PromptShape<D, G>::kv_tile : 0);
// lo + step * code, biased codes as Pair16, as a number and what its rounding left: both
// parts of that are exact, their sum is rounded, 2^-22 of |step code| + |value|
__device__ __forceinline__ void value_exact(uint32_t c, uint32_t step, uint32_t lo, uint32_t* big, uint32_t* small) {
  const uint32_t bias = 0x54005400u;
  auto h = [](const uint32_t& w) { return *reinterpret_cast<const __half2*>(&w); };
  const __half2 n = __hsub2(h(c), h(bias)), p = __hmul2(n, h(step)), q = __hfma2(n, h(step), __hneg2(p));  // p + q, exactly
  const __half2 s = __hadd2(p, h(lo)), b = __hsub2(s, p);
  const __half2 r = __hadd2(q, __hadd2(__hsub2(p, __hsub2(s, b)), __hsub2(h(lo), b)));  // the product's error, and the sum's
  *big = *reinterpret_cast<const uint32_t*>(&s);
  *small = *reinterpret_cast<const uint32_t*>(&r);
}

template <typename T, int D, int G>
__global__ void __launch_bounds__(kPromptThreads, 1) k_kv4_seen(Kv4Dev kv, const __grid_constant__ AttnArgs a, LocalDev dc) {
  using Shape = PromptShape<D, G>;
  constexpr bool FP16 = std::is_same<T, __half>::value;
  constexpr int NG = D / G, BLK = Shape::block, R = kPromptRing, JW = D / 32;
  constexpr float kShift = 6.0f;  // P is 2^6 times what ref says: fp16 keeps it normal down to 2^-20
  extern __shared__ unsigned char prompt_raw[];
  __shared__ uint32_t tmem_slot;
  __shared__ uint32_t s_absent[8];  // by step: bits of pages that are not there
  // bf16 cache, by step and page: 1 where a key of K has its own scale, 2 where V stays bf16
  __shared__ __align__(2) uint8_t s_range[8][2];
  __shared__ int8_t s_exp[4][128];  // by step: K's powers of two
  // the pieces, found by the warp that loads, ahead of the others; what comes after the
  // last one has row_hi 0
  __shared__ SeenWalk s_walk;
  __shared__ PromptPiece s_piece[kSeenRing];
  __shared__ __align__(8) uint64_t s_piece_bars[2 * kSeenRing];
  auto piece_full = [&](int k) { return smem_addr_u32(&s_piece_bars[k % kSeenRing]); };
  auto piece_free = [&](int k) { return smem_addr_u32(&s_piece_bars[kSeenRing + k % kSeenRing]); };
  const uint32_t base = (smem_addr_u32(prompt_raw) + 1023u) & ~1023u;
  const uint32_t sq = base, sk = sq + 2 * Shape::q_tile, sv = sk + 2 * Shape::kv_tile;
  constexpr bool EXACT = kSeenExactK<T, D>;
  const uint32_t sk2 = sv + 2 * Shape::kv_tile, raw = sk2 + (EXACT ? 2 * Shape::kv_tile : 0);  // (K's second numbers)
  unsigned char* raw_g_rw = prompt_raw + (raw - smem_addr_u32(prompt_raw));
  const unsigned char* raw_g = raw_g_rw;
  const uint32_t bars = raw + (uint32_t)(R * BLK);
  auto rawf = [&](int s) { return bars + 8u * (uint32_t)s; };
  auto rawe = [&](int s) { return bars + 8u * (uint32_t)(R + s); };
  auto ready = [&](int s) { return bars + 8u * (uint32_t)(2 * R + 16 + s); };
  auto two = [&](int kind, int i) { return bars + 8u * (uint32_t)(2 * R + 2 * kind + i); };
  const uint32_t last = bars + 8u * (uint32_t)(3 * R + 16);  // the products in flight when a wait gave up
  enum { kFull = 0, kFree, vFull, vFree, sFull, pFull, pvDone, qFull };  // the last: one for both
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    mma_mbar_init(last, 1);
    for (int i = 0; i < R; ++i) {
      mma_mbar_init(rawf(i), 1);
      mma_mbar_init(rawe(i), 4);
      mma_mbar_init(ready(i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mma_mbar_init(two(kFull, i), 4);
      mma_mbar_init(two(kFree, i), 1);
      mma_mbar_init(two(vFull, i), 4);
      mma_mbar_init(two(vFree, i), 1);
      mma_mbar_init(two(sFull, i), 1);
      mma_mbar_init(two(pFull, i), 4);
      mma_mbar_init(two(pvDone, i), 1);
      mma_mbar_init(two(qFull, i), 4);
    }
    for (int i = 0; i < kSeenRing; ++i) {
      mma_mbar_init(piece_full(i), 1);
      mma_mbar_init(piece_free(i), FP16 ? 13 : 15);  // one each from the warps that read it
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  pdl_wait();

  // ---- the line of steps, and this CTA's run of it
  {
    __shared__ long long s_sum[kPromptThreads / 32];
    const int nh = kv.n * kv.heads, cta = (int)blockIdx.x;
    auto steps_of = [&](int s) {
      if (s >= kv.seqs) return 0ll;
      const DecSeq q = dec_seq<true>(kv, a, s, kPromptRows);
      return q.tiles > 0 ? (long long)q.tiles * seen_tile_steps(a, q) : 0ll;
    };
    auto scan = [&](long long mine, long long* total) {  // exclusive, over the CTA
      long long x = mine;
#pragma unroll
      for (int m = 1; m < 32; m <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, m);
        if (lane >= m) x += y;
      }
      __syncthreads();
      if (lane == 31) s_sum[warp] = x;
      __syncthreads();
      long long first = x - mine;
      *total = 0;
      for (int w = 0; w < kPromptThreads / 32; ++w) {
        if (w < warp) first += s_sum[w];
        *total += s_sum[w];
      }
      return first;
    };
    long long units = 0, first0 = 0, mine0 = 0;
    for (int s0 = 0; s0 < kv.seqs; s0 += kPromptThreads) {
      const long long mine = steps_of(s0 + (int)threadIdx.x);
      long long total;
      const long long first = scan(mine, &total);
      if (s0 == 0) first0 = first, mine0 = mine;
      units += total;
    }
    units *= nh;
    const int C = units < (long long)gridDim.x ? (int)units : (int)gridDim.x;
    if (cta >= C) {
      if (threadIdx.x == 0) seen_joins(a)[cta].parts = 0;
      return;
    }
    const long long c0 = units * cta / C, c1 = units * (cta + 1) / C;
    long long before = 0;
    for (int s0 = 0; s0 < kv.seqs && before * nh <= c0; s0 += kPromptThreads) {
      const int s = s0 + (int)threadIdx.x;
      long long mine = mine0, first = first0;
      if (kv.seqs > kPromptThreads) {
        mine = steps_of(s);
        long long total;
        first = before + scan(mine, &total);
        before += total;
      } else {
        before = units;
      }
      if (mine && first * nh <= c0 && c0 < (first + mine) * nh) {
        const int steps = seen_tile_steps(a, dec_seq<true>(kv, a, s, kPromptRows));
        const long long in = c0 - first * nh;
        s_walk = SeenWalk{c0, c1, units, C, s, (int)(in / steps), (int)(in % steps), false};
      }
    }
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr_u32(&tmem_slot)),
                 "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  pdl_trigger();  // not before the allocation
  tc_fence_after();
  const uint32_t tmem = tmem_slot;  // S / P of the two row tiles, then O: 128 columns each
  auto range = [&](int j) { return FP16 ? 0u : (uint32_t)*reinterpret_cast<const volatile uint16_t*>(s_range[j & 7]); };
  auto wide_v = [&](int j, int h) { return (range(j) & (2u << 8 * h)) != 0; };
  auto wait = [&](uint32_t bar, int phase) {
    return local_wait(bar, (uint32_t)phase & 1u, dc, 0, (int)blockIdx.x);
  };
  // Calls `work` for every piece with the steps before it, until one returns false
  // (one thread, or a whole warp).
  auto pieces = [&](bool whole_warp, auto&& work) {
    for (int k = 0, done = 0;; ++k) {
      if (!wait(piece_full(k), k / kSeenRing)) return false;
      const PromptPiece& p = s_piece[k % kSeenRing];
      if (p.row_hi == 0) return true;
      if (!work(p, done)) return false;
      done += p.j1 - p.j0;
      if (whole_warp) __syncwarp();
      if (!whole_warp || lane == 0) mbar_arrive(piece_free(k));
    }
  };
  // the table's slot of a tile's page
  auto slot_at = [&](const PromptPiece& p, int v) { return v < p.kept ? v : p.page0 + v; };

  if (warp == 0) {  // ---- loads
    int unfinished = 0;
    auto load = [&](const PromptPiece& pc, int before) {
      int ids = -1, ids_at = -(1 << 30);
      const int ahead = 2 * (before - pc.j0);  // of the ring, against the tile's pages
      for (int v = 2 * pc.j0; v < 2 * pc.j1; ++v) {
        const int p = v + ahead;
        if (v - ids_at >= 32) {
          ids_at = v;
          ids = v + lane < pc.pages ? kv4_page(kv, pc.seq, slot_at(pc, v + lane)) : -1;
        }
        const int page = __shfl_sync(0xffffffffu, ids, v - ids_at), slot = p % R;
        if (p >= R && !wait(rawe(slot), p / R - 1)) return false;
        if (lane == 0) {
          uint32_t& absent = s_absent[(p / 2) & 7];
          absent = (p & 1 ? absent : 0u) | (page < 0 ? 1u << (p & 1) : 0u);
          mma_mbar_expect(rawf(slot), page < 0 ? 0u : (uint32_t)BLK);
          if (page >= 0)
            asm volatile(
                "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                    raw + (uint32_t)(slot * BLK)),
                "l"(kv4_block(kv, pc.rank, a.layer, page, pc.head, BLK)), "r"((uint32_t)BLK), "r"(rawf(slot))
                : "memory");
        }
        ++unfinished;
      }
      return true;
    };
    // Piece k + 1 is made known before piece k's pages are asked for.  A slot of the
    // ring is free once piece k + 1 - kSeenRing has been worked off, whose pages
    // have been loaded.
    auto publish = [&](int k) {
      if (k >= kSeenRing && !wait(piece_free(k), k / kSeenRing - 1)) return false;
      if (s_walk.over) {  // on to the next sequence that has rows
        const int s = next_with_rows(kv, a, s_walk.s);
        __syncwarp();  // all have read the walk
        if (lane == 0) s_walk.s = s, s_walk.seg = 0, s_walk.over = false;
      }
      __syncwarp();
      if (lane == 0) {
        PromptPiece& p = s_piece[k % kSeenRing];
        if (!seen_next(kv, a, s_walk, p)) p.row_hi = 0;
        mbar_arrive(piece_full(k));
      }
      __syncwarp();
      return true;
    };
    bool ok = publish(0);
    for (int k = 0, before = 0; ok; ++k) {
      const PromptPiece pc = s_piece[k % kSeenRing];
      if (pc.row_hi == 0) break;
      ok = publish(k + 1) && load(pc, before);
      before += pc.j1 - pc.j0;
    }
    // a copy in flight when a wait gave up ends before the CTA does
    for (int p = max(0, unfinished - R); p < unfinished; ++p) local_drain(rawf(p % R), (uint32_t)(p / R) & 1u);
  } else if (warp == 1) {  // ---- MMAs
    if (lane == 0) {
      const uint32_t id = (1u << 4) | ((uint32_t)(128 >> 4) << 24);  // fp16 operands; bf16: bits 7 and 10
      const uint32_t id_s = id | ((uint32_t)(128 >> 3) << 17), id_o = id | ((uint32_t)(D >> 3) << 17);
      uint32_t rg0 = 0, rg1 = 0;  // of even and odd steps
      bool ok = true;
      int had[2] = {0, 0}, qs[2] = {0, 0};  // by row tile: steps and tiles of Q so far
      pieces(false, [&](const PromptPiece& pc, int before) {
        const int steps = pc.j1 - pc.j0, nt = pc.row_hi - pc.row_lo > 128 ? 2 : 1;
        if (steps == 0) return true;
        auto scores = [&](int g, int jj) {
          const int j = before + jj;
          ok = ok && wait(two(kFull, j & 1), j >> 1);
          if (!ok) return;
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = (uint32_t)(kk / 4) * 16384u + (uint32_t)(kk % 4) * 32u;
            const uint64_t ad = mma_smem_desc(sq + (uint32_t)(g * Shape::q_tile) + off);
            const uint64_t bd = mma_smem_desc(sk + (uint32_t)((j & 1) * Shape::kv_tile) + off);
            asm volatile(
                "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem + (uint32_t)g * 128u),
                "l"(ad), "l"(bd), "r"(id_s), "r"(kk > 0 ? 1u : 0u)
                : "memory");
            if constexpr (EXACT)
              asm volatile(
                  "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                  "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem + (uint32_t)g * 128u),
                  "l"(ad), "l"(mma_smem_desc(sk2 + (uint32_t)((j & 1) * Shape::kv_tile) + off)), "r"(id_s), "r"(1u)
                  : "memory");
          }
          tc_commit(two(sFull, g));
          if (g == nt - 1) tc_commit(two(kFree, j & 1));
          (j & 1 ? rg1 : rg0) = range(j);
        };
        for (int g = 0; g < nt; ++g) ok = ok && wait(two(qFull, g), qs[g]);
        for (int g = 0; g < nt; ++g) scores(g, 0);
        for (int jj = 0; jj < steps && ok; ++jj)
          for (int g = 0; g < nt && ok; ++g) {
            const int j = before + jj;
            ok = wait(two(pFull, g), had[g] + jj) && wait(two(vFull, j & 1), j >> 1);
            if (!ok) break;
            tc_fence_after();
            const uint32_t bf = (1u << 7) | (1u << 10);
            const uint32_t ids[2] = {id_o | ((j & 1 ? rg1 : rg0) & 2u ? bf : 0u), id_o | ((j & 1 ? rg1 : rg0) & 0x200u ? bf : 0u)};
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) {
              const uint32_t off = (uint32_t)(kk / 4) * (D * 128u) + (uint32_t)(kk % 4) * 32u;
              const uint64_t bd = mma_smem_desc(sv + (uint32_t)((j & 1) * Shape::kv_tile) + off);
              asm volatile(
                  "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                  "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(tmem + 256u + (uint32_t)g * 128u),
                  "r"(tmem + (uint32_t)g * 128u + (uint32_t)kk * 8u), "l"(bd), "r"(ids[kk / 4]), "r"(jj > 0 || kk > 0 ? 1u : 0u)
                  : "memory");
            }
            if (g == nt - 1) tc_commit(two(vFree, j & 1));
            tc_commit(two(pvDone, g));
            if (jj + 1 < steps) scores(g, jj + 1);
          }
        for (int g = 0; g < nt; ++g) {
          had[g] += steps;
          ++qs[g];
        }
        return ok;
      });
      if (!ok) {
        tc_commit(last);
        local_drain(last, 0);
      }
    }
    __syncwarp();
  } else if (warp < 6) {  // ---- unpack
    const int tid = (int)threadIdx.x - 64;
    bool ok = true;
    auto done_with = [&](int p) {
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(rawe(p % R));
    };
    pieces(true, [&](const PromptPiece& pc, int before) {
      const int len = pc.len, ahead = before - pc.j0;
      for (int j = before; j < before + (pc.j1 - pc.j0) && ok; ++j) {
        const int buf = j & 1;
        auto key_at = [&](int p) { return slot_at(pc, p - 2 * ahead) * kKv4Page; };  // of a page of the ring
        const uint32_t kt = sk + (uint32_t)(buf * Shape::kv_tile), vt = sv + (uint32_t)(buf * Shape::kv_tile);
        if (j >= 2) ok = wait(two(kFree, buf), (j >> 1) - 1);
        uint32_t absent = 0;
#pragma unroll 1
        for (int h = 0; h < 2 && ok; ++h) {  // K of the two pages
          const int p = 2 * j + h, slot = p % R;
          ok = wait(rawf(slot), p / R) && (FP16 || wait(ready(slot), p / R));
          if (!ok) break;
          absent = s_absent[j & 7];
          const bool there = !((absent >> h) & 1u);
          const unsigned char* blk = raw_g + slot * BLK;
          const uint32_t* par = reinterpret_cast<const uint32_t*>(blk + 2 * kv4_codes_bytes(D));
          if (!there) continue;
          // eight neighbouring lanes take the four quarters of rows r and r ^ 5
          // (other half of the banks, other half of the swizzled chunks): no
          // bank conflicts on either side
          const int t = tid & 3;
#pragma unroll 1
          for (int pass = 0; pass < 2; ++pass) {
            const int key = (2 * ((tid >> 3) + 16 * pass)) ^ ((tid & 4) ? 5 : 0);
            const uint32_t row = kt + (uint32_t)(64 * h + key) * 128u;
            const unsigned char* src = blk + key * (D / 2) + t * (JW * 4);
            uint32_t step[NG], lo[NG], w[JW];
            uint32_t odd = 0;  // fp16: large or not finite, K or V (the bf16 cache's parameters have been seen to)
#pragma unroll
            for (int gr = 0; gr < NG; ++gr) {
              const uint32_t pw = par[key * NG + gr];
              if (FP16) odd |= param_large(par[(kKv4Page + key) * NG + gr]) | param_large(pw);
              step[gr] = __byte_perm(pw, pw, 0x1010);
              lo[gr] = __byte_perm(pw, pw, 0x3232);
            }
            if (FP16 && (odd & kBad)) {  // rare, so little code: a pair at a time, in fp32
              uint32_t bad = 0;
#pragma unroll
              for (int gr = 0; gr < NG; ++gr) bad |= param_bad<T>(par[(kKv4Page + key) * NG + gr]);
#pragma unroll 1
              for (int i = 0; i < 4 * JW; ++i) {
                const int u = 4 * (i >> 2) + t;
                const uint32_t c = reinterpret_cast<const uint32_t*>(src)[i >> 2] >> (4 * (i & 3));
                const uint32_t pw = par[key * NG + 8 * u / G];
                const float2 f = Half16<T>::widen2(pw);
                const float2 v = make_float2(fmaf((float)(c & 15u), f.x, f.y), fmaf((float)((c >> 16) & 15u), f.x, f.y));
                const uint32_t pair = (bad | param_bad<T>(pw)) & kBad ? 0xffffffffu /* NaN */ : narrow_finite<T>(v.x, v.y);
                asm volatile("st.shared.b32 [%0], %1;" ::"r"(row + (uint32_t)(u / 8) * 16384u +
                                                             (uint32_t)(((u % 8) ^ (key & 7)) * 16 + 4 * (i & 3))),
                             "r"(pair)
                             : "memory");
                if constexpr (EXACT) {
                  // what the first number left: at most 16, or 32 of a last code an ulp past
                  // the type's largest number; nothing of a NaN, or of a value further out
                  const float2 b = Half16<T>::widen2(pair), r = make_float2(v.x - b.x, v.y - b.y);
                  asm volatile("st.shared.b32 [%0], %1;" ::"r"(row + (sk2 - sk) + (uint32_t)(u / 8) * 16384u +
                                                               (uint32_t)(((u % 8) ^ (key & 7)) * 16 + 4 * (i & 3))),
                               "r"(Half16<T>::narrow2(fabsf(r.x) <= 32.0f ? r.x : 0.0f, fabsf(r.y) <= 32.0f ? r.y : 0.0f))
                               : "memory");
                }
              }
              continue;
            }
            if constexpr (JW == 4) {
              const uint4 v = *reinterpret_cast<const uint4*>(src);
              w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
            } else {
              const uint2 v = *reinterpret_cast<const uint2*>(src);
              w[0] = v.x, w[1] = v.y;
            }
#pragma unroll
            for (int jj = 0; jj < JW; ++jj) {
              const int u = 4 * jj + t, gr = 32 * jj / G;  // channels 8 u ..
              const uint32_t at = row + (uint32_t)(u / 8) * 16384u + (uint32_t)(((u % 8) ^ (key & 7)) * 16);
              if constexpr (EXACT) {
                uint4 a, b;
                value_exact(Pair16<__half>::code<0>(w[jj]), step[gr], lo[gr], &a.x, &b.x);
                value_exact(Pair16<__half>::code<1>(w[jj]), step[gr], lo[gr], &a.y, &b.y);
                value_exact(Pair16<__half>::code<2>(w[jj]), step[gr], lo[gr], &a.z, &b.z);
                value_exact(Pair16<__half>::code<3>(w[jj]), step[gr], lo[gr], &a.w, &b.w);
                sts128(at, a);
                sts128(at + (sk2 - sk), b);
                continue;
              }
              const uint4 v = make_uint4(Pair16<__half>::value(Pair16<__half>::code<0>(w[jj]), step[gr], lo[gr]),
                                         Pair16<__half>::value(Pair16<__half>::code<1>(w[jj]), step[gr], lo[gr]),
                                         Pair16<__half>::value(Pair16<__half>::code<2>(w[jj]), step[gr], lo[gr]),
                                         Pair16<__half>::value(Pair16<__half>::code<3>(w[jj]), step[gr], lo[gr]));
              sts128(at, v);
            }
          }
        }
        if (!ok) break;
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(two(kFull, buf));
        if (j >= 2) ok = wait(two(vFree, buf), (j >> 1) - 1);
        if (!ok) break;
        // V: a thread takes a chunk's word of 8 neighbouring keys (at D = 128 every
        // other run of keys in swapped order, so that the two runs a warp works
        // on lie in different banks); D = 64 has one word a chunk, so each half
        // of the threads takes a page
#pragma unroll 1
        for (int h = D == 128 ? 0 : tid >> 6; h < 2; h += D == 128 ? 1 : 2) {
          const int p = 2 * j + h;
          if (D == 128 && h) done_with(p - 1);
          const unsigned char* blk = raw_g + (p % R) * BLK;
          const int c = tid & 7, oct = D == 128 ? tid >> 4 : (tid >> 3) & 7, ws = D == 128 ? (tid >> 3) & 1 : 0;
          const int swap = D == 128 ? oct & 1 : 0;
          const uint32_t sel0 = swap ? 0x1054u : 0x5410u, sel1 = swap ? 0x3276u : 0x7632u;
          const uint32_t* par = reinterpret_cast<const uint32_t*>(blk + 2 * kv4_codes_bytes(D)) + kKv4Page * NG;
          const bool there = !((absent >> h) & 1u);
          bool wide = !FP16 && wide_v(j, h);
          // the word's channels lie in one group (G = 64) or two (32)
          const int g0 = 64 * ws / G;
          constexpr int GW = G == 32 ? 2 : 1;
          auto by_pairs = [&]() {  // rare, so little code rather than fast: two keys of a channel at a time, in fp32
#pragma unroll 1
            for (int i = 0; i < 32; ++i) {
              const int n = i >> 2, gr = g0 + (GW > 1 ? n >> 2 : 0), d = 64 * ws + 16 * (n >> 1) + c + 8 * (n & 1);
              float v[2];
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                const int key = 8 * oct + 2 * (i & 3) + x;
                const uint32_t word = *reinterpret_cast<const uint32_t*>(blk + kv4_codes_bytes(D) + key * (D / 2) +
                                                                         kv4_v_chunk(D, c, key) * (D / 16) + ws * 4);
                const uint32_t pw = par[key * NG + gr];
                const float2 f = Half16<T>::widen2(pw);
                const bool none = (param_bad<T>(pw) & kBad) || !there || key_at(p) + key >= len;
                v[x] = none ? 0.0f : fmaf((float)((word >> (4 * n)) & 15u), f.x, f.y);
              }
              const uint32_t pair = narrow_finite<T>(v[0], v[1]);
              asm volatile("st.shared.b32 [%0], %1;" ::"r"(vt + (uint32_t)h * (D * 128u) + (uint32_t)d * 128u +
                                                           (uint32_t)((oct ^ (d & 7)) * 16 + 4 * (i & 3))),
                           "r"(pair)
                           : "memory");
            }
          };
          if (!FP16 && wide) {
            by_pairs();
            continue;
          }
          uint32_t w[8], pr[8][GW], bad = 0;
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int key = 8 * oct + (k ^ swap);
            w[k] = *reinterpret_cast<const uint32_t*>(blk + kv4_codes_bytes(D) + key * (D / 2) +
                                                      kv4_v_chunk(D, c, key) * (D / 16) + ws * 4);
#pragma unroll
            for (int x = 0; x < GW; ++x) {
              pr[k][x] = par[key * NG + g0 + x];
              bad |= FP16 ? param_large(pr[k][x]) : param_bad<__half>(pr[k][x]);
            }
          }
          if ((bad & kBad) || !there || key_at(p) + 8 * oct + 7 >= len) {  // some key must be zero
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const int key = 8 * oct + (k ^ swap);
              uint32_t any = 0;  // (another group of the key may be bad: its own unit sees to it)
#pragma unroll
              for (int x = 0; x < GW; ++x) any |= param_bad<__half>(pr[k][x]);
              if ((any & kBad) || !there || key_at(p) + key >= len)
#pragma unroll
                for (int x = 0; x < GW; ++x) pr[k][x] = 0u;
#pragma unroll
              for (int x = 0; x < GW; ++x) wide |= FP16 && (param_large(pr[k][x]) & kBad);  // or is large
            }
            if (FP16 && wide) {
              by_pairs();
              continue;
            }
          }
          uint32_t out[8][4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {  // pairs of keys
            const int k0 = 2 * e, k1 = 2 * e + 1;
            const uint32_t step0 = __byte_perm(pr[k0][0], pr[k1][0], sel0), lo0 = __byte_perm(pr[k0][0], pr[k1][0], sel1);
            const uint32_t step1 = GW > 1 ? __byte_perm(pr[k0][GW - 1], pr[k1][GW - 1], sel0) : step0;
            const uint32_t lo1 = GW > 1 ? __byte_perm(pr[k0][GW - 1], pr[k1][GW - 1], sel1) : lo0;
            const uint32_t x0 = __byte_perm(w[k0], w[k1], sel0), x1 = __byte_perm(w[k0], w[k1], sel1);
            out[0][e] = Pair16<__half>::value(Pair16<__half>::template code<0>(x0), step0, lo0);
            out[1][e] = Pair16<__half>::value(Pair16<__half>::template code<1>(x0), step0, lo0);
            out[2][e] = Pair16<__half>::value(Pair16<__half>::template code<2>(x0), step0, lo0);
            out[3][e] = Pair16<__half>::value(Pair16<__half>::template code<3>(x0), step0, lo0);
            out[4][e] = Pair16<__half>::value(Pair16<__half>::template code<0>(x1), step1, lo1);
            out[5][e] = Pair16<__half>::value(Pair16<__half>::template code<1>(x1), step1, lo1);
            out[6][e] = Pair16<__half>::value(Pair16<__half>::template code<2>(x1), step1, lo1);
            out[7][e] = Pair16<__half>::value(Pair16<__half>::template code<3>(x1), step1, lo1);
          }
#pragma unroll
          for (int n = 0; n < 8; ++n) {
            const int d = 64 * ws + 16 * (n >> 1) + c + 8 * (n & 1);
            sts128(vt + (uint32_t)h * (D * 128u) + (uint32_t)d * 128u + (uint32_t)((oct ^ (d & 7)) * 16),
                   make_uint4(out[n][0], out[n][1], out[n][2], out[n][3]));
          }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(two(vFull, buf));
          if (D == 64) mbar_arrive(rawe((2 * j) % R));
          mbar_arrive(rawe((2 * j + 1) % R));
        }
      }
      return ok;
    });
  } else if (warp >= 14) {  // ---- the bf16 cache's parameters, in place as fp16
    if constexpr (!FP16) {
      // a slot's pages are all one warp's: one that skipped a page of a slot could
      // take the barrier's state before that page for the next page's arrival
      pieces(true, [&](const PromptPiece& pc, int before) {
        const int ahead = 2 * (before - pc.j0), len = pc.len;
        for (int p = 2 * pc.j0 + ahead; p < 2 * pc.j1 + ahead; ++p) {
          const int slot = p % R, j = p >> 1, h = p & 1;
          if ((slot == 1) != (warp == 15)) continue;
          if (!wait(rawf(slot), p / R)) return false;
          uint32_t ranges = 0;
          if (!((s_absent[j & 7] >> h) & 1u)) {
            uint32_t* par = reinterpret_cast<uint32_t*>(raw_g_rw + slot * BLK + 2 * kv4_codes_bytes(D));
            uint32_t k[2][NG], v[2][NG], most = 0, least = 0xffffffffu;
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
              for (int gr = 0; gr < NG; ++gr) {
                k[x][gr] = par[(lane + 32 * x) * NG + gr];
                v[x][gr] = par[(kKv4Page + lane + 32 * x) * NG + gr];
                const uint32_t a = k[x][gr] & 0x7fff7fffu, b = v[x][gr] & 0x7fff7fffu;
                most = __vmaxu2(most, __vmaxu2(a, b));
                least = __vminu2(least, __vminu2(a, b));
              }
            // Mostly all are far inside: steps of 2^-10 .. 2^6 and lo up to 2^10
            // make groups of 2^-8 .. 2^11.
            const bool inside = (least & 0xffffu) >= 0x3a80u && (most & 0xffffu) <= 0x4280u && (most >> 16) <= 0x4480u;
            if (!__all_sync(0xffffffffu, inside)) {
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                const int key = lane + 32 * x;
                const bool counts = slot_at(pc, p - ahead) * kKv4Page + key < len;
                uint32_t bad = 0;
                float m = 0.0f;
                bool fits = true;
#pragma unroll
                for (int gr = 0; gr < NG; ++gr) {
                  m = fmaxf(m, param_top(k[x][gr]));
                  fits = fits && fp16_fits(param_top(v[x][gr]), kTopV);
                  bad |= param_bad<T>(v[x][gr]);
                }
                const int e = fp16_fits(m, kTopK) ? 0 : max(-120, min(126, (int)(__float_as_uint(m) >> 23) - 127));
                s_exp[j & 3][64 * h + key] = (int8_t)e;
                ranges |= counts ? (e ? 1u : 0u) | (fits ? 0u : 2u) : 0u;
#pragma unroll
                for (int gr = 0; gr < NG; ++gr) {
                  const float2 f = param_floats(k[x][gr]);
                  par[key * NG + gr] = (bad & kBad) ? 0xffffffffu : Half16<__half>::narrow2(f.x * power2(-e), f.y * power2(-e));
                }
              }
              ranges = __reduce_or_sync(0xffffffffu, ranges);
            } else {
#pragma unroll
              for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int gr = 0; gr < NG; ++gr) par[(lane + 32 * x) * NG + gr] = param_half(k[x][gr]);
            }
            if (!(ranges & 2u))
#pragma unroll
              for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int gr = 0; gr < NG; ++gr) par[(kKv4Page + lane + 32 * x) * NG + gr] = param_half(v[x][gr]);
          }
          if (lane == 0) s_range[j & 7][h] = (uint8_t)ranges;
          // (the fence before a new page comes over these is the readers')
          __syncwarp();
          if (lane == 0) mbar_arrive(ready(slot));
        }
        return true;
      });
    }
  } else {  // ---- P, one row per thread
    const int g = (warp - 6) >> 2, quad = warp & 3, r = quad * 32 + lane;
    const uint32_t lanes = (uint32_t)(quad * 32) << 16;
    const uint32_t ts = tmem + lanes + (uint32_t)g * 128u, to = tmem + lanes + 256u + (uint32_t)g * 128u;
    // Q into its tile, channels in the codes' order, with the scale's sign; returns
    // what scores are multiplied with
    auto load_q = [&](const PromptPiece& pc) {
      // Straight into shared memory, all loads in flight, neighbouring lanes a row's
      // 16-byte units (a few lines a load, not 32); then in place, a lane a row.  Loops
      // stay loops: this runs once a piece, and much of its time is fetching its code.
      constexpr int UPR = D / 8, RPI = 32 / UPR;
      const int row = pc.row_lo + 128 * g + r, tok = row / a.share, gh = row - tok * a.share;
      const long long own = row < pc.row_hi
                                ? (long long)((size_t)(pc.begin + tok) * a.q_stride + (size_t)(pc.head * a.share + gh) * D)
                                : -1;
      const T* src = static_cast<const T*>(a.q[pc.rank]);
      const int u = lane % UPR, sub = lane / UPR;
      const uint32_t tile = sq + (uint32_t)(g * Shape::q_tile) + (uint32_t)(u / 8) * 16384u;
      auto place = [&](int i) {
        const int x = quad * 32 + i * RPI + sub;
        return tile + (uint32_t)x * 128u + (uint32_t)(((u % 8) ^ (x & 7)) * 16);
      };
#pragma unroll 1
      for (int i = 0; i < UPR; ++i) {
        const long long at = __shfl_sync(0xffffffffu, own, i * RPI + sub);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(place(i)), "l"(src + (at < 0 ? 0 : at + 8 * u)),
                     "r"(at < 0 ? 0 : 16)  // (rows that are not there: zeros)
                     : "memory");
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      __syncwarp();  // (a lane's row has come through all of them)
      const uint32_t own_row = sq + (uint32_t)(g * Shape::q_tile) + (uint32_t)r * 128u;
      auto unit = [&](int x) { return own_row + (uint32_t)(x / 8) * 16384u + (uint32_t)(((x % 8) ^ (r & 7)) * 16); };
      auto get = [&](int x) {
        uint4 v;
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(unit(x)) : "memory");
        return v;
      };
      float c = fabsf(a.scale) * 1.44269504088896341f, f = 1.0f;
      const uint32_t flip = a.scale < 0.0f ? 0x80008000u : 0u;
      if constexpr (!FP16) {  // a bf16 row as fp16: its largest value goes to 2^8 .. 2^9, exactly
        uint32_t top = 0;
#pragma unroll 4
        for (int x = 0; x < UPR; ++x) {
          const uint4 v = get(x);
          top = __vmaxu2(__vmaxu2(__vmaxu2(top, v.x & 0x7fff7fffu), __vmaxu2(v.y & 0x7fff7fffu, v.z & 0x7fff7fffu)),
                         v.w & 0x7fff7fffu);
        }
        top = max(top & 0xffffu, top >> 16);
        const int e = top ? max(-100, min(119, (int)(top >> 7) - 127 - 8)) : 0;
        f = power2(-e);
        c *= power2(e);
      }
      auto half = [&](uint32_t w) {  // two values
        if constexpr (FP16) return w ^ flip;
        const float2 x = param_floats(w);
        return Half16<__half>::narrow2(x.x * f, x.y * f) ^ flip;
      };
#pragma unroll 4
      for (int x = 0; x < UPR; ++x) {
        const uint4 v = get(x);
        sts128(unit(x), make_uint4(half(__byte_perm(v.x, v.z, 0x5410)), half(__byte_perm(v.x, v.z, 0x7632)),
                                   half(__byte_perm(v.y, v.w, 0x5410)), half(__byte_perm(v.y, v.w, 0x7632))));
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(two(qFull, g));
      return c;
    };
    auto mine = [&](const PromptPiece& pc) { return pc.row_hi - pc.row_lo > 128 * g && pc.j1 > pc.j0; };
    // One piece.  before: steps of the CTA so far, had: of this row tile; next() comes
    // between the last scores and the results.
    auto piece = [&](const PromptPiece& pc, int before, int had, float c, auto&& next) {
      const int row = pc.row_lo + 128 * g + r, steps = pc.j1 - pc.j0;
      const bool in = row < pc.row_hi;
      const int tok = row / a.share, gh = row - tok * a.share;
      int hi = in ? pc.pos0 + tok : -1, lo = a.window > 0 ? pc.pos0 + tok - a.window + 1 : 0;
      // the keys that every row of this warp sees need no test
      const int first = pc.row_lo + 128 * g + quad * 32, last = min(first + 31, pc.row_hi - 1);
      int all_hi = first < pc.row_hi ? pc.pos0 + first / a.share : 0x7fffffff;
      int all_lo = a.window > 0 && first < pc.row_hi ? pc.pos0 + last / a.share - a.window + 1 : 0;
      if (a.mask) {
        const SeenRow x = seen_row(a, pc.pos0, in ? pc.news : 0, tok, in ? pc.begin + tok : 0);
        hi = in ? x.hi : -1;
        lo = x.lo;
        all_hi = first < pc.row_hi ? pc.pos0 - 1 : 0x7fffffff;
        all_lo = __reduce_max_sync(0xffffffffu, in ? lo : -(1 << 30));
      }
      if (c == 0.0f) c = 0x1p-140f;  // 0 times the hidden scores' infinity would be NaN
      float ref = 0.0f, l = 0.0f;
      bool any = false, ok = true;
      for (int jj = 0; jj < steps; ++jj) {
        if (!(ok = wait(two(sFull, g), had + jj))) break;
        tc_fence_after();
        const int j = before + jj;
        const int key0 = slot_at(pc, 2 * (pc.j0 + jj)) * kKv4Page;
        const uint32_t absent = s_absent[j & 7];
        const uint32_t rg = range(j);
        const int key1 = slot_at(pc, 2 * (pc.j0 + jj) + 1) * kKv4Page;
        auto whole = [&](int k) { return k + kKv4Page - 1 <= all_hi && (k >= all_lo || k + kKv4Page <= a.sinks); };
        const bool hides = absent || !whole(key0) || !whole(key1);
        const bool wide_p = !FP16 && (rg & 0x202u) != 0;  // a page's V in bf16, so P too
        if (rg & 0x101u) {  // keys with scales of their own
#pragma unroll 1
          for (int c0 = rg & 1u ? 0 : 64; c0 < (rg & 0x100u ? 128 : 64); c0 += 16) {
            uint32_t v[16];
            tmem_ld16(ts + (uint32_t)c0, v);
            tmem_ld_wait16(v);
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * power2(s_exp[j & 3][c0 + i]));
            tmem_st16(ts + (uint32_t)c0, v);
          }
          tmem_st_wait();
        }
        if (hides) {
          // Hidden scores become -infinity in tensor memory, so that one form of what
          // follows serves all steps: two would not stay in the instruction cache.
          const SeenRow x = {hi, lo, pc.pos0, pc.news, a.mask && in ? a.mask + (size_t)(pc.begin + tok) * a.words : nullptr};
#pragma unroll 1
          for (int c0 = 0; c0 < 128; c0 += 32) {
            const uint32_t w = (absent >> (c0 >> 6)) & 1u ? 0u : seen_word(x, a, (c0 < 64 ? key0 : key1) + (c0 & 32));
            uint32_t v[32];
            tmem_ld32(ts + (uint32_t)c0, v);
            tmem_ld_wait32(v);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (!((w >> i) & 1u)) v[i] = 0xff800000u;
            tmem_st16(ts + (uint32_t)c0, v);
            tmem_st16(ts + (uint32_t)c0 + 16u, v + 16);
          }
          tmem_st_wait();
        }
        // Loops over 32 columns stay loops (the roles' code together must stay
        // in the instruction cache); the next columns load under the current.
        uint32_t s[2][32];
        float m0 = -INFINITY, m1 = -INFINITY;
        tmem_ld32(ts, s[0]);
        auto top = [&](const uint32_t* v, int c0) {
#pragma unroll
          for (int i = 0; i < 32; i += 4) {
            m0 = max3(m0, __uint_as_float(v[i]), __uint_as_float(v[i + 1]));
            m1 = max3(m1, __uint_as_float(v[i + 2]), __uint_as_float(v[i + 3]));
          }
        };
#pragma unroll 1
        for (int c0 = 0; c0 < 128; c0 += 64) {
          tmem_ld_wait32(s[0]);
          tmem_ld32(ts + (uint32_t)c0 + 32u, s[1]);
          top(s[0], c0);
          tmem_ld_wait32(s[1]);
          tmem_ld32(ts + ((uint32_t)c0 + 64u) % 128u, s[0]);  // in the end the first columns again
          top(s[1], c0 + 32);
        }
        const float m = fmaxf(m0, m1), mc = m * c;
        const bool grows = m != -INFINITY && (!any || mc > ref + 8.0f);
        if (__any_sync(0xffffffffu, grows && any)) {  // rescale the sums so far
          const float fix = grows && any ? exp2_approx(ref - mc) : 1.0f;
          l *= fix;
          if (!(ok = wait(two(pvDone, g), had + jj - 1))) break;
          tc_fence_after();
#pragma unroll 1
          for (int c0 = 0; c0 < D; c0 += 16) {
            uint32_t v[16];
            tmem_ld16(to + (uint32_t)c0, v);
            tmem_ld_wait16(v);
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * fix);
            tmem_st16(to + (uint32_t)c0, v);
          }
        }
        if (grows) {
          ref = mc;
          any = true;
        }
        const float2 off = make_float2(kShift - ref, kShift - ref), cc = make_float2(c, c);
        float2 sum = make_float2(0.0f, 0.0f);
        auto pair = [&](const uint32_t* v, int i) {
          const float2 x = fma2(make_float2(__uint_as_float(v[i]), __uint_as_float(v[i + 1])), cc, off);
          return make_float2(exp2_approx(x.x), exp2_approx(x.y));
        };
        auto make = [&](const uint32_t* v, int c0) {
          uint32_t w[16];
          if (wide_p) {  // tested once, not per element
            const bool wide = (rg & (c0 < 64 ? 2u : 0x200u)) != 0;
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              const float2 p = pair(v, i);
              sum = add2(sum, p);
              w[i / 2] = wide ? Half16<T>::narrow2(p.x, p.y) : Half16<__half>::narrow2(p.x, p.y);
            }
          } else {
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              const float2 p = pair(v, i);
              sum = add2(sum, p);
              w[i / 2] = Half16<__half>::narrow2(p.x, p.y);
            }
          }
          tmem_st16(ts + (uint32_t)(c0 / 2), w);  // over scores that have been read
        };
#pragma unroll 1
        for (int c0 = 0; c0 < 128; c0 += 64) {
          tmem_ld_wait32(s[0]);
          tmem_ld32(ts + (uint32_t)c0 + 32u, s[1]);
          make(s[0], c0);
          tmem_ld_wait32(s[1]);
          if (c0 == 0) tmem_ld32(ts + 64u, s[0]);
          make(s[1], c0 + 32);
        }
        l += sum.x + sum.y;
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(two(pFull, g));
      }
      if (ok) next();
      const bool some = steps > 0;
      if (ok && some) ok = wait(two(pvDone, g), had + steps - 1);
      tc_fence_after();
      if (pc.slot >= 0) {  // a part of the tile
        float* part = seen_parts(a, D, (int)blockIdx.x, pc.slot);
        const int at = 128 * g + r;
        if (in) {
          part[at] = any || l != 0.0f ? ref : -INFINITY;  // (NaN is seen)
          part[kPromptRows + at] = l;
        }
        float* dst = part + 2 * kPromptRows + 4 * at;
        if (some)
#pragma unroll 1
          for (int c0 = 0; c0 < D; c0 += 16) {
            uint32_t v[16];
            tmem_ld16(to + (uint32_t)c0, v);
            tmem_ld_wait16(v);
            if (in && ok)
#pragma unroll
              for (int i = 0; i < 16; i += 4)
                *reinterpret_cast<uint4*>(dst + (size_t)(c0 + i) * kPromptRows) = make_uint4(v[i], v[i + 1], v[i + 2], v[i + 3]);
          }
        return ok;
      }
      const float inv = l == 0.0f ? 0.0f : __frcp_rn(l);
      const bool wide_out = (reinterpret_cast<uintptr_t>(a.out[pc.rank]) & 31u) == 0;
      const size_t at = (size_t)(pc.begin + tok) * a.q_heads + pc.head * a.share + gh;
#pragma unroll 1
      for (int c0 = 0; c0 < D; c0 += 16) {
        uint32_t v[16], w[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        if (some) {
          tmem_ld16(to + (uint32_t)c0, v);
          tmem_ld_wait16(v);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            w[i] = Half16<T>::narrow2(__uint_as_float(v[2 * i]) * inv, __uint_as_float(v[2 * i + 1]) * inv);
        }
        if (in && ok) {
          uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(a.out[pc.rank]) + at * D + c0);
          if (wide_out) {  // each store of a warp touches 32 lines: half as many
            asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                         "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                         : "memory");
          } else {
            dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
            dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
          }
        }
      }
      if (in && ok && a.lse[pc.rank])
        a.lse[pc.rank][at] = l == 0.0f ? -INFINITY : (ref - kShift + log2f(l)) * 0.69314718055994531f;
      return ok;
    };
    {
      // the next piece's Q is loaded before this one's results are written
      SeenJoin join = {};
      float c_next = 0.0f;
      bool ok = true;
      auto fetch = [&](int k) {
        if (!(ok = wait(piece_full(k), k / kSeenRing))) return;
        const PromptPiece& p = s_piece[k % kSeenRing];
        if (p.row_hi > 0 && mine(p)) c_next = load_q(p);
      };
      fetch(0);
      for (int k = 0, before = 0, had = 0; ok; ++k) {
        const PromptPiece& pc = s_piece[k % kSeenRing];
        if (pc.row_hi == 0) break;
        if (pc.parts) join = SeenJoin{pc.parts, pc.rank, pc.head, pc.row_lo, pc.row_hi, pc.begin, {0, 0}};
        const int steps = pc.j1 - pc.j0;
        if (pc.row_hi - pc.row_lo > 128 * g) {
          const bool done = piece(pc, before, had, c_next, [&] { fetch(k + 1); });
          ok = ok && done;
          had += steps;
        } else {
          fetch(k + 1);
        }
        before += steps;
        __syncwarp();
        if (lane == 0) mbar_arrive(piece_free(k));
      }
      if (warp == 6 && lane == 0) seen_joins(a)[blockIdx.x] = join;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
}

// Joins the parts of the tiles that were cut.  A CTA takes 32 rows, a lane each, its
// warps the channels; the results go through shared memory to whole lines.
constexpr int kSeenJoinThreads = 256, kSeenJoinRows = 32;
template <typename T, int D>
__global__ void __launch_bounds__(kSeenJoinThreads, 3) k_kv4_seen_join(const __grid_constant__ AttnArgs a, int ctas) {
  constexpr int W = kSeenJoinThreads / 32, PER = D / 4 / W, kBatch = 4;  // 16-byte units of a row a warp takes; parts in flight
  constexpr float kShift = 6.0f;
  __shared__ int s_list[kDecMaxCtas], s_warp[W];
  __shared__ uint2 s_out[kSeenJoinRows][D / 4 + 1];
  pdl_prologue();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const SeenJoin* joins = seen_joins(a);
  // the tiles that were cut, in order: the same list in every CTA
  static_assert(kDecMaxCtas <= kSeenJoinThreads, "a thread each");
  const bool mine = (int)threadIdx.x < ctas && joins[threadIdx.x].parts > 0;
  const uint32_t there = __ballot_sync(0xffffffffu, mine);
  if (lane == 0) s_warp[warp] = __popc(there);
  __syncthreads();
  int count = 0, before = 0;
#pragma unroll
  for (int w = 0; w < W; ++w) {
    if (w < warp) before += s_warp[w];
    count += s_warp[w];
  }
  if (mine) s_list[before + __popc(there & ((1u << lane) - 1u))] = (int)threadIdx.x;
  __syncthreads();
  constexpr int kChunks = kPromptRows / kSeenJoinRows;
  for (int item = blockIdx.x; item < count * kChunks; item += gridDim.x) {
    const int cta = s_list[item / kChunks], row0 = item % kChunks * kSeenJoinRows, row = row0 + lane;
    const SeenJoin j = joins[cta];
    if (j.row_lo + row0 >= j.row_hi) continue;
    const bool in = j.row_lo + row < j.row_hi;
    auto part = [&](int i) { return seen_parts(a, D, cta + i, i == 0 ? 1 : 0); };
    float m = -INFINITY;  // the row's largest reference
    for (int i0 = 0; i0 < j.parts; i0 += 8) {
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = in && i0 + i < j.parts ? part(i0 + i)[row] : -INFINITY;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = fmaxf(m, x[i]);
    }
    const float mu = m == -INFINITY ? 0.0f : m;
    float l = 0.0f;
    float4 o[PER];
#pragma unroll
    for (int x = 0; x < PER; ++x) o[x] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int i0 = 0; i0 < j.parts; i0 += kBatch) {
      float f[kBatch], pl[kBatch];
      float4 v[kBatch][PER];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const bool has = in && i0 + b < j.parts;
        const float* p = part(has ? i0 + b : 0);
        const float ref = has ? p[row] : -INFINITY;
        const bool some = ref != -INFINITY;  // (nothing was written where no key was seen)
        f[b] = some ? ref : -INFINITY;
        pl[b] = some ? p[kPromptRows + row] : 0.0f;
#pragma unroll
        for (int x = 0; x < PER; ++x)
          v[b][x] = some ? *reinterpret_cast<const float4*>(p + 2 * kPromptRows + 4 * ((size_t)(warp + W * x) * kPromptRows + row))
                         : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      }
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const float w = exp2_approx(f[b] - mu);
        l = fmaf(w, pl[b], l);
#pragma unroll
        for (int x = 0; x < PER; ++x) {
          o[x].x = fmaf(w, v[b][x].x, o[x].x);
          o[x].y = fmaf(w, v[b][x].y, o[x].y);
          o[x].z = fmaf(w, v[b][x].z, o[x].z);
          o[x].w = fmaf(w, v[b][x].w, o[x].w);
        }
      }
    }
    const float inv = l == 0.0f ? 0.0f : __frcp_rn(l);
#pragma unroll
    for (int x = 0; x < PER; ++x)
      s_out[lane][warp + W * x] = make_uint2(Half16<T>::narrow2(o[x].x * inv, o[x].y * inv), Half16<T>::narrow2(o[x].z * inv, o[x].w * inv));
    auto at = [&](int x) {
      const int y = j.row_lo + row0 + x, tok = y / a.share;
      return (size_t)(j.begin + tok) * a.q_heads + j.head * a.share + (y - tok * a.share);
    };
    if (warp == 0 && in && a.lse[j.rank]) a.lse[j.rank][at(lane)] = l == 0.0f ? -INFINITY : (mu - kShift + log2f(l)) * 0.69314718055994531f;
    __syncthreads();
    for (int e = threadIdx.x; e < kSeenJoinRows * (D / 4); e += kSeenJoinThreads) {
      const int x = e / (D / 4), d4 = e % (D / 4);
      if (j.row_lo + row0 + x < j.row_hi)
        *reinterpret_cast<uint2*>(static_cast<T*>(a.out[j.rank]) + at(x) * D + 4 * d4) = s_out[x][d4];
    }
    __syncthreads();
  }
}

}  // namespace dcc
