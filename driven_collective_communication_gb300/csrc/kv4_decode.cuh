// kv4_decode.cuh -- attention of a few query rows over the 4-bit paged cache
// (single tokens, drafted tokens to verify).
//
// With s_j = c q.K_j (c = scale * log2 e), one pass over the cache keeps, per
// query row, the running maximum m, l = sum 2^(s_j - m) and O = sum 2^(s_j -
// m) V_j.  K_j = lo + step * code per group of G channels, so
//   q.K_j = sum_groups step_jg (q_g . code_jg) + lo_jg (sum q_g),
//   O_d   = sum_j (p_j step_jg) code_jd + sum_j p_j lo_jg.
// The products with the codes run on the tensor cores in fp16 with fp32 sums;
// everything that carries lo is fp32.  The codes are exact.  So is Q: a row is
// scaled by a power of two that brings its largest channel to 2^14, which
// keeps all bits of a bf16 or fp16 channel down to 2^-28 of it.  p * step is
// the one operand that is rounded, to fp16's 11 bits; its scale follows the
// running maximum of s_j and of the steps (R below: l, O and all sums are in
// units of 2^R), so it neither overflows nor falls into the subnormals unless it
// is 2^-28 of the largest seen.  In pages where a mask begins or ends it is two
// bf16 numbers, 16 bits: there a row may see a handful of keys, whose errors do
// not average, beside keys of any size that only other rows see.  Codes enter O
// as n - 8, about the middle of their range, so that what is rounded is about
// half of the group's range at most.
//
// Bound by reading the cache (0.56 bytes a channel at G = 64) if the
// instructions that unpack it stay below the memory's time, above all the
// integer pipe's (half rate).  A nibble in bits 4..7 of a 16-bit lane, with
// the exponent of 64 put around it, is the fp16 number 64 + n: one AND-OR
// makes two codes an operand register, after a shift for three nibbles of
// four (the left one runs on the multiply pipe).  The 64 comes off the scores
// as the accumulators' initial value (-64 sum q), and off O, with the 8, by a
// product of the same rounded p * step with a constant -72 (bf16: 128 + n and -136)
// before each product with codes: nothing is subtracted or converted per code.  (Taken off in the
// end, through one row of ones, it would cost fewer products, but the
// accumulators then carry 72 sum p * step all along, and the tensor core
// truncates its sums: over 131k keys the result lost 3 bits.  Bare nibbles are
// fp16 subnormals and need no exponent, one instruction fewer in seven, but
// the tensor core aligns its sums by nominal exponents: measured, the sums
// lost some 9 bits.)  The fragments take the codes where they lie (kv4.cuh).
// mma.sync with its operands in registers suits this: the tensor work is 8
// rows wide, and tcgen05 would want the unpacked operands written to shared
// or tensor memory first, which costs more than the products.
//
//   S^T[key][row]: A = codes of 16 keys, B = Q^T (8 rows); the accumulator
//   holds keys g, g + 8 and rows 2 t, 2 t + 1 of lane 4 g + t;
//   O^T[channel][row]: A = V codes (16 channels x 16 keys), B = P^T: p * step
//   of the accumulator, packed and transposed 8 x 8 by movmatrix.  Its rows lie
//   in the same lanes, so rescaling needs no exchange.
//
// Work split.  The pages of all (sequence, rank, kv head, row tile) segments
// form one line of units; CTA and warp ranges cut it evenly, so every SM reads
// the same number of bytes whatever the lengths.  A warp streams its pages
// through a ring of its own (one bulk copy per page and head, an mbarrier per
// stage) and never waits for another warp.  Segments cut by a boundary leave
// partial (m, l, O): joined first in the CTA (shared memory, reusing the
// ring), then over the CTAs by whichever comes last, in CTA order, so results
// do not depend on timing.
//
// SEEN: rows that see more than one run of keys (windows with sinks) or a mask's
// drafted tokens.  The line of units then holds the sinks' pages and, behind the
// gap, the window's; in pages that some row does not see in full, each row's 64
// bits take the place of the two comparisons a score.
//
// Measured on GB300, bf16, 8 ranks x 1 kv head x 8 query heads x 128 channels, G
// = 64, one token each: 64 sequences of up to 8192 keys 93 us (326 MB, 3.5 TB/s,
// 52 % of a plain copy's rate); one of 777 keys 13 us.  fp16, 2 kv heads x 4, G =
// 32, one sequence of 131,109 keys: 90 us (336 MB, 3.7 TB/s).  The loads alone
// take 74 and 63 us (65 and 79 % of the copy's rate), loads and scores 82 and 69: of
// the rest about 10 us are the start (plan, page numbers, first pages) and 10 the
// joins and uneven ends, and the loop issues 2.6 of 4 instructions a clock.  Calls
// of few pages a warp are another matter: 16 sequences x 5 drafted tokens in a window
// of 1024 keys, 64 channels, 47 us for 19 MB; the warps have three or four pages each
// and spend 40 % of their cycles waiting for instructions, the unrolled code being
// fetched for the first time.  SEEN: 64 streams of one token, a window of 4000
// keys and 4 sinks of up to 16,384, 8 ranks x 8 query heads, bf16: 91 us (271 MB, 3.0
// TB/s); one stream, window 1024, 64 channels, fp16: 13.7 us.
#pragma once
#include <type_traits>

#include "bulk.cuh"
#include "kv4.cuh"
#include "kv4_plan.h"

namespace dcc {

struct AttnArgs {
  const void* q[DCC_MAX_RANKS];
  void* out[DCC_MAX_RANKS];
  float* lse[DCC_MAX_RANKS];  // all or none
  const int32_t* start;
  char* ws;
  size_t q_stride;
  int tokens, layer, q_heads, share, max_new, window;
  int wide;  // prompt kernel: tiles of 256 rows per segment, before those of 128
  // rows with sets of seen keys of their own (SEEN, below)
  int sinks;             // first tokens that a window does not hide
  int words;             // of a row of mask
  const uint32_t* mask;  // a tree's: drafted token j of the sequence is seen where bit j is set; null: causal rows
  float scale;
  unsigned long long timeout_ns;
};

constexpr int kTreeWords = DCC_TREE_MAX / 32;  // of a row's mask
constexpr int kDecMaxCtas = 160;
constexpr int kDecMaxWarps = 12;
// floats of a partial: m and l per row, then rows of O, padded so that the
// fragments' stores fall into different banks
__host__ __device__ constexpr int dec_slot(int rows, int dim) { return rows * (dim + 6); }
constexpr int kDecMaxSlot = dec_slot(16, 128) > dec_slot(24, 64) ? dec_slot(16, 128) : dec_slot(24, 64);
// workspace: a counter per CTA, two partials per CTA, one per warp
__host__ __device__ constexpr size_t dec_ws_bytes() {
  return 1024 + (size_t)kDecMaxCtas * (2 + kDecMaxWarps) * kDecMaxSlot * 4;
}
static_assert(dec_ws_bytes() == DCC_KV4_ATTENTION_BYTES, "what dcc.h says");

// Warps and stages: as many bytes in flight as shared memory holds, three
// warps to a scheduler where a tile's registers allow (8 rows), two otherwise.
// SMALL: four warps with two stages, two CTAs to an SM, for calls whose pages are
// no more than the warps of one such wave: the next kernel's CTAs then find
// room beside this one's and start under its end (measured on GB300, one
// sequence of 777 keys, 8 ranks, back to back: 13.0 us instead of 13.6).
template <int D, int G, int RT, bool SMALL>
struct DecShape {
  static constexpr int block = kv4_block_bytes(D, G);
  static constexpr int warps = SMALL ? kDecSmallWarps : RT > 1 || 12 * 2 * block > 222 * 1024 ? 8 : 12;
  static constexpr int fit = 222 * 1024 / (warps * block);
  static constexpr int stages = SMALL ? 2 : fit > 4 ? 4 : fit;
  static constexpr size_t smem = (size_t)warps * stages * block + 128;
  static constexpr int ctas = SMALL ? 2 : 1;  // per SM, by registers
};

__device__ __forceinline__ float exp2_approx(float x) {  // 2^x; -inf gives 0
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// D += A B, 16 x 8 x 16, fp32 accumulators
__device__ __forceinline__ void mma_16816(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_16816_from(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1, const float* c) {  // D = C + A B
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}
__device__ __forceinline__ float pow2(int k) { return __int_as_float((k + 127) << 23); }  // -126 <= k <= 127
// the same with bf16 operands
__device__ __forceinline__ void mma_16816_bf16(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                               uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// nibbles P and P + 4 of w as two bf16 numbers 128 + n
template <int P>
__device__ __forceinline__ uint32_t code_pair_bf16(uint32_t w) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w >> (4 * P)), "r"(0x000f000fu), "r"(0x43004300u));
  return r;
}
// nibbles P and P + 4 of w as two fp16 numbers 64 + n
template <int P>
__device__ __forceinline__ uint32_t code_pair(uint32_t w) {
  const uint32_t x = P == 0 ? w * 16u : w >> (4 * (P - (P > 0)));
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(x), "r"(0x00f000f0u), "r"(0x54005400u));  // (x & mask) | 64.0
  return r;
}
// the 8 x 8 matrix of 16-bit elements of which lane 4 r + c holds (r, 2 c) and (r, 2 c + 1), transposed
__device__ __forceinline__ uint32_t transpose8(uint32_t w) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t half2_bits(float a, float b) { return Half16<__half>::narrow2(a, b); }

// ---- SEEN: rows that do not see one run of keys each.  A row sees the keys lo ..
// hi, the sinks up to hi and, of a tree, the drafted tokens of its mask; hi is
// its own position, or in a tree the last one of the context.

// bits 0 .. n - 1 of a word
__device__ __forceinline__ uint32_t bits_below(int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; }
struct SeenRow {
  int hi, lo;      // hi < 0: nothing
  int pos0, news;  // of the sequence: where its drafted tokens begin, and how many there are
  const uint32_t* mask;
};
__device__ __forceinline__ uint32_t seen_mask_word(const SeenRow& r, int words, int i) {
  return i >= 0 && i < words ? r.mask[i] & bits_below(r.news - 32 * i) : 0u;
}
// Of the keys k0 .. k0 + 31, those that the row sees.
__device__ __forceinline__ uint32_t seen_word(const SeenRow& r, const AttnArgs& a, int k0) {
  uint32_t w = bits_below(r.hi + 1 - k0) & (~bits_below(r.lo - k0) | bits_below(a.sinks - k0));
  const int d = k0 - r.pos0;
  if (r.mask && d > -32 && d < r.news)
    w |= __funnelshift_r(seen_mask_word(r, a.words, d >> 5), seen_mask_word(r, a.words, (d >> 5) + 1), (uint32_t)d & 31u);
  return w;
}
// Row of new token `tok` of a sequence: token `at` of the batch.
__device__ __forceinline__ SeenRow seen_row(const AttnArgs& a, int pos0, int news, int tok, int at) {
  SeenRow r = {pos0 + tok, 0, pos0, news, nullptr};
  int own = tok + 1;  // new tokens that it sees: the window is over these and the context
  if (a.mask) {
    r.mask = a.mask + (size_t)at * a.words;
    r.hi = pos0 - 1;
    if (a.window > 0) {
      own = 0;
      for (int i = 0; i < a.words && 32 * i < news; ++i) own += __popc(seen_mask_word(r, a.words, i));
    }
  }
  if (a.window > 0) r.lo = pos0 + own - a.window;
  return r;
}

// One sequence's part of the line of units.
struct DecSeq {
  int begin, rows, pos0, page0, pages, tiles;  // rows: new tokens * share; tiles * pages units per (rank, head)
  bool empty;
  // SEEN: the first `kept` of the pages hold the sinks and are pages 0 .. of the
  // row, the others go on at page0 + kept; and the new tokens
  int kept, news;
};
// The next sequence after s that has rows, or kv.seqs; a whole warp looks.
__device__ __forceinline__ int next_with_rows(const Kv4Dev& kv, const AttnArgs& a, int s) {
  const int lane = threadIdx.x & 31;
  for (int s0 = s + 1; s0 < kv.seqs; s0 += 32) {
    const int x = s0 + lane;
    const unsigned some = __ballot_sync(0xffffffffu, x < kv.seqs && min(a.tokens, a.start[x + 1]) > max(0, a.start[x]));
    if (some) return s0 + __ffs(some) - 1;
  }
  return kv.seqs;
}
// the table's slot of a sequence's page, both counted from page0
__device__ __forceinline__ int dec_slot_of(const DecSeq& q, int slot) { return slot - q.page0 < q.kept ? slot - q.page0 : slot; }
template <bool SEEN>
__device__ __forceinline__ DecSeq dec_seq(const Kv4Dev& kv, const AttnArgs& a, int s, int tile_rows) {
  DecSeq q;
  q.kept = q.news = 0;
  const int b = max(0, a.start[s]), e = min(a.tokens, a.start[s + 1]), len = kv.len[s];
  const int news = max(0, e - b);
  q.begin = b;
  q.pos0 = len - news;
  q.rows = min(news, a.max_new) * a.share;
  q.tiles = (q.rows + tile_rows - 1) / tile_rows;
  // (a row of a tree may see none of the drafted tokens)
  const int first = a.window > 0 ? max(0, q.pos0 - a.window + (SEEN && a.mask ? 0 : 1)) : 0;
  q.page0 = first / kKv4Page;
  if (SEEN) {
    q.news = news;
    q.kept = min((min(a.sinks, len) + kKv4Page - 1) / kKv4Page, q.page0);
    if (q.kept == q.page0) q.kept = 0, q.page0 = 0;  // no gap
    q.page0 -= q.kept;
  }
  // one page past the row at most: it is reported there
  q.pages = len > 0 ? min((len - 1) / kKv4Page, kv.max_pages) - q.page0 + 1 : 0;
  q.empty = q.pages <= 0;
  if (q.empty) {
    q.pages = 1;
    q.page0 = q.kept = 0;
  }
  if (q.rows == 0) q.pages = q.tiles = 0;
  return q;
}

struct DecCursor {
  int s, seg;  // sequence, segment of it: (rank, head), tile
  DecSeq q;
};

// Join `n` partials (by `at`) of one segment and store the result: to `part`
// (a partial again) or to the outputs.  One thread's share: four channels of a
// row (e).  Eight partials' loads are in flight at a time: they come from
// other SMs.
template <typename T, int D, int ROWS, typename At>
__device__ __forceinline__ void dec_join(const AttnArgs& a, int e, int n, At at, float* part, int rank, int head,
                                         int row0, int rows, int begin) {
  constexpr int kBatch = 8;
  {
    const int row = e / (D / 4), d4 = e % (D / 4);
    float m = -INFINITY, l = 0.0f;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int i0 = 0; i0 < n; i0 += kBatch) {
      float pm[kBatch], pl[kBatch];
      float4 v[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const float* p = at(min(i0 + i, n - 1));
        pm[i] = i0 + i < n ? p[row] : -INFINITY;
        pl[i] = i0 + i < n ? p[ROWS + row] : 0.0f;
        v[i] = i0 + i < n ? *reinterpret_cast<const float4*>(p + 2 * ROWS + row * (D + 4) + d4 * 4)
                          : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      }
      float mn = m;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) mn = fmaxf(mn, pm[i]);
      const float mu = mn == -INFINITY ? 0.0f : mn, fix = exp2_approx(m - mu);
      l *= fix;
      o.x *= fix;
      o.y *= fix;
      o.z *= fix;
      o.w *= fix;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const float w = exp2_approx(pm[i] - mu);
        l = fmaf(w, pl[i], l);
        o.x = fmaf(w, v[i].x, o.x);
        o.y = fmaf(w, v[i].y, o.y);
        o.z = fmaf(w, v[i].z, o.z);
        o.w = fmaf(w, v[i].w, o.w);
      }
      m = mn;
    }
    if (part) {
      if (d4 == 0) {
        part[row] = m;
        part[ROWS + row] = l;
      }
      *reinterpret_cast<float4*>(part + 2 * ROWS + row * (D + 4) + d4 * 4) = o;
    } else if (row0 + row < rows) {
      const int t = (row0 + row) / a.share, h = head * a.share + (row0 + row) % a.share;
      const size_t at_row = (size_t)(begin + t) * a.q_heads + h;
      const float inv = l == 0.0f ? 0.0f : __frcp_rn(l);
      uint2 w;
      w.x = Half16<T>::narrow2(o.x * inv, o.y * inv);
      w.y = Half16<T>::narrow2(o.z * inv, o.w * inv);
      *reinterpret_cast<uint2*>(static_cast<T*>(a.out[rank]) + at_row * D + d4 * 4) = w;
      if (d4 == 0 && a.lse[rank])
        a.lse[rank][at_row] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
    }
  }
}

template <typename T, int D, int G, int RT, bool SMALL, bool SEEN>
__global__ void __launch_bounds__(DecShape<D, G, RT, SMALL>::warps * 32, DecShape<D, G, RT, SMALL>::ctas)
    k_kv4_decode(Kv4Dev kv, AttnArgs a) {
  using Shape = DecShape<D, G, RT, SMALL>;
  constexpr int W = Shape::warps, S = Shape::stages, BLK = Shape::block, THREADS = W * 32;
  constexpr int NG = D / G, ROWS = 8 * RT, JW = D / 32, MT = D / 16, SLOT = dec_slot(ROWS, D);
  constexpr float kCenter = 8.0f;
  constexpr uint32_t kBias = 0xd480d480u;      // fp16 -72 = -(64 + kCenter), twice
  constexpr uint32_t kBiasWide = 0xc308c308u;  // bf16 -136 = -(128 + kCenter)
  constexpr int kMinExp = -60;  // steps below 2^-60 count as that: 2^(14 + 60) a key still sums in fp32
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  constexpr uint32_t kFloor = 80u << 7;
  extern __shared__ __align__(128) char dec_smem[];
  __shared__ __align__(8) uint64_t bars[W][S];
  __shared__ long long s_sum[W];
  __shared__ DecCursor s_cur[W][2];  // each warp's two cursors; where its range begins at first
  __shared__ int s_page[W];          // and the page of the segment there
  // what each warp leaves: a segment that began before its range and ended in
  // it (head), one still open at its end (tail); by first and last unit
  __shared__ long long s_seg[2 * W][2];
  __shared__ int s_who[2 * W][5];  // rank, head, first row; rows and first token of the sequence
  __shared__ int s_list[2 * W], s_group[2 * W + 1], s_groups;
  __shared__ int s_open[2];        // CTAs that hold parts of the two segments open at the CTA's ends
  __shared__ int s_last[2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  char* ring = dec_smem + (size_t)warp * S * BLK;
  if (lane < S) mbar_init(&bars[warp][lane], 1);
  if (lane < 2) s_seg[2 * warp + lane][0] = -1;
  fence_mbar_init();
  pdl_prologue();

  // ---- the line of units, and this warp's range of it.  Up to one sequence a
  // thread, the sequences are looked at once.
  const int nh = kv.n * kv.heads;
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
#pragma unroll
    for (int w = 0; w < W; ++w) {
      if (w < warp) first += s_sum[w];
      *total += s_sum[w];
    }
    return first;
  };
  DecSeq sq0 = {};
  long long units = 0, first0 = 0;
  for (int s0 = 0; s0 < kv.seqs; s0 += THREADS) {
    const int s = s0 + (int)threadIdx.x;
    DecSeq q = {};
    if (s < kv.seqs) q = dec_seq<SEEN>(kv, a, s, ROWS);
    long long total;
    const long long first = scan((long long)q.pages * q.tiles, &total);
    if (s0 == 0) {
      sq0 = q;
      first0 = first;
    }
    units += total;
  }
  units *= nh;
  // no more CTAs than units, so that no range between two others is empty
  const int C = units < (long long)gridDim.x ? (int)units : (int)gridDim.x, cta = (int)blockIdx.x;
  if (cta >= C) return;
  const long long c0 = units * cta / C, c1 = units * (cta + 1) / C;
  auto warp_begin = [&](int w) { return c0 + (c1 - c0) * w / W; };
  long long before = 0;
  for (int s0 = 0; s0 < kv.seqs && before * nh <= c1; s0 += THREADS) {
    const int s = s0 + (int)threadIdx.x;
    DecSeq q = sq0;
    long long first = first0;
    if (s0 > 0 || kv.seqs > THREADS) {
      q = DecSeq{};
      if (s < kv.seqs) q = dec_seq<SEEN>(kv, a, s, ROWS);
      long long total;
      first = before + scan((long long)q.pages * q.tiles, &total);
      before += total;
    }
    const long long mine = (long long)q.pages * q.tiles, base = first * nh;
    if (mine && base < c1 && base + mine * nh > c0)
      for (int w = 0; w < W; ++w) {
        const long long u = warp_begin(w);
        if (base <= u && u < base + mine * nh) {
          const int seg = (int)((u - base) / q.pages);
          s_cur[w][0] = s_cur[w][1] = DecCursor{s, seg, q};
          s_page[w] = (int)(u - base - (long long)seg * q.pages);
        }
      }
  }
  __syncthreads();
  const long long u0 = warp_begin(warp), u1 = warp_begin(warp + 1);
  const int count = (int)(u1 - u0);

  // ---- a walk along the units: the loads' cursor runs ahead of the sums'.
  // What changes with the segment only lies in shared memory.
  auto put = [&](DecCursor& c, int s, int seg, const DecSeq& q) {
    __syncwarp();
    if (lane == 0) {
      c.s = s;
      c.seg = seg;
      c.q = q;
    }
    __syncwarp();
  };
  auto next_segment = [&](DecCursor& c) {
    int s = c.s, seg = c.seg + 1;
    DecSeq q = c.q;
    if (seg >= nh * q.tiles) {
      seg = 0;
      if constexpr (SEEN) {
        s = next_with_rows(kv, a, s);
        if (s < kv.seqs) q = dec_seq<SEEN>(kv, a, s, ROWS);
      } else {
        do {
          ++s;
          if (s < kv.seqs) q = dec_seq<SEEN>(kv, a, s, ROWS);
        } while (s < kv.seqs && q.pages == 0);
      }
    }
    put(c, s, seg, q);
  };
  DecCursor& ldc = s_cur[warp][0];
  DecCursor& cuc = s_cur[warp][1];
  int ld_slot = 0, ld_end = 0;     // pages of the sequence's row left to load
  const char* ld_base = nullptr;   // the segment's block of page 0; null: nothing is there to load
  int ids = -1, ids_at = -1;       // 32 page numbers of that row, from this one on
  const size_t page_stride = (size_t)kv.heads * BLK;
  auto ld_open = [&]() {
    const DecSeq q = ldc.q;
    const int rh = ldc.seg / q.tiles, rank = rh / kv.heads;
    ld_slot = q.page0;
    ld_end = q.page0 + q.pages;
    ld_base = q.empty ? nullptr : kv4_block(kv, rank, a.layer, 0, rh - rank * kv.heads, BLK);
  };
  uint32_t missing = 0;  // stages that hold no page
  auto page_at = [&](int slot) { return kv4_page(kv, ldc.s, SEEN ? dec_slot_of(ldc.q, slot) : slot); };
  auto issue = [&](int st) {
    if (ld_slot == ld_end) {
      const int s = ldc.s;
      next_segment(ldc);
      if (ldc.s != s) ids_at = -1;
      ld_open();
    }
    int page = -1;
    if (ld_base) {
      if (ids_at < 0 || ld_slot - ids_at >= 32) {
        ids_at = ld_slot;
        ids = ids_at + lane < ld_end ? page_at(ids_at + lane) : -1;
      }
      if (ld_slot < ids_at) {  // the next segment of the same sequence starts over
        ids_at = ld_slot;
        ids = ids_at + lane < ld_end ? page_at(ids_at + lane) : -1;
      }
      page = __shfl_sync(0xffffffffu, ids, ld_slot - ids_at);
    }
    ++ld_slot;
    if (page < 0) missing |= 1u << st;
    else missing &= ~(1u << st);
    if (lane == 0) {
      mbar_arrive_expect_tx(&bars[warp][st], page < 0 ? 0u : (uint32_t)BLK);
      if (page >= 0) bulk_load(ring + (size_t)st * BLK, ld_base + page * page_stride, BLK, &bars[warp][st]);
    }
  };
  auto wait = [&](int st, uint32_t parity) {
    if (mbar_try_wait(&bars[warp][st], parity)) return true;
    const unsigned long long t0 = global_timer_ns();
    for (unsigned it = 1;; ++it) {
      if (mbar_try_wait(&bars[warp][st], parity)) return true;
      if ((it & 15u) == 0 && global_timer_ns() - t0 > a.timeout_ns) {
        atomicCAS(kv.status + 1, 0ull, pack_status(kStatusTimeout, 0, 0, cta));
        return false;
      }
    }
  };

  // ---- sums of the open segment, for rows 8 x + 2 t + b.  All are in units of
  // 2^R, R = mx * cs + ex - 14 (mx: the largest raw score, before the factor cs)
  uint32_t qf[2 * JW][2 * RT];  // Q^T fragments of each 16-channel step
  float q64[RT][NG][4];         // the scores' accumulators at their start
  float qsum[RT][NG][2], mx[RT][2], l[RT][2], pmid[RT][NG][2], cs[RT][2];
  float o[RT][MT][4];
  int ex = kMinExp, lim_hi[RT][2], lim_lo[RT][2], tile_hi = 0, tile_lo = 0, tile_end = 0;
  int row_at[RT][2];  // SEEN: the rows' tokens of the batch
  auto open = [&]() {
    const DecSeq sq = cuc.q;
    const int rh = cuc.seg / sq.tiles, tile = cuc.seg - rh * sq.tiles, rank = rh / kv.heads, head = rh - rank * kv.heads;
    ex = kMinExp;
#pragma unroll
    for (int x = 0; x < RT; ++x) {
      const int row = tile * ROWS + 8 * x + g, tok = row / a.share;
      const bool in = row < sq.rows;
      const T* q = static_cast<const T*>(a.q[rank]) + (size_t)(sq.begin + tok) * a.q_stride +
                   (size_t)(head * a.share + row - tok * a.share) * D;
      int hi = in ? sq.pos0 + tok : -1, lo = a.window > 0 ? sq.pos0 + tok - a.window + 1 : 0;
      if (SEEN && a.mask) {
        const SeenRow r = seen_row(a, sq.pos0, in ? sq.news : 0, tok, sq.begin + tok);
        hi = in ? r.hi : -1;
        lo = in ? r.lo : -(1 << 30);  // (not among the tile's largest)
      }
      uint4 v[JW];
      float big = 0.0f;
#pragma unroll
      for (int j = 0; j < JW; ++j) {
        v[j] = in ? *reinterpret_cast<const uint4*>(q + 32 * j + 8 * t) : make_uint4(0, 0, 0, 0);
        const uint32_t u[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 f = Half16<T>::widen2(u[e]);
          big = fmaxf(big, fmaxf(fabsf(f.x), fabsf(f.y)));
        }
      }
      big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
      big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
      // the row times 2^k has its largest channel in [2^14, 2^15); it takes the
      // scale's sign, so that a larger raw score is a larger score
      const int eb = (__float_as_int(big) >> 23) - 127;
      const int k = big == 0.0f || eb > 127 ? 0 : min(14 - eb, 110);
      const float up = a.scale < 0.0f ? -pow2(k) : pow2(k);
      const float c = fabsf(a.scale) * 1.44269504088896341f * pow2(-k);
      float qs[NG] = {};
#pragma unroll
      for (int j = 0; j < JW; ++j) {
        const uint32_t u[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
        float f[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 w = Half16<T>::widen2(u[e]);
          f[2 * e] = w.x * up;
          f[2 * e + 1] = w.y * up;
        }
        // channels (e, e + 4) share a register, as two nibbles of a word do
        qf[2 * j][2 * x] = half2_bits(f[0], f[4]);
        qf[2 * j][2 * x + 1] = half2_bits(f[1], f[5]);
        qf[2 * j + 1][2 * x] = half2_bits(f[2], f[6]);
        qf[2 * j + 1][2 * x + 1] = half2_bits(f[3], f[7]);
        qs[32 * j / G] += ((f[0] + f[1]) + (f[2] + f[3])) + ((f[4] + f[5]) + (f[6] + f[7]));
      }
#pragma unroll
      for (int gr = 0; gr < NG; ++gr) {
        qs[gr] += __shfl_xor_sync(0xffffffffu, qs[gr], 1);
        qs[gr] += __shfl_xor_sync(0xffffffffu, qs[gr], 2);
      }
#pragma unroll
      for (int b = 0; b < 2; ++b) {  // of the rows that the accumulators hold here
        const int src = 8 * t + 4 * b;
        cs[x][b] = __shfl_sync(0xffffffffu, c, src);
        lim_hi[x][b] = __shfl_sync(0xffffffffu, hi, src);
        lim_lo[x][b] = __shfl_sync(0xffffffffu, lo, src);
        if (SEEN) row_at[x][b] = __shfl_sync(0xffffffffu, in ? sq.begin + tok : -1, src);
#pragma unroll
        for (int gr = 0; gr < NG; ++gr) {
          qsum[x][gr][b] = __shfl_sync(0xffffffffu, qs[gr], src);
          q64[x][gr][b] = q64[x][gr][2 + b] = -64.0f * qsum[x][gr][b];
          pmid[x][gr][b] = 0.0f;
        }
        mx[x][b] = -INFINITY;
        l[x][b] = 0.0f;
      }
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[x][i][e] = 0.0f;
    }
    // keys from tile_lo to tile_hi are seen by every row of the tile, none past tile_end by any
    const int last = min(tile * ROWS + ROWS, sq.rows) - 1;
    tile_hi = sq.pos0 + tile * ROWS / a.share;
    tile_end = sq.pos0 + last / a.share;
    tile_lo = a.window > 0 ? tile_end - a.window + 1 : 0;
    if (SEEN && a.mask) {
      tile_hi = sq.pos0 - 1;
      tile_end = sq.pos0 + sq.news - 1;
      if (a.window > 0) {
        tile_lo = lim_lo[0][0];
#pragma unroll
        for (int x = 0; x < RT; ++x) tile_lo = max(tile_lo, max(lim_lo[x][0], lim_lo[x][1]));
        tile_lo = __reduce_max_sync(0xffffffffu, tile_lo);
      }
    }
  };

  // One page.  MASKED: some row does not see some key of it.
  // kg: the key of accumulator row g (of 8); ka, kb: those of rows 2 t, 2 t +
  // 1.  The order is the one in which a quad's V rows lie in different banks.
  const int sw = D == 128 ? (t & 1) : (t >> 1);
  const int ka = 2 * t + sw, kb = 2 * t + 1 - sw;
  const int kg = D == 128 ? g ^ ((g >> 1) & 1) : g ^ (g >> 2);
  auto page_pass = [&](auto masked, const char* blk, int key0) {
    constexpr bool MASKED = decltype(masked)::value;
    const uint32_t* par = reinterpret_cast<const uint32_t*>(blk + 2 * kv4_codes_bytes(D)) + kg * NG;
    const uint32_t* vpar = par + kKv4Page * NG;
    float sc[4][RT][4];
    uint32_t vis[RT][2][2];  // SEEN: the page's keys that the rows see
    if constexpr (MASKED && SEEN) {
#pragma unroll
      for (int x = 0; x < RT; ++x)
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const bool tree = a.mask && row_at[x][b] >= 0;
          const SeenRow r = {lim_hi[x][b], lim_lo[x][b], cuc.q.pos0, cuc.q.news,
                             tree ? a.mask + (size_t)row_at[x][b] * a.words : nullptr};
#pragma unroll
          for (int i = 0; i < 2; ++i) vis[x][b][i] = seen_word(r, a, key0 + 32 * i) >> kg;
        }
    }
#pragma unroll
    for (int n = 0; n < 4; ++n) {  // 16 keys each
      uint32_t w[2][JW];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const char* row = blk + (16 * n + 8 * h + kg) * (D / 2) + t * (JW * 4);
        if constexpr (JW == 4) {
          const uint4 v = *reinterpret_cast<const uint4*>(row);
          w[h][0] = v.x, w[h][1] = v.y, w[h][2] = v.z, w[h][3] = v.w;
        } else {
          const uint2 v = *reinterpret_cast<const uint2*>(row);
          w[h][0] = v.x, w[h][1] = v.y;
        }
      }
      float acc[RT][NG][4];
#pragma unroll
      for (int j = 0; j < JW; ++j) {
        const uint32_t a0[4] = {code_pair<0>(w[0][j]), code_pair<0>(w[1][j]), code_pair<1>(w[0][j]), code_pair<1>(w[1][j])};
        const uint32_t a1[4] = {code_pair<2>(w[0][j]), code_pair<2>(w[1][j]), code_pair<3>(w[0][j]), code_pair<3>(w[1][j])};
#pragma unroll
        for (int x = 0; x < RT; ++x) {
          const int gr = 32 * j / G;
          if (32 * j % G == 0)
            mma_16816_from(acc[x][gr], a0[0], a0[1], a0[2], a0[3], qf[2 * j][2 * x], qf[2 * j][2 * x + 1], q64[x][gr]);
          else
            mma_16816(acc[x][gr], a0[0], a0[1], a0[2], a0[3], qf[2 * j][2 * x], qf[2 * j][2 * x + 1]);
          mma_16816(acc[x][gr], a1[0], a1[1], a1[2], a1[3], qf[2 * j + 1][2 * x], qf[2 * j + 1][2 * x + 1]);
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float2 sl[NG];  // step, lo
#pragma unroll
        for (int gr = 0; gr < NG; ++gr) sl[gr] = Half16<T>::widen2(par[(16 * n + 8 * h) * NG + gr]);
#pragma unroll
        for (int x = 0; x < RT; ++x)
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            float s = sl[0].y * qsum[x][0][b];
#pragma unroll
            for (int gr = 1; gr < NG; ++gr) s = fmaf(sl[gr].y, qsum[x][gr][b], s);
#pragma unroll
            for (int gr = 0; gr < NG; ++gr) s = fmaf(sl[gr].x, acc[x][gr][2 * h + b], s);
            if (MASKED && SEEN) {
              if (!((vis[x][b][n >> 1] >> (16 * (n & 1) + 8 * h)) & 1u)) s = -INFINITY;
            } else if (MASKED) {
              const int pos = key0 + 16 * n + 8 * h + kg;
              if (pos > lim_hi[x][b] || pos < lim_lo[x][b]) s = -INFINITY;
            }
            sc[n][x][2 * h + b] = s;
          }
      }
    }
    // The largest step of V (its exponent) and the running maximum; what was summed
    // so far is rescaled where they grew.  In masked pages, where p * step has
    // bf16's range, the smallest that a key has at most: keys that only some rows
    // see may be any size, and their scale is not the others'.
    uint32_t top = 0, low = 0x7fffu;  // by halves: step, lo
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int key = 2 * lane + h;
      uint32_t one = MASKED ? 0u : top;
#pragma unroll
      for (int gr = 0; gr < NG; ++gr) {
        uint32_t w = (vpar - kg * NG)[key * NG + gr] & (kBf16 ? 0x7fff7fffu : 0x7fffu);
        const bool finite = kBf16 ? ((w + 0x00800080u) & 0x80008000u) == 0u : w < 0x7c00u;
        if (!finite || (MASKED && key0 + key > tile_end)) w = 0;
        one = kBf16 ? __vmaxu2(one, w) : max(one, w);
      }
      if (MASKED && (one & 0x7fffu)) low = min(low, one & 0x7fffu);
      if (MASKED) one = kBf16 ? __vmaxu2(top, one) : 0u;
      top = one;
    }
    // A bf16 lo far above all steps (constant groups), and such a step in a masked
    // page, count as 2^-80 of themselves: p times either stays below 2^95, and
    // 2^25 of them still sum in fp32.
    if (kBf16) {
      const uint32_t far = max(max(MASKED ? top & 0xffffu : 0u, top >> 16), kFloor) - kFloor;
      top = MASKED ? far : max(top & 0xffffu, far);
    }
    top = __reduce_max_sync(0xffffffffu, top);
    if (MASKED) {
      low = __reduce_min_sync(0xffffffffu, low);
      if (low < 0x7fffu) top = max(top, low);
    }
    const int ex_new = max(ex, (__float_as_int(Half16<T>::widen((uint16_t)top)) >> 23) - 127);
    bool grew = ex_new > ex;
    float alpha[RT][2], ref[RT][2];
#pragma unroll
    for (int x = 0; x < RT; ++x)
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        float m = mx[x][b];
#pragma unroll
        for (int n = 0; n < 4; ++n) m = fmaxf(m, fmaxf(sc[n][x][b], sc[n][x][2 + b]));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
        grew |= m > mx[x][b];
        // nothing seen so far: the sums are zero (or NaN) and stay so
        alpha[x][b] = mx[x][b] == -INFINITY ? 1.0f : exp2_approx(fmaf(mx[x][b] - m, cs[x][b], (float)(ex - ex_new)));
        mx[x][b] = m;
        ref[x][b] = m == -INFINITY ? 0.0f : m;
      }
    ex = ex_new;
    const float shift = (float)(14 - ex);
    if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
      for (int x = 0; x < RT; ++x)
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          l[x][b] *= alpha[x][b];
#pragma unroll
          for (int gr = 0; gr < NG; ++gr) {
            pmid[x][gr][b] *= alpha[x][b];
          }
#pragma unroll
          for (int i = 0; i < MT; ++i) {
            o[x][i][b] *= alpha[x][b];
            o[x][i][2 + b] *= alpha[x][b];
          }
        }
    }
#pragma unroll
    for (int n = 0; n < 4; ++n) {  // 16 keys each
      // P^T fragments: p * step, and in masked pages what its rounding left
      uint32_t bp[RT][NG][2], bq[RT][NG][2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float2 sv[NG];  // step, centre
#pragma unroll
        for (int gr = 0; gr < NG; ++gr) {
          sv[gr] = Half16<T>::widen2(vpar[(16 * n + 8 * h) * NG + gr]);
          sv[gr].y = fmaf(kCenter, sv[gr].x, sv[gr].y);
        }
#pragma unroll
        for (int x = 0; x < RT; ++x) {
          float p[2];
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            const float s = sc[n][x][2 * h + b];
            p[b] = exp2_approx(fmaf(s - ref[x][b], cs[x][b], shift));
            if (MASKED && s == -INFINITY) p[b] = 0.0f;
            l[x][b] += p[b];
          }
#pragma unroll
          for (int gr = 0; gr < NG; ++gr) {
            float q[2];
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              float c = sv[gr].y;
              q[b] = p[b] * sv[gr].x;
              if (MASKED && p[b] == 0.0f) q[b] = c = 0.0f;  // tokens that are not there may hold anything
              pmid[x][gr][b] = fmaf(p[b], c, pmid[x][gr][b]);
            }
            using Wide = Half16<__nv_bfloat16>;
            const uint32_t w = MASKED ? Wide::narrow2(q[0], q[1]) : half2_bits(q[0], q[1]);
            bp[x][gr][h] = transpose8(w);
            if (MASKED) {
              const float2 f = Wide::widen2(w);
              bq[x][gr][h] = transpose8(Wide::narrow2(q[0] - f.x, q[1] - f.y));
            }
          }
        }
      }
      // V codes of the lane's chunk of 4 tokens: words of (first, second) key
      uint32_t v[2][2][JW / 2];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const int tok = 16 * n + 8 * h + (b ? kb : ka);
          const char* row = blk + kv4_codes_bytes(D) + tok * (D / 2) + kv4_v_chunk(D, g, tok) * (D / 16);
          if constexpr (JW == 4) {
            const uint2 w = *reinterpret_cast<const uint2*>(row);
            v[h][b][0] = w.x, v[h][b][1] = w.y;
          } else {
            v[h][b][0] = *reinterpret_cast<const uint32_t*>(row);
          }
        }
#pragma unroll
      for (int q4 = 0; q4 < MT / 2; ++q4) {  // two 16-channel tiles from each half word
        const int w = q4 >> 1;
        const uint32_t x0 = __byte_perm(v[0][0][w], v[0][1][w], (q4 & 1) ? 0x7632 : 0x5410);
        const uint32_t x1 = __byte_perm(v[1][0][w], v[1][1][w], (q4 & 1) ? 0x7632 : 0x5410);
        if constexpr (MASKED) {
          const uint32_t f0[4] = {code_pair_bf16<0>(x0), code_pair_bf16<1>(x0), code_pair_bf16<0>(x1), code_pair_bf16<1>(x1)};
          const uint32_t f1[4] = {code_pair_bf16<2>(x0), code_pair_bf16<3>(x0), code_pair_bf16<2>(x1), code_pair_bf16<3>(x1)};
#pragma unroll
          for (int x = 0; x < RT; ++x) {
            auto both = [&](const uint32_t* b) {
              mma_16816_bf16(o[x][2 * q4], kBiasWide, kBiasWide, kBiasWide, kBiasWide, b[0], b[1]);
              mma_16816_bf16(o[x][2 * q4 + 1], kBiasWide, kBiasWide, kBiasWide, kBiasWide, b[0], b[1]);
              mma_16816_bf16(o[x][2 * q4], f0[0], f0[1], f0[2], f0[3], b[0], b[1]);
              mma_16816_bf16(o[x][2 * q4 + 1], f1[0], f1[1], f1[2], f1[3], b[0], b[1]);
            };
            both(bp[x][32 * q4 / G]);
            both(bq[x][32 * q4 / G]);
          }
        } else {
          const uint32_t f0[4] = {code_pair<0>(x0), code_pair<1>(x0), code_pair<0>(x1), code_pair<1>(x1)};
          const uint32_t f1[4] = {code_pair<2>(x0), code_pair<3>(x0), code_pair<2>(x1), code_pair<3>(x1)};
#pragma unroll
          for (int x = 0; x < RT; ++x) {
            const uint32_t* b = bp[x][32 * q4 / G];
            mma_16816(o[x][2 * q4], kBias, kBias, kBias, kBias, b[0], b[1]);
            mma_16816(o[x][2 * q4 + 1], kBias, kBias, kBias, kBias, b[0], b[1]);
            mma_16816(o[x][2 * q4], f0[0], f0[1], f0[2], f0[3], b[0], b[1]);
            mma_16816(o[x][2 * q4 + 1], f1[0], f1[1], f1[2], f1[3], b[0], b[1]);
          }
        }
      }
    }
  };

  // The final value of each accumulator: with the fp32 part.  Leaves l summed over the keys' lanes, and mx as R.
  auto settle = [&]() {
#pragma unroll
    for (int x = 0; x < RT; ++x)
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        if (mx[x][b] != -INFINITY) mx[x][b] = fmaf(mx[x][b], cs[x][b], (float)(ex - 14));
#pragma unroll
        for (int m = 4; m < 32; m <<= 1) l[x][b] += __shfl_xor_sync(0xffffffffu, l[x][b], m);
#pragma unroll
        for (int gr = 0; gr < NG; ++gr) {
          float pm = pmid[x][gr][b];
#pragma unroll
          for (int m = 4; m < 32; m <<= 1) pm += __shfl_xor_sync(0xffffffffu, pm, m);
#pragma unroll
          for (int i = gr * G / 16; i < (gr + 1) * G / 16; ++i) {
            o[x][i][b] += pm;
            o[x][i][2 + b] += pm;
          }
        }
      }
  };
  auto store_partial = [&](float* p) {
#pragma unroll
    for (int x = 0; x < RT; ++x)
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int row = 8 * x + 2 * t + b;
        if (g == 0) {
          p[row] = mx[x][b];
          p[ROWS + row] = l[x][b];
        }
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          p[2 * ROWS + row * (D + 4) + 16 * i + g] = o[x][i][b];
          p[2 * ROWS + row * (D + 4) + 16 * i + g + 8] = o[x][i][2 + b];
        }
      }
  };
  auto store_out = [&]() {
    const DecSeq sq = cuc.q;
    const int rh = cuc.seg / sq.tiles, tile = cuc.seg - rh * sq.tiles, rank = rh / kv.heads, head = rh - rank * kv.heads;
#pragma unroll
    for (int x = 0; x < RT; ++x)
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int row = tile * ROWS + 8 * x + 2 * t + b;
        if (row >= sq.rows) continue;
        const float inv = l[x][b] == 0.0f ? 0.0f : __frcp_rn(l[x][b]);
        const size_t at = (size_t)(sq.begin + row / a.share) * a.q_heads + head * a.share + row % a.share;
        uint16_t* dst = static_cast<uint16_t*>(a.out[rank]) + at * D + g;
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          dst[16 * i] = Half16<T>::narrow(o[x][i][b] * inv);
          dst[16 * i + 8] = Half16<T>::narrow(o[x][i][2 + b] * inv);
        }
        if (g == 0 && a.lse[rank])
          a.lse[rank][at] = l[x][b] == 0.0f ? -INFINITY : (mx[x][b] + log2f(l[x][b])) * 0.69314718055994531f;
      }
  };

  float* part_ws = reinterpret_cast<float*>(a.ws + 1024);
  float* head_ws = part_ws + (size_t)kDecMaxCtas * 2 * SLOT + ((size_t)cta * W + warp) * SLOT;

  if (count > 0) {
    long long seg_begin;  // first unit of the open segment
    int left;             // its units still to come
    int key0;             // first key of its next page
    int slot = 0;         // SEEN: that page, counted from the sequence's page0
    auto slot_key = [&]() { return dec_slot_of(cuc.q, slot) * kKv4Page; };
    {
      const int j = s_page[warp];
      const DecSeq q = ldc.q;
      ld_open();
      ld_slot += j;
      seg_begin = u0 - j;
      left = q.pages - j;
      key0 = (q.page0 + j) * kKv4Page;
      if (SEEN) {
        slot = q.page0 + j;
        key0 = slot_key();
      }
    }
    int issued = 0;
    for (; issued < S && issued < count; ++issued) issue(issued);
    bool fresh = true, alive = true;
    int st = 0, i = 0;
    uint32_t parity = 0;
    for (; i < count; ++i) {
      if (fresh) {
        open();
        fresh = false;
      }
      if (!wait(st, parity)) {
        alive = false;
        break;
      }
      if (!((missing >> st) & 1u)) {
        const char* blk = ring + (size_t)st * BLK;
        if (key0 + kKv4Page - 1 > tile_hi || (key0 < tile_lo && !(SEEN && key0 + kKv4Page <= a.sinks)))
          page_pass(std::true_type{}, blk, key0);
        else page_pass(std::false_type{}, blk, key0);
      }
      __syncwarp();  // every lane has read the stage
      if (issued < count) {
        issue(st);
        ++issued;
      }
      key0 += kKv4Page;
      if (SEEN) {
        ++slot;
        key0 = slot_key();
      }
      const bool ends = --left == 0;
      if (ends || i + 1 == count) {  // the segment, or the range, ends
        settle();
        const DecSeq sq = cuc.q;
        if (seg_begin >= u0 && ends) {
          store_out();
        } else {
          const int which = 2 * warp + (ends ? 0 : 1);
          if (ends) store_partial(head_ws);
          if (lane == 0) {
            s_seg[which][0] = seg_begin;
            s_seg[which][1] = seg_begin + sq.pages;
            const int rh = cuc.seg / sq.tiles;
            s_who[which][0] = rh / kv.heads;
            s_who[which][1] = rh % kv.heads;
            s_who[which][2] = (cuc.seg - rh * sq.tiles) * ROWS;
            s_who[which][3] = sq.rows;
            s_who[which][4] = sq.begin;
          }
        }
        if (ends && i + 1 < count) {
          seg_begin += sq.pages;
          next_segment(cuc);
          left = cuc.q.pages;
          key0 = cuc.q.page0 * kKv4Page;
          if (SEEN) {
            slot = cuc.q.page0;
            key0 = slot_key();
          }
          fresh = true;
        }
      }
      if (++st == S) {
        st = 0;
        parity ^= 1u;
      }
    }
    if (!alive)  // a copy never came: wait (bounded) for the others in flight, then leave
      for (int k = i + 1; k < issued; ++k) wait(k % S, (uint32_t)(k / S) & 1u);
  }

  // ---- join what the warps left open
  __syncthreads();  // every ring has been read
  float* tails = reinterpret_cast<float*>(dec_smem);
  float* parts = part_ws + (size_t)cta * 2 * SLOT;  // of the segment open at the CTA's begin, and at its end
  const float* heads = part_ws + (size_t)kDecMaxCtas * 2 * SLOT + (size_t)cta * W * SLOT;
  if (count > 0 && s_seg[2 * warp + 1][0] >= 0) {
    // a tail that no other warp of the CTA shares goes straight to its place
    const long long first = s_seg[2 * warp + 1][0];
    const bool alone = u1 == c1 && s_seg[2 * warp + 1][1] > c1 && (first >= u0 || u0 == c0);
    store_partial(alone ? parts + (first < c0 ? 0 : 1) * SLOT : tails + (size_t)warp * SLOT);
  }
  if (threadIdx.x < 2) s_open[threadIdx.x] = 0;
  __syncthreads();
  int* counters = reinterpret_cast<int*>(a.ws);
  // the segments' lists of partials, in order; all are joined side by side
  if (warp == 0) {
    const long long first = lane < 2 * W ? s_seg[lane][0] : -1;
    const uint32_t there = __ballot_sync(0xffffffffu, first >= 0), below = there & ((1u << lane) - 1u);
    const bool begins = first >= 0 && (below == 0 || s_seg[31 - __clz(below)][0] != first);
    const uint32_t begin = __ballot_sync(0xffffffffu, begins);
    if (first >= 0) s_list[__popc(below)] = lane;
    if (begins) s_group[__popc(begin & ((1u << lane) - 1u))] = __popc(below);
    if (lane == 0) {
      s_groups = __popc(begin);
      s_group[__popc(begin)] = __popc(there);
    }
  }
  __syncthreads();
  const int groups = s_groups;
  constexpr int kShares = ROWS * (D / 4);
  for (int it = threadIdx.x; it < groups * kShares; it += THREADS) {
    const int grp = it / kShares, e = it - grp * kShares, l0 = s_group[grp], n = s_group[grp + 1] - l0, m = s_list[l0];
    const long long first = s_seg[m][0], end = s_seg[m][1];
    auto local = [&](int i) {
      const int x = s_list[l0 + i];
      return (x & 1) ? tails + (size_t)(x >> 1) * SLOT : heads + (size_t)(x >> 1) * SLOT;
    };
    const bool whole = first >= c0 && end <= c1;
    if (!whole && n == 1 && (m & 1) && end > c1) continue;  // went straight to its place
    dec_join<T, D, ROWS>(a, e, n, local, whole ? nullptr : parts + (first < c0 ? 0 : 1) * SLOT, s_who[m][0], s_who[m][1],
                         s_who[m][2], s_who[m][3], s_who[m][4]);
  }
  // the segments open at the CTA's ends are the first and the last
  int open_at[2] = {-1, -1};
  if (groups > 0) {
    const int m = s_list[0], z = s_list[s_group[groups - 1]];
    if (s_seg[m][0] < c0) open_at[0] = m;
    if (s_seg[z][1] > c1 && s_seg[z][0] >= c0) open_at[1] = z;
  }
  if (open_at[0] < 0 && open_at[1] < 0) return;
  // the CTA that comes last to an open segment joins its parts, in CTA order
  __syncthreads();
  if (threadIdx.x < 2) {
    const int side = (int)threadIdx.x;
    s_last[side] = 0;
    if (open_at[side] >= 0) {
      // the CTAs whose ranges hold its first and its last unit
      const long long first = s_seg[open_at[side]][0], end = s_seg[open_at[side]][1];
      const int f = (int)(((first + 1) * C - 1) / units), e = (int)((end * C - 1) / units);
      __threadfence();
      const int old = atomicAdd(&counters[f], 1);
      if (old == e - f) {
        counters[f] = 0;  // as it was found
        s_last[side] = e - f + 1;
        s_open[side] = f;
      }
      __threadfence();
    }
  }
  __syncthreads();
#pragma unroll
  for (int side = 0; side < 2; ++side)
    if (s_last[side]) {
      const int f = s_open[side], m = open_at[side];
      auto remote = [&](int i) { return part_ws + ((size_t)(f + i) * 2 + (i == 0 ? 1 : 0)) * SLOT; };
      for (int e = threadIdx.x; e < kShares; e += THREADS)
        dec_join<T, D, ROWS>(a, e, s_last[side], remote, nullptr, s_who[m][0], s_who[m][1], s_who[m][2], s_who[m][3],
                             s_who[m][4]);
    }
}

}  // namespace dcc
