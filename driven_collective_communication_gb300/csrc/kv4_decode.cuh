// kv4_decode.cuh -- attention of a few query rows over the 4-bit paged cache
// (single tokens, drafted tokens to verify).
//
// With s_j = c q.K_j (c = scale * log2 e), one pass over the cache keeps, per
// query row, the running maximum m, l = sum 2^(s_j - m) and O = sum 2^(s_j -
// m) V_j.  K_j = lo + step * code per group of G channels, so
//   q.K_j = sum_groups step_jg (q_g . code_jg) + lo_jg (sum q_g),
//   O_d   = sum_j (p_j step_jg) code_jd + sum_j p_j lo_jg.
// The products with the codes run on the tensor cores; the codes are exact in
// 16 bits, so the scores lose nothing, and of the second product only p * step
// is rounded (bf16; in two bf16 terms, 16 bits, when the result is fp16: in
// fp16 itself p * step would leave the type's range).  Everything that
// carries lo is fp32.
//
// Bound by reading the cache (0.56 bytes a channel at G = 64), if the
// instructions that unpack it stay below the memory's time.  Codes become
// floats by one AND-OR: nibble n in the mantissa of 128 (bf16) or 64 (fp16)
// is 128 + n (64 + n); that constant is taken off the scores through sum q_g,
// and off O through a product with a row of ones, which sums the same rounded
// p * step -- no subtraction per code, no conversion.  The fragments take the
// codes where they lie (kv4.cuh).  mma.sync with its operands in registers
// suits this: the tensor work is 8 rows wide, and tcgen05 would want the
// unpacked operands written to shared or tensor memory first, which costs
// more than the products.
//
//   S[row][key]: A = Q (16 rows), B = codes of 8 keys; its accumulator holds,
//   in each lane, row g and keys of the quad pair -- exactly the B fragment of
//   O^T[channel][row]: A = V codes (16 channels x 16 keys), B = P^T.
//
// Work split.  The pages of all (sequence, rank, kv head, row tile) segments
// form one line of units; CTA and warp ranges cut it evenly, so every SM reads
// the same number of bytes whatever the lengths.  A warp streams its pages
// through a ring of its own (one bulk copy per page and head, an mbarrier per
// stage) and never waits for another warp.  Segments cut by a boundary leave
// partial (m, l, O): joined first in the CTA (shared memory, reusing the
// ring), then over the CTAs by whichever comes last, in CTA order, so results
// do not depend on timing.
#pragma once
#include "bulk.cuh"
#include "kv4.cuh"

namespace dcc {

struct AttnArgs {
  const void* q[DCC_MAX_RANKS];
  void* out[DCC_MAX_RANKS];
  float* lse[DCC_MAX_RANKS];  // all or none
  const int32_t* start;
  char* ws;
  size_t q_stride;
  int tokens, layer, q_heads, share, max_new, window;
  float scale;
  unsigned long long timeout_ns;
};

constexpr int kDecMaxCtas = 160;
constexpr int kDecMaxWarps = 12;
constexpr int kDecMaxRows = 16;
// floats of a partial: m and l per row, then rows of O, padded so that the
// fragments' stores fall into different banks
__host__ __device__ constexpr int dec_slot(int rows, int dim) { return rows * (dim + 6); }
// workspace: a counter per CTA, two partials per CTA, one per warp
__host__ __device__ constexpr size_t dec_ws_bytes() {
  return 1024 + (size_t)kDecMaxCtas * 2 * dec_slot(kDecMaxRows, 128) * 4 +
         (size_t)kDecMaxCtas * kDecMaxWarps * dec_slot(kDecMaxRows, 128) * 4;
}

// Warps and stages: as many bytes in flight as shared memory holds, three
// warps to a scheduler where a tile's registers allow (8 rows), two otherwise.
template <int D, int G, int RT>
struct DecShape {
  static constexpr int block = kv4_block_bytes(D, G);
  static constexpr int warps = RT > 1 ? 8 : (12 * 2 * block <= 222 * 1024 ? 12 : 10);
  static constexpr int fit = 222 * 1024 / (warps * block);
  static constexpr int stages = fit > 4 ? 4 : fit;
  static constexpr size_t smem = (size_t)warps * stages * block + 128;
};

__device__ __forceinline__ float exp2_approx(float x) {  // 2^x; -inf gives 0
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// D += A B, 16 x 8 x 16, fp32 accumulators
template <bool FP16>
__device__ __forceinline__ void mma_16816(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
  if (FP16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <uint32_t MASK, uint32_t MAGIC>
__device__ __forceinline__ uint32_t and_or(uint32_t w) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w), "n"(MASK), "n"(MAGIC));  // (w & MASK) | MAGIC
  return r;
}
// nibbles P and P + 4 of w as two floats 64 + n (fp16) or 128 + n (bf16)
template <bool FP16, int P>
__device__ __forceinline__ uint32_t unpack_pair(uint32_t w) {
  if (FP16) return and_or<0x00f000f0u, 0x54005400u>(P == 0 ? w << 4 : w >> (4 * (P - 1)));
  return and_or<0x000f000fu, 0x43004300u>(w >> (4 * P));
}
template <bool FP16>
__host__ __device__ constexpr float unpack_bias() { return FP16 ? 64.0f : 128.0f; }

// One sequence's part of the line of units.
struct DecSeq {
  int begin, rows, pos0, page0, pages, tiles;  // rows: new tokens * share; tiles * pages units per (rank, head)
  bool empty;
};
__device__ __forceinline__ DecSeq dec_seq(const Kv4Dev& kv, const AttnArgs& a, int s, int tile_rows) {
  DecSeq q;
  const int b = max(0, a.start[s]), e = min(a.tokens, a.start[s + 1]), len = kv.len[s];
  const int news = max(0, e - b);
  q.begin = b;
  q.pos0 = len - news;
  q.rows = min(news, a.max_new) * a.share;
  q.tiles = (q.rows + tile_rows - 1) / tile_rows;
  const int first = a.window > 0 ? max(0, q.pos0 - a.window + 1) : 0;
  q.page0 = first / kKv4Page;
  // one page past the row at most: it is reported there
  q.pages = len > 0 ? min((len - 1) / kKv4Page, kv.max_pages) - q.page0 + 1 : 0;
  q.empty = q.pages <= 0;
  if (q.empty) {
    q.pages = 1;
    q.page0 = 0;
  }
  if (q.rows == 0) q.pages = q.tiles = 0;
  return q;
}

// Join `n` partials (by `at`) of one segment and store the result: to `part`
// (a partial again) or to the outputs.  All threads of the CTA.
template <typename T, int D, int ROWS, typename At>
__device__ __forceinline__ void dec_join(const AttnArgs& a, int n, At at, float* part, int rank, int head, int row0,
                                         int rows, int begin) {
  for (int e = threadIdx.x; e < ROWS * (D / 4); e += blockDim.x) {
    const int row = e / (D / 4), d4 = e % (D / 4);
    float m = -INFINITY;
    for (int i = 0; i < n; ++i) m = fmaxf(m, at(i)[row]);
    const float mu = m == -INFINITY ? 0.0f : m;
    float l = 0.0f;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
      const float* p = at(i);
      const float w = exp2_approx(p[row] - mu);
      const float4 v = *reinterpret_cast<const float4*>(p + 2 * ROWS + row * (D + 4) + d4 * 4);
      l = fmaf(w, p[ROWS + row], l);
      o.x = fmaf(w, v.x, o.x);
      o.y = fmaf(w, v.y, o.y);
      o.z = fmaf(w, v.z, o.z);
      o.w = fmaf(w, v.w, o.w);
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

template <typename T, int D, int G, int RT>
__global__ void __launch_bounds__(DecShape<D, G, RT>::warps * 32, 1) k_kv4_decode(Kv4Dev kv, AttnArgs a) {
  using Shape = DecShape<D, G, RT>;
  constexpr bool FP16 = sizeof(T) == 2 && !__is_same(T, __nv_bfloat16);
  constexpr int W = Shape::warps, S = Shape::stages, BLK = Shape::block, THREADS = W * 32;
  constexpr int NG = D / G, ROWS = 8 * RT, JW = D / 32, MT = D / 16, SLOT = dec_slot(ROWS, D);
  constexpr float kCenter = 8.0f;  // codes enter O as n - 8: what p * step is rounded against
  extern __shared__ __align__(128) char dec_smem[];
  __shared__ __align__(8) uint64_t bars[W][S];
  __shared__ long long s_sum[W];
  __shared__ int s_seq[W];         // where each warp's range begins: sequence,
  __shared__ long long s_base[W];  // its first unit
  // what each warp leaves: a segment that began before its range and ended in
  // it (head), one still open at its end (tail); by first and last unit
  __shared__ long long s_seg[2 * W][2];
  __shared__ int s_who[2 * W][3];  // sequence, (rank, head), tile
  __shared__ int s_last;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  char* ring = dec_smem + (size_t)warp * S * BLK;
  if (lane < S) mbar_init(&bars[warp][lane], 1);
  if (lane < 2) s_seg[2 * warp + lane][0] = -1;
  fence_mbar_init();
  pdl_prologue();

  // ---- the line of units, and this warp's range of it
  const int nh = kv.n * kv.heads;
  long long sum = 0;
  for (int s = threadIdx.x; s < kv.seqs; s += THREADS) {
    const DecSeq q = dec_seq(kv, a, s, ROWS);
    sum += (long long)q.pages * q.tiles;
  }
  for (int m = 16; m; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
  if (lane == 0) s_sum[warp] = sum;
  __syncthreads();
  long long units = 0;
#pragma unroll
  for (int w = 0; w < W; ++w) units += s_sum[w];
  units *= nh;
  // no more CTAs than units, so that no range between two others is empty
  const int C = units < (long long)gridDim.x ? (int)units : (int)gridDim.x, cta = (int)blockIdx.x;
  if (cta >= C) return;
  const long long c0 = units * cta / C, c1 = units * (cta + 1) / C;
  auto warp_begin = [&](int w) { return c0 + (c1 - c0) * w / W; };
  long long before = 0;
  for (int s0 = 0; s0 < kv.seqs; s0 += THREADS) {
    const int s = s0 + (int)threadIdx.x;
    long long mine = 0;
    if (s < kv.seqs) {
      const DecSeq q = dec_seq(kv, a, s, ROWS);
      mine = (long long)q.pages * q.tiles;
    }
    long long x = mine;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, m);
      if (lane >= m) x += y;
    }
    __syncthreads();
    if (lane == 31) s_sum[warp] = x;
    __syncthreads();
    long long first = before + x - mine;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      if (w < warp) first += s_sum[w];
      before += s_sum[w];
    }
    if (mine)
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const long long u = warp_begin(w);
        if (first * nh <= u && u < (first + mine) * nh) {
          s_seq[w] = s;
          s_base[w] = first * nh;
        }
      }
    if (before * nh > c1) break;
  }
  __syncthreads();
  const long long u0 = warp_begin(warp), u1 = warp_begin(warp + 1);
  const int count = (int)(u1 - u0);

  // ---- a walk along the units: the loads' cursor runs ahead of the sums'
  struct Cursor {
    int s, seg, j;  // sequence, segment of it ((rank, head), tile), page of the segment
    DecSeq q;
  };
  auto seek = [&](Cursor& c) {
    c.s = s_seq[warp];
    c.q = dec_seq(kv, a, c.s, ROWS);
    const long long off = u0 - s_base[warp];
    c.seg = (int)(off / c.q.pages);
    c.j = (int)(off - (long long)c.seg * c.q.pages);
  };
  auto step = [&](Cursor& c) {
    if (++c.j < c.q.pages) return;
    c.j = 0;
    if (++c.seg < nh * c.q.tiles) return;
    c.seg = 0;
    do {
      ++c.s;
      if (c.s < kv.seqs) c.q = dec_seq(kv, a, c.s, ROWS);
    } while (c.s < kv.seqs && c.q.pages == 0);
  };
  Cursor ld = {}, cu = {};
  uint32_t missing = 0;  // stages that hold no page
  int ids = -1, ids_seq = -1, ids_at = -1;
  auto issue = [&](int st) {
    const int slot = ld.q.page0 + ld.j;
    int page = -1;
    if (!ld.q.empty) {
      if (ids_seq != ld.s || ids_at != (slot & ~31)) {  // 32 page numbers at a time
        ids_seq = ld.s;
        ids_at = slot & ~31;
        const int x = ids_at + lane;
        ids = x >= ld.q.page0 && x < ld.q.page0 + ld.q.pages ? kv4_page(kv, ld.s, x) : -1;
      }
      page = __shfl_sync(0xffffffffu, ids, slot & 31);
    }
    if (page < 0) missing |= 1u << st;
    else missing &= ~(1u << st);
    if (lane == 0) {
      const int rh = ld.seg / ld.q.tiles;
      mbar_arrive_expect_tx(&bars[warp][st], page < 0 ? 0u : (uint32_t)BLK);
      if (page >= 0)
        bulk_load(ring + (size_t)st * BLK, kv4_block(kv, rh / kv.heads, a.layer, page, rh % kv.heads, BLK), BLK,
                  &bars[warp][st]);
    }
  };
  auto wait = [&](int st, uint32_t parity) {
    if (mbar_try_wait(&bars[warp][st], parity)) return true;
    const unsigned long long t0 = global_timer_ns();
    for (unsigned it = 1;; ++it) {
      if (mbar_try_wait(&bars[warp][st], parity)) return true;
      if ((it & 15u) == 0 && global_timer_ns() - t0 > a.timeout_ns) {
        atomicCAS(kv.status, 0ull, pack_status(kStatusTimeout, 0, 0, cta));
        return false;
      }
    }
  };

  // ---- sums of the open segment
  uint32_t qf[2 * JW][2 * RT];    // Q fragments of each 16-channel step: a0, a2 (rows g), then a1, a3 (rows g + 8)
  float qsum[RT][NG], mx[RT], l[RT], pmid[RT][NG];
  float o[RT][MT][4], ones[RT][NG][4];
  int lim_hi[RT], lim_lo[RT], tile_hi = 0, tile_lo = 0;
  auto open = [&]() {
    const int rh = cu.seg / cu.q.tiles, tile = cu.seg % cu.q.tiles, rank = rh / kv.heads, head = rh % kv.heads;
#pragma unroll
    for (int x = 0; x < RT; ++x) {
      const int row = tile * ROWS + 8 * x + g, tok = row / a.share;
      const bool in = row < cu.q.rows;
      const T* q = static_cast<const T*>(a.q[rank]) + (size_t)(cu.q.begin + tok) * a.q_stride +
                   (size_t)(head * a.share + row % a.share) * D;
      lim_hi[x] = in ? cu.q.pos0 + tok : -1;
      lim_lo[x] = a.window > 0 ? cu.q.pos0 + tok - a.window + 1 : 0;
#pragma unroll
      for (int gr = 0; gr < NG; ++gr) qsum[x][gr] = 0.0f;
#pragma unroll
      for (int j = 0; j < JW; ++j) {
        const uint4 v = in ? *reinterpret_cast<const uint4*>(q + 32 * j + 8 * t) : make_uint4(0, 0, 0, 0);
        // channels (e, e + 4) share a register, as two nibbles of a word do
        qf[2 * j][2 * x] = __byte_perm(v.x, v.z, 0x5410);
        qf[2 * j][2 * x + 1] = __byte_perm(v.x, v.z, 0x7632);
        qf[2 * j + 1][2 * x] = __byte_perm(v.y, v.w, 0x5410);
        qf[2 * j + 1][2 * x + 1] = __byte_perm(v.y, v.w, 0x7632);
        const float2 f0 = Half16<T>::widen2(v.x), f1 = Half16<T>::widen2(v.y), f2 = Half16<T>::widen2(v.z),
                     f3 = Half16<T>::widen2(v.w);
        qsum[x][32 * j / G] += ((f0.x + f0.y) + (f1.x + f1.y)) + ((f2.x + f2.y) + (f3.x + f3.y));
      }
#pragma unroll
      for (int gr = 0; gr < NG; ++gr) {
        qsum[x][gr] += __shfl_xor_sync(0xffffffffu, qsum[x][gr], 1);
        qsum[x][gr] += __shfl_xor_sync(0xffffffffu, qsum[x][gr], 2);
        pmid[x][gr] = 0.0f;
#pragma unroll
        for (int e = 0; e < 4; ++e) ones[x][gr][e] = 0.0f;
      }
      mx[x] = -INFINITY;
      l[x] = 0.0f;
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[x][i][e] = 0.0f;
    }
    // keys from tile_lo to tile_hi are seen by every row of the tile
    tile_hi = cu.q.pos0 + tile * ROWS / a.share;
    const int last = min(tile * ROWS + ROWS, cu.q.rows) - 1;
    tile_lo = a.window > 0 ? cu.q.pos0 + last / a.share - a.window + 1 : 0;
  };

  // The final value of each accumulator: centre the codes and add the fp32
  // part.  Leaves l and pmid summed over the quad.
  auto settle = [&]() {
#pragma unroll
    for (int x = 0; x < RT; ++x) {
      l[x] += __shfl_xor_sync(0xffffffffu, l[x], 1);
      l[x] += __shfl_xor_sync(0xffffffffu, l[x], 2);
#pragma unroll
      for (int gr = 0; gr < NG; ++gr) {
        float pm = pmid[x][gr];
        pm += __shfl_xor_sync(0xffffffffu, pm, 1);
        pm += __shfl_xor_sync(0xffffffffu, pm, 2);
        const float p0 = __shfl_sync(0xffffffffu, pm, 8 * t), p1 = __shfl_sync(0xffffffffu, pm, 8 * t + 4);
        const float k0 = fmaf(-(128.0f + kCenter), ones[x][gr][0], p0), k1 = fmaf(-(128.0f + kCenter), ones[x][gr][1], p1);
#pragma unroll
        for (int i = gr * G / 16; i < (gr + 1) * G / 16; ++i) {
          o[x][i][0] += k0;
          o[x][i][1] += k1;
          o[x][i][2] += k0;
          o[x][i][3] += k1;
        }
      }
    }
  };
  auto store_partial = [&](float* p) {
#pragma unroll
    for (int x = 0; x < RT; ++x) {
      if (t == 0) {
        p[8 * x + g] = mx[x];
        p[ROWS + 8 * x + g] = l[x];
      }
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) p[2 * ROWS + (8 * x + 2 * t + (e & 1)) * (D + 4) + 16 * i + g + 8 * (e >> 1)] = o[x][i][e];
    }
  };
  auto store_out = [&]() {
    const int rh = cu.seg / cu.q.tiles, tile = cu.seg % cu.q.tiles, rank = rh / kv.heads, head = rh % kv.heads;
#pragma unroll
    for (int x = 0; x < RT; ++x) {
      const float inv = l[x] == 0.0f ? 0.0f : __frcp_rn(l[x]);
      const float inv2[2] = {__shfl_sync(0xffffffffu, inv, 8 * t), __shfl_sync(0xffffffffu, inv, 8 * t + 4)};
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int row = tile * ROWS + 8 * x + 2 * t + b;
        if (row < cu.q.rows) {
          const size_t at = (size_t)(cu.q.begin + row / a.share) * a.q_heads + head * a.share + row % a.share;
          uint16_t* dst = static_cast<uint16_t*>(a.out[rank]) + at * D + g;
#pragma unroll
          for (int i = 0; i < MT; ++i) {
            dst[16 * i] = Half16<T>::narrow(o[x][i][b] * inv2[b]);
            dst[16 * i + 8] = Half16<T>::narrow(o[x][i][2 + b] * inv2[b]);
          }
        }
      }
      const int row = tile * ROWS + 8 * x + g;
      if (t == 0 && row < cu.q.rows && a.lse[rank]) {
        const size_t at = (size_t)(cu.q.begin + row / a.share) * a.q_heads + head * a.share + row % a.share;
        a.lse[rank][at] = l[x] == 0.0f ? -INFINITY : (mx[x] + log2f(l[x])) * 0.69314718055994531f;
      }
    }
  };

  const float c_log2 = a.scale * 1.44269504088896341f;
  float* part_ws = reinterpret_cast<float*>(a.ws + 1024);
  float* head_ws = part_ws + (size_t)kDecMaxCtas * 2 * SLOT + ((size_t)cta * W + warp) * SLOT;

  if (count > 0) {
    seek(ld);
    cu = ld;
    int issued = 0;
    for (; issued < S && issued < count; ++issued) {
      issue(issued);
      step(ld);
    }
    bool fresh = true, alive = true;
    long long seg_begin = u0 - cu.j;  // first unit of the open segment
    int i = 0;
    for (; i < count; ++i) {
      const int st = i % S;
      if (fresh) {
        open();
        fresh = false;
      }
      if (!wait(st, (uint32_t)(i / S) & 1u)) {
        alive = false;
        break;
      }
      if (!((missing >> st) & 1u)) {
        const char* blk = ring + (size_t)st * BLK;
        const int key0 = (cu.q.page0 + cu.j) * kKv4Page;
        const bool masked = key0 + kKv4Page - 1 > tile_hi || key0 < tile_lo;
        const int sw = D == 128 ? (t & 1) : (t >> 1);             // the quad's pair of keys, in the order
        const int ka = 2 * t + sw, kb = 2 * t + 1 - sw;           // in which the V rows' banks differ
        const int kg = D == 128 ? g ^ ((g >> 1) & 1) : g ^ (g >> 2);  // and the key of column g
        float sc[8][2 * RT];
#pragma unroll
        for (int n = 0; n < 8; ++n) {  // 8 keys each
          uint32_t w[JW];
          const char* row = blk + (8 * n + kg) * (D / 2) + t * (JW * 4);
          if constexpr (JW == 4) {
            const uint4 v = *reinterpret_cast<const uint4*>(row);
            w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
          } else {
            const uint2 v = *reinterpret_cast<const uint2*>(row);
            w[0] = v.x, w[1] = v.y;
          }
          float acc[NG][4] = {};
#pragma unroll
          for (int j = 0; j < JW; ++j) {
            float* d = acc[32 * j / G];
            mma_16816<FP16>(d, qf[2 * j][0], RT > 1 ? qf[2 * j][2 * RT - 2] : 0u, qf[2 * j][1],
                            RT > 1 ? qf[2 * j][2 * RT - 1] : 0u, unpack_pair<FP16, 0>(w[j]), unpack_pair<FP16, 1>(w[j]));
            mma_16816<FP16>(d, qf[2 * j + 1][0], RT > 1 ? qf[2 * j + 1][2 * RT - 2] : 0u, qf[2 * j + 1][1],
                            RT > 1 ? qf[2 * j + 1][2 * RT - 1] : 0u, unpack_pair<FP16, 2>(w[j]),
                            unpack_pair<FP16, 3>(w[j]));
          }
          const uint32_t* par = reinterpret_cast<const uint32_t*>(blk + 2 * kv4_codes_bytes(D));
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            const uint32_t* pk = par + (8 * n + (b ? kb : ka)) * NG;
            float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
            for (int gr = 0; gr < NG; ++gr) {
              const float2 sl = Half16<T>::widen2(pk[gr]);  // step, lo
              const float lo = fmaf(-unpack_bias<FP16>(), sl.x, sl.y);
              s0 = fmaf(sl.x, acc[gr][b], fmaf(lo, qsum[0][gr], s0));
              if (RT > 1) s1 = fmaf(sl.x, acc[gr][2 + b], fmaf(lo, qsum[RT - 1][gr], s1));
            }
            sc[n][b] = s0 * c_log2;
            if (RT > 1) sc[n][2 + b] = s1 * c_log2;
            if (masked) {
              const int pos = key0 + 8 * n + (b ? kb : ka);
#pragma unroll
              for (int x = 0; x < RT; ++x)
                if (pos > lim_hi[x] || pos < lim_lo[x]) sc[n][2 * x + b] = -INFINITY;
            }
          }
        }
        // the running maximum; the sums so far are rescaled where it grew
        bool grew = false;
        float alpha[RT];
#pragma unroll
        for (int x = 0; x < RT; ++x) {
          float m = mx[x];
#pragma unroll
          for (int n = 0; n < 8; ++n) m = fmaxf(m, fmaxf(sc[n][2 * x], sc[n][2 * x + 1]));
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
          alpha[x] = m > mx[x] ? exp2_approx(mx[x] - m) : 1.0f;
          grew |= m > mx[x];
          mx[x] = m;
        }
        if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
          for (int x = 0; x < RT; ++x) {
            l[x] *= alpha[x];
            const float a0 = __shfl_sync(0xffffffffu, alpha[x], 8 * t), a1 = __shfl_sync(0xffffffffu, alpha[x], 8 * t + 4);
#pragma unroll
            for (int gr = 0; gr < NG; ++gr) {
              pmid[x][gr] *= alpha[x];
              ones[x][gr][0] *= a0;
              ones[x][gr][1] *= a1;
            }
#pragma unroll
            for (int i2 = 0; i2 < MT; ++i2) {
              o[x][i2][0] *= a0;
              o[x][i2][1] *= a1;
              o[x][i2][2] *= a0;
              o[x][i2][3] *= a1;
            }
          }
        }
        const uint32_t* vpar = reinterpret_cast<const uint32_t*>(blk + 2 * kv4_codes_bytes(D) + kv4_params_bytes(D, G));
#pragma unroll
        for (int k = 0; k < 4; ++k) {  // 16 keys each
          uint32_t bh[RT][NG][2], bl[RT][NG][2];  // P^T fragments: p * step in bf16, and (fp16) what that leaves
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t* pa = vpar + (16 * k + 8 * h + ka) * NG;
            const uint32_t* pb = vpar + (16 * k + 8 * h + kb) * NG;
            float2 va[NG], vb[NG];  // step, centre
#pragma unroll
            for (int gr = 0; gr < NG; ++gr) {
              va[gr] = Half16<T>::widen2(pa[gr]);
              vb[gr] = Half16<T>::widen2(pb[gr]);
              va[gr].y = fmaf(kCenter, va[gr].x, va[gr].y);
              vb[gr].y = fmaf(kCenter, vb[gr].x, vb[gr].y);
            }
#pragma unroll
            for (int x = 0; x < RT; ++x) {
              const float mu = mx[x] == -INFINITY ? 0.0f : mx[x];
              const float p0 = exp2_approx(sc[2 * k + h][2 * x] - mu), p1 = exp2_approx(sc[2 * k + h][2 * x + 1] - mu);
              l[x] += p0 + p1;
#pragma unroll
              for (int gr = 0; gr < NG; ++gr) {
                float q0 = p0 * va[gr].x, q1 = p1 * vb[gr].x, c0 = p0 * va[gr].y, c1 = p1 * vb[gr].y;
                if (masked) {  // rows that hold no token may hold anything
                  if (p0 == 0.0f) q0 = c0 = 0.0f;
                  if (p1 == 0.0f) q1 = c1 = 0.0f;
                }
                pmid[x][gr] += c0 + c1;
                bh[x][gr][h] = Half16<__nv_bfloat16>::narrow2(q0, q1);
                if (FP16) {
                  const float2 f = Half16<__nv_bfloat16>::widen2(bh[x][gr][h]);
                  bl[x][gr][h] = Half16<__nv_bfloat16>::narrow2(q0 - f.x, q1 - f.y);
                }
              }
            }
          }
#pragma unroll
          for (int x = 0; x < RT; ++x)
#pragma unroll
            for (int gr = 0; gr < NG; ++gr) {
              constexpr uint32_t one = 0x3f803f80u;
              mma_16816<false>(ones[x][gr], one, one, one, one, bh[x][gr][0], bh[x][gr][1]);
              if (FP16) mma_16816<false>(ones[x][gr], one, one, one, one, bl[x][gr][0], bl[x][gr][1]);
            }
          // V codes of the lane's chunk of 4 tokens: words of (first, second) key
          uint32_t v[2][2][JW / 2];
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              const int tok = 16 * k + 8 * h + (b ? kb : ka);
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
            const uint32_t f0[4] = {unpack_pair<false, 0>(x0), unpack_pair<false, 1>(x0), unpack_pair<false, 2>(x0),
                                    unpack_pair<false, 3>(x0)};
            const uint32_t f1[4] = {unpack_pair<false, 0>(x1), unpack_pair<false, 1>(x1), unpack_pair<false, 2>(x1),
                                    unpack_pair<false, 3>(x1)};
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const int i2 = 2 * q4 + y, gr = 16 * i2 / G;
#pragma unroll
              for (int x = 0; x < RT; ++x) {
                mma_16816<false>(o[x][i2], f0[2 * y], f0[2 * y + 1], f1[2 * y], f1[2 * y + 1], bh[x][gr][0], bh[x][gr][1]);
                if (FP16)
                  mma_16816<false>(o[x][i2], f0[2 * y], f0[2 * y + 1], f1[2 * y], f1[2 * y + 1], bl[x][gr][0],
                                   bl[x][gr][1]);
              }
            }
          }
        }
      }
      __syncwarp();  // every lane has read the stage
      if (issued < count) {
        issue(st);
        step(ld);
        ++issued;
      }
      if (cu.j + 1 == cu.q.pages || i + 1 == count) {  // the segment, or the range, ends
        settle();
        const bool whole = seg_begin >= u0, ends = cu.j + 1 == cu.q.pages;
        if (whole && ends) {
          store_out();
        } else {
          const int which = 2 * warp + (ends ? 0 : 1);
          if (ends) store_partial(head_ws);
          if (lane == 0) {
            s_seg[which][0] = seg_begin;
            s_seg[which][1] = seg_begin + cu.q.pages;
            s_who[which][0] = cu.s;
            s_who[which][1] = cu.seg / cu.q.tiles;
            s_who[which][2] = cu.seg % cu.q.tiles;
          }
        }
        if (ends) {
          seg_begin += cu.q.pages;
          fresh = true;
        }
      }
      if (i + 1 < count) step(cu);
    }
    if (!alive)  // a copy never came: wait (bounded) for the others in flight, then leave
      for (int k = i + 1; k < issued; ++k) wait(k % S, (uint32_t)(k / S) & 1u);
  }

  // ---- join what the warps left open
  __syncthreads();  // every ring has been read
  float* tails = reinterpret_cast<float*>(dec_smem);
  if (count > 0 && s_seg[2 * warp + 1][0] >= 0) store_partial(tails + (size_t)warp * SLOT);
  __syncthreads();
  int* counters = reinterpret_cast<int*>(a.ws);
  const float* heads = part_ws + (size_t)kDecMaxCtas * 2 * SLOT + (size_t)cta * W * SLOT;
  int m0 = 0;
  while (true) {
    while (m0 < 2 * W && s_seg[m0][0] < 0) ++m0;
    if (m0 >= 2 * W) break;
    const long long first = s_seg[m0][0], end = s_seg[m0][1];
    int list[W + 1], n = 0, m1 = m0;  // the segment's partials, in order
    for (; m1 < 2 * W; ++m1) {
      if (s_seg[m1][0] < 0) continue;
      if (s_seg[m1][0] != first || n > W) break;
      list[n++] = m1;
    }
    const int seq = s_who[m0][0], rh = s_who[m0][1], tile = s_who[m0][2];
    const DecSeq q = dec_seq(kv, a, seq, ROWS);
    auto local = [&](int i) { return (list[i] & 1) ? tails + (size_t)(list[i] >> 1) * SLOT : heads + (size_t)(list[i] >> 1) * SLOT; };
    if (first >= c0 && end <= c1) {
      dec_join<T, D, ROWS>(a, n, local, nullptr, rh / kv.heads, rh % kv.heads, tile * ROWS, q.rows, q.begin);
    } else {
      dec_join<T, D, ROWS>(a, n, local, part_ws + ((size_t)cta * 2 + (first < c0 ? 0 : 1)) * SLOT, 0, 0, 0, 0, 0);
      // the CTAs whose ranges hold its first and its last unit
      const int f = (int)(((first + 1) * C - 1) / units), e = (int)((end * C - 1) / units);
      __threadfence();
      __syncthreads();
      if (threadIdx.x == 0) {
        const int old = atomicAdd(&counters[f], 1);
        s_last = old == e - f;
        if (old == e - f) counters[f] = 0;  // as it was found
        __threadfence();
      }
      __syncthreads();
      if (s_last) {
        auto remote = [&](int i) { return part_ws + ((size_t)(f + i) * 2 + (i == 0 ? 1 : 0)) * SLOT; };
        dec_join<T, D, ROWS>(a, e - f + 1, remote, nullptr, rh / kv.heads, rh % kv.heads, tile * ROWS, q.rows, q.begin);
      }
      __syncthreads();
    }
    m0 = m1;
  }
}

}  // namespace dcc
