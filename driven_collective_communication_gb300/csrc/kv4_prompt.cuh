// kv4_prompt.cuh -- attention of many query rows over the 4-bit paged cache
// (prompt chunks), on the fifth-generation tensor cores.
//
// With hundreds of query rows per kv head the products outweigh the cache's
// bytes: bound by the tensor cores and, as closely, by the exponentials (128
// keys x 256 rows take 2048 clocks of either on an SM).  A CTA owns 256 query
// rows of one (sequence, rank, kv head) -- new tokens times the heads that
// share it -- as two tiles of 128, and walks the keys in steps of 128 (two
// pages).  The pages are unpacked once per step into fp16 tiles in shared
// memory, for both row tiles: K_j and V_j = lo + step * code, rounded once (2^-12
// of a value whose own 4-bit step is a fifteenth of its group's range).  Then per
// row tile
//   S = Q K^T            tcgen05, Q and K in shared memory, S in tensor memory;
//   P = 2^(c S - ref)    fp32, rounded to fp16, over S in tensor memory;
//   O += P V             tcgen05, P in tensor memory, V^T in shared memory.
// ref is a row's reference: it follows the running maximum only when that
// grew by more than 2^8 (then O is rescaled in tensor memory), which is rare
// after the first steps; sums l are fp32, of the unrounded P.  While one row
// tile's P is made, the tensor cores work on the other's.
//
// The bf16 cache's operands are fp16 as well: with bf16 tiles (2^-9) three
// roundings put the output 3.0e-3 off where its own rounding is 1.7e-3 (441
// keys); now it is the latter.  Q's rows are scaled by a power of two, exactly.
// Keys of K out of fp16's range have a power of two of their own, which is put
// back on S; a page with such a V stays bf16, and so do its P.  Neither is met
// in ordinary caches, so their forms are short rather than fast.
//
// Measured on GB300, 2048 new tokens on 8192 keys, 8 ranks x 8 query heads x 128
// channels: fp16 534 us, 0.91 PFLOP/s; bf16 551 us, 0.88 PFLOP/s, 46 % of a
// library product's rate (the MMAs alone: 326 us; bf16 tiles: 521 us).  No unit is
// near its rate: tensor pipe 39 %, issue slots 48 %, integer pipe 37 %, exponentials
// 20 %, shared memory 21 % for the warps and 27 % for the MMAs' operands.  The warps
// wait for tensor memory and for one another: a step is a chain of hand-overs
// (unpack, S, P, O) with two row tiles in turn to cover it.  Tried without gain:
// separate warps for K and V, a row of scores held in registers, P handed over in
// halves, an MMA warp that polls both tiles, rings of K's and V's codes apart (a
// deeper prefetch: 542 us where this took 523).
//
// What it rounds, each to fp16 (2^-12 of the value): K, V and P, where the streaming
// kernel rounds p * step alone.  The errors average over the keys a row sees only as
// fast as the output itself does, so an fp16 output is off by up to 4.1e-4 in its
// 2-norm where its own rounding is 2.1e-4; bf16 outputs show their own rounding only.
// Values of V beyond 2^100 (bf16) may overflow the sums.
//
// Roles (512 threads): warp 0 loads pages (one bulk copy each, three in
// flight); warp 1 issues the MMAs; warps 2..5 unpack; warps 6..9 and 10..13
// make P of the two row tiles, one row per thread; warps 14 and 15 take the bf16
// cache's parameters to fp16, each those of its slots of the ring.
//
// The last wave of CTAs would leave most SMs idle where the row tiles are few
// more than the SMs hold: the host then cuts the rows left over, which see the
// fewest keys, into single tiles of 128 (a CTA with one row tile takes some four
// fifths of one with two).
//
// K is unpacked in the order the codes have (channels e, e + 4 of a word side
// by side), and Q's channels are put in the same order; V is unpacked
// transposed, eight keys of a channel to a 16-byte store, so both operands are
// K-major with the 128-byte swizzle.
//
// A key that no row may see (past the sequence, a missing page) has V = 0, and
// its scores are replaced, not multiplied.  A V row that holds NaN or infinity
// becomes 0 there and makes its K NaN instead, so that rows that see the key
// get NaN and the others nothing.  A value past the type's largest (by an ulp,
// where the step was rounded up) counts as the largest: as an infinity it would
// reach the rows that do not see the key, whose P is 0.  (Looking for such
// groups in the fp16 cache cost 523 -> 530 us.)
#pragma once
#include "fused_mma.cuh"
#include "kv4_decode.cuh"
#include "tcgen05.cuh"

namespace dcc {

constexpr int kPromptThreads = 512;
constexpr int kPromptRing = 3;    // pages in flight

template <int D, int G>
struct PromptShape {
  static constexpr int q_tile = 128 * D * 2;     // one row tile of Q
  static constexpr int kv_tile = 128 * D * 2;    // K, or V^T, of 128 keys
  static constexpr int block = kv4_block_bytes(D, G);
  static constexpr size_t smem = 1024 + 2 * q_tile + 4 * kv_tile + kPromptRing * block + 256;
};

// Arithmetic on two 16-bit values of the cache's type, codes as biased numbers.
template <typename T>
struct Pair16;
template <>
struct Pair16<__half> {
  static constexpr uint32_t kExp = 0x7c00u;
  template <int P>
  __device__ static uint32_t code(uint32_t w) {  // 64 + nibbles P, P + 4
    return code_pair<P>(w);
  }
  __device__ static uint32_t value(uint32_t c, uint32_t step, uint32_t lo) {  // lo + step * code, one rounding
    const uint32_t bias = 0x54005400u;
    const __half2 n = __hsub2(*reinterpret_cast<const __half2*>(&c), *reinterpret_cast<const __half2*>(&bias));
    const __half2 r = __hfma2(n, *reinterpret_cast<const __half2*>(&step), *reinterpret_cast<const __half2*>(&lo));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
};
template <>
struct Pair16<__nv_bfloat16> {
  static constexpr uint32_t kExp = 0x7f80u;
  template <int P>
  __device__ static uint32_t code(uint32_t w) {  // 128 + nibbles P, P + 4
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w >> (4 * P)), "r"(0x000f000fu), "r"(0x43004300u));
    return r;
  }
  __device__ static uint32_t value(uint32_t c, uint32_t step, uint32_t lo) {
    const uint32_t bias = 0x43004300u;
    const __nv_bfloat162 n = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&c), *reinterpret_cast<const __nv_bfloat162*>(&bias));
    const __nv_bfloat162 r = __hfma2(n, *reinterpret_cast<const __nv_bfloat162*>(&step), *reinterpret_cast<const __nv_bfloat162*>(&lo));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
};
// bits 15 or 31 are set where a (step, lo) pair holds a NaN or an infinity
template <typename T>
__device__ __forceinline__ uint32_t param_bad(uint32_t w) {
  constexpr uint32_t one = 0x8000u - Pair16<T>::kExp;  // carries an exponent of all ones into the sign's place
  return (w & 0x7fff7fffu) + (one | one << 16);
}
constexpr uint32_t kBad = 0x80008000u;
// The same for fp16 pairs whose lo + 15 step may be more than fp16 holds: a step
// of 2^11 or a lo of 2^15 on (below both it is at most 63,488 of 65,504).  NaN and
// infinities are among them.
__device__ __forceinline__ uint32_t param_large(uint32_t w) { return (w & 0x7fff7fffu) + 0x08001800u; }

// The bf16 cache's parameters as fp16 operands.  A group's largest magnitude m
// decides: fp16 holds the group to 2^-13 of m for m from 2^-8 up.
__device__ __forceinline__ float2 param_floats(uint32_t w) {  // step, lo
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ float param_top(uint32_t w) {
  const float2 p = param_floats(w);
  return fmaxf(fabsf(p.y), fabsf(fmaf(15.0f, p.x, p.y)));
}
__device__ __forceinline__ bool fp16_fits(float m, float top) { return m == 0.0f || (m >= 0x1p-8f && m <= top); }
__device__ __forceinline__ uint32_t param_half(uint32_t w) {
  const float2 p = param_floats(w);
  return Half16<__half>::narrow2(p.x, p.y);
}
// Two values, none of them NaN, rounded to T and kept finite: a step rounded up may
// put a group's last code past the type's largest number, by an ulp of it (0 ..
// 65,504 in fp16: 15 steps of 4368 are 65,520).
template <typename T>
__device__ __forceinline__ uint32_t narrow_finite(float a, float b) {
  const uint32_t w = Half16<T>::narrow2(a, b), most = std::is_same<T, __half>::value ? 0x7bff7bffu : 0x7f7f7f7fu;
  return (w & 0x80008000u) | __vminu2(w & 0x7fff7fffu, most);
}
__device__ __forceinline__ float power2(int e) { return __int_as_float((127 + e) << 23); }  // e from -126 to 127
constexpr float kTopK = 0x1p15f;  // larger groups of K do not fit fp16
constexpr float kTopV = 0x1p11f;  // the smallest P that fp16 holds, times this, is 2^-12 of a V of 2^-8

template <typename T, int D, int G>
__global__ void __launch_bounds__(kPromptThreads, 1) k_kv4_prompt(Kv4Dev kv, const __grid_constant__ AttnArgs a, LocalDev dc) {
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
  const uint32_t base = (smem_addr_u32(prompt_raw) + 1023u) & ~1023u;
  const uint32_t sq = base, sk = sq + 2 * Shape::q_tile, sv = sk + 2 * Shape::kv_tile, raw = sv + 2 * Shape::kv_tile;
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
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  pdl_wait();

  // ---- this CTA's rows; the last tiles (the most keys) come first
  const int nh = kv.n * kv.heads, per = nh * kv.seqs;
  const int turn = (int)blockIdx.x / per, rest = (int)blockIdx.x % per, seq = rest / nh, rh = rest % nh;
  const int rank = rh / kv.heads, head = rh % kv.heads;
  const DecSeq q = dec_seq<false>(kv, a, seq, kPromptRows);
  // a.wide tiles of 256 rows from the last row down, then tiles of 128
  const int past = min(turn, a.wide), row_hi = q.rows - kPromptRows * past - 128 * (turn - past);
  if (row_hi <= 0) return;
  const int row_lo = max(0, row_hi - (turn < a.wide ? kPromptRows : 128));  // this CTA's rows: row_lo .. row_hi - 1
  const int pos_lo = q.pos0 + row_lo / a.share, pos_hi = q.pos0 + (row_hi - 1) / a.share;
  const int key_lo = a.window > 0 ? max(0, pos_lo - a.window + 1) : 0;
  const int page0 = key_lo / kKv4Page;
  // one page past the row at most: it is reported there
  const int pages = pos_hi < 0 ? 0 : min(pos_hi / kKv4Page, kv.max_pages) - page0 + 1;
  const int steps = (pages + 1) / 2;
  const int nt = row_hi - row_lo > 128 ? 2 : 1;
  if (steps <= 0) {  // nothing to see
    for (int i = threadIdx.x; i < (row_hi - row_lo) * (D / 8); i += kPromptThreads) {
      const int row = row_lo + i / (D / 8);
      const size_t at = (size_t)(q.begin + row / a.share) * a.q_heads + head * a.share + row % a.share;
      *reinterpret_cast<uint4*>(static_cast<T*>(a.out[rank]) + at * D + i % (D / 8) * 8) = make_uint4(0, 0, 0, 0);
      if (i % (D / 8) == 0 && a.lse[rank]) a.lse[rank][at] = -INFINITY;
    }
    return;
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
  const int len = min(kv.len[seq], pos_hi + 1);  // keys that some row may see
  auto wait = [&](uint32_t bar, int phase) { return local_wait(bar, (uint32_t)phase & 1u, dc, rank, head); };

  if (warp == 0) {  // ---- loads
    int ids = -1, ids_at = -(1 << 30), unfinished = 0;
    for (int p = 0; p < 2 * steps; ++p) {
      if (p - ids_at >= 32) {
        ids_at = p;
        ids = p + lane < pages ? kv4_page(kv, seq, page0 + p + lane) : -1;
      }
      const int page = __shfl_sync(0xffffffffu, ids, p - ids_at), slot = p % R;
      if (p >= R && !wait(rawe(slot), p / R - 1)) break;
      if (lane == 0) {
        uint32_t& absent = s_absent[(p / 2) & 7];
        absent = (p & 1 ? absent : 0u) | (page < 0 ? 1u << (p & 1) : 0u);
        mma_mbar_expect(rawf(slot), page < 0 ? 0u : (uint32_t)BLK);
        if (page >= 0)
          asm volatile(
              "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                  raw + (uint32_t)(slot * BLK)),
              "l"(kv4_block(kv, rank, a.layer, page, head, BLK)), "r"((uint32_t)BLK), "r"(rawf(slot))
              : "memory");
      }
      ++unfinished;
    }
    // a copy in flight when a wait gave up ends before the CTA does
    for (int p = max(0, unfinished - R); p < unfinished; ++p) local_drain(rawf(p % R), (uint32_t)(p / R) & 1u);
  } else if (warp == 1) {  // ---- MMAs
    if (lane == 0) {
      const uint32_t id = (1u << 4) | ((uint32_t)(128 >> 4) << 24);  // fp16 operands; bf16: bits 7 and 10
      const uint32_t id_s = id | ((uint32_t)(128 >> 3) << 17), id_o = id | ((uint32_t)(D >> 3) << 17);
      uint32_t rg0 = 0, rg1 = 0;  // of even and odd steps
      bool ok = true;
      auto scores = [&](int g, int j) {
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
        }
        tc_commit(two(sFull, g));
        if (g == nt - 1) tc_commit(two(kFree, j & 1));
        (j & 1 ? rg1 : rg0) = range(j);
      };
      for (int g = 0; g < nt; ++g) ok = ok && wait(two(qFull, g), 0);
      for (int g = 0; g < nt; ++g) scores(g, 0);
      for (int j = 0; j < steps && ok; ++j)
        for (int g = 0; g < nt && ok; ++g) {
          ok = wait(two(pFull, g), j) && wait(two(vFull, j & 1), j >> 1);
          if (!ok) break;
          tc_fence_after();
          const uint32_t bf = (1u << 7) | (1u << 10);
          const uint32_t ids[2] = {id_o | ((j & 1 ? rg1 : rg0) & 2u ? bf : 0u), id_o | ((j & 1 ? rg1 : rg0) & 0x200u ? bf : 0u)};
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            const uint64_t bd = mma_smem_desc(sv + (uint32_t)((j & 1) * Shape::kv_tile) + (uint32_t)(kk / 4) * (D * 128u) +
                                              (uint32_t)(kk % 4) * 32u);
            asm volatile(
                "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(tmem + 256u + (uint32_t)g * 128u),
                "r"(tmem + (uint32_t)g * 128u + (uint32_t)kk * 8u), "l"(bd), "r"(ids[kk / 4]), "r"(j > 0 || kk > 0 ? 1u : 0u)
                : "memory");
          }
          if (g == nt - 1) tc_commit(two(vFree, j & 1));
          tc_commit(two(pvDone, g));
          if (j + 1 < steps) scores(g, j + 1);
        }
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
    for (int j = 0; j < steps && ok; ++j) {
      const int buf = j & 1;
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
              const uint32_t pair = (bad | param_bad<T>(pw)) & kBad
                                        ? 0xffffffffu  // NaN
                                        : narrow_finite<T>(fmaf((float)(c & 15u), f.x, f.y),
                                                           fmaf((float)((c >> 16) & 15u), f.x, f.y));
              asm volatile("st.shared.b32 [%0], %1;" ::"r"(row + (uint32_t)(u / 8) * 16384u +
                                                           (uint32_t)(((u % 8) ^ (key & 7)) * 16 + 4 * (i & 3))),
                           "r"(pair)
                           : "memory");
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
            const uint4 v = make_uint4(Pair16<__half>::value(Pair16<__half>::code<0>(w[jj]), step[gr], lo[gr]),
                                       Pair16<__half>::value(Pair16<__half>::code<1>(w[jj]), step[gr], lo[gr]),
                                       Pair16<__half>::value(Pair16<__half>::code<2>(w[jj]), step[gr], lo[gr]),
                                       Pair16<__half>::value(Pair16<__half>::code<3>(w[jj]), step[gr], lo[gr]));
            sts128(row + (uint32_t)(u / 8) * 16384u + (uint32_t)(((u % 8) ^ (key & 7)) * 16), v);
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
              const bool none = (param_bad<T>(pw) & kBad) || !there || (page0 + p) * kKv4Page + key >= len;
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
        if ((bad & kBad) || !there || (page0 + p) * kKv4Page + 8 * oct + 7 >= len) {  // some key must be zero
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int key = 8 * oct + (k ^ swap);
            uint32_t any = 0;  // (another group of the key may be bad: its own unit sees to it)
#pragma unroll
            for (int x = 0; x < GW; ++x) any |= param_bad<__half>(pr[k][x]);
            if ((any & kBad) || !there || (page0 + p) * kKv4Page + key >= len)
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
  } else if (warp >= 14) {  // ---- the bf16 cache's parameters, in place as fp16
    if constexpr (!FP16) {
      // a slot's pages are all one warp's: one that skipped a page of a slot could
      // take the barrier's state before that page for the next page's arrival
      for (int p = 0; p < 2 * steps; ++p) {
        const int slot = p % R, j = p >> 1, h = p & 1;
        if ((slot == 1) != (warp == 15)) continue;
        if (!wait(rawf(slot), p / R)) break;
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
              const bool counts = (page0 + p) * kKv4Page + key < len;
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
    }
  } else {  // ---- P, one row per thread
    const int g = (warp - 6) >> 2, quad = warp & 3, r = quad * 32 + lane, row = row_lo + 128 * g + r;
    if (g < nt) {
      const bool in = row < row_hi;
      const int tok = row / a.share, gh = row - tok * a.share;
      const int hi = in ? q.pos0 + tok : -1, lo = a.window > 0 ? q.pos0 + tok - a.window + 1 : 0;
      float c = fabsf(a.scale) * 1.44269504088896341f;
      {  // Q into its tile, channels in the codes' order, with the scale's sign
        const T* src = static_cast<const T*>(a.q[rank]) + (size_t)(q.begin + tok) * a.q_stride +
                       (size_t)(head * a.share + gh) * D;
        const uint32_t flip = a.scale < 0.0f ? 0x80008000u : 0u;
        const uint32_t dst = sq + (uint32_t)(g * Shape::q_tile) + (uint32_t)r * 128u;
        float f = 1.0f;
        if constexpr (!FP16) {  // a bf16 row as fp16: its largest value goes to 2^8 .. 2^9, exactly
          uint32_t top = 0;
#pragma unroll 4
          for (int u = 0; u < D / 8; ++u) {
            const uint4 v = in ? *reinterpret_cast<const uint4*>(src + 8 * u) : make_uint4(0, 0, 0, 0);
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
#pragma unroll
        for (int u = 0; u < D / 8; ++u) {
          const uint4 v = in ? *reinterpret_cast<const uint4*>(src + 8 * u) : make_uint4(0, 0, 0, 0);
          const uint4 o = make_uint4(half(__byte_perm(v.x, v.z, 0x5410)), half(__byte_perm(v.x, v.z, 0x7632)),
                                     half(__byte_perm(v.y, v.w, 0x5410)), half(__byte_perm(v.y, v.w, 0x7632)));
          sts128(dst + (uint32_t)(u / 8) * 16384u + (uint32_t)(((u % 8) ^ (r & 7)) * 16), o);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(two(qFull, g));
      }
      const uint32_t lanes = (uint32_t)(quad * 32) << 16;
      const uint32_t ts = tmem + lanes + (uint32_t)g * 128u, to = tmem + lanes + 256u + (uint32_t)g * 128u;
      // the keys that every row of this warp sees need no test
      const int first = row_lo + 128 * g + quad * 32, last = min(first + 31, row_hi - 1);
      const int all_hi = first < row_hi ? q.pos0 + first / a.share : 0x7fffffff;
      const int all_lo = a.window > 0 && first < row_hi ? q.pos0 + last / a.share - a.window + 1 : 0;
      float ref = 0.0f, l = 0.0f;
      bool any = false, ok = true;
      int j = 0;
      for (; j < steps; ++j) {
        if (!(ok = wait(two(sFull, g), j))) break;
        tc_fence_after();
        const int key0 = (page0 + 2 * j) * kKv4Page;
        const uint32_t absent = s_absent[j & 7];
        const uint32_t rg = range(j);
        // (a page's V in bf16, so P too: tested in the masked form only)
        const bool masked = absent || key0 + 127 > all_hi || key0 < all_lo || (rg & 0x202u);
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
        auto seen = [&](int i) {
          const int key = key0 + i;
          return key <= hi && key >= lo && !((absent >> (i >> 6)) & 1u);
        };
        // Loops over 32 columns stay loops (the roles' code together must stay
        // in the instruction cache); the next columns load under the current.
        uint32_t s[2][32];
        float m0 = -INFINITY, m1 = -INFINITY;
        tmem_ld32(ts, s[0]);
        auto top = [&](const uint32_t* v, int c0) {
          if (masked) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (seen(c0 + i)) m0 = fmaxf(m0, __uint_as_float(v[i]));
          } else {
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
              m0 = max3(m0, __uint_as_float(v[i]), __uint_as_float(v[i + 1]));
              m1 = max3(m1, __uint_as_float(v[i + 2]), __uint_as_float(v[i + 3]));
            }
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
          if (!(ok = wait(two(pvDone, g), j - 1))) break;
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
          if (masked) {  // tested once, not per element
            const bool wide = (rg & (c0 < 64 ? 2u : 0x200u)) != 0;
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              float2 p = pair(v, i);
              if (!seen(c0 + i)) p.x = 0.0f;
              if (!seen(c0 + i + 1)) p.y = 0.0f;
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
      if (ok) ok = wait(two(pvDone, g), steps - 1);
      tc_fence_after();
      const float inv = l == 0.0f ? 0.0f : __frcp_rn(l);
      const size_t at = (size_t)(q.begin + tok) * a.q_heads + head * a.share + gh;
#pragma unroll
      for (int c0 = 0; c0 < D; c0 += 16) {
        uint32_t v[16];
        tmem_ld16(to + (uint32_t)c0, v);
        tmem_ld_wait16(v);
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          w[i] = Half16<T>::narrow2(__uint_as_float(v[2 * i]) * inv, __uint_as_float(v[2 * i + 1]) * inv);
        if (in && ok) {
          uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(a.out[rank]) + at * D + c0);
          dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
          dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
        }
      }
      if (in && ok && a.lse[rank])
        a.lse[rank][at] = l == 0.0f ? -INFINITY : (ref - kShift + log2f(l)) * 0.69314718055994531f;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
}

}  // namespace dcc
