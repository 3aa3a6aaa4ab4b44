// kv4_cache.cu -- writing new keys and values into the 4-bit cache, and
// reading them back.
//
// Per token, kv head and group of G channels: lo = min x, step =
// R16((max x - lo) / 15), code = rne((x - lo) / step) in 0..15.  lo is one of
// the inputs, so it is exact in their type; the division is IEEE, so a value
// halfway between two codes goes where the mathematics sends it.
//
// Both kernels ought to be bound by memory: 2 bytes an element on the dense
// side, 1/2 + 4/G in the cache.  Measured on GB300, 12,718 rows x 2 heads x 128
// channels x 8 ranks, fp16, G = 32 (137 MB each way): append 59 us (2.3 TB/s),
// read 32 us (4.2 TB/s).  Both now spend their time on instructions, 33 a value
// appended and 17 read, at 77 % of the issue slots: one value at a time.  D/8 lanes take one (token, head): 16-byte accesses to
// the dense rows, two tokens of a 128-wide head per warp; a group's minimum
// and maximum are three shuffles.  A lane's eight K codes are one word of the
// row; its eight V codes fall into the row's eight chunks, so the row is put
// together in shared memory first and moves as words.
#include "comm.h"
#include "kv4.cuh"

namespace dcc {

constexpr int kKv4RowThreads = 256;
// Tokens a group of lanes takes in large batches: their loads are in flight
// together and the place in the cache is searched for once.
constexpr int kKv4RowTokens = 4;
// From this many (token, head, rank) on: enough groups of lanes to fill the
// GPU (152 SMs x 64) with several tokens each.
constexpr long long kKv4ManyRows = 152ll * 64 * kKv4RowTokens;

struct Kv4RowArgs {
  void* k[DCC_MAX_RANKS];
  void* v[DCC_MAX_RANKS];
  const int32_t* start;
  size_t stride;  // elements between rows of k / v
  int tokens, layer;
};

// Where U rows of the batch, `step` apart, stand in the cache; page < 0: nowhere.
// The first is searched for, the others follow it; their loads overlap.
struct Kv4Place {
  int page, slot;
};
template <int LANES, int U>
__device__ __forceinline__ void kv4_places(const Kv4Dev& kv, const int32_t* start, int tokens, int tok, Kv4Place* at) {
  int s = kv4_seq_of<LANES>(start, kv.seqs, tok);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    at[u] = {-1, 0};
    const int t = tok + u;
    if (t >= tokens) continue;
    if (u > 0) {
      if (s < 0) s = kv4_seq_of<LANES>(start, kv.seqs, t);
      else
        while (s < kv.seqs && t >= start[s + 1]) ++s;
      if (s >= kv.seqs || (s >= 0 && t < start[s])) s = -1;
    }
    if (s < 0) continue;
    const int pos = kv.len[s] - start[s + 1] + t;
    if (pos >= 0) at[u] = {kv4_page(kv, s, pos / kKv4Page), pos % kKv4Page};
  }
}

// The (rank, first of U tokens, head) that D/8 lanes work on.
struct Kv4Item {
  int rank, tok, head;
};
template <int U>
__device__ __forceinline__ Kv4Item kv4_item(const Kv4Dev& kv, int tokens, long long item) {
  const long long per_rank = (long long)((tokens + U - 1) / U) * kv.heads;
  const int rank = (int)(item / per_rank);
  return {rank, (int)(item % per_rank / kv.heads) * U, (int)(item % kv.heads)};
}

// Two values at once, in their 16-bit type.
template <typename T>
struct MinMax;
template <>
struct MinMax<__half> {
  static constexpr uint32_t kOne = 0x0400u;  // the exponent's last bit
  __device__ static uint32_t min2(uint32_t a, uint32_t b) {
    const __half2 r = __hmin2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
};
template <>
struct MinMax<__nv_bfloat16> {
  static constexpr uint32_t kOne = 0x0080u;
  __device__ static uint32_t min2(uint32_t a, uint32_t b) {
    const __nv_bfloat162 r =
        __hmin2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
};

// d / step correctly rounded, as a division would: with inv = 1 / step correctly
// rounded, the remainder of q = d * inv is exact and one step from it lands on
// the correctly rounded quotient (Markstein's theorem; step is no number of
// all-ones mantissa, it has at most 11 bits).  A division per value instead
// took 64 instructions a value and 125 us where this takes 59.
__device__ __forceinline__ float kv4_quotient(float d, float step, float inv) {
  const float q = d * inv;
  return fmaf(fmaf(-q, step, d), inv, q);
}

template <typename T, int D, int G, int U>
__global__ void __launch_bounds__(kKv4RowThreads) k_kv4_append(Kv4Dev kv, Kv4RowArgs a) {
  constexpr int LANES = D / 8, ITEMS = kKv4RowThreads / LANES, GL = G / 8, NG = D / G;
  __shared__ uint32_t vrow[ITEMS][D / 8];
  pdl_prologue();
  const int lane = threadIdx.x % LANES, sub = threadIdx.x / LANES;
  const unsigned mask = ((1ull << LANES) - 1ull) << ((threadIdx.x & 31) / LANES * LANES);
  const Kv4Item it = kv4_item<U>(kv, a.tokens, (long long)blockIdx.x * ITEMS + sub);
  if (it.rank >= kv.n) return;
  uint4 raw[U][2];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const size_t src = (size_t)min(it.tok + u, a.tokens - 1) * a.stride + (size_t)it.head * D + lane * 8;
    raw[u][0] = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.k[it.rank]) + src);
    raw[u][1] = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.v[it.rank]) + src);
  }
  Kv4Place at[U];
  kv4_places<LANES, U>(kv, a.start, a.tokens, it.tok, at);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (at[u].page < 0) continue;
    const int slot = at[u].slot;
    char* blk = kv4_block(kv, it.rank, a.layer, at[u].page, it.head, kv4_block_bytes(D, G));
#pragma unroll
    for (int w = 0; w < 2; ++w) {  // K, then V
      const uint32_t r[4] = {raw[u][w].x, raw[u][w].y, raw[u][w].z, raw[u][w].w};
      // (min, -max) of the group, two values at a time; a NaN or an infinity is
      // an exponent of all ones, which the addition carries into the sign
      uint32_t lo2 = r[0], hi2 = r[0] ^ 0x80008000u, bad = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        constexpr uint32_t one = MinMax<T>::kOne * 0x10001u;
        bad |= (r[j] & 0x7fff7fffu) + one;
        lo2 = MinMax<T>::min2(lo2, r[j]);
        hi2 = MinMax<T>::min2(hi2, r[j] ^ 0x80008000u);
      }
      uint32_t ends = MinMax<T>::min2(__byte_perm(lo2, hi2, 0x5410), __byte_perm(lo2, hi2, 0x7632));
#pragma unroll
      for (int m = 1; m < GL; m <<= 1) ends = MinMax<T>::min2(ends, __shfl_xor_sync(mask, ends, m));
      const unsigned bads = __ballot_sync(mask, (bad & 0x80008000u) != 0u);
      const float2 e2 = Half16<T>::widen2(ends);
      float lo = e2.x;
      uint16_t step16 = Half16<T>::narrow(__fdiv_rn(-e2.y - lo, 15.0f)), lo16 = (uint16_t)ends;
      float step = Half16<T>::widen(step16);
      uint32_t codes = 0;
      if (((bads >> ((threadIdx.x & 31) / GL * GL)) & ((1u << GL) - 1u)) != 0u || !(step - step == 0.0f)) {
        step16 = lo16 = Half16<T>::narrow(__uint_as_float(0x7fc00000u));
      } else if (step > 0.0f) {
        // steps whose reciprocal may overflow: the group times 2^100 (a step is
        // at least 2^-12 of the group's values, so nothing overflows)
        const float up = step < 1e-25f ? 1.2676506002282294e30f : 1.0f;
        step *= up;
        lo *= up;
        const float inv = __fdiv_rn(1.0f, step);
        // adding 1.5 * 2^23 rounds to the nearest even integer, whose bits end
        // the sum's; the constant's own come off all eight at once
        constexpr float kMagic = 12582912.0f;
        constexpr uint32_t kMagicBits = 0x4b400000u * 0x11111111u;
#pragma unroll
        for (int j = 3; j >= 0; --j) {
          const float2 f = Half16<T>::widen2(r[j]);
          const float c0 = fminf(kv4_quotient(fmaf(f.x, up, -lo), step, inv), 15.0f) + kMagic;
          const float c1 = fminf(kv4_quotient(fmaf(f.y, up, -lo), step, inv), 15.0f) + kMagic;
          codes = (codes * 16u + __float_as_uint(c1)) * 16u + __float_as_uint(c0);
        }
        codes -= kMagicBits;
      }
      if (lane % GL == 0)
        *reinterpret_cast<uint32_t*>(blk + 2 * kv4_codes_bytes(D) + w * kv4_params_bytes(D, G) +
                                     (slot * NG + lane / GL) * 4) = (uint32_t)step16 | ((uint32_t)lo16 << 16);
      char* row = blk + w * kv4_codes_bytes(D) + slot * (D / 2);
      if (w == 0) {
        reinterpret_cast<uint32_t*>(row)[kv4_k_word(D, lane)] = codes;
      } else {
        // channels 16 i + 8 half + e, i = lane / 2, half = lane & 1: nibble
        // 2 i + half of chunk e, so lanes 2 i and 2 i + 1 share byte i of it
        const uint32_t other = __shfl_xor_sync(mask, codes, 1);
        const int i = lane >> 1, odd = lane & 1;
        const uint32_t even_c = odd ? other : codes, odd_c = odd ? codes : other;
        uint8_t* bytes = reinterpret_cast<uint8_t*>(vrow[sub]);
        __syncwarp(mask);  // the row before has been read
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int c = 4 * odd + e;
          bytes[kv4_v_chunk(D, c, slot) * (D / 16) + i] =
              (uint8_t)(((even_c >> (4 * c)) & 15u) | (((odd_c >> (4 * c)) & 15u) << 4));
        }
        __syncwarp(mask);
        reinterpret_cast<uint32_t*>(row)[lane] = vrow[sub][lane];
      }
    }
  }
}

template <typename T, int D, int G, int U>
__global__ void __launch_bounds__(kKv4RowThreads) k_kv4_read(Kv4Dev kv, Kv4RowArgs a) {
  constexpr int LANES = D / 8, ITEMS = kKv4RowThreads / LANES, GL = G / 8, NG = D / G;
  __shared__ uint32_t vrow[ITEMS][U][D / 8];
  pdl_prologue();
  const int lane = threadIdx.x % LANES, sub = threadIdx.x / LANES;
  const unsigned mask = ((1ull << LANES) - 1ull) << ((threadIdx.x & 31) / LANES * LANES);
  const Kv4Item it = kv4_item<U>(kv, a.tokens, (long long)blockIdx.x * ITEMS + sub);
  if (it.rank >= kv.n) return;
  Kv4Place at[U];
  kv4_places<LANES, U>(kv, a.start, a.tokens, it.tok, at);
  uint32_t kword[U], vword[U], par[U][2];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    kword[u] = vword[u] = par[u][0] = par[u][1] = 0;
    if (at[u].page < 0) continue;
    const char* blk = kv4_block(kv, it.rank, a.layer, at[u].page, it.head, kv4_block_bytes(D, G));
    kword[u] = reinterpret_cast<const uint32_t*>(blk + at[u].slot * (D / 2))[kv4_k_word(D, lane)];
    vword[u] = reinterpret_cast<const uint32_t*>(blk + kv4_codes_bytes(D) + at[u].slot * (D / 2))[lane];
#pragma unroll
    for (int w = 0; w < 2; ++w)
      par[u][w] = *reinterpret_cast<const uint32_t*>(blk + 2 * kv4_codes_bytes(D) + w * kv4_params_bytes(D, G) +
                                                     (at[u].slot * NG + lane / GL) * 4);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) vrow[sub][u][lane] = vword[u];
  __syncwarp(mask);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (at[u].page < 0) continue;
    uint32_t vcodes = 0;
    const uint8_t* bytes = reinterpret_cast<const uint8_t*>(vrow[sub][u]);
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const uint32_t b = bytes[kv4_v_chunk(D, c, at[u].slot) * (D / 16) + (lane >> 1)];
      vcodes |= ((b >> (4 * (lane & 1))) & 15u) << (4 * c);
    }
    const size_t dst = (size_t)(it.tok + u) * a.stride + (size_t)it.head * D + lane * 8;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const float step = Half16<T>::widen((uint16_t)par[u][w]), lo = Half16<T>::widen((uint16_t)(par[u][w] >> 16));
      const uint32_t codes = w ? vcodes : kword[u];
      float x[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = fmaf(step, (float)((codes >> (4 * j)) & 15u), lo);
      const uint4 out = make_uint4(Half16<T>::narrow2(x[0], x[1]), Half16<T>::narrow2(x[2], x[3]),
                                   Half16<T>::narrow2(x[4], x[5]), Half16<T>::narrow2(x[6], x[7]));
      *reinterpret_cast<uint4*>(static_cast<T*>(w ? a.v[it.rank] : a.k[it.rank]) + dst) = out;
    }
  }
}

template <typename T, int D, int G>
static const void* row_kernel_of(bool read, bool several) {
  if (several) return read ? (const void*)&k_kv4_read<T, D, G, kKv4RowTokens> : (const void*)&k_kv4_append<T, D, G, kKv4RowTokens>;
  return read ? (const void*)&k_kv4_read<T, D, G, 1> : (const void*)&k_kv4_append<T, D, G, 1>;
}
template <typename T>
static const void* row_kernel_for(bool read, int dim, int group, bool several) {
  if (dim == 128) return group == 64 ? row_kernel_of<T, 128, 64>(read, several) : row_kernel_of<T, 128, 32>(read, several);
  return group == 64 ? row_kernel_of<T, 64, 64>(read, several) : row_kernel_of<T, 64, 32>(read, several);
}
const void* kv4_row_kernel(bool fp16, bool read, int dim, int group, bool several) {
  return fp16 ? row_kernel_for<__half>(read, dim, group, several) : row_kernel_for<__nv_bfloat16>(read, dim, group, several);
}

}  // namespace dcc

namespace {

int rows_call(bool read, const dcc_kv4_t* kv, int layer, void* const* k, void* const* v, size_t tokens, size_t stride,
              const int32_t* start, dcc_stream_t s) {
  dcc::Kv4Dev d{};
  int rc = dcc_host::kv4_view(kv, false, &d);
  if (rc != DCC_OK) return rc;
  if (!k || !v || !start || layer < 0 || layer >= kv->layers) return DCC_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(start) & 3u) return DCC_ERR_MISALIGNED;
  const size_t width = (size_t)kv->kv_heads * kv->head_dim;
  if (tokens > (size_t)1 << 30 || stride > (size_t)1 << 32 || (tokens > 1 && stride < width)) return DCC_ERR_INVALID_ARG;
  if (stride % 8) return DCC_ERR_MISALIGNED;  // every row 16-byte aligned
  if (tokens == 0) return DCC_OK;
  dcc::Kv4RowArgs a{};
  const size_t bytes = ((tokens - 1) * stride + width) * 2;
  const size_t pool = (size_t)kv->layers * kv->pages * width / kv->head_dim *
                      dcc::kv4_block_bytes(kv->head_dim, kv->group);
  for (int r = 0; r < kv->n_ranks; ++r)
    if (!k[r] || !v[r]) return DCC_ERR_INVALID_ARG;
  for (int r = 0; r < kv->n_ranks; ++r) {
    if ((reinterpret_cast<uintptr_t>(k[r]) | reinterpret_cast<uintptr_t>(v[r])) & 15u) return DCC_ERR_MISALIGNED;
    for (int p = 0; p < kv->n_ranks; ++p)
      if (dcc_host::overlaps(k[r], bytes, kv->pool[p], pool) || dcc_host::overlaps(v[r], bytes, kv->pool[p], pool))
        return DCC_ERR_INVALID_ARG;
    for (int p = 0; read && p < kv->n_ranks; ++p) {  // outputs
      if (dcc_host::rows_overlap(k[r], v[p], tokens, stride * 2, width * 2) ||
          (p < r && (dcc_host::rows_overlap(k[r], k[p], tokens, stride * 2, width * 2) ||
                     dcc_host::rows_overlap(v[r], v[p], tokens, stride * 2, width * 2))))
        return DCC_ERR_INVALID_ARG;
    }
    a.k[r] = k[r];
    a.v[r] = v[r];
  }
  a.start = start;
  a.stride = stride;
  a.tokens = (int)tokens;
  a.layer = layer;
  const int per_cta = dcc::kKv4RowThreads / (kv->head_dim / 8);
  const bool several = (long long)tokens * kv->kv_heads * kv->n_ranks >= dcc::kKv4ManyRows;
  const long long per = several ? dcc::kKv4RowTokens : 1;
  const long long items = ((long long)tokens + per - 1) / per * kv->kv_heads * kv->n_ranks;
  const long long grid = (items + per_cta - 1) / per_cta;
  if (grid > 0x7fffffffll) return DCC_ERR_INVALID_ARG;
  if ((rc = dcc_host::kv4_ready(&d)) != DCC_OK) return rc;
  void* args[] = {&d, &a};
  return dcc_host::launch(dcc::kv4_row_kernel(kv->dtype == DCC_FP16, read, kv->head_dim, kv->group, several), (int)grid,
                          dcc::kKv4RowThreads, false, args, static_cast<cudaStream_t>(s), 0, true);
}

}  // namespace

extern "C" {

int dcc_kv4_append(const dcc_kv4_t* kv, int layer, void* const* k, void* const* v, size_t tokens, size_t stride,
                   const int32_t* start, dcc_stream_t s) {
  return rows_call(false, kv, layer, k, v, tokens, stride, start, s);
}
int dcc_kv4_read(const dcc_kv4_t* kv, int layer, void* const* k, void* const* v, size_t tokens, size_t stride,
                 const int32_t* start, dcc_stream_t s) {
  return rows_call(true, kv, layer, k, v, tokens, stride, start, s);
}

}  // extern "C"
