// kv4.cuh -- the 4-bit key/value cache: its layout, and what the kernels and
// host files that work on it share.
//
// Every rank holds a pool of pages, [layer][page][kv head][block]; a page
// holds 64 tokens.  One block is one kv head's share of a page:
//
//   K codes  64 rows of D/2 bytes      V codes  64 rows of D/2 bytes
//   K params 64 rows of D/G pairs      V params 64 rows of D/G pairs
//
// A row is one token.  A pair (step, lo) of the cache's 16-bit type belongs to
// G consecutive channels: value = lo + step * code, code 0..15.  A block is
// contiguous (9,216 bytes at D = 128, G = 64), so one bulk copy brings a page
// of one head into shared memory.
//
// Within a row the codes lie in the order in which the attention kernel's
// matrix fragments take them, so that it loads whole words without bank
// conflicts and no code is moved between lanes:
//   K  word t * (D/32) + j (t = 0..3) holds channels 32 j + 8 t .. + 7: lane
//      t of a fragment's quad reads its D/32 words at once, and word j of the
//      four lanes covers one run of 32 channels (never two groups);
//   V  D/8 codes per chunk c = 0..7: nibble m holds channel 16 (m / 2) + c +
//      8 (m mod 2), rows c and c + 8 of fragment m / 2.  At D = 128 the
//      chunks of tokens with bit 2 set are exchanged in halves (c ^ 4), so
//      the four tokens a quad reads together lie in different banks.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "dcc.h"
#include "dcc_internal.h"
#include "memory_channel.cuh"

namespace dcc {

constexpr int kKv4Page = DCC_KV4_PAGE;  // tokens per page

__host__ __device__ constexpr int kv4_codes_bytes(int dim) { return kKv4Page * dim / 2; }  // K or V codes of a block
__host__ __device__ constexpr int kv4_params_bytes(int dim, int group) { return kKv4Page * (dim / group) * 4; }
__host__ __device__ constexpr int kv4_block_bytes(int dim, int group) {
  return 2 * kv4_codes_bytes(dim) + 2 * kv4_params_bytes(dim, group);
}

// word of a K row that holds channels 8 u .. 8 u + 7
__host__ __device__ constexpr int kv4_k_word(int dim, int u) { return (u & 3) * (dim / 32) + (u >> 2); }
// place of V chunk c in the row of token `tok`
__host__ __device__ constexpr int kv4_v_chunk(int dim, int c, int tok) {
  return dim == 128 ? c ^ (((tok >> 2) & 1) * 4) : c;
}

// Device view of a cache, passed by value.
struct Kv4Dev {
  char* pool[DCC_MAX_RANKS];
  int32_t* table;  // [seqs][max_pages], -1 past a sequence's pages
  int32_t* len;    // [seqs]
  int32_t* refs;   // [pages] (page calls only)
  int n, layers, pages, seqs, max_pages, heads;
  unsigned long long* status;  // first number out of range, first wait that gave up; 0 = none
};

template <typename T>
struct Half16;
template <>
struct Half16<__half> {
  __device__ static float widen(uint16_t b) { return __half2float(__ushort_as_half(b)); }
  __device__ static uint16_t narrow(float f) { return __half_as_ushort(__float2half_rn(f)); }
  __device__ static float2 widen2(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }
  __device__ static uint32_t narrow2(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
};
template <>
struct Half16<__nv_bfloat16> {
  __device__ static float widen(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }
  __device__ static uint16_t narrow(float f) { return __bfloat16_as_ushort(__float2bfloat16_rn(f)); }
  __device__ static float2 widen2(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
  __device__ static uint32_t narrow2(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
};

// A page number read from a table, or -1 (recorded) where it is none of the pool's.
__device__ __forceinline__ int kv4_page(const Kv4Dev& kv, int seq, int slot) {
  const int p = slot < kv.max_pages ? kv.table[(size_t)seq * kv.max_pages + slot] : -1;
  if (p >= 0 && p < kv.pages) return p;
  atomicCAS(kv.status, 0ull, kStatusBounds | ((unsigned long long)(uint32_t)seq << 32));
  return -1;
}
__device__ __forceinline__ char* kv4_block(const Kv4Dev& kv, int rank, int layer, int page, int head, int block_bytes) {
  return kv.pool[rank] + (((size_t)layer * kv.pages + page) * kv.heads + head) * (size_t)block_bytes;
}

// Sequence of row `row` of a ragged batch (start[0..seqs], ascending): the s
// with start[s] <= row < start[s+1], or -1.  WIDTH neighbouring lanes search
// together (all call with the same arguments): each round of loads narrows
// the range WIDTH-fold, two rounds for 256 sequences with 16 lanes.
template <int WIDTH>
__device__ __forceinline__ int kv4_seq_of(const int32_t* start, int seqs, int row) {
  const int lane = threadIdx.x & (WIDTH - 1), first = (threadIdx.x & 31) & ~(WIDTH - 1);
  const unsigned mask = WIDTH == 32 ? 0xffffffffu : ((1u << (WIDTH & 31)) - 1u) << first;
  int lo = 0, n = seqs;
  while (true) {
    const int step = (n + WIDTH - 1) / WIDTH, p = lane * step;
    const bool below = p < n && start[lo + p] <= row;
    const int cnt = __popc(__ballot_sync(mask, below) & mask);
    if (cnt == 0) return -1;
    lo += (cnt - 1) * step;
    n = min(step, n - (cnt - 1) * step);
    if (step == 1) break;
  }
  return start[lo] <= row && row < start[lo + 1] ? lo : -1;
}

}  // namespace dcc

namespace dcc {
struct LocalDev;
}
namespace dcc_host {
// Status words of the calls that use no communicator, on the current device
// (ops_status.cu); null after a CUDA error.
unsigned long long* local_status();
// What the kernels of one such call wait with, given the status words.
dcc::LocalDev local_dev(unsigned long long* status);
// Checks a cache descriptor and makes its device view, without any CUDA call;
// kv4_ready adds what a launch needs (ops_status.cu).
int kv4_view(const dcc_kv4_t* kv, bool need_refs, dcc::Kv4Dev* out);
int kv4_ready(dcc::Kv4Dev* d);
// A buffer of a call; one that is written overlaps no other.
struct Extent {
  const void* p;
  size_t bytes;
  bool written;
};
bool disjoint(const Extent* e, int n);
// Whether rows of `width` bytes, `stride` apart (both alike), meet: slices of one buffer may interleave.
bool rows_overlap(const void* a, const void* b, size_t rows, size_t stride, size_t width);
}  // namespace dcc_host
