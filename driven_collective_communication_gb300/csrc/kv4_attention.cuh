// kv4_attention.cuh -- causal attention over the 4-bit paged cache.
#pragma once
#include "kv4.cuh"

namespace dcc {

constexpr int kAttnThreads = 256;

struct AttnArgs {
  const void* q[DCC_MAX_RANKS];
  void* out[DCC_MAX_RANKS];
  float* lse[DCC_MAX_RANKS];  // all or none
  const int32_t* start;
  size_t q_stride;
  int tokens, layer, q_heads, max_new, window;
  float scale;
};

// One warp per (rank, row, query head): 32 keys at a time, a lane's key for
// the scores, a lane's channels for the sum.
template <typename T, int D, int G>
__global__ void __launch_bounds__(kAttnThreads) k_kv4_attention(Kv4Dev kv, AttnArgs a) {
  constexpr int NG = D / G, CH = D / 32;  // channels per lane
  pdl_prologue();
  const int lane = threadIdx.x & 31;
  const long long item = (long long)blockIdx.x * (kAttnThreads / 32) + (threadIdx.x >> 5);
  const long long per_rank = (long long)a.tokens * a.q_heads;
  const int rank = (int)(item / per_rank);
  if (rank >= kv.n) return;
  const int tok = (int)(item % per_rank / a.q_heads), qh = (int)(item % a.q_heads);
  const int seq = kv4_seq_of<32>(a.start, kv.seqs, tok);
  if (seq < 0 || tok - a.start[seq] >= a.max_new) return;
  const int pos = kv.len[seq] - a.start[seq + 1] + tok;
  const int head = qh / (a.q_heads / kv.heads);
  const uint16_t* q = static_cast<const uint16_t*>(a.q[rank]) + (size_t)tok * a.q_stride + (size_t)qh * D;
  float m = -INFINITY, l = 0.0f, acc[CH] = {};
  const int first = a.window > 0 && pos - a.window + 1 > 0 ? pos - a.window + 1 : 0;
  for (int j0 = first / 32 * 32; j0 <= pos; j0 += 32) {
    const int page = kv4_page(kv, seq, j0 / kKv4Page);
    if (page < 0) continue;
    const char* blk = kv4_block(kv, rank, a.layer, page, head, kv4_block_bytes(D, G));
    const int slot = j0 % kKv4Page + lane, j = j0 + lane;
    const uint32_t* kp = reinterpret_cast<const uint32_t*>(blk + 2 * kv4_codes_bytes(D));
    const uint32_t* vp = kp + kKv4Page * NG;
    float s = -INFINITY;
    if (j >= first && j <= pos) {
      const uint32_t* row = reinterpret_cast<const uint32_t*>(blk + slot * (D / 2));
      s = 0.0f;
      for (int u = 0; u < D / 8; ++u) {
        const uint32_t w = row[kv4_k_word(D, u)], par = kp[slot * NG + u * 8 / G];
        const float step = Half16<T>::widen((uint16_t)par), lo = Half16<T>::widen((uint16_t)(par >> 16));
#pragma unroll
        for (int e = 0; e < 8; ++e)
          s = fmaf(Half16<T>::widen(q[u * 8 + e]), fmaf(step, (float)((w >> (4 * e)) & 15u), lo), s);
      }
      s *= a.scale;
    }
    float top = s;
    for (int x = 16; x; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
    if (top == -INFINITY) continue;
    const float mn = fmaxf(m, top), fix = expf(m - mn), p = expf(s - mn);
    m = mn;
    float sum = p;
    for (int x = 16; x; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
    l = l * fix + sum;
#pragma unroll
    for (int c = 0; c < CH; ++c) acc[c] *= fix;
    for (int t = 0; t < 32; ++t) {
      const float pt = __shfl_sync(0xffffffffu, p, t);
      if (j0 + t < first || j0 + t > pos) continue;
      const int sl = j0 % kKv4Page + t;
      const uint8_t* row = reinterpret_cast<const uint8_t*>(blk + kv4_codes_bytes(D) + sl * (D / 2));
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int d = lane + 32 * c, nib = 2 * (d / 16) + (d % 16) / 8;
        const uint32_t b = row[kv4_v_chunk(D, d & 7, sl) * (D / 16) + nib / 2];
        const uint32_t par = vp[sl * NG + d / G];
        const float v = fmaf(Half16<T>::widen((uint16_t)par), (float)((b >> (4 * (nib & 1))) & 15u),
                             Half16<T>::widen((uint16_t)(par >> 16)));
        acc[c] = fmaf(pt, v, acc[c]);
      }
    }
  }
  const size_t o = (size_t)tok * a.q_heads + qh;
#pragma unroll
  for (int c = 0; c < CH; ++c)
    static_cast<uint16_t*>(a.out[rank])[o * D + lane + 32 * c] =
        Half16<T>::narrow(l > 0.0f ? __fdiv_rn(acc[c], l) : (l == 0.0f ? 0.0f : l));
  if (lane == 0 && a.lse[rank]) a.lse[rank][o] = m == -INFINITY ? m : m + logf(l);
}

}  // namespace dcc
