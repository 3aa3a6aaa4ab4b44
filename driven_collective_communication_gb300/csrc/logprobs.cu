// logprobs.cu -- log probabilities of given tokens, entropy and the top
// alternatives of vocabulary-parallel logits.
//
// With d_j = scale (x_j - m), m the row's largest logit, Z = sum e^d_j and U =
// sum d_j e^d_j:
//   log p_j = d_j - ln Z,   H = -sum p_j ln p_j = ln Z - U / Z
// (both terms of H are positive: nothing cancels).  One pass keeps m, Z and U per
// thread, rescaled when m grows (U' = f (U + d Z), f = e^d, d the step of m); the
// sums of threads, slices and ranks join by the same rule, in a fixed order.
//
// Top alternatives.  A token's place is one 64-bit key, the value's bits in
// ascending order above the complement of the token's number: equal values go to
// the lowest number, keys are all different, and the k largest do not depend on the
// order in which they were met.  A CTA holds a threshold (a key that k others are
// known to reach) and a buffer of the keys above it.  The first threshold comes
// from the first batch: each thread's largest value, of these the largest few of
// each warp, of those the k-th, which k tokens reach.  After the first batch, and
// where the buffer has grown, it is cut to its k largest (a key's place is the
// number of keys above it), and the k-th becomes the threshold: about k (1 + ln of
// the batches) tokens a row pass it, and the others cost one comparison a batch.
//
// Work split.  A row is cut into batches that each lie in one rank's shard, and a
// CTA takes a run of them (a whole row, where rows fill the GPU): nothing is
// exchanged but 16 bytes and k keys a run, joined by the CTA that comes last.
//
// Bound by reading the logits once (6.8 TB/s) if the instructions per token stay
// below some 8; measured on GB300, fp16, 2048 rows of 152,008 tokens: 122 us
// without alternatives (5.1 TB/s), 146 with one, 178 with 20 (3.5 TB/s); bf16, 256
// rows of 131,072: 20, 26 and 36 us; one row: 8 to 15 us.  What is left is the
// instructions (63 % of the issue slots) and the threads' waits for one another,
// one a batch.  CTAs of 128 threads, seven to an SM: 256 threads with about the
// same registers took 213 us (more warps wait at a barrier), 64 threads 208, and
// 64 registers a thread, which spill, 243 (the first case with 20).
#include <cfloat>

#include "comm.h"
#include "kv4.cuh"
#include "tcgen05.cuh"

namespace dcc {

constexpr int kLpThreads = 128, kLpWarps = kLpThreads / 32;
constexpr int kLpCap = 1024;      // keys of the buffer
constexpr int kLpCut = 192;       // keys after a batch from which the buffer is cut
constexpr int kLpMaxRuns = 1064;  // CTAs of a call whose rows are cut: one wave of 7 to an SM

struct LpArgs {
  const void* x[DCC_MAX_RANKS];
  const int32_t* target;
  float* logprob;
  float* entropy;
  int32_t* ids;
  float* top_lp;
  int* counters;              // one a row
  float4* sums;               // [row][run]: m, Z, U
  unsigned long long* keys;   // [row][run][top]
  unsigned long long* status;
  size_t stride;
  int n, columns, vocab, top, runs, batches /* of a rank's shard */;
  float scale;
};

// The numbers of 16 bytes: as pairs, their maximum, and one of them.
template <typename T>
struct LpVec;
template <>
struct LpVec<float> {
  static constexpr int N = 4;
  __device__ static float2 pair(uint4 v, int i) {
    return i == 0 ? make_float2(__uint_as_float(v.x), __uint_as_float(v.y)) : make_float2(__uint_as_float(v.z), __uint_as_float(v.w));
  }
  template <int VPT>
  __device__ static float top(const uint4* v) {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      m = max3(m, __uint_as_float(v[i].x), __uint_as_float(v[i].y));
      m = max3(m, __uint_as_float(v[i].z), __uint_as_float(v[i].w));
    }
    return m;
  }
  // a bit for each number that is `least` or more; the numbers of the first n vectors
  template <int VPT>
  __device__ static uint32_t reach(const uint4* v, float least) {
    uint32_t r = 0;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      if (__uint_as_float(v[i].x) >= least) r |= 1u << (4 * i);
      if (__uint_as_float(v[i].y) >= least) r |= 2u << (4 * i);
      if (__uint_as_float(v[i].z) >= least) r |= 4u << (4 * i);
      if (__uint_as_float(v[i].w) >= least) r |= 8u << (4 * i);
    }
    return r;
  }
  __device__ static uint32_t lanes(int n) { return (1u << (4 * n)) - 1u; }
  // the number of bit x, and its column after the thread's first one
  template <int VPT>
  __device__ static float at(const uint4* v, int x, int* col) {
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      if (x == 4 * i) w = v[i].x;
      if (x == 4 * i + 1) w = v[i].y;
      if (x == 4 * i + 2) w = v[i].z;
      if (x == 4 * i + 3) w = v[i].w;
    }
    *col = x / 4 * (kLpThreads * N) + x % 4;
    return __uint_as_float(w);
  }
  static constexpr uint32_t kNegInf = 0xff800000u;
  __device__ static float load(const float* p) { return __ldg(p); }
};
template <typename T16>
struct LpVec16 {
  static constexpr int N = 8;
  static constexpr uint32_t kNegInf = std::is_same<T16, __half>::value ? 0xfc00fc00u : 0xff80ff80u;
  __device__ static uint32_t word(uint4 v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }
  __device__ static float2 pair(uint4 v, int i) { return Half16<T16>::widen2(word(v, i)); }
  __device__ static uint32_t max2(uint32_t a, uint32_t b) {  // (a NaN loses: it shows in Z)
    if constexpr (std::is_same<T16, __half>::value) {
      const __half2 m = __hmax2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
      return *reinterpret_cast<const uint32_t*>(&m);
    } else {
      const __nv_bfloat162 m = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
      return *reinterpret_cast<const uint32_t*>(&m);
    }
  }
  template <int VPT>
  __device__ static float top(const uint4* v) {
    uint32_t m = kNegInf;
#pragma unroll
    for (int i = 0; i < VPT; ++i) m = max2(m, max2(max2(v[i].x, v[i].y), max2(v[i].z, v[i].w)));
    const float2 f = Half16<T16>::widen2(m);
    return fmaxf(fmaxf(f.x, f.y), -INFINITY);
  }
  // As for 32 bits; bits w and w + 16 are the halves of word w.  `least` is one of
  // the type's numbers.
  template <int VPT>
  __device__ static uint32_t reach(const uint4* v, float least) {
    const uint32_t l = Half16<T16>::narrow2(least, least);
    uint32_t r = 0;
#pragma unroll
    for (int i = 0; i < 4 * VPT; ++i) r |= reach2(word(v[i / 4], i % 4), l) & (0x00010001u << i);
    return r;
  }
  __device__ static uint32_t reach2(uint32_t a, uint32_t l) {
    if constexpr (std::is_same<T16, __half>::value)
      return __hge2_mask(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&l));
    else
      return __hge2_mask(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&l));
  }
  __device__ static uint32_t lanes(int n) { return 0x00010001u * ((1u << (4 * n)) - 1u); }
  template <int VPT>
  __device__ static float at(const uint4* v, int x, int* col) {
    const int i = x & 15;
    uint32_t w = 0;
#pragma unroll
    for (int y = 0; y < 4 * VPT; ++y)
      if (y == i) w = word(v[y / 4], y % 4);
    *col = i / 4 * (kLpThreads * N) + i % 4 * 2 + (x >> 4);
    return Half16<T16>::widen((uint16_t)(x >> 4 ? w >> 16 : w));
  }
  __device__ static float load(const T16* p) { return Half16<T16>::widen(__ldg(reinterpret_cast<const uint16_t*>(p))); }
};
template <>
struct LpVec<__half> : LpVec16<__half> {};
template <>
struct LpVec<__nv_bfloat16> : LpVec16<__nv_bfloat16> {};

__device__ __forceinline__ float lp_exp2(float x) {  // 2^x; -inf gives 0
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// a value's bits in ascending order (both zeros alike); 0 is below all of them
__device__ __forceinline__ uint32_t lp_order(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float lp_value(uint32_t o) { return __uint_as_float(o ^ ((o >> 31) ? 0x80000000u : 0xffffffffu)); }
__device__ __forceinline__ unsigned long long lp_key(float x, uint32_t id) {
  return (unsigned long long)lp_order(x) << 32 | (uint32_t)~id;
}

struct LpSum {
  float m, z, u;  // u in units of log2
};
// the sums of both, c = scale * log2 e
__device__ __forceinline__ LpSum lp_join(LpSum a, LpSum b, float c) {
  const float m = fmaxf(a.m, b.m);
  LpSum r = {m, 0.0f, 0.0f};
  const LpSum* s[2] = {&a, &b};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const bool none = s[i]->m == -INFINITY;  // z is 0, or NaN
    const float d = none ? 0.0f : (s[i]->m - m) * c, f = lp_exp2(d);
    r.z = fmaf(f, s[i]->z, r.z);
    r.u = fmaf(f, fmaf(fmaxf(d, -1000.0f), s[i]->z, s[i]->u), r.u);
  }
  return r;
}
// over the CTA's threads, in a fixed order; all get it
__device__ __forceinline__ LpSum lp_join_cta(LpSum x, float c, LpSum* smem /* kLpWarps */) {
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (int o = 16; o > 0; o >>= 1) {
    const LpSum other = {__shfl_xor_sync(0xffffffffu, x.m, o), __shfl_xor_sync(0xffffffffu, x.z, o),
                         __shfl_xor_sync(0xffffffffu, x.u, o)};
    x = lane & o ? lp_join(other, x, c) : lp_join(x, other, c);
  }
  if (lane == 0) smem[threadIdx.x >> 5] = x;
  __syncthreads();
  x = smem[0];
#pragma unroll 1
  for (int w = 1; w < kLpWarps; ++w) x = lp_join(x, smem[w], c);
  return x;
}

struct LpTop {
  unsigned long long keys[2][kLpCap];
  unsigned long long thr;  // only keys above it count
  uint32_t est[kLpWarps * 32];
  int count, now;          // keys in buffer `now`
};
// Cuts the buffer to its k largest keys, in descending order, and raises the
// threshold to the k-th.  All threads call, between two barriers without additions;
// returns the keys left (read from the buffer instead, another thread might have
// added to it already).
__device__ __forceinline__ int lp_cut(LpTop& s, int k) {
  const int n = min(s.count, kLpCap), now = s.now;
  const unsigned long long* from = s.keys[now];
  unsigned long long* to = s.keys[now ^ 1];
  for (int i = threadIdx.x; i < n; i += kLpThreads) {
    const unsigned long long key = from[i];
    int above = 0;
    int j = 0;
#pragma unroll 4
    for (; j + 1 < n; j += 2) {
      const ulonglong2 two = *reinterpret_cast<const ulonglong2*>(from + j);
      above += two.x > key;
      above += two.y > key;
    }
    if (j < n) above += from[j] > key;
    if (above < k) to[above] = key;
    if (above == k - 1) s.thr = key;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    s.count = min(n, k);
    s.now = now ^ 1;
  }
  __syncthreads();
  return min(n, k);
}
__device__ __forceinline__ bool lp_add(LpTop& s, unsigned long long key) {
  const int at = atomicAdd(&s.count, 1);
  if (at < kLpCap) s.keys[s.now][at] = key;
  return at < kLpCap;
}
// A first threshold: each warp's j largest of one value a thread (0: none), of all
// warps' the k-th.  All threads call.
__device__ __forceinline__ void lp_first(LpTop& s, uint32_t mine, int k) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int j = min(32, (k + kLpWarps - 1) / kLpWarps + (k > 1 ? 2 : 0)), n = kLpWarps * j;
  uint32_t keep = 0;
#pragma unroll 1
  for (int i = 0; i < j; ++i) {
    const uint32_t best = __reduce_max_sync(0xffffffffu, mine);
    const unsigned who = __ballot_sync(0xffffffffu, mine == best);
    if (lane == __ffs(who) - 1) mine = 0u;
    if (lane == i) keep = best;
  }
  if (lane < j) s.est[warp * j + lane] = keep;
  __syncthreads();
  if ((int)threadIdx.x < n) {
    const uint32_t x = s.est[threadIdx.x];
    int above = 0;  // before it in descending order
#pragma unroll 4
    for (int i = 0; i < n; ++i) above += s.est[i] > x || (s.est[i] == x && i < (int)threadIdx.x);
    if (above == k - 1 && x) s.thr = ((unsigned long long)x << 32) - 1;
  }
  __syncthreads();
}

template <typename T, int VPT>
__global__ void __launch_bounds__(kLpThreads, 7) k_token_logprobs(const __grid_constant__ LpArgs a) {
  using Vec = LpVec<T>;
  constexpr int E = Vec::N;
  __shared__ __align__(16) LpTop s;
  __shared__ LpSum s_sum[kLpWarps];
  __shared__ int s_last;
  const int k = a.top;
  const int row = (int)(blockIdx.x / (unsigned)a.runs), run = (int)(blockIdx.x % (unsigned)a.runs);
  const float c = a.scale * 1.44269504088896341f;
  if (threadIdx.x == 0) {
    s.thr = 0;
    s.count = s.now = 0;
  }
  pdl_prologue();
  __syncthreads();

  const int all = a.n * a.batches;
  const int b0 = (int)((long long)all * run / a.runs), b1 = (int)((long long)all * (run + 1) / a.runs);
  LpSum sum = {-INFINITY, 0.0f, 0.0f};
  // A rank's part of the row: `head` columns up to the first whole vector, nv vectors,
  // and what is left.  Batch g holds the vectors from g * kGroup on; the one that is
  // not full, also the columns outside the vectors, one a thread.
  constexpr int kGroup = kLpThreads * VPT;
  struct Part {
    const T* p;
    int rank, valid, head, nv;
  };
  auto part = [&](int rank) {
    Part x;
    x.rank = rank;
    x.p = static_cast<const T*>(a.x[rank]) + (size_t)row * a.stride;
    x.valid = max(0, min(a.columns, a.vocab - rank * a.columns));
    x.head = min(x.valid, (int)((16u - (reinterpret_cast<uintptr_t>(x.p) & 15u)) % 16u / sizeof(T)));
    x.nv = (x.valid - x.head) / E;
    return x;
  };
  struct Batch {
    int rank, first, mine;  // the thread's first column, and vectors
    int extra;              // its column outside the vectors, or -1
    float x;
  };
  uint4 next[VPT];
  Batch then;
  auto fetch = [&](const Part& x, int g) {
    const int v0 = g * kGroup, left = x.nv - v0;
    const uint4* q = reinterpret_cast<const uint4*>(x.p + x.head) + v0 + (int)threadIdx.x;
    then.rank = x.rank;
    then.first = x.head + (v0 + (int)threadIdx.x) * E;
    then.extra = -1;
    then.x = -INFINITY;
    if (left >= kGroup) {
      then.mine = VPT;
#pragma unroll
      for (int i = 0; i < VPT; ++i) next[i] = __ldcs(q + i * kLpThreads);
    } else {
      then.mine = max(0, min(VPT, (left - (int)threadIdx.x + kLpThreads - 1) / kLpThreads));
#pragma unroll
      for (int i = 0; i < VPT; ++i)
        if (i < then.mine) next[i] = __ldcs(q + i * kLpThreads);
      if (left >= 0 && (int)threadIdx.x < x.valid - x.nv * E) {
        then.extra = (int)threadIdx.x < x.head ? (int)threadIdx.x : x.nv * E + (int)threadIdx.x;
        then.x = Vec::load(x.p + then.extra);
      }
    }
  };
  int held = 0;  // keys of the buffer, at most
  Part at = part(b0 / a.batches);
  int g = b0 % a.batches;
  fetch(at, g);  // (every run has a batch)
  for (int b = b0; b < b1; ++b) {
    uint4 v[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) v[i] = next[i];
    const Batch now = then;
    if (b + 1 < b1) {
      if (++g == a.batches) {
        g = 0;
        at = part(at.rank + 1);
      }
      fetch(at, g);
    }
    if (now.mine < VPT) {
#pragma unroll
      for (int i = 0; i < VPT; ++i)
        if (i >= now.mine) v[i] = make_uint4(Vec::kNegInf, Vec::kNegInf, Vec::kNegInf, Vec::kNegInf);
    }
    const float top = fmaxf(Vec::template top<VPT>(v), now.x);
    // sums (the difference first: the values may be as large as the type holds)
    const float m = fmaxf(sum.m, top), ref = m == -INFINITY ? 0.0f : m;
    if (m > sum.m) {
      const float d = sum.m == -INFINITY ? 0.0f : (sum.m - m) * c, f = lp_exp2(d);
      sum.u = f * fmaf(fmaxf(d, -1000.0f), sum.z, sum.u);
      sum.z *= f;
      sum.m = m;
    }
    if (now.extra >= 0) {
      const float d = (now.x - ref) * c, e = lp_exp2(d);
      sum.z += e;
      sum.u = fmaf(e, fmaxf(d, -1000.0f), sum.u);
    }
    float2 z = make_float2(0.0f, 0.0f), u = z;
    const float2 cc = make_float2(c, c), nr = make_float2(-ref, -ref);
#pragma unroll
    for (int i = 0; i < VPT; ++i)
      if (i < now.mine)
#pragma unroll
        for (int e = 0; e < E / 2; ++e) {
          const float2 d = mul2(add2(Vec::pair(v[i], e), nr), cc);
          const float2 w = make_float2(lp_exp2(d.x), lp_exp2(d.y));
          z = add2(z, w);
          u = fma2(w, d, u);
        }
    const float zb = z.x + z.y;
    float ub = u.x + u.y;
    if (!(ub - ub == 0.0f)) {  // 0 times a hidden token's infinity, or NaN: once more, with care
      u = make_float2(0.0f, 0.0f);
#pragma unroll
      for (int i = 0; i < VPT; ++i)
        if (i < now.mine)
#pragma unroll
          for (int e = 0; e < E / 2; ++e) {
            const float2 d = mul2(add2(Vec::pair(v[i], e), nr), cc);
            u = fma2(make_float2(lp_exp2(d.x), lp_exp2(d.y)), make_float2(fmaxf(d.x, -1000.0f), fmaxf(d.y, -1000.0f)), u);
          }
      ub = u.x + u.y;
    }
    sum.z += zb;
    sum.u += ub;
    if (k == 0) continue;
    // top alternatives
    if (s.thr == 0) lp_first(s, now.mine > 0 || now.extra >= 0 ? lp_order(top) : 0u, k);
    uint32_t pending = 0;
    bool extra = false;
    const uint32_t first = (uint32_t)((s.thr + 1) >> 32);  // the least value that may count
    if (lp_order(top) >= first) {
      const float least = first ? lp_value(first) : -INFINITY;
      pending = Vec::template reach<VPT>(v, least);
      if (now.mine < VPT) pending &= Vec::lanes(now.mine);
      extra = now.extra >= 0 && now.x >= least;
    }
    // The bits go as their tokens are added.  Only where the buffer might be too small
    // the threads look together whether it was: then it is cut, and those that are
    // left try again.
    int adders = __syncthreads_count(pending != 0 || extra);
    while (adders) {
      const unsigned long long thr = s.thr;
      const uint32_t id0 = (uint32_t)(now.rank * a.columns);
      while (pending) {
        const int x = __ffs(pending) - 1;
        int col;
        const float f = Vec::template at<VPT>(v, x, &col);
        const unsigned long long key = lp_key(f, id0 + (uint32_t)(now.first + col));
        if (key > thr && !lp_add(s, key)) break;
        pending &= pending - 1;
      }
      if (extra) {
        const unsigned long long key = lp_key(now.x, id0 + (uint32_t)now.extra);
        extra = key > thr && !lp_add(s, key);
      }
      held += adders * (VPT * E + 1);
      if (held <= kLpCap) break;
      adders = __syncthreads_count(pending != 0 || extra);
      held = s.count;
      if (adders || held > kLpCut || held > k + k / 2) held = lp_cut(s, k);
    }
  }

  // ---- the CTA's sums
  sum = lp_join_cta(sum, c, s_sum);  // (and everything is in the buffer)
  if (k) lp_cut(s, k);

  if (a.runs > 1) {  // join the runs of the row
    const size_t at = (size_t)row * a.runs + run;
    if (threadIdx.x == 0) a.sums[at] = make_float4(sum.m, sum.z, sum.u, 0.0f);
    for (int i = threadIdx.x; i < k; i += kLpThreads) a.keys[at * k + i] = i < s.count ? s.keys[s.now][i] : 0ull;
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) {
      s_last = atomicAdd(&a.counters[row], 1) == a.runs - 1;
      if (s_last) a.counters[row] = 0;  // as it was found
    }
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    sum = LpSum{-INFINITY, 0.0f, 0.0f};
    for (int i = threadIdx.x; i < a.runs; i += kLpThreads) {
      const float4 p = __ldcg(&a.sums[(size_t)row * a.runs + i]);
      sum = lp_join(sum, LpSum{p.x, p.y, p.z}, c);
    }
    sum = lp_join_cta(sum, c, s_sum);
    if (k) {
      const unsigned long long* keys = a.keys + (size_t)row * a.runs * k;
      if (threadIdx.x == 0) {
        s.count = 0;
        s.thr = 0;
      }
      __syncthreads();
      // k tokens reach the k-th of the runs' first keys, and the largest of their k-th
      uint32_t best = 0;
      unsigned long long last = 0;
      // (neighbouring runs in different warps)
      for (int i = (threadIdx.x & 31) * kLpWarps + (threadIdx.x >> 5); i < a.runs; i += kLpThreads) {
        best = max(best, (uint32_t)(__ldcg(keys + (size_t)i * k) >> 32));
        last = max(last, __ldcg(keys + (size_t)i * k + k - 1));
      }
      lp_first(s, best, k);
      if (last) atomicMax(&s.thr, last - 1);
      __syncthreads();
      for (int i0 = 0; i0 < a.runs * k; i0 += kLpThreads) {
        const unsigned long long thr = s.thr;
        const int i = i0 + (int)threadIdx.x;
        const unsigned long long key = i < a.runs * k ? __ldcg(keys + i) : 0ull;
        if (key > thr) lp_add(s, key);
        __syncthreads();
        const bool full = s.count > kLpCap - kLpThreads;
        __syncthreads();  // all have read the count
        if (full) lp_cut(s, k);
      }
      lp_cut(s, k);
    }
  }

  // ---- results
  const bool none = !(sum.z > 0.0f) || !(sum.z < INFINITY) || sum.m == INFINITY;  // no distribution
  const float lz = logf(sum.z), nan = __int_as_float(0x7fffffff);
  if (threadIdx.x == 0) {
    if (a.entropy) a.entropy[row] = none ? nan : lz - sum.u * 0.69314718055994531f / sum.z;
    if (a.logprob) {
      const int t = a.target[row];
      float lp = 0.0f;
      if (t >= a.vocab) {
        atomicCAS(a.status, 0ull, kStatusBounds | ((unsigned long long)(uint32_t)t << 32));
        lp = nan;
      } else if (t >= 0) {
        const int rank = t / a.columns;
        const float x = Vec::load(static_cast<const T*>(a.x[rank]) + (size_t)row * a.stride + (t - rank * a.columns));
        lp = none ? nan : fmaf(x - sum.m, a.scale, -lz);
      }
      a.logprob[row] = lp;
    }
  }
  for (int i = threadIdx.x; i < k; i += kLpThreads) {
    const unsigned long long key = s.keys[s.now][i];
    const size_t at = (size_t)row * k + i;
    a.ids[at] = none ? -1 : (int)~(uint32_t)key;
    a.top_lp[at] = none ? nan : fmaf(lp_value((uint32_t)(key >> 32)) - sum.m, a.scale, -lz);
  }
}

const void* logprobs_kernel(int which) {  // 2 * type + (vectors of a thread: 4, 1)
  switch (which) {
    case 0: return (const void*)&k_token_logprobs<float, 4>;
    case 1: return (const void*)&k_token_logprobs<float, 1>;
    case 2: return (const void*)&k_token_logprobs<__half, 4>;
    case 3: return (const void*)&k_token_logprobs<__half, 1>;
    case 4: return (const void*)&k_token_logprobs<__nv_bfloat16, 4>;
    case 5: return (const void*)&k_token_logprobs<__nv_bfloat16, 1>;
    default: return nullptr;
  }
}

}  // namespace dcc

namespace {
constexpr size_t kLpCounters = ((size_t)dcc::kLpMaxRuns * 4 + 15) / 16 * 16;
size_t lp_ws_bytes(int top) { return kLpCounters + (size_t)dcc::kLpMaxRuns * (sizeof(float4) + 8 * (size_t)top); }
}  // namespace

extern "C" {

int dcc_token_logprobs_workspace(int n_ranks, size_t tokens, size_t columns, int top, size_t* bytes) {
  if (!bytes || n_ranks < 1 || n_ranks > DCC_MAX_RANKS || top < 0 || top > DCC_TOP_MAX || columns < 1)
    return DCC_ERR_INVALID_ARG;
  (void)tokens;  // rows are cut only where there are few of them
  *bytes = lp_ws_bytes(top);
  return DCC_OK;
}

int dcc_token_logprobs(int n_ranks, const void* const* logits, size_t tokens, size_t columns, size_t stride, size_t vocab,
                       const int32_t* target, float scale, int top, float* logprob, float* entropy, int32_t* top_ids,
                       float* top_logprob, void* workspace, size_t workspace_bytes, dcc_dtype_t t, dcc_stream_t s) {
  size_t need = 0;
  int rc = dcc_token_logprobs_workspace(n_ranks, tokens, columns, top, &need);
  if (rc != DCC_OK) return rc;
  if (t != DCC_FP32 && t != DCC_FP16 && t != DCC_BF16) return DCC_ERR_UNSUPPORTED;
  // the kernel's exponentials take scale log2 e, in fp32
  if (!logits || !workspace || workspace_bytes < need || !(scale > 0.0f) || !(scale * 1.44269504088896341f <= FLT_MAX))
    return DCC_ERR_INVALID_ARG;
  if (tokens &&  // (empty buffers have no address)
      ((logprob != nullptr) != (target != nullptr) || (top > 0 && (!top_ids || !top_logprob)) ||
       (top == 0 && (top_ids || top_logprob)) || (!logprob && !entropy && top == 0)))
    return DCC_ERR_INVALID_ARG;
  if (tokens > (size_t)1 << 24 || columns > (size_t)1 << 27 || stride > (size_t)1 << 32 || (tokens > 1 && stride < columns) ||
      columns * n_ranks > (size_t)1 << 30 || vocab < 1 || vocab > columns * n_ranks || (size_t)top > vocab)
    return DCC_ERR_INVALID_ARG;
  const size_t size = t == DCC_FP32 ? 4 : 2;
  const uintptr_t words = reinterpret_cast<uintptr_t>(target) | reinterpret_cast<uintptr_t>(logprob) |
                          reinterpret_cast<uintptr_t>(entropy) | reinterpret_cast<uintptr_t>(top_ids) |
                          reinterpret_cast<uintptr_t>(top_logprob);
  if ((words & 3u) || (reinterpret_cast<uintptr_t>(workspace) & 15u)) return DCC_ERR_MISALIGNED;
  if (tokens == 0) return DCC_OK;
  dcc::LpArgs a{};
  const size_t span = ((tokens - 1) * stride + columns) * size, out = tokens * 4;
  for (int r = 0; r < n_ranks; ++r) {
    if (!logits[r]) return DCC_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(logits[r]) & (size - 1)) return DCC_ERR_MISALIGNED;
    const dcc_host::Extent e[] = {{workspace, need, true}, {logprob, out, true},          {entropy, out, true},
                                  {top_ids, out * top, true}, {top_logprob, out * top, true}, {logits[r], span, false},
                                  {target, out, false}};
    if (!dcc_host::disjoint(e, 7)) return DCC_ERR_INVALID_ARG;
    a.x[r] = logits[r];
  }
  if (!(a.status = dcc_host::local_status())) return DCC_ERR_CUDA;
  a.target = target;
  a.logprob = logprob;
  a.entropy = entropy;
  a.ids = top_ids;
  a.top_lp = top_logprob;
  char* ws = static_cast<char*>(workspace);
  a.counters = reinterpret_cast<int*>(ws);  // in front: their place is the same whatever the call
  a.sums = reinterpret_cast<float4*>(ws + kLpCounters);
  a.keys = reinterpret_cast<unsigned long long*>(ws + kLpCounters + (size_t)dcc::kLpMaxRuns * sizeof(float4));
  a.stride = tokens > 1 ? stride : 0;
  a.n = n_ranks;
  a.columns = (int)columns;
  a.vocab = (int)vocab;
  a.top = top;
  a.scale = scale;
  // A shard's vectors in batches of four a thread, or one where the GPU would not be
  // full otherwise; the last one is not full.
  const long long vectors = (long long)((columns * size + 15) / 16), runs_wanted = dcc::kLpMaxRuns / (long long)tokens;  // of a row
  const auto batches = [&](int per) { return (vectors + per * dcc::kLpThreads - 1) / (per * dcc::kLpThreads); };
  const int per = n_ranks * batches(4) < runs_wanted ? 1 : 4;
  a.batches = (int)batches(per);
  const long long all = (long long)n_ranks * a.batches;
  a.runs = (int)(runs_wanted < 1 ? 1 : runs_wanted < all ? runs_wanted : all);
  const int type = t == DCC_FP32 ? 0 : t == DCC_FP16 ? 1 : 2;
  void* args[] = {&a};
  return dcc_host::launch(dcc::logprobs_kernel(2 * type + (per == 1)), (int)((long long)tokens * a.runs), dcc::kLpThreads,
                          false, args, static_cast<cudaStream_t>(s), 0, true);
}

}  // extern "C"
