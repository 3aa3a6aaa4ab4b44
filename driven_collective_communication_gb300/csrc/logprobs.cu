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
// from the first batch: of each warp's 32 largest (one a lane) the j-th, and of the
// warps' the smallest, is reached by 8 j >= k tokens.  Where the buffer fills, it
// is cut to its k largest (a key's place is the number of keys above it), and the
// k-th becomes the threshold; so most batches only compare their maximum with it.
//
// Work split.  A row is cut into batches that each lie in one rank's shard, and a
// CTA takes a run of them (a whole row, where rows fill the GPU): nothing is
// exchanged but 16 bytes and k keys a run, joined by the CTA that comes last.
// Bound by reading the logits once.
#include "comm.h"
#include "kv4.cuh"

namespace dcc {

constexpr int kLpThreads = 256, kLpWarps = kLpThreads / 32;
constexpr int kLpCap = 1024;      // keys of the buffer
constexpr int kLpCut = 192;       // keys after a batch from which the buffer is cut
constexpr int kLpMaxRuns = 1216;  // CTAs of a call whose rows are cut (8 to an SM)

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
  int n, columns, vocab, top, runs, batches /* of a rank's shard */, span /* vectors of a batch */;
  float scale;
};

template <typename T>
struct LpVec;  // the numbers of 16 bytes
template <>
struct LpVec<float> {
  static constexpr int N = 4;
  __device__ static void widen(uint4 v, float* f) {
    f[0] = __uint_as_float(v.x), f[1] = __uint_as_float(v.y), f[2] = __uint_as_float(v.z), f[3] = __uint_as_float(v.w);
  }
};
template <typename T16>
struct LpVec16 {
  static constexpr int N = 8;
  __device__ static void widen(uint4 v, float* f) {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 p = Half16<T16>::widen2(u[i]);
      f[2 * i] = p.x, f[2 * i + 1] = p.y;
    }
  }
};
template <>
struct LpVec<__half> : LpVec16<__half> {};
template <>
struct LpVec<__nv_bfloat16> : LpVec16<__nv_bfloat16> {};
template <typename T>
struct LpNegInf {
  static constexpr uint32_t word = std::is_same<T, float>::value ? 0xff800000u
                                   : std::is_same<T, __half>::value ? 0xfc00fc00u : 0xff80ff80u;
};

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

struct LpTop {
  unsigned long long keys[2][kLpCap];
  unsigned long long thr;
  uint32_t est[kLpWarps];
  int count, now;  // keys in buffer `now`
};
// Cuts the buffer to its k largest keys, in descending order, and raises the
// threshold to the k-th.  All threads call; the buffer is theirs before and after.
__device__ __forceinline__ void lp_cut(LpTop& s, int k) {
  const int n = min(s.count, kLpCap), now = s.now;
  const unsigned long long* from = s.keys[now];
  unsigned long long* to = s.keys[now ^ 1];
  for (int i = threadIdx.x; i < n; i += kLpThreads) {
    const unsigned long long key = from[i];
    int above = 0;
#pragma unroll 4
    for (int j = 0; j < n; ++j) above += from[j] > key;
    if (above < k) to[above] = key;
    if (above == k - 1) s.thr = key;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    s.count = min(n, k);
    s.now = now ^ 1;
  }
  __syncthreads();
}
__device__ __forceinline__ bool lp_add(LpTop& s, unsigned long long key) {
  const int at = atomicAdd(&s.count, 1);
  if (at < kLpCap) s.keys[s.now][at] = key;
  return at < kLpCap;
}

template <typename T, int VPT>
__global__ void __launch_bounds__(kLpThreads, 4) k_token_logprobs(const __grid_constant__ LpArgs a) {
  constexpr int E = LpVec<T>::N;
  __shared__ LpTop s;
  __shared__ LpSum s_sum[kLpWarps];
  __shared__ int s_last;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, k = a.top;
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
  uint4 next[VPT];
  // a batch's 16-byte vectors; what does not belong to the row is -infinity
  auto fetch = [&](int b) {
    const int rank = b / a.batches, v0 = (b - rank * a.batches) * a.span;
    const T* p = static_cast<const T*>(a.x[rank]) + (size_t)row * a.stride;
    const int before = (int)((reinterpret_cast<uintptr_t>(p) & 15u) / sizeof(T));  // of the first vector, not the row's
    const int valid = max(0, min(a.columns, a.vocab - rank * a.columns));
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = i * kLpThreads + (int)threadIdx.x, e0 = (v0 + v) * E - before;
      uint4 w = make_uint4(LpNegInf<T>::word, LpNegInf<T>::word, LpNegInf<T>::word, LpNegInf<T>::word);
      if (v < a.span && e0 < valid && e0 + E > 0) {
        if (e0 >= 0 && e0 + E <= valid) {
          w = __ldcs(reinterpret_cast<const uint4*>(p + e0));
        } else {
          uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int e = 0; e < E; ++e)
            if (e0 + e >= 0 && e0 + e < valid) {
              if constexpr (sizeof(T) == 4) {
                u[e] = __ldg(reinterpret_cast<const uint32_t*>(p) + e0 + e);
              } else {
                const uint32_t h = __ldg(reinterpret_cast<const uint16_t*>(p) + e0 + e);
                u[e / 2] = e & 1 ? (u[e / 2] & 0xffffu) | h << 16 : (u[e / 2] & 0xffff0000u) | h;
              }
            }
          w = make_uint4(u[0], u[1], u[2], u[3]);
        }
      }
      next[i] = w;
    }
  };
  if (b0 < b1) fetch(b0);
  for (int b = b0; b < b1; ++b) {
    uint4 v[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) v[i] = next[i];
    if (b + 1 < b1) fetch(b + 1);
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      float f[E];
      LpVec<T>::widen(v[i], f);
#pragma unroll
      for (int e = 0; e < E; ++e) top = fmaxf(top, f[e]);
    }
    // sums
    const float m = fmaxf(sum.m, top), ref = m == -INFINITY ? 0.0f : m;
    if (m > sum.m) {
      const float d = sum.m == -INFINITY ? 0.0f : (sum.m - m) * c, f = lp_exp2(d);
      sum.u = f * fmaf(fmaxf(d, -1000.0f), sum.z, sum.u);
      sum.z *= f;
      sum.m = m;
    }
    float z0 = 0.0f, z1 = 0.0f, u0 = 0.0f, u1 = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      float f[E];
      LpVec<T>::widen(v[i], f);
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        const float da = (f[e] - ref) * c, db = (f[e + 1] - ref) * c, pa = lp_exp2(da), pb = lp_exp2(db);
        z0 += pa;
        z1 += pb;
        u0 = fmaf(pa, fmaxf(da, -1000.0f), u0);  // (0 times infinity)
        u1 = fmaf(pb, fmaxf(db, -1000.0f), u1);
      }
    }
    sum.z += z0 + z1;
    sum.u += u0 + u1;
    if (k == 0) continue;
    // top alternatives
    const int rank = b / a.batches, v0 = (b - rank * a.batches) * a.span;
    const int before =
        (int)((reinterpret_cast<uintptr_t>(static_cast<const T*>(a.x[rank]) + (size_t)row * a.stride) & 15u) / sizeof(T));
    const int valid = max(0, min(a.columns, a.vocab - rank * a.columns));
    if (b == b0) {
      const int j = (k + kLpWarps - 1) / kLpWarps;
      bool some = false;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int x = i * kLpThreads + (int)threadIdx.x, e0 = (v0 + x) * E - before;
        some |= x < a.span && e0 < valid && e0 + E > 0;
      }
      uint32_t mine = some ? lp_order(top) : 0u, best = 0u;
      for (int i = 0; i < j; ++i) {
        best = __reduce_max_sync(0xffffffffu, mine);
        const unsigned who = __ballot_sync(0xffffffffu, mine == best);
        if (lane == __ffs(who) - 1) mine = 0u;
      }
      if (lane == 0) s.est[warp] = best;
      __syncthreads();
      if (threadIdx.x == 0) {
        uint32_t least = 0xffffffffu;
        int warps = 0;
        for (int w = 0; w < kLpWarps; ++w)
          if (s.est[w]) {
            least = min(least, s.est[w]);
            ++warps;
          }
        if (warps * j >= k) s.thr = ((unsigned long long)least << 32) - 1;  // least > 0
      }
      __syncthreads();
    }
    unsigned long long thr = s.thr;
    uint32_t pending = 0;
    if (lp_order(top) >= (uint32_t)(thr >> 32)) {
      const float least = lp_value((uint32_t)(thr >> 32));
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        float f[E];
        LpVec<T>::widen(v[i], f);
#pragma unroll
        for (int e = 0; e < E; ++e)
          if (!(f[e] < least)) pending |= 1u << (i * E + e);
      }
    }
    // the places of pending tokens go down as they are added; where the buffer is
    // full it is cut, and those that are left try again
    bool again;
    do {
      thr = s.thr;
      __syncthreads();  // all have read it, and the count after the last batch
      while (pending) {
        const int x = __ffs(pending) - 1, i = x / E, e = x % E;
        uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
        for (int y = 0; y < VPT; ++y)
          if (y == i) w[0] = v[y].x, w[1] = v[y].y, w[2] = v[y].z, w[3] = v[y].w;
        float f;
        if constexpr (sizeof(T) == 4) {
          f = __uint_as_float(e == 0 ? w[0] : e == 1 ? w[1] : e == 2 ? w[2] : w[3]);
        } else {
          const uint32_t p = e < 2 ? w[0] : e < 4 ? w[1] : e < 6 ? w[2] : w[3];
          f = Half16<T>::widen((uint16_t)(e & 1 ? p >> 16 : p));
        }
        const int q = i * kLpThreads + (int)threadIdx.x, col = (v0 + q) * E - before + e;
        if (q < a.span && col >= 0 && col < valid) {
          const unsigned long long key = lp_key(f, (uint32_t)(rank * a.columns + col));
          if (key > thr && !lp_add(s, key)) break;
        }
        pending &= pending - 1;
      }
      again = __syncthreads_or(pending != 0);
      if (again || s.count > kLpCut) lp_cut(s, k);
    } while (again);
  }

  // ---- the CTA's sums
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const LpSum other = {__shfl_xor_sync(0xffffffffu, sum.m, o), __shfl_xor_sync(0xffffffffu, sum.z, o),
                         __shfl_xor_sync(0xffffffffu, sum.u, o)};
    sum = lane & o ? lp_join(other, sum, c) : lp_join(sum, other, c);
  }
  if (lane == 0) s_sum[warp] = sum;
  if (k) {
    __syncthreads();
    lp_cut(s, k);
  }
  __syncthreads();
  sum = s_sum[0];
#pragma unroll
  for (int w = 1; w < kLpWarps; ++w) sum = lp_join(sum, s_sum[w], c);

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
    for (int i = 0; i < a.runs; ++i) {
      const float4 p = __ldcg(&a.sums[(size_t)row * a.runs + i]);
      sum = lp_join(sum, LpSum{p.x, p.y, p.z}, c);
    }
    if (k) {
      const unsigned long long* keys = a.keys + (size_t)row * a.runs * k;
      if (threadIdx.x == 0) {
        s.count = 0;
        s.thr = 0;
      }
      __syncthreads();
      // k tokens reach the largest of the runs' k-th keys
      for (int i = threadIdx.x; i < a.runs; i += kLpThreads) {
        const unsigned long long last = __ldcg(keys + (size_t)i * k + k - 1);
        if (last) atomicMax(&s.thr, last - 1);
      }
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
        const T* p = static_cast<const T*>(a.x[rank]) + (size_t)row * a.stride + (t - rank * a.columns);
        float x;
        if constexpr (sizeof(T) == 4) x = __ldg(reinterpret_cast<const float*>(p));
        else x = Half16<T>::widen(__ldg(reinterpret_cast<const uint16_t*>(p)));
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
  if (!logits || !workspace || workspace_bytes < need || !(scale > 0.0f) || !(scale - scale == 0.0f))
    return DCC_ERR_INVALID_ARG;
  if ((logprob != nullptr) != (target != nullptr) || (top > 0 && (!top_ids || !top_logprob)) ||
      (top == 0 && (top_ids || top_logprob)) || (!logprob && !entropy && top == 0))
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
  // A shard's vectors, and one more where rows do not begin on one.  Batches are
  // four vectors a thread, or one where the GPU would not be full otherwise.
  const long long vectors = (long long)((columns * size + 15) / 16 + 1);
  const long long runs_wanted = dcc::kLpMaxRuns / (long long)tokens;  // of a row
  const auto batches = [&](int per) { return (vectors + per * dcc::kLpThreads - 1) / (per * dcc::kLpThreads); };
  const int per = n_ranks * batches(4) < runs_wanted ? 1 : 4;
  a.batches = (int)batches(per);
  a.span = (int)((vectors + a.batches - 1) / a.batches);
  const long long all = (long long)n_ranks * a.batches;
  a.runs = (int)(runs_wanted < 1 ? 1 : runs_wanted < all ? runs_wanted : all);
  const int type = t == DCC_FP32 ? 0 : t == DCC_FP16 ? 1 : 2;
  void* args[] = {&a};
  return dcc_host::launch(dcc::logprobs_kernel(2 * type + (per == 1)), (int)((long long)tokens * a.runs), dcc::kLpThreads,
                          false, args, static_cast<cudaStream_t>(s), 0, true);
}

}  // extern "C"
