// linear.cuh -- the column-parallel linear layer: matrix product with bias,
// activation and residual in its epilogue.
#pragma once
#include "kv4.cuh"

namespace dcc {

struct LinArgs {
  const void* w[DCC_MAX_RANKS];     // rows x k
  const void* x[DCC_MAX_RANKS];     // tokens x k
  const void* bias[DCC_MAX_RANKS];  // rows, all or none
  const void* res[DCC_MAX_RANKS];   // tokens x rows, all or none
  void* y[DCC_MAX_RANKS];           // tokens x rows
  int n, tokens, rows, k, act;
};

// The activation of one fp32 sum.
__device__ __forceinline__ float lin_act(float z, int act) {
  switch (act) {
    case DCC_ACT_RELU: return z > 0.0f ? z : (z - z == 0.0f || z < 0.0f ? 0.0f : z);  // NaN stays
    case DCC_ACT_GELU: return 0.5f * z * (1.0f + erff(z * 0.70710678118654752f));
    case DCC_ACT_GELU_TANH: return 0.5f * z * (1.0f + tanhf(0.79788456080286536f * (z + 0.044715f * z * z * z)));
    case DCC_ACT_SILU: return __fdiv_rn(z, 1.0f + expf(-z));
    default: return z;
  }
}

constexpr int kLinThreads = 256;

// One warp per (rank, row, 8 tokens); lanes along k.
template <typename T>
__global__ void __launch_bounds__(kLinThreads) k_linear(LinArgs a) {
  pdl_prologue();
  const int lane = threadIdx.x & 31;
  const long long item = (long long)blockIdx.x * (kLinThreads / 32) + (threadIdx.x >> 5);
  const int tiles = (a.tokens + 7) / 8;
  const int row = (int)(item % a.rows), rank = (int)(item / a.rows / tiles), t0 = (int)(item / a.rows % tiles) * 8;
  if (rank >= a.n) return;
  const T* w = static_cast<const T*>(a.w[rank]) + (size_t)row * a.k;
  float acc[8] = {};
  for (int k0 = lane * 8; k0 < a.k; k0 += 256) {
    const uint4 wv = *reinterpret_cast<const uint4*>(w + k0);
    const uint32_t wu[4] = {wv.x, wv.y, wv.z, wv.w};
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      if (t0 + t >= a.tokens) break;
      const uint4 xv = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.x[rank]) + (size_t)(t0 + t) * a.k + k0);
      const uint32_t xu[4] = {xv.x, xv.y, xv.z, xv.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 p = Half16<T>::widen2(wu[j]), q = Half16<T>::widen2(xu[j]);
        acc[t] = fmaf(p.x, q.x, acc[t]);
        acc[t] = fmaf(p.y, q.y, acc[t]);
      }
    }
  }
#pragma unroll
  for (int t = 0; t < 8; ++t) {
    for (int m = 16; m; m >>= 1) acc[t] += __shfl_xor_sync(0xffffffffu, acc[t], m);
    if (lane == t && t0 + t < a.tokens) {
      float z = acc[t];
      if (a.bias[0]) z += Half16<T>::widen(static_cast<const uint16_t*>(a.bias[rank])[row]);
      z = lin_act(z, a.act);
      const size_t o = (size_t)(t0 + t) * a.rows + row;
      if (a.res[0]) z += Half16<T>::widen(static_cast<const uint16_t*>(a.res[rank])[o]);
      static_cast<uint16_t*>(a.y[rank])[o] = Half16<T>::narrow(z);
    }
  }
}

}  // namespace dcc
