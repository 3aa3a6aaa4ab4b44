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

}  // namespace dcc
