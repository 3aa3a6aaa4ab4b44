// linear.cu -- host side of the column-parallel linear layer.
#include "comm.h"
#include "linear.cuh"

namespace dcc {
const void* linear_kernel(bool fp16) {
  return fp16 ? (const void*)&k_linear<__half> : (const void*)&k_linear<__nv_bfloat16>;
}
}  // namespace dcc

extern "C" int dcc_linear(int n_ranks, void* const* weight, void* const* x, void* const* bias, void* const* residual,
                          void* const* y, size_t tokens, size_t rows, size_t k, dcc_act_t act, dcc_dtype_t t,
                          dcc_stream_t s) {
  if (n_ranks < 1 || n_ranks > DCC_MAX_RANKS || !weight || !x || !y) return DCC_ERR_INVALID_ARG;
  if ((int)act < DCC_ACT_NONE || (int)act > DCC_ACT_SILU) return DCC_ERR_INVALID_ARG;
  if (t != DCC_BF16 && t != DCC_FP16) return DCC_ERR_UNSUPPORTED;
  if (rows % 8 || k % 8) return DCC_ERR_UNSUPPORTED;  // the documented shape rule
  if (tokens > (size_t)1 << 26 || rows > (size_t)1 << 26 || k > (size_t)1 << 26) return DCC_ERR_INVALID_ARG;
  if (tokens == 0 || rows == 0) return DCC_OK;
  if (k == 0) return DCC_ERR_INVALID_ARG;
  const size_t wb = rows * k * 2, xb = tokens * k * 2, yb = tokens * rows * 2, bb = rows * 2;
  dcc::LinArgs a{};
  for (int r = 0; r < n_ranks; ++r) {
    if (!weight[r] || !x[r] || !y[r] || (bias && !bias[r]) || (residual && !residual[r])) return DCC_ERR_INVALID_ARG;
    uintptr_t low = reinterpret_cast<uintptr_t>(weight[r]) | reinterpret_cast<uintptr_t>(x[r]) |
                    reinterpret_cast<uintptr_t>(y[r]);
    if (bias) low |= reinterpret_cast<uintptr_t>(bias[r]);
    if (residual) low |= reinterpret_cast<uintptr_t>(residual[r]);
    if (low & 15u) return DCC_ERR_MISALIGNED;
    for (int p = 0; p < n_ranks; ++p) {
      if (dcc_host::overlaps(y[r], yb, weight[p], wb) || dcc_host::overlaps(y[r], yb, x[p], xb) ||
          (p != r && dcc_host::overlaps(y[r], yb, y[p], yb)) || (bias && dcc_host::overlaps(y[r], yb, bias[p], bb)) ||
          (residual && dcc_host::overlaps(y[r], yb, residual[p], yb) && !(p == r && residual[r] == y[r])))
        return DCC_ERR_INVALID_ARG;
    }
    a.w[r] = weight[r];
    a.x[r] = x[r];
    a.bias[r] = bias ? bias[r] : nullptr;
    a.res[r] = residual ? residual[r] : nullptr;
    a.y[r] = y[r];
  }
  a.n = n_ranks;
  a.tokens = (int)tokens;
  a.rows = (int)rows;
  a.k = (int)k;
  a.act = (int)act;
  const long long items = (long long)n_ranks * (long long)rows * (long long)((tokens + 7) / 8);
  const long long grid = (items + dcc::kLinThreads / 32 - 1) / (dcc::kLinThreads / 32);
  if (grid > 0x7fffffffll) return DCC_ERR_INVALID_ARG;
  void* args[] = {&a};
  return dcc_host::launch(dcc::linear_kernel(t == DCC_FP16), (int)grid, dcc::kLinThreads, false, args,
                          static_cast<cudaStream_t>(s), 0, true);
}
