// kv4_seen_fp16.cu -- the attention's kernels over fp16 caches for rows with sets of
// seen keys of their own: trees of drafted tokens, windows with sinks.
#include "kv4_attention.cuh"

namespace dcc {
AttnKernel attn_seen_kernel_fp16(int dim, int group, int which) { return attn_kernel_for<__half, true>(dim, group, which); }
}  // namespace dcc
