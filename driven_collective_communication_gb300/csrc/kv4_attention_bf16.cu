// kv4_attention_bf16.cu -- the attention's kernels over bf16 caches.
#include "kv4_attention.cuh"

namespace dcc {
AttnKernel attn_kernel_bf16(int dim, int group, int which) { return attn_kernel_for<__nv_bfloat16>(dim, group, which); }
}  // namespace dcc
