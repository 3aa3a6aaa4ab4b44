// kv4_attention_fp16.cu -- the attention's kernels over fp16 caches.
#include "kv4_attention.cuh"

namespace dcc {
AttnKernel attn_kernel_fp16(int dim, int group, int which) { return attn_kernel_for<__half>(dim, group, which); }
}  // namespace dcc
