// kv4_attention.cuh -- the attention's kernels by type, head size and group; the
// two types compile in a unit each (kv4_attention_bf16.cu, kv4_attention_fp16.cu),
// and so do those for rows with sets of seen keys of their own (kv4_seen_*.cu).
#pragma once
#include "kv4_seen.cuh"

namespace dcc {

struct AttnKernel {
  const void* fn;
  int threads;
  size_t smem;
};
// which: 1 to 3 row tiles of the streaming kernel (3: 64-wide heads only), its
// small form, the prompt kernel, or what joins its parts (SEEN)
constexpr int kAttnPrompt = 0, kAttnSmall = 4, kAttnJoin = 5;
AttnKernel attn_kernel_bf16(int dim, int group, int which);
AttnKernel attn_kernel_fp16(int dim, int group, int which);
AttnKernel attn_seen_kernel_bf16(int dim, int group, int which);
AttnKernel attn_seen_kernel_fp16(int dim, int group, int which);

template <typename T, int D, int G, bool SEEN>
AttnKernel attn_kernel_of(int which) {
  auto decode = [](auto tiles, auto small) {
    constexpr int RT = decltype(tiles)::value;
    constexpr bool SMALL = decltype(small)::value;
    using S = DecShape<D, G, RT, SMALL>;
    return AttnKernel{(const void*)&k_kv4_decode<T, D, G, RT, SMALL, SEEN>, S::warps * 32, S::smem};
  };
  using No = std::false_type;
  switch (which) {
    case kAttnPrompt:
      if constexpr (SEEN) return {(const void*)&k_kv4_seen<T, D, G>, kPromptThreads, kSeenSmem<T, D, G>};
      else return {(const void*)&k_kv4_prompt<T, D, G>, kPromptThreads, PromptShape<D, G>::smem};
    case kAttnJoin:
      if constexpr (SEEN) return {(const void*)&k_kv4_seen_join<T, D>, kSeenJoinThreads, 0};
      else return {};
    case kAttnSmall: return decode(std::integral_constant<int, 1>{}, std::true_type{});
    case 1: return decode(std::integral_constant<int, 1>{}, No{});
    default: break;
  }
  if constexpr (D == 64)  // 24 rows: 64-wide heads have the registers
    if (which == 3) return decode(std::integral_constant<int, 3>{}, No{});
  return decode(std::integral_constant<int, 2>{}, No{});
}
template <typename T, bool SEEN = false>
AttnKernel attn_kernel_for(int dim, int group, int which) {
  if (dim == 128) return group == 64 ? attn_kernel_of<T, 128, 64, SEEN>(which) : attn_kernel_of<T, 128, 32, SEEN>(which);
  return group == 64 ? attn_kernel_of<T, 64, 64, SEEN>(which) : attn_kernel_of<T, 64, 32, SEEN>(which);
}

}  // namespace dcc
