// kv4_attention.cu -- host side of the attention over the 4-bit cache.
#include "comm.h"
#include "kv4_attention.cuh"

namespace dcc {
AttnKernel attn_kernel(bool fp16, bool seen, int dim, int group, int which) {
  if (seen) return fp16 ? attn_seen_kernel_fp16(dim, group, which) : attn_seen_kernel_bf16(dim, group, which);
  return fp16 ? attn_kernel_fp16(dim, group, which) : attn_kernel_bf16(dim, group, which);
}
const void* kv4_attention_kernel(bool fp16, bool seen, int dim, int group, int which) {
  return attn_kernel(fp16, seen, dim, group, which).fn;
}
}  // namespace dcc

namespace {

// What the three calls share.  Of a tree: mask, `words` to a row; else null and 0.
int attention_call(const dcc_kv4_t* kv, int layer, void* const* q, void* const* out, float* const* lse, int q_heads,
                   size_t tokens, size_t q_stride, const int32_t* start, int max_new, bool tree, const uint32_t* mask,
                   int words, float scale, int window, int sinks, void* workspace, size_t workspace_bytes, dcc_stream_t s);

}  // namespace

extern "C" {

int dcc_kv4_attention_workspace(const dcc_kv4_t* kv, int q_heads, size_t* bytes) {
  if (!kv || !bytes || q_heads < 1 || kv->kv_heads < 1 || q_heads % kv->kv_heads) return DCC_ERR_INVALID_ARG;
  const size_t seen = dcc::seen_ws_bytes(kv->head_dim), dec = dcc::dec_ws_bytes();
  *bytes = seen > dec ? seen : dec;
  return DCC_OK;
}

int dcc_kv4_attention(const dcc_kv4_t* kv, int layer, void* const* q, void* const* out, float* const* lse, int q_heads,
                      size_t tokens, size_t q_stride, const int32_t* start, int max_new, float scale, int window,
                      void* workspace, size_t workspace_bytes, dcc_stream_t s) {
  return attention_call(kv, layer, q, out, lse, q_heads, tokens, q_stride, start, max_new, false, nullptr, 0, scale, window,
                        0, workspace, workspace_bytes, s);
}

int dcc_kv4_attention_sinks(const dcc_kv4_t* kv, int layer, void* const* q, void* const* out, float* const* lse,
                            int q_heads, size_t tokens, size_t q_stride, const int32_t* start, int max_new, float scale,
                            int window, int sinks, void* workspace, size_t workspace_bytes, dcc_stream_t s) {
  return attention_call(kv, layer, q, out, lse, q_heads, tokens, q_stride, start, max_new, false, nullptr, 0, scale, window,
                        sinks, workspace, workspace_bytes, s);
}

int dcc_kv4_attention_tree(const dcc_kv4_t* kv, int layer, void* const* q, void* const* out, float* const* lse,
                           int q_heads, size_t tokens, size_t q_stride, const int32_t* start, int max_new,
                           const uint32_t* mask, int mask_words, float scale, int window, int sinks, void* workspace,
                           size_t workspace_bytes, dcc_stream_t s) {
  return attention_call(kv, layer, q, out, lse, q_heads, tokens, q_stride, start, max_new, true, mask, mask_words, scale,
                        window, sinks, workspace, workspace_bytes, s);
}

}  // extern "C"

namespace {

int attention_call(const dcc_kv4_t* kv, int layer, void* const* q, void* const* out, float* const* lse, int q_heads,
                   size_t tokens, size_t q_stride, const int32_t* start, int max_new, bool tree, const uint32_t* mask,
                   int words, float scale, int window, int sinks, void* workspace, size_t workspace_bytes, dcc_stream_t s) {
  dcc::Kv4Dev d{};
  int rc = dcc_host::kv4_view(kv, false, &d);
  if (rc != DCC_OK) return rc;
  if (!q || !out || !start || !workspace || layer < 0 || layer >= kv->layers || q_heads < 1 || max_new < 1 ||
      window < 0 || sinks < 0 || !(scale - scale == 0.0f))
    return DCC_ERR_INVALID_ARG;
  if (q_heads % kv->kv_heads || q_heads / kv->kv_heads > 128) return DCC_ERR_INVALID_ARG;
  // positions stay below 2^30 (kv4_view), so a window that long hides nothing;
  // kept, position - window + 1 would leave 32 bits for rows before position zero
  if (window >= 1 << 30) window = 0;
  if (window == 0) sinks = 0;
  const bool seen = tree || sinks > 0;  // else causal rows, one run of keys each
  size_t need = dcc::dec_ws_bytes();
  if (seen && (rc = dcc_kv4_attention_workspace(kv, q_heads, &need)) != DCC_OK) return rc;
  if (workspace_bytes < need) return DCC_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(start) & 3u) || (reinterpret_cast<uintptr_t>(workspace) & 15u) || q_stride % 8)
    return DCC_ERR_MISALIGNED;
  const size_t width = (size_t)q_heads * kv->head_dim;
  if (tokens > (size_t)1 << 26 || q_stride > (size_t)1 << 32 || (tokens > 1 && q_stride < width))
    return DCC_ERR_INVALID_ARG;
  if (tokens * (size_t)(q_heads / kv->kv_heads) > (size_t)1 << 30) return DCC_ERR_INVALID_ARG;  // rows are 32-bit
  if (tree) {
    // a row's words hold all of its sequence's drafted tokens that rows of this call stand for
    if ((!mask && tokens) || words < 1 || words > dcc::kTreeWords) return DCC_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(mask) & 3u) return DCC_ERR_MISALIGNED;
    if (((size_t)max_new < tokens ? (size_t)max_new : tokens) > (size_t)words * 32) return DCC_ERR_INVALID_ARG;
  }
  if (tokens == 0) return DCC_OK;
  if ((size_t)max_new > tokens) max_new = (int)tokens;
  const size_t qb = ((tokens - 1) * q_stride + width) * 2, ob = tokens * width * 2, lb = tokens * q_heads * 4;
  const size_t pool = (size_t)kv->layers * kv->pages * kv->kv_heads * dcc::kv4_block_bytes(kv->head_dim, kv->group);
  dcc::AttnArgs a{};
  for (int r = 0; r < kv->n_ranks; ++r) {
    if (!q[r] || !out[r] || (lse && !lse[r])) return DCC_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(q[r]) | reinterpret_cast<uintptr_t>(out[r])) & 15u) return DCC_ERR_MISALIGNED;
    if (lse && (reinterpret_cast<uintptr_t>(lse[r]) & 3u)) return DCC_ERR_MISALIGNED;
    for (int p = 0; p < kv->n_ranks; ++p) {
      if (dcc_host::overlaps(out[r], ob, q[p], qb) || dcc_host::overlaps(out[r], ob, kv->pool[p], pool) ||
          (p < r && dcc_host::overlaps(out[r], ob, out[p], ob)))
        return DCC_ERR_INVALID_ARG;
      if (lse && (dcc_host::overlaps(lse[r], lb, q[p], qb) || dcc_host::overlaps(lse[r], lb, kv->pool[p], pool) ||
                  dcc_host::overlaps(lse[r], lb, out[p], ob) || (p < r && dcc_host::overlaps(lse[r], lb, lse[p], lb))))
        return DCC_ERR_INVALID_ARG;
    }
    // the small buffers of the call, against what it writes (and the workspace against all)
    const size_t table = (size_t)kv->seqs * kv->max_pages * 4, seqs = (size_t)kv->seqs * 4;
    const dcc_host::Extent e[] = {{workspace, need, true},   {out[r], ob, true},       {lse ? lse[r] : nullptr, lb, true},
                                  {q[r], qb, false},         {kv->pool[r], pool, false}, {kv->table, table, false},
                                  {kv->len, seqs, false},    {start, seqs + 4, false}, {mask, tokens * words * 4, false}};
    if (!dcc_host::disjoint(e, 9)) return DCC_ERR_INVALID_ARG;
    a.q[r] = q[r];
    a.out[r] = out[r];
    a.lse[r] = lse ? lse[r] : nullptr;
  }
  a.start = start;
  a.q_stride = q_stride;
  a.tokens = (int)tokens;
  a.layer = layer;
  a.q_heads = q_heads;
  a.max_new = max_new;
  a.window = window;
  a.sinks = sinks < (1 << 30) ? sinks : 1 << 30;
  a.mask = mask;
  a.words = words;
  a.scale = scale;
  a.share = q_heads / kv->kv_heads;
  a.ws = static_cast<char*>(workspace);
  a.timeout_ns = 2000000000ull;
  if ((rc = dcc_host::kv4_ready(&d)) != DCC_OK) return rc;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return DCC_ERR_CUDA;
  }
  const bool fp16 = kv->dtype == DCC_FP16;
  cudaStream_t st = static_cast<cudaStream_t>(s);
  const long long heads = (long long)kv->n_ranks * kv->kv_heads;
  dcc::AttnPlan p = {};
  if (seen)
    p = dcc::seen_plan(heads, kv->seqs, kv->max_pages, kv->head_dim, a.share, (long long)tokens, max_new, a.window, a.sinks, sms);
  else
    p = dcc::attn_plan(heads, kv->seqs, kv->max_pages, kv->head_dim, a.share, (long long)tokens, max_new, sms);
  if (p.prompt) {
    const dcc::AttnKernel k = dcc::attn_kernel(fp16, seen, kv->head_dim, kv->group, dcc::kAttnPrompt);
    if (dcc_host::max_active_per_sm(k.fn, k.threads, k.smem) < 1) return DCC_ERR_LAUNCH;
    if (seen) {
      int ctas = sms < dcc::kDecMaxCtas ? sms : dcc::kDecMaxCtas;
      dcc::LocalDev dc = dcc_host::local_dev(d.status);
      void* args[] = {&d, &a, &dc};
      rc = dcc_host::launch(k.fn, ctas, k.threads, false, args, st, k.smem, true);
      if (rc != DCC_OK) return rc;
      const dcc::AttnKernel j = dcc::attn_kernel(fp16, true, kv->head_dim, kv->group, dcc::kAttnJoin);
      void* join[] = {&a, &ctas};
      return dcc_host::launch(j.fn, 3 * ctas, j.threads, false, join, st, 0, true);
    }
    if (p.wide > (1 << 24)) return DCC_ERR_INVALID_ARG;
    a.wide = (int)p.wide;
    const long long grid = (p.wide + p.narrow) * heads * kv->seqs;
    if (grid > 0x7fffffffll) return DCC_ERR_INVALID_ARG;
    dcc::LocalDev dc = dcc_host::local_dev(d.status);
    void* args[] = {&d, &a, &dc};
    return dcc_host::launch(k.fn, (int)grid, k.threads, false, args, st, k.smem, true);
  }
  const dcc::AttnKernel k = dcc::attn_kernel(fp16, seen, kv->head_dim, kv->group, p.small ? dcc::kAttnSmall : p.tiles);
  if (dcc_host::max_active_per_sm(k.fn, k.threads, k.smem) < 1) return DCC_ERR_LAUNCH;
  void* args[] = {&d, &a};
  return dcc_host::launch(k.fn, sms < dcc::kDecMaxCtas ? sms : dcc::kDecMaxCtas, k.threads, false, args, st, k.smem,
                          true);
}

}  // namespace
