// kv4_plan.h -- which kernel an attention call over the 4-bit cache launches,
// from what the host knows (no CUDA in here).
//
// Two kernels.  The prompt kernel keeps the tensor cores busy but does not split
// a segment's keys over CTAs; the streaming kernel spreads any work evenly but
// goes over the cache once per row tile.  Per key, on GB300: a wave of the prompt
// kernel takes 0.017 us, a pass of the streaming kernel over one segment
// 5.6e-5 us, a 300th; with few pages its latency shows and it is a 100th.
// (Segments: ranks x kv heads x sequences.)  Measured, streaming / prompt, us, 8
// heads per kv head of 128 channels: 8 segments of 8192 keys, 64 tokens 121 / 154,
// 128 tokens 224 / 154; 1 segment of 60,000 keys, 128 tokens 200 / 1027; 128
// segments of up to 4096 keys, 4 tokens 68 / 75, 8 tokens 115 / 75, 128 tokens
// 1876 / 235; 8 segments of 700 keys x 4 heads, 64 tokens 29.8 / 29.5, 128 tokens
// 43 / 30.
//
// The lengths are on the device, and a slot may be idle or bring one token
// beside another's chunk, so slots are not counted: `tokens` rows of which no
// sequence has more than max_new are at most as much work as tokens / max_new
// sequences of max_new rows each.
#pragma once

namespace dcc {

constexpr int kPromptRows = 256;  // per CTA of the prompt kernel: two tiles of 128
constexpr int kDecSmallWarps = 4;

struct AttnPlan {
  bool prompt;
  // prompt kernel: tiles of 256 rows of each slot, then of 128
  long long wide, narrow;
  // streaming kernel: row tiles of 8, or its small form
  int tiles;
  bool small;
};

// Row tiles of the streaming kernel: as few passes over the cache as the registers
// allow, then the fewest rows that make that many.
inline void stream_plan(AttnPlan* p, long long n_heads, long long seqs, long long max_pages, int dim, long long rows,
                        long long sms) {
  const long long most = dim == 64 ? 3 : 2, times = (rows + 8 * most - 1) / (8 * most);
  p->tiles = (int)((rows + 8 * times - 1) / (8 * times));
  p->small = rows <= 8 && n_heads * seqs * max_pages <= sms * kDecSmallWarps;
}

// Rows with sets of seen keys of their own (trees, windows with sinks).  Their
// kernel of many rows splits any call evenly over the SMs, so what counts is how
// often the streaming kernel goes over the keys: once, it is the faster one; twice,
// it is where an SM has more than some 16 steps of 128 keys (the other's start
// and joins no longer show); three times, never.  Measured, streaming / other, us, 8
// heads per kv head: 128 channels, 32 rows, 8 x 700 keys (segments x keys) 20.7 /
// 17.5, 8 x 8192 32.9 / 30.7, 128 x 2048 65 / 61, 512 x 4096 254 / 312, 8 x 65,536 75
// / 84; 48 rows (three times) 23.0 / 17.8, 34.8 / 32.4, 87 / 62, 370 / 315, 102 / 87.
// 64 channels, 48 rows, the same: 19.4 / 13.6, 29.3 / 22.7, 53 / 43, 194 / 218, 58 / 63.
inline AttnPlan seen_plan(long long n_heads, long long seqs, long long max_pages, int dim, long long share, long long tokens,
                          long long max_new, long long window, long long sinks, long long sms) {
  AttnPlan p = {};
  const long long rows = max_new * share, tile = dim == 64 ? 24 : 16, passes = (rows + tile - 1) / tile;
  long long full = (tokens + max_new - 1) / max_new, pages = max_pages;  // sequences, as below
  if (full > seqs) full = seqs;
  if (window > 0 && (window + sinks + max_new) / 64 + 1 < pages) pages = (window + sinks + max_new) / 64 + 1;
  p.prompt = passes > 2 || (passes == 2 && n_heads * full * pages <= 32 * sms);
  if (!p.prompt) stream_plan(&p, n_heads, seqs, max_pages, dim, rows, sms);
  return p;
}

inline AttnPlan attn_plan(long long n_heads /* ranks x kv heads */, long long seqs, long long max_pages, int dim,
                          long long share, long long tokens, long long max_new, long long sms) {
  AttnPlan p = {};
  const long long rows = max_new * share, tile = dim == 64 ? 24 : 16, passes = (rows + tile - 1) / tile;
  long long full = (tokens + max_new - 1) / max_new;
  if (full > seqs) full = seqs;
  const long long segments = n_heads * full;
  long long wide = (rows + kPromptRows - 1) / kPromptRows;
  const long long waves = (segments * wide + sms - 1) / sms;
  p.prompt = rows > 16 && segments * passes > (max_pages <= 32 ? 100 : 300) * waves;
  if (p.prompt) {
    // whole waves of 256-row tiles; what is left in 128-row tiles if they fit one
    // wave.  Here slots count: each has a CTA for every tile that it may have.
    const long long slots = n_heads * seqs;
    const long long whole = slots * wide / sms * sms / slots, left = (rows - whole * kPromptRows + 127) / 128;
    if (whole < wide && slots * left <= sms) {
      wide = whole;
      p.narrow = left;
    }
    p.wide = wide;
    return p;
  }
  stream_plan(&p, n_heads, seqs, max_pages, dim, rows, sms);
  return p;
}

}  // namespace dcc
