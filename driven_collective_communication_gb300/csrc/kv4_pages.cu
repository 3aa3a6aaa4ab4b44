// kv4_pages.cu -- the pages of the 4-bit cache: giving them out, sharing,
// copying, compacting and freeing them.
//
// All bookkeeping is whole numbers in device memory, and the outcome does not
// depend on timing: free pages are taken lowest first and requests are served
// in order, both by prefix sums; reference counts change by atomic adds,
// whose order does not show.
//
// Two kernels.  The first is one CTA, or for large pools one cluster of 8: each
// CTA owns one eighth of the pages (and strides over the sequences), the
// phases are separated by barriers, and the CTAs' totals are exchanged through
// their workspace words -- the scan of the counts is the only long part, and
// eight SMs read them eight times as fast as one, without a launch per phase.
// It is bound by latency, and a cluster's barrier with its fence costs more
// than a CTA's: a fork of 64 beams out of 128 with its copies takes 19 us on
// GB300 with one CTA (a host that issues slowly: up to 25), 27 with the cluster.  It writes the list of page copies to
// the workspace.  The second kernel copies:
// the number of copies is only known on the device, so its CTAs (as many as
// the GPU holds) stride over (copy, rank, layer, chunk), 16 bytes a thread and
// several loads in flight; it is bound by memory (GB300: 0.98 GB read and
// written in 162 us with the books, 6.0 TB/s, 89 % of a plain copy's rate).
#include <initializer_list>

#include "comm.h"
#include "kv4.cuh"

namespace dcc {

constexpr int kBookCtas = 8;       // one portable cluster
constexpr int kBookThreads = 1024;
// Up to this many page counts, and as many table entries to go through, one CTA
// keeps the books: 4 to a thread.
constexpr long long kBookOneCta = 4 * kBookThreads;
constexpr int kCopyThreads = 256;
constexpr int kCopyUnroll = 4;     // 16-byte vectors a thread has in flight

// Workspace, int32 words: totals, then the copies and the lists.
constexpr int kWsWords = 64;
enum { kWsCopies = 0, kWsTotal = 8 /* + 8 j + CTA, j = 0..2 */, kWsFails = 40, kWsFreed = 41 };
struct PagesWs {
  int32_t* w;     // kWsWords
  int32_t* from;  // [pages]: page copied / moved
  int32_t* to;    // [pages]: page it goes to; also the list of free pages given out
  int32_t* mark;  // [seqs]: which request named the sequence first
  int32_t* pre;   // [seqs + 1]: pages wanted before request i
};

enum BookMode { kBookFree = 0, kBookFork = 1, kBookReserve = 2 };
struct BookArgs {
  const int32_t* src;  // fork
  const int32_t* dst;  // fork, free: the sequences given up; reserve: tokens to add
  int count;
  int32_t* info;
  PagesWs ws;
};

template <int CTAS>
__device__ __forceinline__ void book_sync() {  // the whole grid is one CTA or one cluster
  if (CTAS == 1) {
    __syncthreads();
    return;
  }
  __threadfence();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Exclusive prefix sum over the CTA's threads, and the total.
template <typename V>
__device__ __forceinline__ V cta_scan(V v, V* total, V* smem /* 32 */) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  V x = v;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const V y = __shfl_up_sync(0xffffffffu, x, m);
    if (lane >= m) x += y;
  }
  __syncthreads();
  if (lane == 31) smem[warp] = x;
  __syncthreads();
  if (warp == 0) {
    V s = lane < (int)(blockDim.x >> 5) ? smem[lane] : 0;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const V y = __shfl_up_sync(0xffffffffu, s, m);
      if (lane >= m) s += y;
    }
    smem[lane] = s;
  }
  __syncthreads();
  *total = smem[31];
  return x - v + (warp ? smem[warp - 1] : 0);
}
// Sum over the CTA's threads of a value each holds.
__device__ __forceinline__ int cta_sum(int v, int* smem) {
  int total;
  cta_scan(v, &total, smem);
  return total;
}

__device__ __forceinline__ void book_bad(const Kv4Dev& kv, int what) {
  atomicCAS(kv.status, 0ull, kStatusBounds | ((unsigned long long)(uint32_t)what << 32));
}

// The pages this CTA looks after: an equal part of them, in order.
struct Span {
  int b, e;
};
template <int CTAS>
__device__ __forceinline__ Span my_pages(int pages, int cta) {
  return {(int)((long long)pages * cta / CTAS), (int)((long long)pages * (cta + 1) / CTAS)};
}
// Counts are read past L1: other CTAs' atomics change them.
__device__ __forceinline__ int ld_count(const int32_t* p) { return __ldcg(p); }

// Writes the free pages of rank base.. (in ascending page order) below `need`
// to list; base: free pages of the CTAs before this one.
__device__ __forceinline__ void list_free(const Kv4Dev& kv, Span my, int base, int need, int32_t* list, int* smem) {
  for (int p0 = my.b; p0 < my.e && base < need; p0 += kBookThreads) {
    const int p = p0 + (int)threadIdx.x;
    const int f = p < my.e && ld_count(kv.refs + p) == 0 ? 1 : 0;
    int total;
    const int at = base + cta_scan(f, &total, smem);
    if (f && at < need) list[at] = p;
    base += total;
  }
}

// Pages request i asks for: of a fork, one if src holds a partial page; of a
// reservation, those its sequence lacks.  ok: the request can be served at all.
__device__ __forceinline__ int book_want(const Kv4Dev& kv, const BookArgs& a, int mode, int i, bool* ok) {
  if (mode == kBookFork) {
    const int d = a.dst[i], s = a.src[i];
    *ok = d >= 0 && d < kv.seqs && __ldcg(a.ws.mark + d) == i && s >= 0 && s < kv.seqs &&
          __ldcg(a.ws.mark + s) == 0x7fffffff;
    if (!*ok) return 0;
    const int len = kv.len[s];  // no dst: nothing in this kernel changes it
    *ok = len >= 0 && (len + kKv4Page - 1) / kKv4Page <= kv.max_pages;
    return *ok && len % kKv4Page > 0 ? 1 : 0;
  }
  const int len = kv.len[i], add = a.dst[i];
  const long long pages = ((long long)len + (add > 0 ? add : 0) + kKv4Page - 1) / kKv4Page;
  *ok = add <= 0 || (len >= 0 && pages <= kv.max_pages);
  return *ok && add > 0 ? (int)pages - (len + kKv4Page - 1) / kKv4Page : 0;
}

template <int CTAS>
__global__ void __launch_bounds__(kBookThreads) k_kv4_book(Kv4Dev kv, BookArgs a, int mode) {
  __shared__ int smem[32];
  pdl_prologue();
  const int cta = (int)blockIdx.x, tid = cta * kBookThreads + (int)threadIdx.x;
  constexpr int kAll = CTAS * kBookThreads;
  constexpr long long kCap = 1 << 30;
  const PagesWs ws = a.ws;
  const int n_req = mode == kBookReserve ? kv.seqs : a.count;
  const int mp = kv.max_pages;

  for (int i = tid; i < kWsWords; i += kAll) ws.w[i] = 0;
  if (mode != kBookReserve) {
    for (int i = tid; i < kv.seqs; i += kAll) ws.mark[i] = 0x7fffffff;
    book_sync<CTAS>();
    for (int i = tid; i < n_req; i += kAll) {
      const int d = a.dst[i];
      if (d >= 0 && d < kv.seqs) atomicMin(&ws.mark[d], i);
      else book_bad(kv, d);
    }
    book_sync<CTAS>();
    // the dropped sequences give up their pages: one warp per sequence
    int skipped = 0;
    for (int i = tid >> 5; i < n_req; i += kAll / 32) {
      const int d = a.dst[i];
      const bool mine = d >= 0 && d < kv.seqs && __ldcg(ws.mark + d) == i;
      if (!mine) {
        skipped += (threadIdx.x & 31) == 0;
        continue;
      }
      int32_t* row = kv.table + (size_t)d * mp;
      for (int j = threadIdx.x & 31; j < mp; j += 32) {
        const int p = row[j];
        if (p < 0) continue;
        if (p < kv.pages) atomicSub(kv.refs + p, 1);
        else book_bad(kv, d);
        row[j] = -1;
      }
      if ((threadIdx.x & 31) == 0) kv.len[d] = 0;
    }
    if (skipped && mode == kBookFree) atomicAdd(&ws.w[kWsFails], skipped);
  }
  book_sync<CTAS>();

  // free pages, by CTA
  const Span my = my_pages<CTAS>(kv.pages, cta);
  int mine = 0;
  for (int p = my.b + (int)threadIdx.x; p < my.e; p += kBookThreads) mine += ld_count(kv.refs + p) == 0;
  mine = cta_sum(mine, smem);
  if (threadIdx.x == 0) ws.w[kWsTotal + cta] = mine;
  // pages wanted before each request: CTA 0, in 64 bits, capped (a request
  // past the cap is past any pool's end and fails)
  if (mode != kBookFree && cta == 0) {
    __shared__ long long smem64[32];
    long long base = 0;
    for (int i0 = 0; i0 < n_req; i0 += kBookThreads) {
      const int i = i0 + (int)threadIdx.x;
      bool ok;
      const long long want = i < n_req ? book_want(kv, a, mode, i, &ok) : 0;
      long long total;
      const long long at = base + cta_scan(want, &total, smem64);
      if (i < n_req) ws.pre[i] = (int)(at < kCap ? at : kCap);
      base += total;
    }
    if (threadIdx.x == 0) ws.pre[n_req] = (int)(base < kCap ? base : kCap);
  }
  book_sync<CTAS>();
  int nfree = 0, before = 0;
  for (int c = 0; c < CTAS; ++c) {
    const int t = __ldcg(ws.w + kWsTotal + c);
    if (c < cta) before += t;
    nfree += t;
  }
  if (mode == kBookFree) {
    if (tid == 0 && a.info) {
      a.info[0] = nfree;
      a.info[1] = __ldcg(ws.w + kWsFails);
      a.info[2] = 0;
    }
    return;
  }
  const int wanted = __ldcg(ws.pre + n_req);
  list_free(kv, my, before, wanted < nfree ? wanted : nfree, ws.to, smem);
  book_sync<CTAS>();

  // serve the requests: one warp each
  int fails = 0, given = 0;
  for (int i = tid >> 5; i < n_req; i += kAll / 32) {
    const int lane = threadIdx.x & 31;
    bool ok;
    const int want = book_want(kv, a, mode, i, &ok), at = __ldcg(ws.pre + i);
    __syncwarp();  // every lane has read the length that lane 0 changes below
    if (mode == kBookFork && (a.src[i] < 0 || a.src[i] >= kv.seqs)) book_bad(kv, a.src[i]);
    if (!ok || (want && at + want > nfree)) {
      fails += lane == 0;
      continue;
    }
    if (mode == kBookFork) {
      const int d = a.dst[i], s = a.src[i], len = kv.len[s], full = len / kKv4Page;
      const int32_t* from = kv.table + (size_t)s * mp;
      int32_t* row = kv.table + (size_t)d * mp;
      for (int j = lane; j < full; j += 32) {
        const int p = from[j];
        if (p >= 0 && p < kv.pages) atomicAdd(kv.refs + p, 1);
        else book_bad(kv, s);
        row[j] = p;
      }
      if (lane == 0) {
        if (want) {
          const int q = __ldcg(ws.to + at), p = from[full];
          row[full] = q;
          kv.refs[q] = 1;
          // a source outside the pool copies nothing (the new page on itself)
          const bool in = p >= 0 && p < kv.pages;
          if (!in) book_bad(kv, s);
          ws.from[at] = in ? p : q;
          ++given;
        }
        kv.len[d] = len;
      }
    } else if (a.dst[i] > 0) {
      const int len = kv.len[i], held = (len + kKv4Page - 1) / kKv4Page;
      int32_t* row = kv.table + (size_t)i * mp;
      for (int j = lane; j < want; j += 32) {
        const int q = __ldcg(ws.to + at + j);
        row[held + j] = q;
        kv.refs[q] = 1;
      }
      __syncwarp();
      if (lane == 0) {
        kv.len[i] = len + a.dst[i];
        given += want;
      }
    }
  }
  if (fails) atomicAdd(&ws.w[kWsFails], fails);
  if (given) atomicAdd(&ws.w[kWsFreed], given);
  // forks are served in order of their place in the list, so the copies are its first entries
  book_sync<CTAS>();
  if (tid == 0) {
    const int g = __ldcg(ws.w + kWsFreed);
    ws.w[kWsCopies] = mode == kBookFork ? g : 0;
    if (a.info) {
      a.info[0] = nfree - g;
      a.info[1] = __ldcg(ws.w + kWsFails);
      a.info[2] = g;
    }
  }
}

struct CompactArgs {
  int32_t* new_table;
  int32_t* new_refs;
  int32_t* remap;
  int32_t* info;
  PagesWs ws;
};

template <int CTAS>
__global__ void __launch_bounds__(kBookThreads) k_kv4_compact_book(Kv4Dev kv, CompactArgs a) {
  __shared__ int smem[32];
  pdl_prologue();
  const int cta = (int)blockIdx.x, tid = cta * kBookThreads + (int)threadIdx.x;
  constexpr int kAll = CTAS * kBookThreads;
  const PagesWs ws = a.ws;
  const Span my = my_pages<CTAS>(kv.pages, cta);
  int mine = 0;
  for (int p = my.b + (int)threadIdx.x; p < my.e; p += kBookThreads) mine += kv.refs[p] > 0;
  mine = cta_sum(mine, smem);
  if (threadIdx.x == 0) ws.w[kWsTotal + cta] = mine;
  book_sync<CTAS>();
  int live = 0, live_before = 0;
  for (int c = 0; c < CTAS; ++c) {
    const int t = __ldcg(ws.w + kWsTotal + c);
    if (c < cta) live_before += t;
    live += t;
  }
  // Free pages below `live` and used pages from `live` on, before this CTA's
  // span: of the pages below min(b, live), those not in use; of the used
  // pages before b, those from `live` on.  Used pages below `live`: counted
  // once more, by the CTA whose span holds the boundary.
  int low = 0;  // used pages of my span below `live`
  for (int p = my.b + (int)threadIdx.x; p < my.e && p < live; p += kBookThreads) low += kv.refs[p] > 0;
  low = cta_sum(low, smem);
  if (threadIdx.x == 0) ws.w[kWsTotal + 8 + cta] = low;
  book_sync<CTAS>();
  int low_before = 0, low_all = 0;
  for (int c = 0; c < CTAS; ++c) {
    const int t = __ldcg(ws.w + kWsTotal + 8 + c);
    if (c < cta) low_before += t;
    low_all += t;
  }
  int slot = (my.b < live ? my.b : live) - low_before;  // free slots before mine
  int mover = live_before - low_before;                 // moving pages before mine
  const int moves = live - low_all;
  for (int p0 = my.b; p0 < my.e; p0 += kBookThreads) {
    const int p = p0 + (int)threadIdx.x;
    const bool in = p < my.e;
    const int r = in ? kv.refs[p] : 0;
    const int is_slot = in && p < live && r <= 0, is_mover = in && p >= live && r > 0;
    int ts, tm;
    const int as = slot + cta_scan(is_slot, &ts, smem);
    const int am = mover + cta_scan(is_mover, &tm, smem);
    if (is_slot) ws.to[as] = p;
    if (is_mover) ws.from[am] = p;
    if (in && !is_mover) {
      a.remap[p] = r > 0 ? p : -1;
      if (r > 0) a.new_refs[p] = r;  // p < live
    }
    slot += ts;
    mover += tm;
  }
  book_sync<CTAS>();
  for (int i = tid; i < moves; i += kAll) {
    const int p = __ldcg(ws.from + i), q = __ldcg(ws.to + i);
    a.remap[p] = q;
    a.new_refs[q] = kv.refs[p];
  }
  book_sync<CTAS>();  // (new_refs may be refs) the movers' counts have been read
  for (int p = live + tid; p < kv.pages; p += kAll) a.new_refs[p] = 0;
  if (tid == 0) {
    ws.w[kWsCopies] = moves;
    if (a.info) {
      a.info[0] = kv.pages - live;
      a.info[1] = moves;
    }
  }
}

struct CopyArgs {
  const int32_t* from;
  const int32_t* to;
  const int32_t* count_dev;  // copies, or null: count
  int count;
  // compact: the table that follows
  int32_t* new_table;
  const int32_t* remap;
  unsigned vecs;    // 16-byte vectors of one page in one layer
  unsigned chunks;  // pieces of kCopyThreads * kCopyUnroll vectors
};

__global__ void __launch_bounds__(kCopyThreads) k_kv4_copy(Kv4Dev kv, CopyArgs a) {
  pdl_prologue();
  if (a.new_table) {
    const size_t total = (size_t)kv.seqs * kv.max_pages;
    for (size_t i = (size_t)blockIdx.x * kCopyThreads + threadIdx.x; i < total; i += (size_t)gridDim.x * kCopyThreads) {
      const int p = kv.table[i];
      if (p >= kv.pages) book_bad(kv, p);
      a.new_table[i] = p >= 0 && p < kv.pages ? a.remap[p] : -1;
    }
  }
  const long long copies = a.count_dev ? *a.count_dev : a.count;
  const long long units = copies * kv.n * kv.layers * a.chunks;
  for (long long u = blockIdx.x; u < units; u += gridDim.x) {
    long long x = u;
    const unsigned chunk = (unsigned)(x % a.chunks);
    x /= a.chunks;
    const int i = (int)(x % copies);
    x /= copies;
    const int layer = (int)(x % kv.layers), rank = (int)(x / kv.layers);
    const int p = a.from[i], q = a.to[i];
    if (p < 0 || p >= kv.pages || q < 0 || q >= kv.pages) {
      if (threadIdx.x == 0) book_bad(kv, i);
      continue;
    }
    const uint4* src = reinterpret_cast<const uint4*>(kv.pool[rank]) + ((size_t)layer * kv.pages + p) * a.vecs;
    uint4* dst = reinterpret_cast<uint4*>(kv.pool[rank]) + ((size_t)layer * kv.pages + q) * a.vecs;
    const unsigned v0 = chunk * (kCopyThreads * kCopyUnroll) + threadIdx.x;
    uint4 r[kCopyUnroll];
#pragma unroll
    for (int j = 0; j < kCopyUnroll; ++j)
      if (v0 + j * kCopyThreads < a.vecs) r[j] = __ldcs(src + v0 + j * kCopyThreads);
#pragma unroll
    for (int j = 0; j < kCopyUnroll; ++j)
      if (v0 + j * kCopyThreads < a.vecs) __stcs(dst + v0 + j * kCopyThreads, r[j]);
  }
}

const void* kv4_pages_kernel(int i) {
  switch (i) {
    case 0: return (const void*)&k_kv4_book<1>;
    case 1: return (const void*)&k_kv4_book<kBookCtas>;
    case 2: return (const void*)&k_kv4_compact_book<1>;
    case 3: return (const void*)&k_kv4_compact_book<kBookCtas>;
    case 4: return (const void*)&k_kv4_copy;
    default: return nullptr;
  }
}

}  // namespace dcc

namespace {
using dcc_host::launch;

size_t ws_bytes(const dcc_kv4_t* kv) {
  return 4 * ((size_t)dcc::kWsWords + 2 * (size_t)kv->pages + 2 * (size_t)kv->seqs + 4);
}

int page_view(const dcc_kv4_t* kv, bool need_refs, void* ws, size_t bytes, dcc::Kv4Dev* d, dcc::PagesWs* out) {
  const int rc = dcc_host::kv4_view(kv, need_refs, d);
  if (rc != DCC_OK) return rc;
  if (!out) return DCC_OK;
  if (!ws || bytes < ws_bytes(kv)) return DCC_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(ws) & 15u) return DCC_ERR_MISALIGNED;
  out->w = static_cast<int32_t*>(ws);
  out->from = out->w + dcc::kWsWords;
  out->to = out->from + kv->pages;
  out->mark = out->to + kv->pages;
  out->pre = out->mark + kv->seqs;
  return DCC_OK;
}

bool odd_word(const void* p) { return reinterpret_cast<uintptr_t>(p) & 3u; }

int copy_launch(const dcc_kv4_t* kv, dcc::Kv4Dev& d, dcc::CopyArgs& a, cudaStream_t s) {
  a.vecs = (unsigned)((size_t)kv->kv_heads * dcc::kv4_block_bytes(kv->head_dim, kv->group) / 16);
  constexpr unsigned per = dcc::kCopyThreads * dcc::kCopyUnroll;
  a.chunks = (a.vecs + per - 1) / per;
  const void* fn = dcc::kv4_pages_kernel(4);
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return DCC_ERR_CUDA;
  }
  const int per_sm = dcc_host::max_active_per_sm(fn, dcc::kCopyThreads);
  if (per_sm < 1) return DCC_ERR_LAUNCH;
  void* args[] = {&d, &a};
  return launch(fn, sms * per_sm, dcc::kCopyThreads, false, args, s, 0, true);
}

// What a page call reads and writes lies apart: the cache's books, the pools, the
// workspace, info and `more` (at most 4 of the call's own).
bool books_apart(const dcc_kv4_t* kv, const void* ws, const int32_t* info,
                 std::initializer_list<dcc_host::Extent> more) {
  const size_t pool = (size_t)kv->layers * kv->pages * kv->kv_heads * dcc::kv4_block_bytes(kv->head_dim, kv->group);
  dcc_host::Extent e[9] = {{kv->table, (size_t)kv->seqs * kv->max_pages * 4, true},
                           {kv->len, (size_t)kv->seqs * 4, true},
                           {kv->refs, (size_t)kv->pages * 4, true},
                           {ws, ws_bytes(kv), true},
                           {info, 16, true}};
  int n = 5;
  for (const dcc_host::Extent& x : more) e[n++] = x;
  if (!dcc_host::disjoint(e, n)) return false;
  for (int r = 0; r < kv->n_ranks; ++r)
    for (int i = 0; i < n; ++i)
      if (e[i].p && dcc_host::overlaps(e[i].p, e[i].bytes, kv->pool[r], pool)) return false;
  return true;
}

// Kernel `which` for one CTA, which + 1 for a cluster, by the numbers to go through.
int launch_book(int which, long long numbers, void** args, cudaStream_t s) {
  const bool one = numbers <= dcc::kBookOneCta;
  return launch(dcc::kv4_pages_kernel(one ? which : which + 1), one ? 1 : dcc::kBookCtas, dcc::kBookThreads, false, args,
                s, 0, true, one ? 0 : dcc::kBookCtas);
}

int book_call(const dcc_kv4_t* kv, int mode, const int32_t* src, const int32_t* dst, size_t count, int32_t* info,
              void* ws, size_t bytes, cudaStream_t s) {
  dcc::Kv4Dev d{};
  dcc::BookArgs a{};
  int rc = page_view(kv, true, ws, bytes, &d, &a.ws);
  if (rc != DCC_OK) return rc;
  if (count > (size_t)kv->seqs) return DCC_ERR_INVALID_ARG;
  if ((count && !dst) || (mode == dcc::kBookFork && count && !src)) return DCC_ERR_INVALID_ARG;
  if (odd_word(src) || odd_word(dst) || odd_word(info)) return DCC_ERR_MISALIGNED;
  if (!books_apart(kv, ws, info, {{src, count * 4, false}, {dst, count * 4, false}})) return DCC_ERR_INVALID_ARG;
  a.src = src;
  a.dst = dst;
  a.count = (int)count;
  a.info = info;
  if ((rc = dcc_host::kv4_ready(&d)) != DCC_OK) return rc;
  void* args[] = {&d, &a, &mode};
  const long long rows = mode == dcc::kBookReserve ? 0 : (long long)count * kv->max_pages;
  rc = launch_book(0, kv->pages > rows ? kv->pages : rows, args, s);
  if (rc != DCC_OK || mode != dcc::kBookFork || count == 0) return rc;
  dcc::CopyArgs c{};
  c.from = a.ws.from;
  c.to = a.ws.to;
  c.count_dev = a.ws.w + dcc::kWsCopies;
  return copy_launch(kv, d, c, s);
}

}  // namespace

extern "C" {

int dcc_kv4_pages_workspace(const dcc_kv4_t* kv, size_t* bytes) {
  if (!kv || !bytes || kv->pages < 1 || kv->seqs < 1) return DCC_ERR_INVALID_ARG;
  *bytes = ws_bytes(kv);
  return DCC_OK;
}

int dcc_kv4_reserve(const dcc_kv4_t* kv, const int32_t* add, int32_t* info, void* workspace, size_t workspace_bytes,
                    dcc_stream_t s) {
  if (!kv || !add) return DCC_ERR_INVALID_ARG;
  return book_call(kv, dcc::kBookReserve, nullptr, add, kv->seqs > 0 ? (size_t)kv->seqs : 0, info, workspace,
                   workspace_bytes, static_cast<cudaStream_t>(s));
}

int dcc_kv4_free(const dcc_kv4_t* kv, const int32_t* seqs, size_t count, int32_t* info, void* workspace,
                 size_t workspace_bytes, dcc_stream_t s) {
  return book_call(kv, dcc::kBookFree, nullptr, seqs, count, info, workspace, workspace_bytes,
                   static_cast<cudaStream_t>(s));
}

int dcc_kv4_fork(const dcc_kv4_t* kv, const int32_t* src, const int32_t* dst, size_t count, int32_t* info,
                 void* workspace, size_t workspace_bytes, dcc_stream_t s) {
  return book_call(kv, dcc::kBookFork, src, dst, count, info, workspace, workspace_bytes,
                   static_cast<cudaStream_t>(s));
}

int dcc_kv4_copy(const dcc_kv4_t* kv, const int32_t* src, const int32_t* dst, size_t count, dcc_stream_t s) {
  dcc::Kv4Dev d{};
  int rc = page_view(kv, false, nullptr, 0, &d, nullptr);
  if (rc != DCC_OK) return rc;
  if (count > (size_t)kv->pages || (count && (!src || !dst))) return DCC_ERR_INVALID_ARG;
  if (odd_word(src) || odd_word(dst)) return DCC_ERR_MISALIGNED;
  if (count == 0) return DCC_OK;
  dcc::CopyArgs c{};
  if ((rc = dcc_host::kv4_ready(&d)) != DCC_OK) return rc;
  c.from = src;
  c.to = dst;
  c.count = (int)count;
  return copy_launch(kv, d, c, static_cast<cudaStream_t>(s));
}

int dcc_kv4_compact(const dcc_kv4_t* kv, int32_t* new_table, int32_t* new_refs, int32_t* remap, int32_t* info,
                    void* workspace, size_t workspace_bytes, dcc_stream_t s) {
  dcc::Kv4Dev d{};
  dcc::CompactArgs a{};
  int rc = page_view(kv, true, workspace, workspace_bytes, &d, &a.ws);
  if (rc != DCC_OK) return rc;
  if (!new_table || !new_refs || !remap) return DCC_ERR_INVALID_ARG;
  if (odd_word(new_table) || odd_word(new_refs) || odd_word(remap) || odd_word(info)) return DCC_ERR_MISALIGNED;
  // the new table and counts may be the cache's own
  const size_t table_bytes = (size_t)kv->seqs * kv->max_pages * 4, pages_bytes = (size_t)kv->pages * 4;
  if (!books_apart(kv, workspace, info,
                   {{new_table == kv->table ? nullptr : new_table, table_bytes, true},
                    {new_refs == kv->refs ? nullptr : new_refs, pages_bytes, true},
                    {remap, pages_bytes, true}}))
    return DCC_ERR_INVALID_ARG;
  a.new_table = new_table;
  a.new_refs = new_refs;
  a.remap = remap;
  a.info = info;
  if ((rc = dcc_host::kv4_ready(&d)) != DCC_OK) return rc;
  void* args[] = {&d, &a};
  cudaStream_t st = static_cast<cudaStream_t>(s);
  rc = launch_book(2, kv->pages, args, st);
  if (rc != DCC_OK) return rc;
  dcc::CopyArgs c{};
  c.from = a.ws.from;
  c.to = a.ws.to;
  c.count_dev = a.ws.w + dcc::kWsCopies;
  c.new_table = new_table;
  c.remap = remap;
  return copy_launch(kv, d, c, st);
}

}  // extern "C"
