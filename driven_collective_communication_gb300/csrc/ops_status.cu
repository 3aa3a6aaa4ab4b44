// ops_status.cu -- what the calls without a communicator share on the host:
// the status word their kernels record failures in, and the checks of a cache
// descriptor.
#include <cuda_runtime.h>

#include <atomic>
#include <mutex>

#include "comm.h"
#include "kv4.cuh"
#include "tcgen05.cuh"

namespace {
// Words per device: the first number out of range, the first wait that gave up,
// the tag of the last call in which one did (LocalDev).  The address comes from
// cudaGetSymbolAddress.
static __device__ unsigned long long g_local_status[6];  // and what the last check took of them
constexpr int kMaxDevices = 64;
std::mutex g_mu, g_check_mu;
unsigned long long* g_addr[kMaxDevices];

// Takes the record and leaves none, one word at a time in one step each: what a
// kernel on another stream records meanwhile is either taken or left.
__global__ void k_local_take(unsigned long long* status) { status[3 + threadIdx.x] = atomicExch(status + threadIdx.x, 0ull); }
}  // namespace

namespace dcc {
const void* local_take_kernel() { return (const void*)&k_local_take; }
}  // namespace dcc

namespace dcc_host {

unsigned long long* local_status() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
    cudaGetLastError();
    return nullptr;
  }
  std::lock_guard<std::mutex> lock(g_mu);
  if (!g_addr[dev]) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_local_status) != cudaSuccess) {
      cudaGetLastError();
      return nullptr;
    }
    g_addr[dev] = static_cast<unsigned long long*>(p);
  }
  return g_addr[dev];
}

dcc::LocalDev local_dev(unsigned long long* status) {
  static std::atomic<unsigned long long> calls{0};
  return {2000000000ull, ++calls, status + 1};
}

int kv4_view(const dcc_kv4_t* kv, bool need_refs, dcc::Kv4Dev* out) {
  if (!kv || !kv->pool || !kv->table || !kv->len || (need_refs && !kv->refs)) return DCC_ERR_INVALID_ARG;
  if (kv->n_ranks < 1 || kv->n_ranks > DCC_MAX_RANKS || kv->layers < 1 || kv->pages < 1 || kv->seqs < 1 ||
      kv->max_pages < 1 || kv->kv_heads < 1)
    return DCC_ERR_INVALID_ARG;
  // positions and page numbers are 32-bit; pool offsets are not
  if (kv->max_pages > (1 << 24) || kv->pages > (1 << 28) || kv->seqs > (1 << 20) || kv->kv_heads > (1 << 12) ||
      kv->layers > (1 << 12))
    return DCC_ERR_INVALID_ARG;
  if (kv->dtype != DCC_FP16 && kv->dtype != DCC_BF16) return DCC_ERR_UNSUPPORTED;
  if ((kv->head_dim != 64 && kv->head_dim != 128) || (kv->group != 32 && kv->group != 64)) return DCC_ERR_UNSUPPORTED;
  if (((reinterpret_cast<uintptr_t>(kv->table) | reinterpret_cast<uintptr_t>(kv->len) |
        reinterpret_cast<uintptr_t>(kv->refs)) & 3u))
    return DCC_ERR_MISALIGNED;
  const size_t bytes = (size_t)kv->layers * kv->pages * kv->kv_heads * dcc::kv4_block_bytes(kv->head_dim, kv->group);
  for (int r = 0; r < kv->n_ranks; ++r) {
    const char* p = static_cast<const char*>(kv->pool[r]);
    if (!p) return DCC_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(p) & 15u) return DCC_ERR_MISALIGNED;
    for (int q = 0; q < r; ++q) {
      const char* o = static_cast<const char*>(kv->pool[q]);
      if (p < o + bytes && o < p + bytes) return DCC_ERR_INVALID_ARG;  // two ranks' pools overlap
    }
    out->pool[r] = const_cast<char*>(p);
  }
  out->table = kv->table;
  out->len = kv->len;
  out->refs = kv->refs;
  out->n = kv->n_ranks;
  out->layers = kv->layers;
  out->pages = kv->pages;
  out->seqs = kv->seqs;
  out->max_pages = kv->max_pages;
  out->heads = kv->kv_heads;
  out->status = nullptr;  // kv4_ready
  return DCC_OK;
}

int kv4_ready(dcc::Kv4Dev* d) {
  d->status = local_status();
  return d->status ? DCC_OK : DCC_ERR_CUDA;
}

bool disjoint(const Extent* e, int n) {
  for (int i = 0; i < n; ++i)
    for (int j = 0; j < i; ++j)
      if ((e[i].written || e[j].written) && e[i].p && e[j].p && overlaps(e[i].p, e[i].bytes, e[j].p, e[j].bytes))
        return false;
  return true;
}

bool rows_overlap(const void* a, const void* b, size_t rows, size_t stride, size_t width) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b), d = x < y ? y - x : x - y;
  if (rows <= 1) return rows == 1 && d < width;
  const uintptr_t i = d / stride, m = d % stride;  // row j of one lies m past row j + i of the other
  return (m < width && i < rows) || (stride - m < width && i + 1 < rows);
}

}  // namespace dcc_host

extern "C" {

int dcc_kv4_block_bytes(int head_dim, int group, size_t* bytes) {
  if (!bytes) return DCC_ERR_INVALID_ARG;
  if ((head_dim != 64 && head_dim != 128) || (group != 32 && group != 64)) return DCC_ERR_UNSUPPORTED;
  *bytes = (size_t)dcc::kv4_block_bytes(head_dim, group);
  return DCC_OK;
}

int dcc_local_check(dcc_stream_t s) {
  unsigned long long* p = dcc_host::local_status();
  if (!p) return DCC_ERR_CUDA;
  unsigned long long st[3] = {0, 0, 0};
  cudaStream_t stream = static_cast<cudaStream_t>(s);
  if (cudaStreamSynchronize(stream) != cudaSuccess) {
    cudaGetLastError();
    return DCC_ERR_CUDA;
  }
  std::lock_guard<std::mutex> lock(g_check_mu);  // what was taken lies in one place
  void* args[] = {&p};
  const int rc = dcc_host::launch(dcc::local_take_kernel(), 1, 3, false, args, stream);
  if (rc != DCC_OK) return rc;
  if (cudaMemcpyAsync(st, p + 3, sizeof st, cudaMemcpyDeviceToHost, stream) != cudaSuccess ||
      cudaStreamSynchronize(stream) != cudaSuccess) {
    cudaGetLastError();
    return DCC_ERR_CUDA;
  }
  if (st[0] == 0 && st[1] == 0) return DCC_OK;
  return (st[1] & 0xffull) == dcc::kStatusTimeout ? DCC_ERR_TIMEOUT : DCC_ERR_BOUNDS;
}

}  // extern "C"
