// linear.cu -- host side of the column-parallel linear layer.
#include <algorithm>
#include <map>
#include <mutex>
#include <tuple>

#include "comm.h"
#include "linear_big.cuh"

namespace dcc {
const void* linear_kernel(int which) {
  switch (which) {
    case 0: return (const void*)&k_linear_mma<kMmaPairThreads>;
    case 1: return (const void*)&k_linear_mma<kMmaThreads>;
    case 2: return (const void*)&k_linear_big;
    default: return nullptr;
  }
}
}  // namespace dcc

namespace {
using dcc_host::launch;

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn encode_tiled() {
  static const EncodeTiledFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    const bool ok = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                        cudaSuccess &&
                    q == cudaDriverEntryPointSuccess;
    cudaGetLastError();
    return ok ? reinterpret_cast<EncodeTiledFn>(p) : nullptr;
  }();
  return fn;
}
// outer x inner 16-bit elements, box 64 (one 128-byte swizzle row) x box_rows, zeros outside
int make_map(const void* ptr, size_t inner, size_t outer, unsigned box_rows, bool fp16, CUtensorMap* out) {
  EncodeTiledFn enc = encode_tiled();
  if (!enc) return DCC_ERR_UNSUPPORTED;
  const cuuint64_t dims[2] = {(cuuint64_t)inner, (cuuint64_t)outer}, strides[1] = {(cuuint64_t)inner * 2};
  const cuuint32_t box[2] = {(cuuint32_t)dcc::kMmaBK, (cuuint32_t)box_rows}, estr[2] = {1, 1};
  return enc(out, fp16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(ptr),
             dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? DCC_OK
             : DCC_ERR_INVALID_ARG;
}

// What a device holds at once: clusters of a kernel, by (device, kernel,
// cluster size, shared memory).  A property of the device, asked once.
struct Room {
  int sms = 0, smem_sm = 0, smem_reserved = 0, dev = -1;
};
int room(Room* r) {
  static std::mutex mu;
  static Room known[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
    cudaGetLastError();
    return DCC_ERR_CUDA;
  }
  std::lock_guard<std::mutex> lock(mu);
  Room& k = known[dev];
  if (k.dev < 0) {
    if (cudaDeviceGetAttribute(&k.sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&k.smem_sm, cudaDevAttrMaxSharedMemoryPerMultiprocessor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&k.smem_reserved, cudaDevAttrReservedSharedMemoryPerBlock, dev) != cudaSuccess) {
      cudaGetLastError();
      return DCC_ERR_CUDA;
    }
    k.dev = dev;
  }
  *r = k;
  return DCC_OK;
}
int clusters(const Room& r, const void* fn, int threads, int size, size_t smem) {
  static std::mutex mu;
  static std::map<std::tuple<int, const void*, int, size_t>, int> known;
  std::lock_guard<std::mutex> lock(mu);
  const auto key = std::make_tuple(r.dev, fn, size, smem);
  const auto it = known.find(key);
  if (it != known.end()) return it->second;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)size);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)size;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  int num = 0;
  if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, 226 * 1024) != cudaSuccess ||
      cudaFuncSetAttribute(fn, cudaFuncAttributePreferredSharedMemoryCarveout, 100) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&num, fn, &cfg) != cudaSuccess) {
    cudaGetLastError();
    num = 0;
  }
  known[key] = num;
  return num;
}

// Launch plan of the kernel for up to 256 tokens: the row tile's height and
// the K split of one form, by the rule of the row-parallel layer's plan: the
// deepest split whose grid fits the GPU at once and has at least three
// quarters of the CTAs of the fullest such grid; where no grid fits, tiles of
// 128 rows in several waves.
struct Plan {
  const void* fn = nullptr;
  int threads = 0, stages = 0, bm = dcc::kMmaBM, ks = 1, rounds = 0;
  size_t smem = 0;
  bool one_wave = false;
};
Plan plan(const Room& r, bool pair, int n, int ntile, int rows, int k) {
  Plan p;
  p.threads = pair ? dcc::kMmaPairThreads : dcc::kMmaThreads;
  p.fn = dcc::linear_kernel(pair ? 0 : 1);
  p.stages = dcc::mma_stages(ntile, 1, pair ? dcc::kMmaPairStageBudget : dcc::kMmaStageBudget);
  p.smem = dcc::mma_smem_bytes(ntile, p.stages, 1);
  const bool two = pair && 2 * (p.smem + (size_t)r.smem_reserved) <= (size_t)r.smem_sm;
  const int kblocks = (k + dcc::kMmaBK - 1) / dcc::kMmaBK;
  auto tiles = [&](int bm) { return (long long)n * ((rows + bm - 1) / bm); };
  int bms[dcc::kMmaMaxSplit + 1] = {};
  long long ctas[dcc::kMmaMaxSplit + 1] = {}, most = 0;
  for (int ks = 1; ks <= dcc::kMmaMaxSplit && ks <= kblocks; ks *= 2) {
    if (!dcc::mma_epilogue_fits(ntile, p.stages, 1, ks)) break;
    const long long cap = (long long)clusters(r, p.fn, p.threads, ks, p.smem) * (two ? 2 : 1);
    for (int bm = 64; bm <= dcc::kMmaBM; bm += 8) {
      if (tiles(bm) > cap) continue;
      int tall = bm;
      while (tall + 8 <= dcc::kMmaBM && tiles(tall + 8) == tiles(bm)) tall += 8;
      bms[ks] = tall;
      ctas[ks] = tiles(bm) * ks;
      most = std::max(most, ctas[ks]);
      break;
    }
  }
  for (int ks = dcc::kMmaMaxSplit; ks >= 1; ks /= 2)
    if (bms[ks] && 4 * ctas[ks] >= 3 * most) {
      p.bm = bms[ks];
      p.ks = ks;
      p.one_wave = true;
      break;
    }
  p.rounds = dcc::mma_epilogue_rounds(ntile, p.stages, 1, p.ks);
  return p;
}

int run_mma(const dcc::LinArgs& l, bool fp16, dcc::LocalDev& dc, cudaStream_t s) {
  Room r;
  int rc = room(&r);
  if (rc != DCC_OK) return rc;
  const int ntile = l.tokens <= 16 ? 16 : (l.tokens + 15) / 16 * 16;
  const Plan one = plan(r, false, l.n, ntile, l.rows, l.k), pair = plan(r, true, l.n, ntile, l.rows, l.k);
  // a grid in one wave first, then an epilogue in one round, then the deeper split
  const bool better = pair.one_wave != one.one_wave           ? pair.one_wave
                      : (pair.rounds == 1) != (one.rounds == 1) ? pair.rounds == 1
                                                                : pair.ks > one.ks;
  const Plan& p = better ? pair : one;
  if (p.rounds < 1 || clusters(r, p.fn, p.threads, p.ks, p.smem) < 1) return DCC_ERR_LAUNCH;
  dcc::LinMaps maps;
  std::memset(&maps, 0, sizeof maps);
  for (int i = 0; i < l.n; ++i) {
    rc = make_map(l.w[i], (size_t)l.k, (size_t)l.rows, (unsigned)p.bm, fp16, &maps.w[i]);
    if (rc == DCC_OK && (i == 0 || l.x[i] != l.x[i - 1]))
      rc = make_map(l.x[i], (size_t)l.k, (size_t)l.tokens, (unsigned)ntile, fp16, &maps.x[i]);
    else if (rc == DCC_OK)
      maps.x[i] = maps.x[i - 1];
    if (rc != DCC_OK) return rc;
  }
  dcc::LinMmaArgs a{};
  a.l = l;
  a.ntile = ntile;
  a.ks = p.ks;
  a.stages = p.stages;
  a.bm = p.bm;
  a.tiles = (l.rows + p.bm - 1) / p.bm;
  a.rounds = p.rounds;
  a.fp16 = fp16;
  const long long grid = (long long)l.n * a.tiles * p.ks;
  if (grid > 0x7fffffffll) return DCC_ERR_INVALID_ARG;
  void* args[] = {&maps, &dc, &a};
  return launch(p.fn, (int)grid, p.threads, false, args, s, p.smem, true, p.ks > 1 ? p.ks : 0);
}

int run_big(const dcc::LinArgs& l, bool fp16, dcc::LocalDev& dc, cudaStream_t s) {
  Room r;
  int rc = room(&r);
  if (rc != DCC_OK) return rc;
  dcc::LinBigArgs a{};
  a.l = l;
  a.tok_tiles = (l.tokens + dcc::kBigTokens - 1) / dcc::kBigTokens;
  a.ntile = ((l.tokens + a.tok_tiles - 1) / a.tok_tiles + 15) / 16 * 16;
  a.row_tiles = (l.rows + dcc::kBigRows - 1) / dcc::kBigRows;
  a.fp16 = fp16;
  const void* fn = dcc::linear_kernel(2);
  const size_t smem = dcc::big_smem_bytes(a.ntile);
  const int pairs = clusters(r, fn, dcc::kBigThreads, 2, smem);
  if (pairs < 1) return DCC_ERR_LAUNCH;
  const long long tiles = (long long)l.n * a.row_tiles * a.tok_tiles;
  if (tiles > 0x3fffffffll) return DCC_ERR_INVALID_ARG;
  dcc::LinMaps maps;
  std::memset(&maps, 0, sizeof maps);
  for (int i = 0; i < l.n; ++i) {
    rc = make_map(l.w[i], (size_t)l.k, (size_t)l.rows, 128, fp16, &maps.w[i]);
    if (rc == DCC_OK && (i == 0 || l.x[i] != l.x[i - 1]))
      rc = make_map(l.x[i], (size_t)l.k, (size_t)l.tokens, (unsigned)a.ntile / 2, fp16, &maps.x[i]);
    else if (rc == DCC_OK)
      maps.x[i] = maps.x[i - 1];
    if (rc != DCC_OK) return rc;
  }
  void* args[] = {&maps, &dc, &a};
  return launch(fn, 2 * (int)std::min<long long>(tiles, pairs), dcc::kBigThreads, false, args, s, smem, true, 2);
}

}  // namespace

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
  unsigned long long* status = dcc_host::local_status();
  if (!status) return DCC_ERR_CUDA;
  dcc::LocalDev dc = dcc_host::local_dev(status);
  cudaStream_t st = static_cast<cudaStream_t>(s);
  return tokens <= (size_t)dcc::kMmaMaxTokens ? run_mma(a, t == DCC_FP16, dc, st) : run_big(a, t == DCC_FP16, dc, st);
}
