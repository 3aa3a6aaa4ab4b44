// linear_big.cuh -- the column-parallel linear layer for more than 256 tokens
// (prompt chunks), on the fifth-generation tensor cores.
//
// Bound by the tensor cores.  Two CTAs of a cluster work as a pair on one
// 256-row tile of W and up to 256 tokens (cta_group::2): each holds its 128
// rows of W and half of the tokens, so a tile's operands cross from L2 to the
// SMs once per pair -- 64 bytes a clock and SM at the full MMA rate, where
// single CTAs with 128 x 256 tiles would ask for 96.  Tokens are cut into equal
// tiles of a multiple of 16, so a ragged count wastes at most 15 columns a
// tile.  Persistent: one pair per two SMs takes every 76th tile, token tiles
// of one weight tile side by side (the weights then come from memory once),
// and the accumulator is doubled in tensor memory, so the epilogue of one tile
// runs under the products of the next.  Measured on GB300, 8 ranks, 2048 tokens x
// 3584 rows x 8192, bias and GELU: 590-610 us by the clock that the power limit
// leaves, 1.6 PFLOP/s (a library product alone: 1.9 in a burst, 1.7 sustained); the
// tensor pipe is active 81 % of the time.  All of K goes into one accumulator, whose
// adds truncate: some more results fall an ulp of their type off than with K split.
// Roles (192 threads):
//   warp 0, one thread       TMA into this CTA's stage; the bytes of both CTAs
//                             complete on the leader's full barrier;
//   warp 1, one thread       (leader) tcgen05.mma 256 x N x 16; commits free
//                             the stage in both CTAs;
//   warps 2..5               epilogue: lane = row, so the 32 lanes of a warp
//                             read residuals and write results of 32
//                             neighbouring rows of a token.
// Waits run to their limit whatever another wait did (one wave, so that bounds
// the kernel): what the other CTA of a pair had in flight is then long done.
#pragma once
#include "linear_mma.cuh"

namespace dcc {

constexpr int kBigThreads = 192;
constexpr int kBigStages = 6;
constexpr int kBigRows = 256;    // rows of W per pair
constexpr int kBigTokens = 256;  // most tokens per tile

struct LinBigArgs {
  LinArgs l;
  int ntile, row_tiles, tok_tiles, fp16;
};
__host__ __device__ constexpr uint32_t big_stage_bytes(int ntile) { return 128u * 128u + (uint32_t)(ntile / 2) * 128u; }
__host__ __device__ constexpr size_t big_smem_bytes(int ntile) {
  return 1024 + (size_t)kBigStages * big_stage_bytes(ntile) + 16 * kBigStages + 64;
}

__device__ __forceinline__ uint32_t cluster_addr(uint32_t addr, uint32_t cta) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(cta));
  return r;
}
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar,
                                              uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2.L2::cache_hint [%0], "
      "[%1, {%2, %3}], [%4], %5;" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(bar), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void commit_pair(uint32_t bar) {  // arrives at `bar` of both CTAs
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"((uint16_t)3)
      : "memory");
}

// 16 tokens of one row: y + t * rows, r (or null) alike; `live` tokens are there
template <int ACT>
__device__ __forceinline__ void big_store16(const uint32_t* v, float bias, const uint16_t* res, uint16_t* y, size_t rows,
                                            int live, bool fp16) {
  float r[16] = {};
  if (res)
#pragma unroll
    for (int j = 0; j < 16; ++j)
      if (j < live) {
        const uint16_t b = res[j * rows];
        r[j] = fp16 ? Half16<__half>::widen(b) : Half16<__nv_bfloat16>::widen(b);
      }
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    float z = lin_act(__uint_as_float(v[j]) + bias, ACT);
    if (res) z += r[j];
    const uint16_t b = fp16 ? Half16<__half>::narrow(z) : Half16<__nv_bfloat16>::narrow(z);
    if (j < live) y[j * rows] = b;
  }
}

__global__ void __launch_bounds__(kBigThreads, 1)
    k_linear_big(const __grid_constant__ LinMaps maps, LocalDev dc, const __grid_constant__ LinBigArgs a) {
  extern __shared__ unsigned char big_raw[];
  __shared__ uint32_t tmem_slot;
  constexpr int S = kBigStages;
  const uint32_t base = (smem_addr_u32(big_raw) + 1023u) & ~1023u;  // the same in both CTAs
  const int N = a.ntile;
  const uint32_t st_bytes = big_stage_bytes(N), a_bytes = 128u * 128u;
  const uint32_t bars = base + (uint32_t)S * st_bytes;
  auto full = [&](int s) { return bars + 8u * (uint32_t)s; };          // leader: both CTAs' bytes have landed
  auto empty = [&](int s) { return bars + 8u * (uint32_t)(S + s); };   // the products have read the stage
  auto accf = [&](int b) { return bars + 8u * (uint32_t)(2 * S + b); };      // accumulator b is complete
  auto acce = [&](int b) { return bars + 8u * (uint32_t)(2 * S + 2 + b); };  // leader: and has been read
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t cta;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(cta));
  if (warp == 0) {
    if (lane < 2 * S + 2) mma_mbar_init(bars + 8u * (uint32_t)lane, 1);
    else if (lane < 2 * S + 4) mma_mbar_init(bars + 8u * (uint32_t)lane, 8);  // 4 warps of each CTA
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 2) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr_u32(&tmem_slot)),
                 "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  pdl_wait();
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  pdl_trigger();  // not before the allocation
  mma_cluster_sync();  // both CTAs' barriers stand
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = tmem_slot;
  const int kpb = (a.l.k + kMmaBK - 1) / kMmaBK;
  const int tiles = a.l.n * a.row_tiles * a.tok_tiles, first = (int)blockIdx.x / 2, stride = (int)gridDim.x / 2;
  auto place = [&](int w, int* rank, int* row, int* tok) {  // token tiles fastest, then rows, then ranks
    *tok = w % a.tok_tiles * N;
    const int r = w / a.tok_tiles;
    *row = r % a.row_tiles * kBigRows;
    *rank = r / a.row_tiles;
  };

  if (warp == 0 && lane == 0) {  // TMA producer
    const uint64_t pol_w = l2_evict_first(), pol_x = l2_evict_last();
    int it = 0;
    bool ok = true;
    for (int w = first; w < tiles && ok; w += stride) {
      int rank, row, tok;
      place(w, &rank, &row, &tok);
      for (int kb = 0; kb < kpb; ++kb, ++it) {
        const int s = it % S;
        if (it >= S && !local_wait<false>(empty(s), (uint32_t)((it / S - 1) & 1), dc, rank, (int)cta)) {
          ok = false;
          break;
        }
        if (cta == 0) mma_mbar_expect(full(s), 2 * st_bytes);
        const uint32_t sa = base + (uint32_t)s * st_bytes, bar = cluster_addr(full(s), 0);
        tma_load_pair(sa, &maps.w[rank], kb * kMmaBK, row + (int)cta * 128, bar, pol_w);
        tma_load_pair(sa + a_bytes, &maps.x[rank], kb * kMmaBK, tok + (int)cta * (N / 2), bar, pol_x);
      }
    }
  } else if (warp == 1 && lane == 0 && cta == 0) {  // MMA issuer
    const uint32_t ab = a.fp16 ? 0u : 1u;
    const uint32_t idesc = (1u << 4) | (ab << 7) | (ab << 10) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(256 >> 4) << 24);
    int it = 0, i = 0;
    bool ok = true;
    for (int w = first; w < tiles && ok; w += stride, ++i) {
      const int b = i & 1;
      if (i >= 2 && !local_wait<false>(acce(b), (uint32_t)((i / 2 - 1) & 1), dc, 0, 0)) break;
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      for (int kb = 0; kb < kpb; ++kb, ++it) {
        const int s = it % S;
        if (!local_wait<false>(full(s), (uint32_t)((it / S) & 1), dc, 0, 0)) {
          ok = false;
          break;
        }
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const uint32_t sa = base + (uint32_t)s * st_bytes, sb = sa + a_bytes;
#pragma unroll
        for (int kk = 0; kk < kMmaBK / 16; ++kk) {
          const uint64_t ad = mma_smem_desc(sa + (uint32_t)kk * 32u), bd = mma_smem_desc(sb + (uint32_t)kk * 32u);
          asm volatile(
              "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
              "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem + (uint32_t)b * 256u),
              "l"(ad), "l"(bd), "r"(idesc), "r"((kb > 0 || kk > 0) ? 1u : 0u)
              : "memory");
        }
        commit_pair(empty(s));
      }
      if (ok) commit_pair(accf(b));
    }
  } else if (warp >= 2) {  // epilogue
    const int quad = warp & 3;
    int i = 0;
    for (int w = first; w < tiles; w += stride, ++i) {
      int rank, row0, tok;
      place(w, &rank, &row0, &tok);
      const int b = i & 1, row = row0 + (int)cta * 128 + quad * 32 + lane;
      const bool in = row < a.l.rows;
      const bool fp16 = a.fp16 != 0;
      float bias = 0.0f;
      if (a.l.bias[0] && in) {
        const uint16_t v = static_cast<const uint16_t*>(a.l.bias[rank])[row];
        bias = fp16 ? Half16<__half>::widen(v) : Half16<__nv_bfloat16>::widen(v);
      }
      if (!local_wait<false>(accf(b), (uint32_t)((i / 2) & 1), dc, rank, (int)cta)) break;
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      for (int c0 = 0; c0 < N; c0 += 16) {
        uint32_t v[16];
        tmem_ld16(tmem + ((uint32_t)(quad * 32) << 16) + (uint32_t)b * 256u + (uint32_t)c0, v);
        tmem_ld_wait16(v);
        if (c0 + 16 >= N) {  // the accumulator may be overwritten
          asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
          __syncwarp();
          if (lane == 0)
            asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr(acce(b), 0))
                         : "memory");
        }
        const int live = min(16, a.l.tokens - (tok + c0));
        if (!in || live <= 0) continue;
        const size_t off = (size_t)(tok + c0) * a.l.rows + row;
        const uint16_t* res = a.l.res[0] ? static_cast<const uint16_t*>(a.l.res[rank]) + off : nullptr;
        uint16_t* y = static_cast<uint16_t*>(a.l.y[rank]) + off;
        switch (a.l.act) {
          case DCC_ACT_RELU: big_store16<DCC_ACT_RELU>(v, bias, res, y, a.l.rows, live, fp16); break;
          case DCC_ACT_GELU: big_store16<DCC_ACT_GELU>(v, bias, res, y, a.l.rows, live, fp16); break;
          case DCC_ACT_GELU_TANH: big_store16<DCC_ACT_GELU_TANH>(v, bias, res, y, a.l.rows, live, fp16); break;
          case DCC_ACT_SILU: big_store16<DCC_ACT_SILU>(v, bias, res, y, a.l.rows, live, fp16); break;
          default: big_store16<DCC_ACT_NONE>(v, bias, res, y, a.l.rows, live, fp16); break;
        }
      }
    }
  }
  __syncwarp();
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  mma_cluster_sync();  // neither CTA leaves while the other may still reach its barriers
  if (warp == 2) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
}

}  // namespace dcc
