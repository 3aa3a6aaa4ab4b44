// linear_mma.cuh -- the column-parallel linear layer for up to 256 tokens, on
// the fifth-generation tensor cores.
//
// Per rank p, Y_p = act(X_p W_p^T + b_p) + R_p.  Up to 256 tokens the weights
// are read once and the layer is bound by that stream (at 64 tokens and K =
// 8192 some 125 flops a byte, a third of what the tensor cores could do in the
// time).  So, as in the row-parallel layer (fused_mma.cuh), the weights are the
// A operand: a CTA owns up to 128 rows of one rank's W (the MMA's M) for all
// tokens (its N) and a slice of K; the KS CTAs of a cluster split K, so that
// enough CTAs stream when the rows alone are few, and join their partial tiles
// through distributed shared memory, in split order.  Then bias, activation,
// residual and the one rounding follow in registers.  Measured on GB300, 8
// ranks, K = 8192: 1 token x 1024 rows 23.1 us (134 MB, 5.8 TB/s, 86 % of a plain
// copy's rate), 64 tokens x 3584 rows with bias, GELU and residual 81.5 us (478 MB,
// 5.9 TB/s, 87 %).  Roles per CTA (128
// threads, two CTAs to an SM, or 256):
//   warp 0, one thread   TMA: per 64 channels, the rows x 64 tile of W and the
//                         tokens x 64 tile of X (128-byte swizzled, K-major)
//                         onto a stage mbarrier;
//   warp 1, one thread   four tcgen05.mma per stage into fp32 tensor memory;
//   all                  the epilogue.
#pragma once
#include "fused_mma.cuh"
#include "linear.cuh"
#include "tcgen05.cuh"

namespace dcc {

struct LinMaps {
  CUtensorMap w[DCC_MAX_RANKS];  // rows x k, box 64 x bm
  CUtensorMap x[DCC_MAX_RANKS];  // tokens x k, box 64 x ntile
};
struct LinMmaArgs {
  LinArgs l;
  int ntile, ks, stages, bm, tiles, rounds, fp16;  // tiles: row tiles of one rank
};

// 8 sums of neighbouring rows -> bias, activation, residual, one rounding
__device__ __forceinline__ uint4 lin_finish8(float* v, const uint4* bias, const uint4* res, int act, bool fp16) {
  if (bias) {
    float b[8];
    mma_widen8(*bias, fp16, b);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += b[j];
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = lin_act(v[j], act);
  if (res) {
    float r[8];
    mma_widen8(*res, fp16, r);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += r[j];
  }
  return mma_narrow8(v, fp16);
}

// The partial tiles' way: tokens in `rounds` ranges of W, each dealt out to
// the KS CTAs in slices of T; slice o goes to CTA o by one bulk copy into its
// inbox (see mma_epilogue in fused_mma.cuh, whose buffers and barriers these
// are).  part and inbox reuse the stage buffers.
template <int KSC, int THREADS>
__device__ __forceinline__ void lin_epilogue(const LocalDev& dc, const LinMmaArgs& a, uint32_t tmem, float* part,
                                             uint32_t inbar, unsigned split, int rank, int m0, bool acc_ok) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, quad = warp & 3, row = quad * 32 + lane;
  const int R = a.rounds, W = a.ntile / R, T = W / KSC;
  float* inbox = part + (size_t)W * kMmaBM;
  const uint32_t slice_bytes = (uint32_t)T * kMmaBM * 4u;
  const bool fp16 = a.fp16 != 0;
  bool ok = acc_ok;
  for (int r = 0; r < R; ++r) {
    const int w_lo = r * W, t_lo = w_lo + (int)split * T;
    if (r > 0) {
      if (KSC > 1) mma_cluster_sync();
      else __syncthreads();
    }
    if (KSC > 1) {
      if (threadIdx.x == 0) mma_mbar_expect(inbar, (uint32_t)(KSC - 1) * slice_bytes);
      mma_cluster_arrive();
    }
    for (int c0 = w_lo + (warp >> 2) * 16; c0 < w_lo + W; c0 += 16 * (THREADS / 128)) {
      uint32_t v[16];
      tmem_ld16(tmem + ((uint32_t)(quad * 32) << 16) + (uint32_t)c0, v);
      tmem_ld_wait16(v);
#pragma unroll
      for (int j = 0; j < 16; ++j) part[(c0 - w_lo + j) * kMmaBM + row] = acc_ok ? __uint_as_float(v[j]) : 0.0f;
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    if (KSC > 1) {
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncthreads();
      mma_cluster_wait();
      if (threadIdx.x == 0) {
        for (int o = 0; o < KSC; ++o) {
          if (o == (int)split) continue;
          const int slot = (int)split < o ? (int)split : (int)split - 1;
          uint32_t dst, bar;
          const uint32_t ldst = smem_addr_u32(inbox + (size_t)slot * T * kMmaBM);
          asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(dst) : "r"(ldst), "r"((uint32_t)o));
          asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(bar) : "r"(inbar), "r"((uint32_t)o));
          asm volatile(
              "cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
              "r"(smem_addr_u32(part + (size_t)o * T * kMmaBM)), "r"(slice_bytes), "r"(bar)
              : "memory");
        }
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
      }
      if (!local_wait(inbar, (uint32_t)(r & 1), dc, rank, (int)split)) {
        local_drain(inbar, (uint32_t)(r & 1));
        ok = false;
      }
    } else {
      __syncthreads();
    }
    for (int w = threadIdx.x; w < T * (kMmaBM / 8); w += THREADS) {
      const int tl = w / (kMmaBM / 8), r8 = (w % (kMmaBM / 8)) * 8, t = t_lo + tl, mr = m0 + r8;
      if (t >= a.l.tokens || r8 >= a.bm || mr >= a.l.rows) continue;
      const size_t off = (size_t)t * a.l.rows + mr;
      uint4 bias, res;
      if (a.l.bias[0]) bias = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.l.bias[rank]) + mr);
      if (a.l.res[0]) res = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.l.res[rank]) + off);
      float acc[8];
#pragma unroll
      for (int s = 0; s < KSC; ++s) {  // split order
        const float* src = s == (int)split ? &part[((int)split * T + tl) * kMmaBM + r8]
                                           : &inbox[((s < (int)split ? s : s - 1) * T + tl) * kMmaBM + r8];
        const float4 lo = *reinterpret_cast<const float4*>(src), hi = *reinterpret_cast<const float4*>(src + 4);
        const float v8[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] = s == 0 ? v8[j] : acc[j] + v8[j];
      }
      const uint4 out = lin_finish8(acc, a.l.bias[0] ? &bias : nullptr, a.l.res[0] ? &res : nullptr, a.l.act, fp16);
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.l.y[rank]) + off) = out;
    }
    // my copies have read part before it is overwritten or the CTA exits
    if (KSC > 1 && threadIdx.x == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
  }
  (void)ok;
}

template <int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS == kMmaPairThreads ? 2 : 1)
    k_linear_mma(const __grid_constant__ LinMaps maps, LocalDev dc, const __grid_constant__ LinMmaArgs a) {
  extern __shared__ unsigned char lin_raw[];
  __shared__ uint32_t tmem_slot;
  const uint32_t raw_u32 = smem_addr_u32(lin_raw);
  const uint32_t base = (raw_u32 + 1023u) & ~1023u;  // 128-byte swizzle wants 1024-byte alignment
  unsigned char* gbase = lin_raw + (base - raw_u32);
  const int S = a.stages, NTILE = a.ntile, KS = a.ks;
  const uint32_t a_bytes = kMmaBM * kMmaBK * 2, st_bytes = (uint32_t)mma_stage_bytes(NTILE, 1);
  const uint32_t bars = base + (uint32_t)S * st_bytes;  // full[S], empty[S], accumulator ready, inbox full
  auto full = [&](int s) { return bars + 8u * (uint32_t)s; };
  auto empty = [&](int s) { return bars + 8u * (uint32_t)(S + s); };
  const uint32_t accf = bars + 16u * (uint32_t)S, inbar = accf + 8u;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  unsigned split = 0;
  if (KS > 1) asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(split));
  const int tile = (int)blockIdx.x / KS, rank = tile / a.tiles, m0 = (tile - rank * a.tiles) * a.bm;
  // 64-channel blocks; past k the TMA fills both tiles with zeros
  const int kpb = (a.l.k + kMmaBK - 1) / kMmaBK;
  const int b0 = (int)((long long)split * kpb / KS), b1 = (int)((long long)(split + 1) * kpb / KS), nk = b1 - b0;
  const uint32_t ncols = NTILE <= 32 ? 32u : NTILE <= 64 ? 64u : NTILE <= 128 ? 128u : 256u;
  if (warp == 0) {
    for (int j = lane; j < 2 * S + 2; j += 32) mma_mbar_init(bars + 8u * (uint32_t)j, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 2) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr_u32(&tmem_slot)),
                 "r"(ncols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  // overlaps the end of the previous kernel on the stream, as do these prefetches into L2
  if (warp == 3 && lane == 0)
    for (int i = 0; i < nk && i < S; ++i) tma_prefetch_2d(&maps.w[rank], (b0 + i) * kMmaBK, m0);
  pdl_wait();
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  pdl_trigger();  // not before the allocation
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = tmem_slot;

  if (warp == 0 && lane == 0) {  // TMA producer
    const uint32_t tx = st_bytes - (uint32_t)(kMmaBM - a.bm) * (kMmaBK * 2);  // the weight box has bm rows
    const uint64_t pol_w = l2_evict_first(), pol_x = l2_evict_last();
    int i = 0;
    for (; i < nk; ++i) {
      const int s = i % S;
      if (i >= S && !local_wait(empty(s), (uint32_t)(((i / S) - 1) & 1), dc, rank, (int)split)) break;
      const uint32_t sa = base + (uint32_t)s * st_bytes;
      mma_mbar_expect(full(s), tx);
      tma_load_2d_hint(sa, &maps.w[rank], (b0 + i) * kMmaBK, m0, full(s), pol_w);
      tma_load_2d_hint(sa + a_bytes, &maps.x[rank], (b0 + i) * kMmaBK, 0, full(s), pol_x);
    }
    // none is in flight when the CTA leaves, whoever gave up
    for (int j = i > S ? i - S : 0; j < i; ++j) local_drain(full(j % S), (uint32_t)((j / S) & 1));
  } else if (warp == 1 && lane == 0) {  // MMA issuer
    const uint32_t idesc = mma_instr_desc(NTILE, a.fp16 != 0);
    for (int i = 0; i < nk; ++i) {
      const int s = i % S;
      if (!local_wait(full(s), (uint32_t)((i / S) & 1), dc, rank, (int)split)) break;
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      const uint32_t sa = base + (uint32_t)s * st_bytes, sb = sa + a_bytes;
#pragma unroll
      for (int kk = 0; kk < kMmaBK / 16; ++kk) {
        const uint64_t ad = mma_smem_desc(sa + (uint32_t)kk * 32u), bd = mma_smem_desc(sb + (uint32_t)kk * 32u);
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem),
            "l"(ad), "l"(bd), "r"(idesc), "r"((i > 0 || kk > 0) ? 1u : 0u)
            : "memory");
      }
      asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(empty(s))
                   : "memory");
    }
    // arrives once every MMA issued above has completed (at once if none)
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(accf) : "memory");
  }
  __syncwarp();
  const bool acc_ok = nk > 0 && local_wait(accf, 0, dc, rank, (int)split);
  if (!acc_ok) local_drain(accf, 0);
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  float* part = reinterpret_cast<float*>(gbase);  // reuses the stage buffers (all loads consumed)
  if (mma_round_fits(NTILE, S, 1, KS, a.rounds)) {  // the host's plan always does
    switch (KS) {
      case 1: lin_epilogue<1, THREADS>(dc, a, tmem, part, inbar, split, rank, m0, acc_ok); break;
      case 2: lin_epilogue<2, THREADS>(dc, a, tmem, part, inbar, split, rank, m0, acc_ok); break;
      case 4: lin_epilogue<4, THREADS>(dc, a, tmem, part, inbar, split, rank, m0, acc_ok); break;
      default: lin_epilogue<8, THREADS>(dc, a, tmem, part, inbar, split, rank, m0, acc_ok); break;
    }
  } else if (threadIdx.x == 0) {
    atomicCAS(dc.status, 0ull, pack_bounds(rank, kBufScratch, 0));
  }
  __syncthreads();
  if (warp == 2) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(ncols) : "memory");
}

}  // namespace dcc
