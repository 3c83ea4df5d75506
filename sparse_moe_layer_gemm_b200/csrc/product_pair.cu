// The stand-alone products on CTA pairs (2-SM MMA, M = 256): 256 features x
// up to 256 rows per tile, for problems with enough tiles to be bound by the
// tensor cores.  Same orientation, operands and epilogue as product_gemm.cu.
//
// Operand split of the pair MMA: CTA r supplies features [128 r, 128 r + 128)
// of the tile and rows [r N/2, (r + 1) N/2), and holds its features x all N
// rows of the accumulator.  One instruction keeps both SMs' tensor cores busy
// for N / 2 cycles, above its issue cost of about 100 from N = 208 on, and a
// byte loaded into shared memory feeds twice the MMAs of a one-CTA tile.
//
// Roles per CTA (10 warps): warp 0 TMA producer (own halves; every load
// completes on the leader's full barrier), warp 1 tensor memory and (leader)
// MMA issue, warps 2-9 epilogue, two per accumulator lane quadrant on
// alternate 16-row chunks, so the epilogue of one tile stays below the next
// tile's mainloop.  Every wait is bounded.  No TMA multicast.
//
// Weight gradient: the rows behind the group's last one in its last slot are
// cleared by each CTA's producer warp, which waits for that slot's loads on a
// barrier of its own, clears, and then signals the leader's full barrier (two
// arrivals per phase: both producers for such a slot, else twice the leader).
#include <algorithm>

#include "moe_internal.h"
#include "pair_common.cuh"
#include "product_device.cuh"

namespace moe {

namespace {

using namespace product;

constexpr int kPairBM = 2 * kProductBM;
constexpr int kThreads = 32 * 10;
constexpr int kEpiWarps = 8;
constexpr int kStages = 6;
constexpr int kOperand = 2 * kSubBytes;  // 128 rows or features of 64 steps
constexpr int kSlot = 2 * kOperand;
constexpr int kAccCols = 256;
constexpr int kBarBytes = (2 * kStages + 6) * 8 + 16;

template <int MODE, typename T>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    product_pair_kernel(const __grid_constant__ CUtensorMap tmA,
                        const __grid_constant__ CUtensorMap tmB, const ProductParams p) {
  constexpr bool kAMn = MODE != kProductDx;
  constexpr bool kBMn = MODE == kProductDw;
  // this CTA's bytes of a slot: its features, and half of the tile's rows
  const uint32_t box_bytes =
      kOperand + (kBMn ? (p.bn / 2 + 63) / 64 * kSubBytes : p.bn / 2 * 128);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kStages * kSlot + kEpiWarps * kEpiWarpBytes);
  const uint32_t full0 = smem_u32(bars);
  const uint32_t empty0 = full0 + 8 * kStages;
  const uint32_t tfull0 = empty0 + 8 * kStages;
  const uint32_t tempty0 = tfull0 + 16;
  const uint32_t drain = tempty0 + 16;
  const uint32_t tail = drain + 8;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * kStages + 6);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* tab_mem = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(bars) + kBarBytes);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int pair = blockIdx.x >> 1;
  const int n_pairs = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full0 + 8 * s, 2);
      mbar_init(empty0 + 8 * s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull0 + 8 * b, 1);
      mbar_init(tempty0 + 8 * b, 2 * kEpiWarps);
    }
    mbar_init(drain, 1);
    mbar_init(tail, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tmA);
    prefetch_tmap(&tmB);
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(tmem_slot), 2 * kAccCols);
    tmem_relinquish_pair();
  }
  pdl_wait();
  const GroupTable tab = build_group_table(tab_mem, p.offsets, p.groups, p.rows, p.bn);
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // both CTAs' barriers are ready before remote use
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int f_tiles = (p.feats + kPairBM - 1) / kPairBM;
  const int total = MODE == kProductDw
                        ? p.groups * f_tiles * ((p.cols + p.bn - 1) / p.bn)
                        : tab.block_start[p.groups] * f_tiles;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    const uint64_t pol = l2_policy_evict_normal();
    const uint32_t full_leader = mapa_shared(full0, 0);
    uint32_t it = 0, tails = 0;
    bool ok = true;
    for (int w = pair; w < total && ok; w += n_pairs) {
      const Tile t = decode<MODE, kPairBM>(p, tab, w);
      const int nkb = (t.depth + 63) >> 6;
      const int half = ((t.n_valid + 15) & ~15) >> 1;  // this CTA's rows of the MMA
      const int f = t.f0 + static_cast<int>(rank) * kProductBM;
      const int j = t.j0 + static_cast<int>(rank) * half;
      for (int kb = 0; kb < nkb; ++kb) {
        const uint32_t s = it % kStages;
        const int left = t.depth - kb * 64;
        const bool clear = MODE == kProductDw && left < 64 && (left & 15) != 0 &&
                           t.c0 + t.depth < p.rows;
        int go = 1;
        if (lane == 0) {
          go = mbar_wait(empty0 + 8 * s, ((it / kStages) & 1u) ^ 1u, abort_flag, p.status) ? 1 : 0;
          if (go) {
            if (clear) {
              mbar_arrive_expect_tx(tail, box_bytes);
            } else if (rank == 0) {
              mbar_arrive_expect_tx(full0 + 8 * s, 2 * box_bytes);
              mbar_arrive(full0 + 8 * s);
            }
            const uint32_t bar = clear ? mapa_shared(tail, rank) : full_leader + 8 * s;
            const uint32_t sa = smem_u32(smem + s * kSlot);
            const uint32_t sb = sa + kOperand;
            const int c = t.c0 + kb * 64;
            if (MODE == kProductForward) {
              tma_load_3d_pair(sa, &tmA, bar, f, c, t.g, pol);
              tma_load_3d_pair(sa + kSubBytes, &tmA, bar, f + 64, c, t.g, pol);
            } else if (MODE == kProductDx) {
              tma_load_3d_pair(sa, &tmA, bar, c, f, t.g, pol);
            } else {
              tma_load_2d_pair(sa, &tmA, bar, f, c, pol);
              tma_load_2d_pair(sa + kSubBytes, &tmA, bar, f + 64, c, pol);
            }
            if (kBMn) {
              tma_load_2d_pair(sb, &tmB, bar, j, c, pol);
              if (p.bn > 128) tma_load_2d_pair(sb + kSubBytes, &tmB, bar, j + 64, c, pol);
            } else {
              tma_load_2d_pair(sb, &tmB, bar, c, j, pol);
            }
            if (clear) go = mbar_wait(tail, tails & 1u, abort_flag, p.status) ? 1 : 0;
          }
        }
        if (!__shfl_sync(0xffffffffu, go, 0)) {
          ok = false;
          break;
        }
        if (clear) {
          const int n16 = (((left + 15) & ~15) - left) * 8;  // 16-byte pieces per box
          const int boxes = static_cast<int>(box_bytes) / kSubBytes;
          uint8_t* slot = smem + s * kSlot;
          for (int i = lane; i < n16 * boxes; i += 32) {
            const int box = i / n16;
            *reinterpret_cast<uint4*>(slot + box * kSubBytes + left * 128 + (i - box * n16) * 16) =
                make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(full_leader + 8 * s);
          ++tails;
        }
        ++it;
      }
    }
    // the leader sees every armed slot complete (both CTAs' loads); the peer is
    // held by the cluster barrier at the end
    if (rank == 0 && lane == 0) {
      const uint32_t used = it < static_cast<uint32_t>(kStages) ? it : kStages;
      for (uint32_t s = 0; s < used; ++s) {
        const uint32_t last = (it - 1u) - ((it - 1u - s) % kStages);
        mbar_wait(full0 + 8 * s, (last / kStages) & 1u, nullptr, p.status);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (rank == 0 && lane == 0) {
      constexpr uint64_t kStepA = (kAMn ? 2048 : 32) >> 4;
      constexpr uint64_t kStepB = (kBMn ? 2048 : 32) >> 4;
      const uint32_t sa = smem_u32(smem);
      const uint64_t ad0 = kAMn ? sdesc_mn_sw128(sa) : sdesc_k_sw<128>(sa);
      const uint64_t bd0 = kBMn ? sdesc_mn_sw128(sa + kOperand) : sdesc_k_sw<128>(sa + kOperand);
      uint32_t it = 0, tc = 0;
      bool ok = true;
      for (int w = pair; w < total && ok; w += n_pairs) {
        const Tile t = decode<MODE, kPairBM>(p, tab, w);
        const int nkb = (t.depth + 63) >> 6;
        if (nkb == 0) continue;  // an empty group's gradient: the epilogue takes zeros
        const uint32_t idesc =
            product_idesc(is_bf16<T>(), kAMn, kBMn, kPairBM, (t.n_valid + 15) & ~15);
        const uint32_t buf = tc & 1u;
        if (!mbar_wait_cluster(tempty0 + 8 * buf, ((tc >> 1) & 1u) ^ 1u, abort_flag, p.status)) break;
        tc_fence_after();
        const uint32_t d = tmem_base + buf * kAccCols;
        for (int kb = 0; kb < nkb; ++kb) {
          const uint32_t s = it % kStages;
          const uint32_t ph = (it / kStages) & 1u;
          // a cleared slot's zeros come from the peer's threads: cluster scope
          if (!(MODE == kProductDw ? mbar_wait_cluster(full0 + 8 * s, ph, abort_flag, p.status)
                                   : mbar_wait(full0 + 8 * s, ph, abort_flag, p.status))) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t ad = ad0 + static_cast<uint64_t>((s * kSlot) >> 4);
          const uint64_t bd = bd0 + static_cast<uint64_t>((s * kSlot) >> 4);
          const int steps = min(4, (t.depth - kb * 64 + 15) >> 4);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (i < steps)
              gemm::mma_issue_pair(d, ad + i * kStepA, bd + i * kStepB, idesc,
                                   (kb > 0 || i > 0) ? 1u : 0u);
          tc_commit_pair_mc(empty0 + 8 * s, 3);  // frees the slot in both CTAs
          ++it;
        }
        if (!ok) break;
        tc_commit_pair_mc(tfull0 + 8 * buf, 3);
        ++tc;
      }
      if (it > 0) {  // no MMA may still be writing TMEM at deallocation
        tc_commit_pair(drain);
        mbar_wait(drain, 0, nullptr, p.status);
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;           // the TMEM lane quadrant this warp may read
    const int part = (warp - 2) >> 2;  // which of its quadrant's two warps
    const uint32_t tempty_leader = mapa_shared(tempty0, 0);
    uint8_t* stg = smem + kStages * kSlot + (warp - 2) * kEpiWarpBytes;
    uint32_t tc = 0;
    for (int w = pair; w < total; w += n_pairs) {
      const Tile t = decode<MODE, kPairBM>(p, tab, w);
      const bool empty = t.depth <= 0;
      const uint32_t buf = tc & 1u;
      const int64_t row0 = MODE == kProductDw
                               ? static_cast<int64_t>(t.g) * p.cols + t.j0
                               : static_cast<int64_t>(t.j0);
      if (!empty) {
        int go = 1;
        if (lane == 0)
          go = mbar_wait(tfull0 + 8 * buf, (tc >> 1) & 1u, abort_flag, p.status) ? 1 : 0;
        if (!__shfl_sync(0xffffffffu, go, 0)) break;
        tc_fence_after();
      }
      const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + buf * kAccCols;
      store_tile<MODE, T>(p, taddr, 16 * part, 32, t.n_valid, row0,
                          t.f0 + static_cast<int>(rank) * kProductBM + q * 32, t.g, empty, stg, lane);
      if (!empty) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(tempty_leader + 8 * buf);
        ++tc;
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  // neither CTA leaves (nor frees TMEM) while its peer may still use its
  // shared memory, barriers or TMEM
  cluster_sync_all();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 2 * kAccCols);
  }
}

template <int MODE, typename T>
cudaError_t launch(const ProductMaps& m, const ProductParams& p, size_t smem, int grid,
                   cudaStream_t st) {
  cudaError_t e = cudaFuncSetAttribute(product_pair_kernel<MODE, T>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
  if (e != cudaSuccess) return e;
  return launch_pdl(product_pair_kernel<MODE, T>, dim3(static_cast<unsigned>(grid)), dim3(kThreads),
                    smem, st, m.a, m.b, p);
}

}  // namespace

cudaError_t launch_product_pair(int mode, bool bf16, const ProductMaps& m, const ProductParams& p,
                                int num_sms, cudaStream_t st) {
  const size_t smem = 1024 + static_cast<size_t>(kStages) * kSlot +
                      kEpiWarps * kEpiWarpBytes + kBarBytes +
                      static_cast<size_t>(group_table_bytes(p.groups));
  const int64_t f_tiles = (p.feats + kPairBM - 1) / kPairBM;
  int64_t tiles;
  if (mode == kProductDw)
    tiles = p.groups * f_tiles * ((p.cols + p.bn - 1) / p.bn);
  else if (p.offsets == nullptr)
    tiles = f_tiles * ((p.rows + p.bn - 1) / p.bn);
  else
    tiles = f_tiles * std::min<int64_t>(p.rows, p.rows / p.bn + p.groups);
  if (tiles <= 0) return cudaSuccess;
  if (tiles > (1LL << 30)) return cudaErrorInvalidValue;
  const int grid = static_cast<int>(std::min<int64_t>(2 * tiles, num_sms & ~1));
  if (bf16) {
    if (mode == kProductForward) return launch<kProductForward, __nv_bfloat16>(m, p, smem, grid, st);
    if (mode == kProductDx) return launch<kProductDx, __nv_bfloat16>(m, p, smem, grid, st);
    return launch<kProductDw, __nv_bfloat16>(m, p, smem, grid, st);
  }
  if (mode == kProductForward) return launch<kProductForward, __half>(m, p, smem, grid, st);
  if (mode == kProductDx) return launch<kProductDx, __half>(m, p, smem, grid, st);
  return launch<kProductDw, __half>(m, p, smem, grid, st);
}

}  // namespace moe
