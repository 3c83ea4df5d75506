// The stand-alone products on one-CTA tiles (see products.h for the three
// forms): 128 features x up to 128 rows per tile, tcgen05 MMAs into tensor
// memory, TMA-fed slots of 64 contraction steps.
//
// Operands come straight from the caller's tensors.  A tile whose contraction
// index is contiguous in memory is K-major (rows of 128 swizzled bytes); one
// whose feature / row index is contiguous is MN-major: boxes of 64 elements x
// 64 contraction steps, 1024-byte groups of 8 steps (stride offset) and 8 KB
// from one 64-element chunk to the next (leading offset).  So W [K, N] serves
// the forward and dx, and x and dz the weight gradient, with no transposed
// copies.
//
// Few tiles (a decode batch, some hundred rows): `split` CTAs of a cluster share
// a tile, each taking a part of its contraction; see Split in
// product_device.cuh for how their partials meet.
//
// Roles per CTA (12 warps): warps 0 and 1 TMA producers, warp 2 tensor memory,
// warps 2 and 3 MMA issue, warps 4-11 epilogue (two per accumulator lane
// quadrant).  Persistent over tiles w = cluster, cluster + clusters, ...; the
// accumulators are double-buffered.  A producer and an MMA warp are a pipeline
// of their own, with its slots and its accumulator: the first takes the even
// slots of a tile's contraction, the second the odd ones, and the epilogue adds
// the two sums.  With one pipeline a turn of its MMA warp (wait, issue, commit)
// bounds small tiles, whatever their rows: 173 ns per 64 steps at 16 rows, 215 at
// 128 (16 CTAs alone), 135 and 162 with two.  Before that, 16 rows took 475 ns
// with one-lane loops and 350 with whole-warp loops and elect.  With enough tiles HBM is the bound: 512
// rows over 288 groups, 4096 -> 1280, read their weights at 6.6 TB/s; with
// weights in L2 its delivery, 16 bytes a picosecond (512 rows 4096 -> 4096 on 128
// CTAs: 22 us).  Every wait is bounded (moe_ptx.cuh).
//
// Weight gradient: the contraction runs over the group's rows, which end
// inside a slot; the rows behind the last one belong to the next group.  The
// issuing warp clears them in shared memory (both operands: 0 x NaN is NaN)
// up to the MMA's 16 steps before it issues that slot.
#include <algorithm>

#include "moe_internal.h"
#include "product_device.cuh"

namespace moe {

namespace {

using namespace product;

constexpr int kPipes = 2;     // pipelines of a CTA: a producer and an MMA warp each
constexpr int kEpiWarps = 8;  // two per accumulator lane quadrant, on alternate chunks of rows
constexpr int kThreads = 32 * (2 * kPipes + kEpiWarps);
constexpr int kABytes = 2 * kSubBytes;
constexpr int kMaxStages = 4;  // per pipeline: what 64 rows leave room for, the most of all
// sub-slots of 64 contraction steps per slot: two up to 32 rows (32 rows 1280 ->
// 4096 6.8 us with two, 7.3 with one; 64 rows 4096 -> 4096 in 4 parts 11.0 and 9.6)
// where that leaves two slots, so that loads run below MMAs; else one (32 rows
// 4096 -> 1280 in 8 parts 8.0 us with one slot of two, 7.5 with three of one; dw of
// 8000 rows 64 x 72 10.5 and 9.3)
constexpr int subs_of(int bn, size_t room, size_t sub) {
  return bn <= 32 && room >= 4 * sub ? 2 : 1;
}

constexpr int kAhead = 2;  // residual chunks on their way
// staging of the epilogue
__host__ __device__ __forceinline__ int epi_bytes(const ProductParams& p) {
  return kEpiWarps * epi_warp_bytes(p, 16, kAhead);
}
constexpr int kBars = 2 * kPipes * kMaxStages + 4 + kPipes + 1;
constexpr int kBarBytes = (kBars + 1) / 2 * 16 + 16;

// bytes of the B operand of one slot
__host__ __device__ constexpr int b_bytes(int mode, int bn) {
  return mode == kProductDw ? (bn + 63) / 64 * kSubBytes : bn * 128;
}

// The two halves of cluster_sync_all.
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// This CTA's sub-slots [kb0, kb1) of a contraction shared by `split` CTAs.
__device__ __forceinline__ void my_slots(int depth, int rank, int split, int* kb0, int* kb1) {
  const int nkb = (depth + 63) >> 6;
  *kb0 = static_cast<int>(static_cast<int64_t>(nkb) * rank / split);
  *kb1 = static_cast<int>(static_cast<int64_t>(nkb) * (rank + 1) / split);
}

template <int MODE, typename T>
__global__ void __launch_bounds__(kThreads, 1)
    product_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                   const ProductParams p) {
  constexpr bool kAMn = MODE != kProductDx;
  constexpr bool kBMn = MODE == kProductDw;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int stages = p.stages;
  const int sub_bytes = kABytes + b_bytes(MODE, p.bn);
  // what a sub-slot's loads bring: of a problem with fewer rows than the tile
  // only those (what lies behind them in shared memory reaches no kept result)
  const int load_bytes = kABytes + (kBMn ? b_bytes(MODE, p.bn) : p.box_rows * 128);
  const int subs = p.subs;
  const int slot_bytes = subs * sub_bytes;
  uint8_t* epi = smem + kPipes * stages * slot_bytes;
  uint8_t* received = epi + epi_bytes(p);  // of a split tile: what the other CTAs send
  uint64_t* bars = reinterpret_cast<uint64_t*>(received + split_bytes(p.bn, p.split));
  const uint32_t full_all = smem_u32(bars);  // [pipeline][kMaxStages]
  const uint32_t empty_all = full_all + 8 * kPipes * kMaxStages;
  const uint32_t tfull0 = empty_all + 8 * kPipes * kMaxStages;
  const uint32_t tempty0 = tfull0 + 16;
  const uint32_t drain0 = tempty0 + 16;
  const uint32_t xfull = drain0 + 8 * kPipes;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + kBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* tab_mem = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(bars) + kBarBytes);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int split = p.split;
  const int rank = split > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int cluster = blockIdx.x / split;
  const int clusters = gridDim.x / split;
  // accumulator columns, two buffers of one accumulator per pipeline (a power of
  // two, at least 32)
  uint32_t acc_cols = 16;
  while (acc_cols < static_cast<uint32_t>(p.bn)) acc_cols <<= 1;
  const uint32_t buf_cols = kPipes * acc_cols;
  const uint32_t tmem_cols = 2 * buf_cols;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kPipes * kMaxStages; ++s) {
      mbar_init(full_all + 8 * s, 1);
      mbar_init(empty_all + 8 * s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull0 + 8 * b, kPipes);
      mbar_init(tempty0 + 8 * b, kEpiWarps);
    }
    for (int u = 0; u < kPipes; ++u) mbar_init(drain0 + 8 * u, 1);
    mbar_init(xfull, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tmA);
    prefetch_tmap(&tmB);
  }
  if (warp == kPipes) {
    tmem_alloc(smem_u32(tmem_slot), tmem_cols);
    tmem_relinquish();
  }
  begin_ordered(p.order);
  const GroupTable tab = build_group_table(tab_mem, p.offsets, p.groups, p.rows, p.bn);
  tc_fence_before();
  __syncthreads();
  pdl_trigger();
  // this CTA's barriers are ready; the peers' are needed only where the partials
  // meet, so the loads do not wait for them
  if (split > 1) cluster_arrive();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int total = p.f_tiles * (MODE == kProductDw ? p.groups * p.dw_blocks
                                                    : tab.block_start[p.groups]);

  // this warp has passed the cluster barrier above, and has arrived at the next
  bool peers_ready = false, left = false;
  if (warp < kPipes) {
    // ------------------------------------------------------------ producers
    const uint32_t full0 = full_all + 8 * kMaxStages * warp;
    const uint32_t empty0 = empty_all + 8 * kMaxStages * warp;
    const uint32_t ring = smem_u32(smem) + warp * stages * slot_bytes;
    const uint64_t pol = l2_policy_evict_normal();
    uint32_t it = 0, s = 0, ph = 0;
    bool ok = true;
    for (int w = cluster; w < total && ok; w += clusters) {
      const Tile t = decode<MODE, kProductBM>(p, tab, w);
      int kb0, kb1;
      my_slots(t.depth, rank, split, &kb0, &kb1);
      for (int kb = kb0 + warp * subs; kb < kb1; kb += kPipes * subs) {
        if (!(ok = warp_wait(empty0 + 8 * s, ph ^ 1u, abort_flag, p.status))) break;
        const int n = min(subs, kb1 - kb);
        if (elect_one()) {
          const uint32_t bar = full0 + 8 * s;
          mbar_arrive_expect_tx(bar, n * load_bytes);
          uint32_t sa = ring + s * slot_bytes;
          int c = t.c0 + kb * 64;
          for (int i = 0; i < n; ++i, sa += sub_bytes, c += 64) {
            const uint32_t sb = sa + kABytes;
            if (MODE == kProductForward) {
              if (p.wide_a) {
                tma_load_4d(sa, &tmA, bar, 0, c, t.f0 >> 6, t.g, pol);
              } else {
                tma_load_3d(sa, &tmA, bar, t.f0, c, t.g, pol);
                tma_load_3d(sa + kSubBytes, &tmA, bar, t.f0 + 64, c, t.g, pol);
              }
            } else if (MODE == kProductDx) {
              tma_load_3d(sa, &tmA, bar, c, t.f0, t.g, pol);
            } else {
              tma_load_2d(sa, &tmA, bar, t.f0, c, pol);
              tma_load_2d(sa + kSubBytes, &tmA, bar, t.f0 + 64, c, pol);
            }
            if (kBMn) {
              tma_load_2d(sb, &tmB, bar, t.j0, c, pol);
              if (p.bn > 64) tma_load_2d(sb + kSubBytes, &tmB, bar, t.j0 + 64, c, pol);
            } else {
              tma_load_2d(sb, &tmB, bar, c, t.j0, pol);
            }
          }
        }
        __syncwarp();
        ++it;
        if (++s == static_cast<uint32_t>(stages)) {
          s = 0;
          ph ^= 1u;
        }
      }
    }
    // every load issued lands before the CTA can end
    if (lane == 0) {
      const uint32_t used = it < static_cast<uint32_t>(stages) ? it : stages;
      for (uint32_t q = 0; q < used; ++q) {
        const uint32_t last = (it - 1u) - ((it - 1u - q) % stages);
        mbar_wait(full0 + 8 * q, (last / stages) & 1u, nullptr, p.status);
      }
    }
  } else if (warp < 2 * kPipes) {
    // ------------------------------------------------------------ MMA issuers
    const int pipe = warp - kPipes;
    const uint32_t full0 = full_all + 8 * kMaxStages * pipe;
    const uint32_t empty0 = empty_all + 8 * kMaxStages * pipe;
    uint8_t* ring = smem + pipe * stages * slot_bytes;
    constexpr uint64_t kStepA = (kAMn ? 2048 : 32) >> 4;
    constexpr uint64_t kStepB = (kBMn ? 2048 : 32) >> 4;
    const uint32_t sa0 = smem_u32(ring);
    const uint64_t ad0 = kAMn ? sdesc_mn_sw128(sa0) : sdesc_k_sw<128>(sa0);
    const uint64_t bd0 = kBMn ? sdesc_mn_sw128(sa0 + kABytes) : sdesc_k_sw<128>(sa0 + kABytes);
    uint32_t s = 0, ph = 0, tc = 0;
    bool any = false, ok = true;
    for (int w = cluster; w < total && ok; w += clusters) {
      const Tile t = decode<MODE, kProductBM>(p, tab, w);
      int kb0, kb1;
      my_slots(t.depth, rank, split, &kb0, &kb1);
      if (kb0 == kb1) continue;  // nothing to add: the epilogue takes zeros
      const uint32_t idesc =
          product_idesc(is_bf16<T>(), kAMn, kBMn, kProductBM, (t.n_valid + 15) & ~15);
      const uint32_t buf = tc & 1u;
      if (!warp_wait(tempty0 + 8 * buf, ((tc >> 1) & 1u) ^ 1u, abort_flag, p.status)) break;
      tc_fence_after();
      ++tc;
      const int first = kb0 + pipe * subs;
      if (first >= kb1) {  // all of it is the first pipeline's
        if (lane == 0) mbar_arrive(tfull0 + 8 * buf);
        __syncwarp();
        continue;
      }
      any = true;
      const uint32_t d = tmem_base + buf * buf_cols + pipe * acc_cols;
      uint32_t acc = 0;
      for (int kb = first; kb < kb1; kb += kPipes * subs) {
        if (!(ok = warp_wait(full0 + 8 * s, ph, abort_flag, p.status))) break;
        // contraction steps of this CTA that exist from here on
        const int left = min(t.depth, kb1 * 64) - kb * 64;
        if (MODE == kProductDw && (left & 15) != 0 && left < 64 * subs &&
            t.c0 + t.depth < p.rows) {
          // up to the next multiple of 16 the steps are another group's rows (behind
          // the tensor's last row the load fills zeros): clear them in every box
          uint8_t* sub = ring + s * slot_bytes + (left >> 6) * sub_bytes;
          const int from = left & 63;
          const int n16 = (((from + 15) & ~15) - from) * 8;  // 16-byte pieces per box
          const int boxes = sub_bytes / kSubBytes;
          for (int i = lane; i < n16 * boxes; i += 32) {
            const int box = i / n16;
            *reinterpret_cast<uint4*>(sub + box * kSubBytes + from * 128 + (i - box * n16) * 16) =
                make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        tc_fence_after();
        if (elect_one()) {
          uint64_t ad = ad0 + static_cast<uint64_t>((s * slot_bytes) >> 4);
          uint64_t bd = bd0 + static_cast<uint64_t>((s * slot_bytes) >> 4);
          if (left > 64 * subs - 16) {
            for (int h = 0; h < subs; ++h) {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                tc_mma_bf16(d, ad + i * kStepA, bd + i * kStepB, idesc, h + i > 0 ? 1u : acc);
              ad += sub_bytes >> 4;
              bd += sub_bytes >> 4;
            }
          } else {
            for (int i = 0; i < (left + 15) >> 4; ++i) {
              if (i == 4) {
                ad += (sub_bytes >> 4) - 4 * kStepA;
                bd += (sub_bytes >> 4) - 4 * kStepB;
              }
              tc_mma_bf16(d, ad + i * kStepA, bd + i * kStepB, idesc, i > 0 ? 1u : acc);
            }
          }
          tc_commit(empty0 + 8 * s);
          if (kb + kPipes * subs >= kb1) tc_commit(tfull0 + 8 * buf);
        }
        __syncwarp();
        acc = 1;
        if (++s == static_cast<uint32_t>(stages)) {
          s = 0;
          ph ^= 1u;
        }
      }
    }
    if (any) {  // no MMA may still be writing TMEM at deallocation
      if (elect_one()) tc_commit(drain0 + 8 * pipe);
      __syncwarp();
      mbar_wait(drain0 + 8 * pipe, 0, nullptr, p.status);
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;  // the TMEM lane quadrant this warp may read
    uint32_t tc = 0;
    const int epi_warp = warp - 2 * kPipes;
    const int part = epi_warp >> 2;  // which of its quadrant's warps
    uint8_t* stg = epi + epi_warp * (epi_bytes(p) / kEpiWarps);
    for (int w = cluster; w < total; w += clusters) {
      const Tile t = decode<MODE, kProductBM>(p, tab, w);
      int kb0, kb1;
      my_slots(t.depth, rank, split, &kb0, &kb1);
      const bool empty = kb0 == kb1;
      const uint32_t buf = tc & 1u;
      const int64_t row0 = MODE == kProductDw
                               ? static_cast<int64_t>(t.g) * p.cols + t.j0
                               : static_cast<int64_t>(t.j0);
      const Split x(t.n_valid, split, rank, 0, 1, smem_u32(smem), smem_u32(received),
                    xfull);
      if (split > 1) {
        if (epi_warp == 0 && lane == 0) split_expect(x);
        cluster_wait();
        peers_ready = true;
      }
      if (!empty) {
        int go = 1;
        if (lane == 0)
          go = mbar_wait(tfull0 + 8 * buf, (tc >> 1) & 1u, abort_flag, p.status) ? 1 : 0;
        if (!__shfl_sync(0xffffffffu, go, 0)) {
          if (split > 1) split_settle(p, x);
          break;
        }
        tc_fence_after();
      }
      const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + buf * buf_cols;
      // the second pipeline's accumulator, if it had a part
      const uint32_t second = kb1 - kb0 > subs ? acc_cols : 0;
      if (split == 1) {
        store_tile<MODE, T, 16, kAhead, true, false>(p, taddr, second, part, kEpiWarps / 4, t.n_valid, row0,
                                              t.f0 + q * 32, t.g, empty, stg, lane, Alone{});
        if (!empty) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(tempty0 + 8 * buf);
          ++tc;
        }
        continue;
      }
      // one tile per cluster in this form (the launch has a cluster per tile)
      split_send(x, taddr, second, q, part, empty, lane);
      // (the warp of the first features waits for all that is sent here as it joins)
      if (!store_tile<MODE, T, 16, kAhead, true, false>(
              p, taddr + x.first(), second, part, kEpiWarps / 4, x.rows(rank), row0 + x.first(),
              t.f0 + q * 32, t.g, empty, stg, lane, Joined{x, q, lane, abort_flag, p.status, false}))
        split_settle(p, x);
      cluster_arrive();
      left = true;
      break;
    }
  }

  tc_fence_before();
  if (split > 1 && !peers_ready) cluster_wait();
  if (split > 1 && !left) cluster_arrive();
  __syncthreads();
  if (warp == kPipes) {
    tc_fence_after();
    tmem_dealloc(tmem_base, tmem_cols);
  }
  if (split > 1) cluster_wait();  // what this CTA sent has been received
  end_ordered(p.order);
}

template <int MODE, typename T>
cudaError_t launch(const ProductMaps& m, const ProductParams& p, size_t smem, int grid,
                   cudaStream_t st) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(p.split);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, product_kernel<MODE, T>, m.a, m.b, p);
}

}  // namespace

cudaError_t product_configure_device() {
  cudaError_t e = cudaSuccess;
  auto set = [&](auto kernel) {
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
  };
  set(product_kernel<kProductForward, __nv_bfloat16>);
  set(product_kernel<kProductDx, __nv_bfloat16>);
  set(product_kernel<kProductDw, __nv_bfloat16>);
  set(product_kernel<kProductForward, __half>);
  set(product_kernel<kProductDx, __half>);
  set(product_kernel<kProductDw, __half>);
  return e;
}

cudaError_t product_cluster_room(int cluster, int* ctas) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = 227 * 1024;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  const cudaError_t e =
      cudaOccupancyMaxActiveClusters(&n, product_kernel<kProductForward, __nv_bfloat16>, &cfg);
  *ctas = n * cluster;
  return e;
}

size_t product_slots(int mode, ProductParams* p) {
  const size_t fixed = 1024 + static_cast<size_t>(epi_bytes(*p) + split_bytes(p->bn, p->split)) +
                       kBarBytes + static_cast<size_t>(group_table_bytes(p->groups));
  const size_t sub = kPipes * (kABytes + static_cast<size_t>(b_bytes(mode, p->bn)));
  const size_t room = static_cast<size_t>(227) * 1024 - fixed;
  p->subs = subs_of(p->bn, room, sub);
  const size_t slot = p->subs * sub;
  p->stages = static_cast<int>(std::min<size_t>(kMaxStages, room / slot));
  return p->stages < 1 || p->stages * slot < static_cast<size_t>(split_out_bytes(p->bn, p->split))
             ? 0
             : fixed + p->stages * slot;
}

cudaError_t launch_product(int mode, bool bf16, const ProductMaps& m, const ProductParams& p0,
                           int num_sms, cudaStream_t st) {
  ProductParams p = p0;
  const int64_t tiles = product_tile_order(mode, kProductBM, &p);
  if (tiles <= 0) return cudaSuccess;
  if (tiles > (1LL << 30)) return cudaErrorInvalidValue;
  const size_t smem = product_slots(mode, &p);
  if (smem == 0) return cudaErrorInvalidConfiguration;
  const int grid =
      p.split > 1 ? static_cast<int>(tiles) * p.split : static_cast<int>(std::min<int64_t>(tiles, num_sms));
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
