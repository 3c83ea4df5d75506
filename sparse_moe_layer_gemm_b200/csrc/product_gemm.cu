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
// Few tiles (a decode batch): `split` CTAs of a cluster share a tile, each
// taking a part of its contraction.  The parts meet in shared memory over the
// cluster: the rows of the tile are dealt out to the CTAs, every CTA sends
// its fp32 partial of a row to the row's owner, and the owner adds them in
// rank order (the same sum on every run; no workspace, no counters) and
// finishes the row.
//
// MMAs into one accumulator follow one another only every ~250 cycles at these
// tile sizes (64 slots of a 16-row tile took 35 us, 16 KB per 1000 cycles,
// below what one SM's share of HBM delivers), so a tile keeps 2 or 4
// accumulators, takes them in turn step by step and adds them at the end.
//
// Roles per CTA (6 warps): warp 0 TMA producer, warp 1 tensor memory and MMA
// issue, warps 2-5 epilogue (one accumulator lane quadrant each).  Persistent
// over tiles w = cluster, cluster + clusters, ...; the accumulator is
// double-buffered.  Every wait is bounded (moe_ptx.cuh).
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

constexpr int kThreads = 32 * 6;
constexpr int kABytes = 2 * kSubBytes;
constexpr int kMaxStages = 12;
constexpr int kBarBytes = (2 * kMaxStages + 6) * 8 + 16;

// bytes of the B operand of one slot
__host__ __device__ constexpr int b_bytes(int mode, int bn) {
  return mode == kProductDw ? (bn + 63) / 64 * kSubBytes : bn * 128;
}

// fp32 partials received for this CTA's share of a tile's rows (split), or the
// epilogue warps' staged chunks
__host__ __device__ constexpr int exchange_bytes(int split, int bn) {
  return split > 1 ? split * ((bn + split - 1) / split) * kProductBM * 4 : 4 * kEpiWarpBytes;
}

__device__ __forceinline__ void st_cluster_f32(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// This CTA's slots [kb0, kb1) of a contraction shared by `split` CTAs.
__device__ __forceinline__ void my_slots(int depth, int rank, int split, int* kb0, int* kb1) {
  const int nkb = (depth + 63) >> 6;
  *kb0 = static_cast<int>(static_cast<int64_t>(nkb) * rank / split);
  *kb1 = static_cast<int>(static_cast<int64_t>(nkb) * (rank + 1) / split);
}

template <int MODE, typename T>
__global__ void __launch_bounds__(kThreads, 2)
    product_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                   const ProductParams p) {
  constexpr bool kAMn = MODE != kProductDx;
  constexpr bool kBMn = MODE == kProductDw;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int stages = p.stages;
  const int slot_bytes = kABytes + b_bytes(MODE, p.bn);
  float* xch = reinterpret_cast<float*>(smem + stages * slot_bytes);
  uint64_t* bars = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(xch) +
                                               exchange_bytes(p.split, p.bn));
  const uint32_t full0 = smem_u32(bars);
  const uint32_t empty0 = full0 + 8 * kMaxStages;
  const uint32_t tfull0 = empty0 + 8 * kMaxStages;
  const uint32_t tempty0 = tfull0 + 16;
  const uint32_t drain = tempty0 + 16;
  const uint32_t xfull = drain + 8;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * kMaxStages + 6);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* tab_mem = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(bars) + kBarBytes);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int split = p.split;
  const int rank = split > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int cluster = blockIdx.x / split;
  const int clusters = gridDim.x / split;
  // columns of one accumulator (a power of two); a tile's accumulators, and two
  // sets of them except where the CTA has one tile
  uint32_t chain_cols = 16;
  while (chain_cols < static_cast<uint32_t>(p.bn)) chain_cols <<= 1;
  const int chains = p.bn <= 64 ? 4 : 2;
  const uint32_t acc_cols = chains * chain_cols;
  const uint32_t tmem_cols = split > 1 ? acc_cols : 2 * acc_cols;

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull0 + 8 * b, 1);
      mbar_init(tempty0 + 8 * b, 4);
    }
    mbar_init(drain, 1);
    mbar_init(xfull, 4 * split);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tmA);
    prefetch_tmap(&tmB);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), tmem_cols);
    tmem_relinquish();
  }
  pdl_wait();
  const GroupTable tab = build_group_table(tab_mem, p.offsets, p.groups, p.rows, p.bn);
  tc_fence_before();
  __syncthreads();
  if (split > 1) cluster_sync_all();  // every CTA's barriers are ready before remote use
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int f_tiles = (p.feats + kProductBM - 1) / kProductBM;
  const int total = MODE == kProductDw
                        ? p.groups * f_tiles * ((p.cols + p.bn - 1) / p.bn)
                        : tab.block_start[p.groups] * f_tiles;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      const uint64_t pol = l2_policy_evict_normal();
      uint32_t it = 0, s = 0, ph = 0;
      bool ok = true;
      for (int w = cluster; w < total && ok; w += clusters) {
        const Tile t = decode<MODE, kProductBM>(p, tab, w);
        int kb0, kb1;
        my_slots(t.depth, rank, split, &kb0, &kb1);
        for (int c = t.c0 + kb0 * 64, c1 = t.c0 + kb1 * 64; c < c1; c += 64) {
          if (!mbar_wait(empty0 + 8 * s, ph ^ 1u, abort_flag, p.status)) {
            ok = false;
            break;
          }
          const uint32_t bar = full0 + 8 * s;
          mbar_arrive_expect_tx(bar, slot_bytes);
          const uint32_t sa = smem_u32(smem) + s * slot_bytes;
          const uint32_t sb = sa + kABytes;
          if (MODE == kProductForward) {
            tma_load_3d(sa, &tmA, bar, t.f0, c, t.g, pol);
            tma_load_3d(sa + kSubBytes, &tmA, bar, t.f0 + 64, c, t.g, pol);
          } else if (MODE == kProductDx) {
            tma_load_3d(sa, &tmA, bar, c, t.f0, t.g, pol);
          } else {
            tma_load_2d(sa, &tmA, bar, t.f0, c, pol);
            tma_load_2d(sa + kSubBytes, &tmA, bar, t.f0 + 64, c, pol);
          }
          if (kBMn) {
            for (int h = 0; h < p.bn; h += 64)
              tma_load_2d(sb + h * 128, &tmB, bar, t.j0 + h, c, pol);
          } else {
            tma_load_2d(sb, &tmB, bar, c, t.j0, pol);
          }
          ++it;
          if (++s == static_cast<uint32_t>(stages)) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
      // every load issued lands before the CTA can end
      const uint32_t used = it < static_cast<uint32_t>(stages) ? it : stages;
      for (uint32_t s = 0; s < used; ++s) {
        const uint32_t last = (it - 1u) - ((it - 1u - s) % stages);
        mbar_wait(full0 + 8 * s, (last / stages) & 1u, nullptr, p.status);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    constexpr uint64_t kStepA = (kAMn ? 2048 : 32) >> 4;
    constexpr uint64_t kStepB = (kBMn ? 2048 : 32) >> 4;
    const uint32_t sa0 = smem_u32(smem);
    const uint64_t ad0 = kAMn ? sdesc_mn_sw128(sa0) : sdesc_k_sw<128>(sa0);
    const uint64_t bd0 = kBMn ? sdesc_mn_sw128(sa0 + kABytes) : sdesc_k_sw<128>(sa0 + kABytes);
    uint32_t s = 0, ph = 0, tc = 0;
    bool any = false, ok = true;
    // (the whole warp walks the tiles for dw, whose last slots it clears)
    for (int w = cluster; w < total && ok && (MODE == kProductDw || lane == 0); w += clusters) {
      const Tile t = decode<MODE, kProductBM>(p, tab, w);
      int kb0, kb1;
      my_slots(t.depth, rank, split, &kb0, &kb1);
      if (kb0 == kb1) continue;  // nothing to add: the epilogue takes zeros
      const uint32_t idesc =
          product_idesc(is_bf16<T>(), kAMn, kBMn, kProductBM, (t.n_valid + 15) & ~15);
      const uint32_t buf = tc & 1u;
      int go = 1;
      if (lane == 0)
        go = mbar_wait(tempty0 + 8 * buf, ((tc >> 1) & 1u) ^ 1u, abort_flag, p.status) ? 1 : 0;
      if (MODE == kProductDw) go = __shfl_sync(0xffffffffu, go, 0);
      if (!go) break;
      tc_fence_after();
      any = true;
      const uint32_t d = tmem_base + buf * acc_cols;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (lane == 0) go = mbar_wait(full0 + 8 * s, ph, abort_flag, p.status) ? 1 : 0;
        if (MODE == kProductDw) go = __shfl_sync(0xffffffffu, go, 0);
        if (!go) {
          ok = false;
          break;
        }
        const int left = t.depth - kb * 64;  // contraction steps that exist from here on
        const int steps = min(4, (left + 15) >> 4);
        if (MODE == kProductDw && (left & 15) != 0 && left < 64 && t.c0 + t.depth < p.rows) {
          // steps [left, steps * 16) are another group's rows (behind the tensor's last
          // row the load fills zeros): clear them in every box
          uint8_t* slot = smem + s * slot_bytes;
          const int n16 = (steps * 16 - left) * 8;  // 16-byte pieces per box
          const int boxes = slot_bytes / kSubBytes;
          for (int i = lane; i < n16 * boxes; i += 32) {
            const int box = i / n16;
            *reinterpret_cast<uint4*>(slot + box * kSubBytes + left * 128 + (i - box * n16) * 16) =
                make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        if (lane == 0) {
          tc_fence_after();
          const uint64_t at = static_cast<uint64_t>((s * slot_bytes) >> 4);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (i < steps)
              tc_mma_bf16(d + (chains == 4 ? i : i & 1) * chain_cols, ad0 + at + i * kStepA,
                          bd0 + at + i * kStepB, idesc, (kb > kb0 || i >= chains) ? 1u : 0u);
          tc_commit(empty0 + 8 * s);
          if (kb == kb1 - 1) tc_commit(tfull0 + 8 * buf);
        }
        if (++s == static_cast<uint32_t>(stages)) {
          s = 0;
          ph ^= 1u;
        }
      }
      ++tc;
    }
    if (lane == 0 && any) {  // no MMA may still be writing TMEM at deallocation
      tc_commit(drain);
      mbar_wait(drain, 0, nullptr, p.status);
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;  // the TMEM lane quadrant this warp may read
    uint32_t tc = 0;
    const T* bias = static_cast<const T*>(p.bias);
    uint8_t* stg = reinterpret_cast<uint8_t*>(xch) + (warp - 2) * kEpiWarpBytes;
    for (int w = cluster; w < total; w += clusters) {
      const Tile t = decode<MODE, kProductBM>(p, tab, w);
      int kb0, kb1;
      my_slots(t.depth, rank, split, &kb0, &kb1);
      const bool empty = kb0 == kb1;
      // accumulators in use: all, unless the only slot has fewer steps
      const int used = kb1 - kb0 > 1 ? chains : min(chains, (t.depth - kb0 * 64 + 15) >> 4);
      const uint32_t buf = tc & 1u;
      const int feat = t.f0 + q * 32 + lane;
      const bool live = feat < p.feats;
      const int64_t row0 = MODE == kProductDw
                               ? static_cast<int64_t>(t.g) * p.cols + t.j0
                               : static_cast<int64_t>(t.j0);
      const float b = (MODE == kProductForward && bias != nullptr && live)
                          ? to_f32<T>(bias[static_cast<int64_t>(t.g) * p.feats + feat])
                          : 0.f;
      if (!empty) {
        int go = 1;
        if (lane == 0)
          go = mbar_wait(tfull0 + 8 * buf, (tc >> 1) & 1u, abort_flag, p.status) ? 1 : 0;
        if (!__shfl_sync(0xffffffffu, go, 0)) break;
        tc_fence_after();
      }
      const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + buf * acc_cols;
      const int share = (t.n_valid + split - 1) / split;  // rows each CTA of the cluster finishes
      // where the row's owner takes this CTA's partial of this lane's feature
      const uint32_t xch_addr = smem_u32(xch) + (rank * share * kProductBM + q * 32 + lane) * 4;
      if (split == 1) {
        store_tile<MODE, T>(p, taddr, 0, 16, t.n_valid, row0, t.f0 + q * 32, t.g, empty, stg, lane,
                            used, chain_cols);
      } else {
        int owner = 0, local = 0;  // the row's CTA and its place there
        uint32_t at = mapa_shared(xch_addr, 0);
        for (int c = 0; c < t.n_valid; c += 16) {
          float v[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] = 0.f;
          if (!empty) {
            for (int h = 0; h < used; ++h) {
              uint32_t r[16];
              tmem_ld_x16(taddr + h * chain_cols + c, r);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 16; ++i) v[i] += __uint_as_float(r[i]);
            }
          }
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            if (c + i >= t.n_valid) break;
            st_cluster_f32(at + local * (kProductBM * 4), v[i]);
            if (++local == share) {
              local = 0;
              if (++owner < split) at = mapa_shared(xch_addr, owner);
            }
          }
        }
      }
      if (!empty) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(tempty0 + 8 * buf);
        ++tc;
      }
      if (split > 1) {
        // one tile per cluster in this form (the launch has a cluster per
        // tile), so the exchange area is written once
        __syncwarp();
        if (lane < split) mbar_arrive_cluster(mapa_shared(xfull, lane));
        int go = 1;
        if (lane == 0) go = mbar_wait_cluster(xfull, 0, abort_flag, p.status) ? 1 : 0;
        if (!__shfl_sync(0xffffffffu, go, 0)) break;
        // the waiting lane's acquire orders the other lanes' reads too
        __syncwarp();
        const int mine = min(share, t.n_valid - rank * share);
        for (int j = 0; j < mine; ++j) {
          float part[kProductMaxSplit];
#pragma unroll
          for (int s = 0; s < kProductMaxSplit; ++s)
            part[s] = s < split ? xch[(s * share + j) * kProductBM + q * 32 + lane] : 0.f;
          float v = 0.f;
#pragma unroll
          for (int s = 0; s < kProductMaxSplit; ++s) v += part[s];
          if (live) finish_value<MODE, T>(p, row0 + rank * share + j, feat, b, v);
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (split > 1) cluster_sync_all();  // no CTA leaves while its peers may still reach it
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, tmem_cols);
  }
}

template <int MODE, typename T>
cudaError_t launch(const ProductMaps& m, const ProductParams& p, size_t smem, int grid,
                   cudaStream_t st) {
  cudaError_t e = cudaFuncSetAttribute(product_kernel<MODE, T>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
  if (e != cudaSuccess) return e;
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

size_t product_slot_bytes(int mode, int bn) {
  return static_cast<size_t>(kABytes) + b_bytes(mode, bn);
}

cudaError_t launch_product(int mode, bool bf16, const ProductMaps& m, const ProductParams& p0,
                           int num_sms, cudaStream_t st) {
  ProductParams p = p0;
  const size_t fixed = 1024 + exchange_bytes(p.split, p.bn) + kBarBytes +
                       static_cast<size_t>(group_table_bytes(p.groups));
  const size_t slot = product_slot_bytes(mode, p.bn);
  const int64_t f_tiles = (p.feats + kProductBM - 1) / kProductBM;
  // the most tiles the launch can have (a ragged problem's count is known on the device only)
  int64_t tiles;
  if (mode == kProductDw) {
    tiles = p.groups * f_tiles * ((p.cols + p.bn - 1) / p.bn);
  } else {
    const int64_t blocks = p.offsets == nullptr
                               ? (p.rows + p.bn - 1) / p.bn
                               : std::min<int64_t>(p.rows, p.rows / p.bn + p.groups);
    tiles = blocks * f_tiles;
  }
  if (tiles <= 0) return cudaSuccess;
  if (tiles > (1LL << 30)) return cudaErrorInvalidValue;
  p.stages = static_cast<int>(
      std::min<size_t>(kMaxStages, (static_cast<size_t>(227) * 1024 - fixed) / slot));
  const size_t smem = fixed + p.stages * slot;
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
