// The stand-alone products on CTA pairs (2-SM MMA, M = 256): 256 features x
// up to 512 rows per tile, for problems with enough tiles to be bound by the
// tensor cores.  Same orientation, operands and epilogue as product_gemm.cu.
//
// Operand split of the pair MMA: CTA r supplies features [128 r, 128 r + 128)
// of the tile and half of its rows, and holds its features x all rows of the
// accumulator.
//
// HALVES = 1: tiles of up to 256 rows, the accumulator double-buffered, so the
// epilogue runs below the next tile's mainloop.  At 256 rows an SM's share of a
// slot is 32 KB to load and 512 cycles of MMAs (4096^3: 94 to 98 us, 23 us per
// wave of tiles; the library's product 91 to 93).  Problems of few such tiles
// share them: the pairs of a cluster each take a part of a tile's contraction
// (Split in product_device.cuh; 512 rows 4096 -> 4096 18.6 us in 2 parts, 21.8 on
// one-CTA tiles).
// HALVES = 2: tiles of up to 512 rows in two even accumulators that share the
// features' loads, a quarter less per flop.  They fill tensor memory, so the
// epilogue overlaps the next tile only by skewing them: a tile's first kLead
// slots go to the first accumulator before the second (which still drains),
// its last kLead slots too (the first drains while the second finishes).
// Worth it where it saves a wave of tiles (the choice is in products_api.cu).
//
// Roles per CTA (10 warps): warp 0 TMA producer (own halves; every load
// completes on the leader's full barrier), warp 1 tensor memory and (leader)
// MMA issue, warps 2-9 epilogue, two per accumulator lane quadrant on
// alternate chunks of rows.  Accumulators are taken in turn, one per half, so
// tiles of one half still double-buffer.  Every wait is bounded.  No TMA
// multicast.
//
// Weight gradient: the rows behind the group's last one in its last slot are
// cleared by a warp of their own (warp 10) in each CTA, which waits for that
// slot's loads on a barrier of the slot's, clears, and then signals the
// leader's full barrier (two arrivals per phase: both CTAs' for such a slot,
// else twice the leader's).  (By the producer warp itself the next tile's
// loads waited a load's latency per tile: 198 us against 190 for 16384 rows
// in 36 groups, 4096 x 1280 gradients.)
#include <algorithm>

#include "moe_internal.h"
#include "pair_common.cuh"
#include "product_device.cuh"

namespace moe {

namespace {

using namespace product;

constexpr int kPairBM = 2 * kProductBM;
// warps: producer, MMA, 8 epilogue, and for dw the clearing one
constexpr int threads_of(int mode) { return 32 * (mode == kProductDw ? 11 : 10); }
constexpr int kEpiWarps = 8;
constexpr int kOperand = 2 * kSubBytes;  // 128 rows or features of 64 steps
constexpr int kAccCols = 256;
constexpr int kLead = 2;  // slots by which the first accumulator leads at a tile's ends

// residual chunks on their way; of a split tile, where a pair has few
constexpr int kAhead = 4, kAheadSplit = 2;

template <int HALVES>
struct PairShape {
  static constexpr int kMaxStages = HALVES == 1 ? 8 : 4;
  static constexpr int kBars = 3 * kMaxStages + 6;
  static constexpr int kBarBytes = (kBars + 1) / 2 * 16 + 16;
};

// an accumulator's rows are rounded up to this for the MMA, so that each CTA
// supplies a multiple of 8 (MN-major: of 16; a half of 8 rows more is slow to
// read, 58 us against 45 for 4096 x 1280 gradients)
__host__ __device__ constexpr int pair_unit(int mode) { return mode == kProductDw ? 32 : 16; }
// bytes of a slot's rows per CTA and half, and of a slot
__host__ __device__ constexpr int pair_half_bytes(int mode, int bn) {
  const int rows = product_pair_half(bn, pair_unit(mode)) / 2;
  return mode == kProductDw ? (rows + 63) / 64 * kSubBytes : rows * 128;
}
__host__ __device__ constexpr int pair_slot_bytes(int mode, int halves, bool splits, int bn) {
  return splits ? kOperand + pair_half_bytes(mode, bn) : (1 + halves) * kOperand;
}

__host__ __device__ __forceinline__ int epi_bytes(const ProductParams& p) {
  return kEpiWarps * (p.split > 1 ? epi_warp_bytes(p, 16, kAheadSplit) : epi_warp_bytes(p, 32, kAhead));
}

// Whether the rows behind a dw tile's last one, up to a multiple of 16, are
// another group's (behind the tensor's last row the load fills zeros).
__device__ __forceinline__ bool cleared(const Tile& t, int rows) {
  return (t.depth & 15) != 0 && t.c0 + t.depth < rows;
}

// Rank k of `split` takes a part of the tile's contraction.
__device__ __forceinline__ void take_part(Tile* t, int k, int split) {
  const int64_t nkb = (t->depth + 63) >> 6;
  const int from = static_cast<int>(nkb * k / split) * 64;
  const int to = min(t->depth, static_cast<int>(nkb * (k + 1) / split) * 64);
  t->c0 += from;
  t->depth = to - from;
}

// SPLITS: the tiles' contractions may be shared (a kernel of its own: below the
// others' epilogue its code cost 1 us per call, 1024 rows 4096 -> 4096 27.9 us
// for 26.9, 4096 rows 4096 -> 11264 with gelu 258 for 250).
template <int MODE, int HALVES, typename T, bool SPLITS>
__global__ void __launch_bounds__(threads_of(MODE), 1)
    product_pair_kernel(const __grid_constant__ CUtensorMap tmA,
                        const __grid_constant__ CUtensorMap tmB, const ProductParams p) {
  constexpr bool kAMn = MODE != kProductDx;
  constexpr bool kBMn = MODE == kProductDw;
  // (dw is not split: its contraction may be empty, and ends inside a slot)
  static_assert(!SPLITS || (HALVES == 1 && MODE != kProductDw), "split");
  const int slot_bytes = pair_slot_bytes(MODE, HALVES, SPLITS, p.bn);
  const uint32_t stages = static_cast<uint32_t>(p.stages);
  constexpr int kMaxStages = PairShape<HALVES>::kMaxStages;
  constexpr int kBarBytes = PairShape<HALVES>::kBarBytes;
  constexpr int kUnit = pair_unit(MODE);
  // most rows per accumulator, and this CTA's bytes of one half's rows in a slot
  const int hn_max = product_pair_half(p.bn, kUnit);
  const uint32_t half_bytes = pair_half_bytes(MODE, p.bn);
  // rows per accumulator of a tile: all in one if they fit, else two even halves
  auto half_rows = [&](int n_valid) {
    return HALVES == 1 || n_valid <= hn_max ? n_valid : round_up((n_valid + 1) / 2, kUnit);
  };
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* epi = smem + stages * slot_bytes;
  uint8_t* received = epi + epi_bytes(p);  // of a split tile: what the other pairs send
  uint64_t* bars =
      reinterpret_cast<uint64_t*>(received + (SPLITS ? split_bytes(p.bn, p.split) : 0));
  const uint32_t full0 = smem_u32(bars);
  const uint32_t empty0 = full0 + 8 * kMaxStages;
  const uint32_t tfull0 = empty0 + 8 * kMaxStages;
  const uint32_t tempty0 = tfull0 + 16;
  const uint32_t drain = tempty0 + 16;
  const uint32_t tail0 = drain + 8;
  const uint32_t xfull = tail0 + 8 * kMaxStages;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + PairShape<HALVES>::kBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* tab_mem = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(bars) + kBarBytes);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  // the pairs of a cluster share one tile
  const int split = SPLITS ? p.split : 1;
  const uint32_t in_cluster = cluster_ctarank();
  const uint32_t rank = in_cluster & 1u, leader = in_cluster & ~1u;
  const int pair = blockIdx.x / (2 * split);
  const int n_pairs = gridDim.x / (2 * split);
  const uint16_t both = static_cast<uint16_t>(3u << leader);

  if (threadIdx.x == 0) {
    for (uint32_t s = 0; s < stages; ++s) {
      mbar_init(full0 + 8 * s, 2);
      mbar_init(empty0 + 8 * s, 1);
      mbar_init(tail0 + 8 * s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull0 + 8 * b, 1);
      mbar_init(tempty0 + 8 * b, 2 * kEpiWarps);
    }
    mbar_init(drain, 1);
    mbar_init(xfull, 1);
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
  begin_ordered(p.order);
  const GroupTable tab = build_group_table(tab_mem, p.offsets, p.groups, p.rows, p.bn);
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // both CTAs' barriers are ready before remote use
  pdl_trigger();
  tc_fence_after();
  auto tile_of = [&](int w) {
    Tile t = decode<MODE, kPairBM>(p, tab, w);
    if (SPLITS) take_part(&t, static_cast<int>(in_cluster >> 1), split);
    return t;
  };
  const uint32_t tmem_base = *tmem_slot;
  const int total = p.f_tiles * (MODE == kProductDw ? p.groups * p.dw_blocks
                                                    : tab.block_start[p.groups]);

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    const uint64_t pol = l2_policy_evict_normal();
    const uint32_t full_leader = mapa_shared(full0, leader);
    uint32_t it = 0, s = 0, ph = 0;
    bool ok = true;
    for (int w = pair; w < total && ok; w += n_pairs) {
      const Tile t = tile_of(w);
      const int f = t.f0 + static_cast<int>(rank) * kProductBM;
      // this CTA's first row in each half's MMA
      int j[HALVES], halves = 0;
      const int hn = half_rows(t.n_valid);
#pragma unroll
      for (int h = 0; h < HALVES; ++h) {
        const int n = min(hn, t.n_valid - h * hn);
        if (n > 0) ++halves;
        j[h] = t.j0 + h * hn + static_cast<int>(rank) * (round_up(n, kUnit) / 2);
      }
      const uint32_t box_bytes = kOperand + halves * half_bytes;
      for (int left = t.depth, c = t.c0; left > 0; left -= 64, c += 64) {
        const bool clear = MODE == kProductDw && left < 64 && cleared(t, p.rows);
        if (!(ok = warp_wait(empty0 + 8 * s, ph ^ 1u, abort_flag, p.status))) break;
        if (elect_one()) {
          if (clear) {
            mbar_arrive_expect_tx(tail0 + 8 * s, box_bytes);
          } else if (rank == 0) {
            mbar_arrive_expect_tx(full0 + 8 * s, 2 * box_bytes);
            mbar_arrive(full0 + 8 * s);
          }
          const uint32_t bar = clear ? mapa_shared(tail0 + 8 * s, in_cluster) : full_leader + 8 * s;
          const uint32_t sa = smem_u32(smem) + s * slot_bytes;
          const uint32_t sb = sa + kOperand;
          if (MODE == kProductForward) {
            if (p.wide_a) {
              tma_load_4d_pair(sa, &tmA, bar, 0, c, f >> 6, t.g, pol);
            } else {
              tma_load_3d_pair(sa, &tmA, bar, f, c, t.g, pol);
              tma_load_3d_pair(sa + kSubBytes, &tmA, bar, f + 64, c, t.g, pol);
            }
          } else if (MODE == kProductDx) {
            tma_load_3d_pair(sa, &tmA, bar, c, f, t.g, pol);
          } else {
            tma_load_2d_pair(sa, &tmA, bar, f, c, pol);
            tma_load_2d_pair(sa + kSubBytes, &tmA, bar, f + 64, c, pol);
          }
#pragma unroll
          for (int h = 0; h < HALVES; ++h) {
            if (h >= halves) break;
            if (kBMn) {
              tma_load_2d_pair(sb + h * kOperand, &tmB, bar, j[h], c, pol);
              if (hn_max > 128)
                tma_load_2d_pair(sb + h * kOperand + kSubBytes, &tmB, bar, j[h] + 64, c, pol);
            } else {
              tma_load_2d_pair(sb + h * kOperand, &tmB, bar, c, j[h], pol);
            }
          }
        }
        __syncwarp();
        ++it;
        if (++s == stages) {
          s = 0;
          ph ^= 1u;
        }
      }
    }
    // the leader sees every armed slot complete (both CTAs' loads); the peer is
    // held by the cluster barrier at the end
    if (rank == 0 && lane == 0) {
      const uint32_t used = it < stages ? it : stages;
      for (uint32_t s = 0; s < used; ++s) {
        const uint32_t last = (it - 1u) - ((it - 1u - s) % stages);
        mbar_wait(full0 + 8 * s, (last / stages) & 1u, nullptr, p.status);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (rank == 0) {
      constexpr uint64_t kStepA = (kAMn ? 2048 : 32) >> 4;
      constexpr uint64_t kStepB = (kBMn ? 2048 : 32) >> 4;
      const uint32_t sa = smem_u32(smem);
      const uint64_t ad0 = kAMn ? sdesc_mn_sw128(sa) : sdesc_k_sw<128>(sa);
      const uint64_t bd0 = kBMn ? sdesc_mn_sw128(sa + kOperand) : sdesc_k_sw<128>(sa + kOperand);
      uint32_t s = 0, ph = 0, tc = 0;
      bool any = false, ok = true;
      // the next tile is decoded below the current one's first MMAs
      Tile next{};
      if (pair < total) next = tile_of(pair);
      for (int w = pair; w < total && ok; w += n_pairs) {
        const Tile t = next;
        auto look_ahead = [&]() {
          if (w + n_pairs < total) next = tile_of(w + n_pairs);
        };
        const int nkb = (t.depth + 63) >> 6;
        if (nkb == 0) look_ahead();
        if (nkb == 0) continue;  // an empty group's gradient: the epilogue takes zeros
        any = true;
        uint32_t idesc[HALVES], d[HALVES];
        int halves = 0;
        const int hn = half_rows(t.n_valid);
#pragma unroll
        for (int h = 0; h < HALVES; ++h) {
          const int n = min(hn, t.n_valid - h * hn);
          if (n > 0) ++halves;
          idesc[h] = product_idesc(is_bf16<T>(), kAMn, kBMn, kPairBM, round_up(n, kUnit));
          d[h] = tmem_base + ((tc + h) & 1u) * kAccCols;
        }
        // half h's accumulator is drained
        auto acquire = [&](int h) {
          const uint32_t c = tc + h;
          const bool r = __all_sync(
              0xffffffffu, mbar_wait_cluster(tempty0 + 8 * (c & 1u), ((c >> 1) & 1u) ^ 1u, abort_flag,
                                             p.status));
          tc_fence_after();
          return r;
        };
        // slot k slots on from the current one holds its loads
        auto wait_slot = [&](uint32_t k) {
          const uint32_t q = s + k;
          const uint32_t bar = full0 + 8 * (q < stages ? q : q - stages);
          const uint32_t par = q < stages ? ph : ph ^ 1u;
          // a cleared slot's zeros come from the peer's threads: cluster scope
          const bool r = __all_sync(
              0xffffffffu, MODE == kProductDw ? mbar_wait_cluster(bar, par, abort_flag, p.status)
                                              : mbar_wait(bar, par, abort_flag, p.status));
          tc_fence_after();
          return r;
        };
        // the MMAs of half h on that slot, `left` contraction steps remaining
        auto issue = [&](int h, uint32_t k, int left) {
          const uint32_t q = s + k;
          const uint64_t at = static_cast<uint64_t>((q < stages ? q : q - stages) * (slot_bytes >> 4));
          const uint64_t ad = ad0 + at;
          const uint64_t bd = bd0 + at + static_cast<uint64_t>(h * (kOperand >> 4));
          const uint32_t acc = left < t.depth ? 1u : 0u;
          if (elect_one()) {
            if (left > 48) {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                gemm::mma_issue_pair(d[h], ad + i * kStepA, bd + i * kStepB, idesc[h],
                                     i > 0 ? 1u : acc);
            } else {
              for (int i = 0; i < (left + 15) >> 4; ++i)
                gemm::mma_issue_pair(d[h], ad + i * kStepA, bd + i * kStepB, idesc[h],
                                     i > 0 ? 1u : acc);
            }
          }
          __syncwarp();
        };
        auto release = [&]() {
          if (elect_one()) tc_commit_pair_mc(empty0 + 8 * s, both);  // frees the slot in both CTAs
          __syncwarp();
          if (++s == stages) {
            s = 0;
            ph ^= 1u;
          }
        };
        auto finish = [&](int h) {
          if (elect_one()) tc_commit_pair_mc(tfull0 + 8 * ((tc + h) & 1u), both);
          __syncwarp();
        };
        if (!(ok = acquire(0))) break;
        int left = t.depth;
        if (HALVES == 1 || halves == 1) {
          for (; left > 0; left -= 64) {
            if (!(ok = wait_slot(0))) break;
            issue(0, 0, left);
            release();
            if (left == t.depth) look_ahead();
          }
          if (!ok) break;
          finish(0);
        } else {
          // kLead slots to the first accumulator, then to the second; both on
          // the slots between; the last kLead slots again one after the other
          const int lead = min(kLead, nkb);
          for (int k = 0; k < lead && ok; ++k)
            if ((ok = wait_slot(k))) issue(0, k, left - 64 * k);
          look_ahead();
          if (ok && nkb <= kLead) finish(0);
          if (!ok || !(ok = acquire(1))) break;
          for (int k = 0; k < lead; ++k, left -= 64) {
            issue(1, 0, left);
            release();
          }
          for (; left > 64 * kLead; left -= 64) {
            if (!(ok = wait_slot(0))) break;
            issue(0, 0, left);
            issue(1, 0, left);
            release();
          }
          if (!ok) break;
          if (left > 0) {
            const int rest = (left + 63) >> 6;
            for (int k = 0; k < rest && ok; ++k)
              if ((ok = wait_slot(k))) issue(0, k, left - 64 * k);
            if (!ok) break;
            finish(0);
            for (; left > 0; left -= 64) {
              issue(1, 0, left);
              release();
            }
          }
          finish(1);
        }
        tc += halves;
      }
      if (any) {  // no MMA may still be writing TMEM at deallocation
        if (elect_one()) tc_commit_pair(drain);
        __syncwarp();
        mbar_wait(drain, 0, nullptr, p.status);
      }
    }
  } else if (MODE == kProductDw && warp == 2 + kEpiWarps) {
    // ------------------------------------------------------------ clearing
    const uint32_t full_leader = mapa_shared(full0, leader);
    uint32_t s = 0, phases = 0;  // the slot, and each slot's phase of its tail barrier
    for (int w = pair; w < total; w += n_pairs) {
      const Tile t = tile_of(w);
      const uint32_t nkb = (t.depth + 63) >> 6;
      if (nkb == 0) continue;
      const uint32_t last = (s + nkb - 1) % stages;
      s = (s + nkb) % stages;
      if (!cleared(t, p.rows)) continue;
      if (!warp_wait(tail0 + 8 * last, (phases >> last) & 1u, abort_flag, p.status)) break;
      phases ^= 1u << last;
      const int left = t.depth & 63;
      const int n16 = (((left + 15) & ~15) - left) * 8;  // 16-byte pieces per box
      uint8_t* slot = smem + last * slot_bytes;
      // (boxes that this tile did not load are cleared too, harmlessly)
      for (int i = lane; i < n16 * (slot_bytes / kSubBytes); i += 32) {
        const int box = i / n16;
        *reinterpret_cast<uint4*>(slot + box * kSubBytes + left * 128 + (i - box * n16) * 16) =
            make_uint4(0, 0, 0, 0);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(full_leader + 8 * last);
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;           // the TMEM lane quadrant this warp may read
    const int part = (warp - 2) >> 2;  // which of its quadrant's two warps
    const uint32_t tempty_leader = mapa_shared(tempty0, leader);
    uint8_t* stg = epi + (warp - 2) * (epi_bytes(p) / kEpiWarps);
    uint32_t tc = 0;
    for (int w = pair; w < total; w += n_pairs) {
      const Tile t = tile_of(w);
      const bool empty = t.depth <= 0;
      const int64_t row0 = MODE == kProductDw
                               ? static_cast<int64_t>(t.g) * p.cols + t.j0
                               : static_cast<int64_t>(t.j0);
      bool ok = true;
      const int hn = half_rows(t.n_valid);
      const int f0 = t.f0 + static_cast<int>(rank) * kProductBM + q * 32;
      const Split x(t.n_valid, split, static_cast<int>(in_cluster >> 1), static_cast<int>(rank), 2,
                    smem_u32(smem), smem_u32(received), xfull);
      if (SPLITS && warp == 2 && lane == 0) split_expect(x);
      for (int h = 0; h * hn < t.n_valid; ++h) {
        const uint32_t buf = tc & 1u;
        if (!empty) {
          int go = 1;
          if (lane == 0)
            go = mbar_wait(tfull0 + 8 * buf, (tc >> 1) & 1u, abort_flag, p.status) ? 1 : 0;
          if (!(ok = __shfl_sync(0xffffffffu, go, 0) != 0)) {
            if (SPLITS) split_settle(p, x);
            break;
          }
          tc_fence_after();
        }
        const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + buf * kAccCols;
        if (SPLITS) {  // the launch has a cluster per tile
          split_send(x, taddr, 0, q, part, empty, lane);
          const bool joined = store_tile<MODE, T, 16, kAheadSplit, false, false>(
              p, taddr + x.first(), 0, part, 2, x.rows(x.rank), row0 + x.first(), f0, t.g, empty, stg,
              lane, Joined{x, q, lane, abort_flag, p.status, false});
          if (!joined || f0 >= p.feats) split_settle(p, x);
          break;
        }
        // (two accumulators: choose() takes them for a bias at most)
        store_tile<MODE, T, 32, kAhead, false, HALVES == 2>(
            p, taddr, 0, part, 2, min(hn, t.n_valid - h * hn), row0 + h * hn, f0, t.g, empty, stg,
            lane, Alone{});
        if (!empty) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(tempty_leader + 8 * buf);
          ++tc;
        }
      }
      if (!ok) break;
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
  end_ordered(p.order);
}

template <int HALVES>
size_t slots(int mode, ProductParams* p) {
  using S = PairShape<HALVES>;
  const int slot = pair_slot_bytes(mode, HALVES, p->split > 1, p->bn);
  // (a residual's staging takes a slot's room)
  const int fixed = 1024 + epi_bytes(*p) + split_bytes(p->bn, p->split) + S::kBarBytes +
                    group_table_bytes(p->groups);
  p->stages = std::min(S::kMaxStages, (227 * 1024 - fixed) / slot);
  return p->stages < (HALVES == 1 ? 2 : kLead + 1) ||
                 p->stages * slot < split_out_bytes(p->bn, p->split)
             ? 0
             : static_cast<size_t>(fixed + p->stages * slot);
}

template <int MODE, int HALVES, typename T, bool SPLITS>
cudaError_t launch(const ProductMaps& m, const ProductParams& p0, int grid, cudaStream_t st) {
  ProductParams p = p0;
  const size_t smem = product_pair_slots(MODE, &p);
  if (smem == 0) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(threads_of(MODE));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(2 * p.split);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, product_pair_kernel<MODE, HALVES, T, SPLITS>, m.a, m.b, p);
}

template <int MODE, typename T>
cudaError_t launch_mode(const ProductMaps& m, const ProductParams& p, int grid, cudaStream_t st) {
  if (p.split > 1) {
    if constexpr (MODE != kProductDw) {
      if (p.bn <= kAccCols) return launch<MODE, 1, T, true>(m, p, grid, st);
    }
    return cudaErrorInvalidConfiguration;
  }
  if (p.bn <= kAccCols) return launch<MODE, 1, T, false>(m, p, grid, st);
  if (p.act != MOE_ACT_NONE || p.residual != nullptr || p.preact != nullptr)
    return cudaErrorInvalidConfiguration;
  return launch<MODE, 2, T, false>(m, p, grid, st);
}

template <typename T>
cudaError_t launch_type(int mode, const ProductMaps& m, const ProductParams& p, int grid,
                        cudaStream_t st) {
  if (mode == kProductForward) return launch_mode<kProductForward, T>(m, p, grid, st);
  if (mode == kProductDx) return launch_mode<kProductDx, T>(m, p, grid, st);
  return launch_mode<kProductDw, T>(m, p, grid, st);
}

template <typename T>
cudaError_t configure() {
  cudaError_t e = cudaSuccess;
  auto set = [&](auto kernel) {
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
  };
  set(product_pair_kernel<kProductForward, 1, T, false>);
  set(product_pair_kernel<kProductForward, 1, T, true>);
  set(product_pair_kernel<kProductForward, 2, T, false>);
  set(product_pair_kernel<kProductDx, 1, T, false>);
  set(product_pair_kernel<kProductDx, 1, T, true>);
  set(product_pair_kernel<kProductDx, 2, T, false>);
  set(product_pair_kernel<kProductDw, 1, T, false>);
  set(product_pair_kernel<kProductDw, 2, T, false>);
  return e;
}

}  // namespace

size_t product_pair_slots(int mode, ProductParams* p) {
  p->subs = 1;
  return p->bn <= kAccCols ? slots<1>(mode, p) : slots<2>(mode, p);
}

cudaError_t product_pair_configure_device() {
  const cudaError_t e = configure<__nv_bfloat16>();
  return e != cudaSuccess ? e : configure<__half>();
}

cudaError_t launch_product_pair(int mode, bool bf16, const ProductMaps& m, const ProductParams& p0,
                                int num_sms, cudaStream_t st) {
  ProductParams p = p0;
  const int64_t tiles = product_tile_order(mode, kPairBM, &p);
  if (tiles <= 0) return cudaSuccess;
  if (tiles > (1LL << 30)) return cudaErrorInvalidValue;
  const int grid = p.split > 1 ? static_cast<int>(2 * tiles) * p.split
                               : static_cast<int>(std::min<int64_t>(2 * tiles, num_sms & ~1));
  return bf16 ? launch_type<__nv_bfloat16>(mode, m, p, grid, st)
              : launch_type<__half>(mode, m, p, grid, st);
}

}  // namespace moe
