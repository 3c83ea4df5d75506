// Device pieces shared by the stand-alone products: the two 16-bit types, the
// activations, the table of a ragged problem's groups.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/moe.h"
#include "moe_ptx.cuh"
#include "products.h"

namespace moe {
namespace product {

// Launch order of the kernels (see LaunchOrder in products.h).
__device__ __forceinline__ void pdl_trigger() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void begin_ordered(LaunchOrder o) {
  if (!o.late_wait) pdl_wait();
}
__device__ __forceinline__ void end_ordered(LaunchOrder o) {
  if (o.late_wait) pdl_wait();
}

template <typename T>
constexpr bool is_bf16() {
  return __is_same(T, __nv_bfloat16);
}

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }

// one rounding to nearest even
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }

// Activations and their slopes in fp32, cheap enough to hide below a tile's
// MMAs (two special-function operations per value at most).
//
// gelu: the normal distribution function from erfc(x) = t Q(t) exp(-x^2),
// t = 1 / (1 + 0.6 x), x >= 0, Q a degree-7 polynomial fitted here to
// exp(x^2) erfc(x) / t over 0 <= x <= 10 by reweighted least squares (relative
// error 3.2e-7 with the coefficients below; gelu as evaluated here 1.9e-6 for
// -6 < z < 0 and 8e-6 down to -13, from the exponent's rounding, 6.7e-7 above
// -1).  The tail keeps its relative accuracy, where 1 + erf cancels.
// (4096 x 4096 -> 11264: 12 us over no activation; erfcf in its place 87 us.)
// gelu_tanh is 0.5 (1 + tanh u) = sigmoid(2 u), for the same reason.
constexpr float kInvSqrt2Pi = 0.39894228040143268f;
constexpr float kTanhScale = 0.79788456080286536f;  // sqrt(2 / pi)
constexpr float kTanhCubic = 0.044715f;

// one special-function instruction each, to a few units of 2^-23
__device__ __forceinline__ float reciprocal(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float exp2_fast(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
constexpr float kLog2e = 1.4426950408889634f;

// 4 / (1 + exp(-z)); an exponential of infinity (z < -88.7) gives 0.  A quarter
// of the sum is inverted, since rcp gives 0 for what passes 2^126 (z < -87.3)
// and silu and its slope are normal numbers there.
__device__ __forceinline__ float sigmoid_times_4(float z) {
  return reciprocal(fmaf(0.25f, exp2_fast(-kLog2e * z), 0.25f));
}
__device__ __forceinline__ float sigmoid(float z) { return 0.25f * sigmoid_times_4(z); }

// Phi(z), and exp(-z^2 / 2)
__device__ __forceinline__ float normal_cdf(float z, float* e) {
  const float a = fabsf(z);
  const float t = reciprocal(fmaf(0.6f * 0.70710678118654752f, a, 1.0f));
  float q = -0.09208406507968903f;
  q = fmaf(q, t, 0.411952942609787f);
  q = fmaf(q, t, -0.6444682478904724f);
  q = fmaf(q, t, 0.28378206491470337f);
  q = fmaf(q, t, 0.07340489327907562f);
  q = fmaf(q, t, 0.2916032075881958f);
  q = fmaf(q, t, 0.3372488021850586f);
  q = fmaf(q, t, 0.3385601043701172f);
  *e = exp2_fast(-0.5f * kLog2e * z * z);
  const float half_erfc = 0.5f * t * q * *e;
  return z < 0.f ? half_erfc : 1.0f - half_erfc;
}

__device__ __forceinline__ float activate(float z, int act) {
  switch (act) {
    case MOE_ACT_RELU:
      return z < 0.f ? 0.f : z;  // NaN stays NaN
    case MOE_ACT_SILU:
      return z * sigmoid(z);
    case MOE_ACT_GELU: {
      float e;
      return z * normal_cdf(z, &e);
    }
    case MOE_ACT_GELU_TANH:
      return z * sigmoid(2.0f * kTanhScale * (z + kTanhCubic * z * z * z));
    default:
      return z;
  }
}

__device__ __forceinline__ float activation_slope(float z, int act) {
  switch (act) {
    case MOE_ACT_RELU:
      return z > 0.f ? 1.f : (z <= 0.f ? 0.f : z);  // NaN stays NaN
    case MOE_ACT_SILU: {
      const float s = sigmoid(z);
      return s * (1.0f + z * (1.0f - s));
    }
    case MOE_ACT_GELU: {
      float e;
      const float c = normal_cdf(z, &e);
      return c + z * kInvSqrt2Pi * e;
    }
    case MOE_ACT_GELU_TANH: {
      // beyond 20 the sigmoid is 0 or 1 in fp32, and z^2 may overflow
      if (fabsf(z) > 20.f) return z > 0.f ? 1.f : 0.f;
      const float z2 = z * z;
      const float s = sigmoid(2.0f * kTanhScale * z * (1.0f + kTanhCubic * z2));
      return s + z * s * (1.0f - s) * 2.0f * kTanhScale * (1.0f + 3.0f * kTanhCubic * z2);
    }
    default:
      return 1.f;
  }
}

// The groups of a ragged problem in shared memory: row0[g] the first row of
// group g, row0[groups] the end of the last, block_start[g] the exclusive
// prefix of ceil(rows of g / unit).  Offsets are clamped into [0, rows] and
// raised to the largest before them, so whatever the device holds the groups
// do not overlap and no row outside the tensors is touched.  All threads of
// the CTA call it; the table is complete after its closing __syncthreads.
struct GroupTable {
  int* block_start;  // [groups + 1]
  int* row0;         // [groups + 1]
  int* block_rows;   // [groups]
  __device__ __forceinline__ int count(int g) const { return row0[g + 1] - row0[g]; }
};

constexpr int group_table_bytes(int groups) { return 3 * (groups + 1) * 4; }

__host__ __device__ constexpr int round_up(int v, int m) { return (v + m - 1) / m * m; }

__device__ __forceinline__ GroupTable build_group_table(int* mem, const int* offsets, int groups,
                                                        int rows, int unit) {
  GroupTable t{mem, mem + groups + 1, mem + 2 * (groups + 1)};
  if (offsets == nullptr) {
    if (threadIdx.x == 0) {
      t.row0[0] = 0;
      t.row0[1] = rows;
      const int blocks = (rows + unit - 1) / unit;
      t.block_start[0] = 0;
      t.block_start[1] = blocks;
      t.block_rows[0] = min(unit, round_up((rows + blocks - 1) / max(blocks, 1), 16));
    }
    __syncthreads();
    return t;
  }
  for (int g = threadIdx.x; g <= groups; g += blockDim.x)
    t.row0[g] = min(max(offsets[g], 0), rows);
  __syncthreads();
  if (threadIdx.x < 32) {
    const int lane = static_cast<int>(threadIdx.x);
    int last = 0, base = 0;  // the largest offset and the blocks before this step's groups
    for (int g0 = 0; g0 <= groups; g0 += 32) {
      const int g = g0 + lane;
      int m = max(last, g <= groups ? t.row0[g] : 0);
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, m, d);
        if (lane >= d) m = max(m, v);
      }
      // blocks of group g - 1, which ends at offset g
      int before = __shfl_up_sync(0xffffffffu, m, 1);
      if (lane == 0) before = g0 == 0 ? m : last;
      int s = (m - before + unit - 1) / unit;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, s, d);
        if (lane >= d) s += v;
      }
      if (g <= groups) {
        t.row0[g] = m;
        t.block_start[g] = base + s;
      }
      last = __shfl_sync(0xffffffffu, m, 31);
      base += __shfl_sync(0xffffffffu, s, 31);
    }
  }
  __syncthreads();
  for (int g = threadIdx.x; g < groups; g += blockDim.x) {
    const int blocks = max(t.block_start[g + 1] - t.block_start[g], 1);
    t.block_rows[g] = min(unit, round_up((t.count(g) + blocks - 1) / blocks, 16));
  }
  __syncthreads();
  return t;
}

// The group whose blocks hold block b (the last g with block_start[g] <= b;
// empty groups are skipped).
__device__ __forceinline__ int group_of_block(const GroupTable& t, int groups, int b) {
  int lo = 0, hi = groups;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (t.block_start[mid] <= b)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// One lane of the (converged) warp, the same at every call.  The tcgen05 and
// TMA instructions take warp-uniform registers: issued inside a loop that the
// whole warp walks, under this predicate, their operands stay there (a loop
// walked by one lane alone cost half as much again: see product_gemm.cu).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}\n"
      : "=r"(p));
  return p != 0;
}

// 4-D tiled TMA load into this CTA's shared memory.  No multicast.
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                            int x, int y, int z, int w, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4, %5}], [%6], %7;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar), "l"(policy)
      : "memory");
}

// mbar_wait by the whole warp, which continues or stops together.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort,
                                          int* status) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, status));
}

constexpr int kSubBytes = 64 * 128;  // one MN-major box: 64 steps x 64 elements

__device__ __forceinline__ bool mbar_try_wait_cluster(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// mbar_wait with cluster scope: what the arriving CTAs wrote here is visible.
__device__ __forceinline__ bool mbar_wait_cluster(uint32_t bar, uint32_t parity,
                                                  volatile int* abort, int* status) {
  if (mbar_try_wait_cluster(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  for (;;) {
#pragma unroll 1
    for (int i = 0; i < 32; ++i)
      if (mbar_try_wait_cluster(bar, parity)) return true;
    if (*abort) return false;
    if (global_timer_ns() - t0 > kWaitLimitNs) {
      *abort = 1;
      atomicOr(status, kDevErrTimeout);
      return false;
    }
  }
}

// Shared-memory matrix descriptor of an MN-major operand with the 128-byte
// swizzle: 64-element chunks 8 KB apart (leading byte offset), groups of 8
// contraction steps 1 KB apart (stride byte offset), descriptor version 1,
// layout type 2.
__device__ __forceinline__ uint64_t sdesc_mn_sw128(uint32_t saddr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(kSubBytes >> 4) << 16;
  d |= static_cast<uint64_t>(1024 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}

// Instruction descriptor of kind::f16 with 128 x n accumulators in fp32.
__device__ __forceinline__ uint32_t product_idesc(bool bf16, bool a_mn, bool b_mn, int m, int n) {
  return (1u << 4) | ((bf16 ? 1u : 0u) << 7) | ((bf16 ? 1u : 0u) << 10) |
         ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
         (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}

struct Tile {
  int g;        // group
  int f0;       // first feature
  int j0;       // first row of the tile: of the tensor (forward, dx) or of the group's output (dw)
  int n_valid;  // rows of the tile
  int c0;       // first contraction index (dw: row of the tensor)
  int depth;    // contraction length
};

__device__ __forceinline__ int divide(int n, const FastDiv& f) {
  return static_cast<int>((__umulhi(static_cast<uint32_t>(n), f.mul) + static_cast<uint32_t>(n)) >>
                          f.shift);
}

// Tile w.  Inside a group, chunks of p.chunk row blocks run feature-major: a
// weight tile's readers follow one another, and the chunk's rows stay in L2
// across its weight tiles.
template <int MODE, int BM>
__device__ __forceinline__ Tile decode(const ProductParams& p, const GroupTable& t, int w) {
  Tile r;
  int local, blocks;
  const int b = divide(w, p.by_group);  // dw: the group, else the row block over all groups
  if (MODE == kProductDw) {
    blocks = p.dw_blocks;
    r.g = b;
    local = w - b * static_cast<int>(p.by_group.d);
  } else {
    r.g = group_of_block(t, p.groups, b);
    local = w - t.block_start[r.g] * p.f_tiles;
    blocks = t.block_start[r.g + 1] - t.block_start[r.g];
  }
  const int c = divide(local, p.by_chunk);
  const int rem = local - c * static_cast<int>(p.by_chunk.d);
  const int first = c * p.chunk;
  const int in_chunk = min(p.chunk, blocks - first);
  // rem < 2^13, in_chunk <= 16: the rounded quotient of rem + 1/2 truncates right
  const int ft = static_cast<int>((static_cast<float>(rem) + 0.5f) *
                                  reciprocal(static_cast<float>(in_chunk)));
  const int nb = first + (rem - ft * in_chunk);
  r.f0 = ft * BM;
  if (MODE == kProductDw) {
    r.j0 = nb * p.dw_rows;
    r.n_valid = min(p.dw_rows, p.cols - r.j0);
    r.c0 = t.row0[r.g];
    r.depth = t.count(r.g);
  } else {
    const int size = t.block_rows[r.g];
    r.j0 = t.row0[r.g] + nb * size;
    r.n_valid = min(size, t.count(r.g) - nb * size);
    r.c0 = 0;
    r.depth = p.depth;
  }
  return r;
}

// ---------------------------------------------------------------- epilogue
// An accumulator holds features on its lanes and output rows on its columns;
// the output is row-major with features contiguous.  A warp takes 32 features
// x 32 rows at a time on pair tiles (16 on one-CTA tiles, or with a residual or
// pre-activation) as two 16x256b tensor-memory loads per 16 rows: the values
// then lie in the registers as 8 x 8 matrices (feature lane / 4, rows 2 (lane %
// 4) and + 1), so after packing two rows into 32 bits one transposing stmatrix
// per 8 rows lays [row][32 features] into shared memory, from where 16-byte
// pieces go out (4 or 2 bytes where the rows' alignment allows no more), 64
// contiguous bytes per row.  The residual comes in the same way backwards.  Against one 2-byte store per value, 4096 rows 64 -> 4096 went
// from 95 to 20 us (33.5 MB written).
constexpr int kEpiPitch = 80;                  // bytes per staged row: 64 + 16 against bank conflicts
constexpr int kEpiChunk = 16 * kEpiPitch;      // one staged chunk
// bytes per warp: `rows` rows, or 16 and a ring of `ahead` chunks of the residual
__host__ __device__ __forceinline__ int epi_warp_bytes(const ProductParams& p, int rows, int ahead) {
  return p.residual != nullptr ? (1 + ahead) * kEpiChunk : rows / 16 * kEpiChunk;
}

__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void tmem_ld_16x256b_x2(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7])
      : "r"(taddr));
}

__device__ __forceinline__ void stmatrix_x4_trans(uint32_t addr, const uint32_t (&r)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
               : "memory");
}

__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// two fp32 values rounded into one register, `lo` in the low half
template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t v);
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t v) {
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&v));
}
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t v) {
  return __half22float2(*reinterpret_cast<const __half2*>(&v));
}

// ROWS staged rows x 32 features <-> global memory at `base` (the chunk's first
// row and this warp's first feature); n rows and nf features exist.  W
// elements per access (8, 2 or 1, as the rows' alignment allows), 32 / W lanes
// per row, eight accesses under way at once.
template <int W>
struct Access;
template <>
struct Access<8> {
  using Type = uint4;
};
template <>
struct Access<2> {
  using Type = uint32_t;
};
template <>
struct Access<1> {
  using Type = uint16_t;
};

template <typename T, int ROWS, int W, bool OUT>
__device__ __forceinline__ void copy_staged(uint8_t* stg, T* base, int64_t ld, int n, int nf,
                                            int lane) {
  using V = typename Access<W>::Type;
  constexpr int kLanes = 32 / W, kPer = 32 / kLanes;  // lanes per row, rows per access
  constexpr int kBatch = ROWS / kPer < 8 ? ROWS / kPer : 8;
  const int col = (lane % kLanes) * W, row = lane / kLanes;
  const bool whole = col + W <= nf;
  uint8_t* s = stg + row * kEpiPitch + col * 2;
  T* at = base + row * ld + col;
#pragma unroll
  for (int k0 = 0; k0 < ROWS / kPer; k0 += kBatch) {
    V v[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int r = (k0 + k) * kPer;
      if (OUT)
        v[k] = *reinterpret_cast<const V*>(s + r * kEpiPitch);
      else if (whole && r + row < n)
        v[k] = *reinterpret_cast<const V*>(at + r * ld);
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int r = (k0 + k) * kPer;
      if (!whole || r + row >= n) continue;
      if (OUT)
        *reinterpret_cast<V*>(at + r * ld) = v[k];
      else
        *reinterpret_cast<V*>(s + r * kEpiPitch) = v[k];
    }
  }
  if (W == 2 && col + 1 == nf) {  // the odd last feature
    for (int r = 0; r + row < n; r += kPer) {
      T* e = reinterpret_cast<T*>(s + r * kEpiPitch);
      if (OUT)
        at[r * ld] = *e;
      else
        *e = at[r * ld];
    }
  }
}

template <typename T, int ROWS, bool OUT>
__device__ __forceinline__ void copy_rows(uint8_t* stg, T* base, int64_t ld, int n, int nf, int width,
                                          int lane) {
  if (width == 8)
    copy_staged<T, ROWS, 8, OUT>(stg, base, ld, n, nf, lane);
  else if (width == 2)
    copy_staged<T, ROWS, 2, OUT>(stg, base, ld, n, nf, lane);
  else
    copy_staged<T, ROWS, 1, OUT>(stg, base, ld, n, nf, lane);
}

// The activation, or its slope, of N values: the choice is made once.
template <int N>
__device__ __forceinline__ void slope_all(float (&v)[N], int act) {
  switch (act) {
    case MOE_ACT_RELU:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = activation_slope(v[i], MOE_ACT_RELU);
      break;
    case MOE_ACT_SILU:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = activation_slope(v[i], MOE_ACT_SILU);
      break;
    case MOE_ACT_GELU:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = activation_slope(v[i], MOE_ACT_GELU);
      break;
    case MOE_ACT_GELU_TANH:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = activation_slope(v[i], MOE_ACT_GELU_TANH);
      break;
    default:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = 1.f;
  }
}

template <int N>
__device__ __forceinline__ void activate_all(float (&v)[N], int act) {
  switch (act) {
    case MOE_ACT_RELU:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = activate(v[i], MOE_ACT_RELU);
      break;
    case MOE_ACT_SILU:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = activate(v[i], MOE_ACT_SILU);
      break;
    case MOE_ACT_GELU:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = activate(v[i], MOE_ACT_GELU);
      break;
    case MOE_ACT_GELU_TANH:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = activate(v[i], MOE_ACT_GELU_TANH);
      break;
    default:
      break;
  }
}

// ------------------------------------------------------ shared contractions
// `split` ranks of a cluster (CTAs, or pairs of them) share a tile, each with a
// part of its contraction.  The tile's rows, 16 at a time, are dealt to the
// ranks; each rank sends the owners its fp32 partials of their rows, and an
// owner adds what it gets to its own, always in the same order: the same sum on
// every run, no workspace, no counters.  A warp sends the chunks of its
// accumulator quadrant in the epilogue's register layout: into the slots of its
// CTA (their MMAs are done), then by a bulk copy that counts its bytes off on
// the owner's mbarrier, and the owner's epilogue adds them as it goes.  The code
// runs once per CTA, so that most of its cost is instructions fetched for the
// first time: 2.5 us over an unsplit tile's end for 16 rows of 4 ranks, and 5.2
// for 128, with rows dealt by fours in loops unrolled eightfold and an epilogue
// of its own; 1.2 and 2.0 as it is (128 rows 4096 -> 4096: 13.3 us, now 10.8).
//
// What comes in: [source][chunk of 16 rows][quadrant] 2 KB, 1 KB per 8 rows.
constexpr int split_chunks(int rows, int split) { return ((rows + 15) / 16 + split - 1) / split; }
constexpr int split_bytes(int bn, int split) {
  return split > 1 ? (split - 1) * split_chunks(bn, split) * 8192 : 0;
}
// What goes out: the most chunks of other ranks, which the slots have to hold.
constexpr int split_out_bytes(int bn, int split) {
  const int others = (split - 1) * split_chunks(bn, split), all = (bn + 15) / 16;
  return split > 1 ? (others < all ? others : all) * 8192 : 0;
}

struct Split {
  int ranks, rank;
  int cta0, step;         // the CTA of rank k in the cluster: cta0 + step k
  uint32_t out, in, bar;  // this CTA's slots, buffer and its mbarrier (one arrival)
  int n_valid, per;       // rows of the tile, chunks of 16 per rank
  __device__ __forceinline__ Split(int n_valid_, int ranks_, int rank_, int cta0_, int step_,
                                   uint32_t out_, uint32_t in_, uint32_t bar_)
      : ranks(ranks_), rank(rank_), cta0(cta0_), step(step_), out(out_), in(in_), bar(bar_),
        n_valid(n_valid_), per(split_chunks(n_valid_, ranks_)) {}
  __device__ __forceinline__ int first() const { return rank * per * 16; }
  // rows of rank k
  __device__ __forceinline__ int rows(int k) const {
    return max(0, min(per * 16, n_valid - k * per * 16));
  }
  __device__ __forceinline__ uint32_t at(int source, int chunk, int q) const {
    return in + ((source * per + chunk) * 4 + q) * 2048;
  }
};

// shared memory of this CTA to one of the cluster's, in 16-byte pieces
__device__ __forceinline__ void bulk_copy_cluster(uint32_t dst, uint32_t src, uint32_t bytes,
                                                  uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
      ::"r"(dst), "r"(src), "r"(bytes), "r"(bar)
      : "memory");
}

// What this rank is sent, announced once.
__device__ __forceinline__ void split_expect(const Split& x) {
  const int mine = x.rows(x.rank);
  if (mine > 0) mbar_arrive_expect_tx(x.bar, (x.ranks - 1) * ((mine + 7) >> 3) * 4096);
}

// Waits, with a limit, for all that the others send: no CTA may end before, not
// even one whose waits gave up or whose features all lie behind the last one.
__device__ __forceinline__ void split_settle(const ProductParams& p, const Split& x) {
  if (x.rows(x.rank) > 0) mbar_wait(x.bar, 0, nullptr, p.status);
}

// The others' rows of this warp's 32 features (accumulator lanes of quadrant q
// at taddr, a second part `second` columns on), every second chunk of them.
// zeros: nothing was added up.
__device__ __forceinline__ void split_send(const Split& x, uint32_t taddr, uint32_t second, int q,
                                           int part, bool zeros, int lane) {
  uint32_t at = x.out + q * 2048;
  int n = 0;
#pragma unroll 1
  for (int o = 1; o < x.ranks; ++o) {
    const int to = (x.rank + o) & (x.ranks - 1);
    const int rows = x.rows(to);
#pragma unroll 1
    for (int c = 0; c < rows; c += 16, at += 8192) {
      if ((n++ & 1) != part) continue;
      uint32_t r[2][8], r2[2][8];
#pragma unroll
      for (int i = 0; i < 16; ++i) r[i >> 3][i & 7] = r2[i >> 3][i & 7] = 0;
      if (!zeros) {
        const uint32_t from = taddr + to * x.per * 16 + c;
        tmem_ld_16x256b_x2(from, r[0]);
        tmem_ld_16x256b_x2(from + (16u << 16), r[1]);
        if (second != 0) {
          tmem_ld_16x256b_x2(from + second, r2[0]);
          tmem_ld_16x256b_x2(from + second + (16u << 16), r2[1]);
        }
        tmem_ld_wait();
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {  // rows 8 (k / 2) on, features 16 (k % 2) on
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          v[e] = __uint_as_float(r[k & 1][4 * (k >> 1) + e]) +
                 __uint_as_float(r2[k & 1][4 * (k >> 1) + e]);
        asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at + k * 512 + lane * 16),
                     "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3])
                     : "memory");
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (elect_one()) {
        const uint32_t cta = x.cta0 + x.step * to;
        bulk_copy_cluster(mapa_shared(x.at(x.rank < to ? x.rank : x.rank - 1, c >> 4, q), cta), at,
                          rows - c > 8 ? 2048 : 1024, mapa_shared(x.bar, cta));
      }
      __syncwarp();
    }
  }
}

// What the epilogue adds to its chunk of 16 rows at row c: nothing, or what the
// other ranks sent, once it has come.  False if it did not come in time.
struct Alone {
  template <int N>
  __device__ __forceinline__ bool operator()(float (&)[N], int) {
    return true;
  }
};
struct Joined {
  const Split& x;
  int q, lane;
  volatile int* abort;
  int* status;
  bool waited;
  template <int N>
  __device__ __forceinline__ bool operator()(float (&v)[N], int c) {
    static_assert(N == 16, "a chunk of 16 rows");
    if (!waited && !__all_sync(0xffffffffu, mbar_wait_cluster(x.bar, 0, abort, status))) return false;
    waited = true;
#pragma unroll 1
    for (int s = 0; s < x.ranks - 1; ++s) {
      const uint32_t at = x.at(s, c >> 4, q) + lane * 16;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float u[4];
        asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(u[0]), "=f"(u[1]), "=f"(u[2]), "=f"(u[3])
                     : "r"(at + k * 512));
#pragma unroll
        for (int e = 0; e < 4; ++e) v[4 * k + e] += u[e];
      }
    }
    return true;
  }
};

// One warp's part of a tile: lanes [32 q, 32 q + 32) of the accumulator at
// taddr (quadrant and buffer included), in chunks of ROWS rows: `part`,
// part + parts, ... below n_valid; row0 the tile's first output row, f0 the
// warp's first feature.  zeros: the contraction was empty.  TWO: a second part
// of the sum may lie `second` columns on (0: it does not).  EXTRA: with a
// residual or the pre-activation.  ACT: the activation may be one.
// False if `join` gave up.
template <int MODE, typename T, int ROWS, bool EXTRA, bool ACT, int AHEAD, bool TWO, typename Join>
__device__ __forceinline__ bool store_chunks(const ProductParams& p, uint32_t taddr,
                                             uint32_t second, int part, int parts, int n_valid,
                                             int64_t row0, int f0, int g, bool zeros, uint8_t* stg,
                                             int lane, Join join) {
  static_assert(!EXTRA || ROWS == 16, "staging");
  const int nf = p.feats - f0;
  if (nf <= 0) return true;
  // matrix m: features 8 m + lane / 4
  float bias[4] = {0.f, 0.f, 0.f, 0.f};
  if (MODE == kProductForward && p.bias != nullptr) {
    const T* b = static_cast<const T*>(p.bias) + static_cast<int64_t>(g) * p.feats + f0;
#pragma unroll
    for (int m = 0; m < 4; ++m)
      if (8 * m + (lane >> 2) < nf) bias[m] = to_f32<T>(b[8 * m + (lane >> 2)]);
  }
  // stmatrix / ldmatrix: lane 8 m + j addresses row j of matrix m
  const uint32_t mat = smem_u32(stg) + (lane & 7) * kEpiPitch + (lane >> 3) * 16;
  T* out = static_cast<T*>(p.out) + row0 * p.ld_out + f0;
  constexpr int kB = ROWS / 16;  // 16-row loads per chunk
  uint32_t r[2 * kB][8], r2[2 * kB][8];
  auto load = [&](int c) {
#pragma unroll
    for (int b = 0; b < kB; ++b) {
      if (c + 16 * b >= n_valid) break;
      tmem_ld_16x256b_x2(taddr + c + 16 * b, r[2 * b]);
      tmem_ld_16x256b_x2(taddr + (16u << 16) + c + 16 * b, r[2 * b + 1]);
      if (TWO && second != 0) {
        tmem_ld_16x256b_x2(taddr + second + c + 16 * b, r2[2 * b]);
        tmem_ld_16x256b_x2(taddr + second + (16u << 16) + c + 16 * b, r2[2 * b + 1]);
      }
    }
  };
#pragma unroll
  for (int i = 0; i < 16 * kB; ++i) r[i >> 3][i & 7] = r2[i >> 3][i & 7] = 0;
  if (!zeros) load(part * ROWS);
  // a residual of 16-byte pieces comes by asynchronous copies AHEAD chunks ahead
  // into a ring of staged chunks (4096 rows 1024 -> 4096 36 us, 31 without a
  // residual; as register loads, whose arrival every later shared-memory read
  // waits for, 49 us one chunk ahead and 47 us four ahead)
  const T* residual = static_cast<const T*>(p.residual) + row0 * p.ld_residual + f0;
  const bool ring = EXTRA && p.residual != nullptr && p.width_residual == 8;
  auto fetch = [&](int c, int slot) {
    const int piece = lane & 3;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int row = 8 * k + (lane >> 2);
      if (piece * 8 < nf && c + row < n_valid)
        cp_async_16(smem_u32(stg) + (1 + slot) * kEpiChunk + row * kEpiPitch + piece * 16,
                    residual + (c + row) * p.ld_residual + piece * 8);
    }
    cp_async_commit();
  };
  if (ring) {
#pragma unroll
    for (int a = 0; a < AHEAD; ++a) fetch((part + a * parts) * ROWS, a);
  }
  int slot = 0;
  for (int c = part * ROWS; c < n_valid; c += parts * ROWS) {
    const int n = min(ROWS, n_valid - c);
    if (EXTRA && p.residual != nullptr && !ring)
      copy_rows<T, 16, false>(stg + kEpiChunk, const_cast<T*>(residual) + c * p.ld_residual,
                              p.ld_residual, n, nf, p.width_residual, lane);
    if (!zeros) tmem_ld_wait();
    // v[8 k + 2 m + e]: rows 8 k + 2 (lane % 4) + e of matrix m
    float v[16 * kB];
#pragma unroll
    for (int k = 0; k < 2 * kB; ++k)
#pragma unroll
      for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int e = 0; e < 2; ++e)
        {
          const int a = 2 * (k >> 1) + (m >> 1), b = 4 * (k & 1) + 2 * (m & 1) + e;
          v[8 * k + 2 * m + e] =
              TWO ? __uint_as_float(r[a][b]) + __uint_as_float(r2[a][b]) : __uint_as_float(r[a][b]);
        }
    // the next chunk's load runs below this one's arithmetic and stores
    if (!zeros && c + parts * ROWS < n_valid) load(c + parts * ROWS);
    if (!join(v, c)) {
      if (ring) cp_async_wait<0>();
      return false;
    }
    if (MODE != kProductForward && !is_bf16<T>()) {
#pragma unroll
      for (int i = 0; i < 16 * kB; ++i) v[i] *= p.out_scale;
    }
#pragma unroll
    for (int i = 0; i < 16 * kB; ++i) v[i] += bias[(i >> 1) & 3];
    auto stage = [&]() {
#pragma unroll
      for (int k = 0; k < 2 * kB; ++k) {
        const uint32_t w[4] = {pack2<T>(v[8 * k], v[8 * k + 1]), pack2<T>(v[8 * k + 2], v[8 * k + 3]),
                               pack2<T>(v[8 * k + 4], v[8 * k + 5]),
                               pack2<T>(v[8 * k + 6], v[8 * k + 7])};
        stmatrix_x4_trans(mat + k * 8 * kEpiPitch, w);
      }
      __syncwarp();
    };
    if (EXTRA && p.preact != nullptr) {
      stage();
      copy_rows<T, ROWS, true>(stg, static_cast<T*>(p.preact) + (row0 + c) * p.ld_preact + f0,
                               p.ld_preact, n, nf, p.width_preact, lane);
      __syncwarp();
    }
    if (ACT) activate_all(v, p.act);
    if (EXTRA && p.residual != nullptr) {
      if (ring) cp_async_wait<AHEAD - 1>();
      __syncwarp();
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        uint32_t w[4];
        ldmatrix_x4_trans(mat + (1 + slot) * kEpiChunk + k * 8 * kEpiPitch, w);
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const float2 f = unpack2<T>(w[m]);
          v[8 * k + 2 * m] += f.x;
          v[8 * k + 2 * m + 1] += f.y;
        }
      }
    }
    stage();
    copy_rows<T, ROWS, true>(stg, out + c * p.ld_out, p.ld_out, n, nf, p.width_out, lane);
    __syncwarp();
    if (ring) {  // (every lane has read its part of this chunk's residual)
      fetch(c + AHEAD * parts * ROWS, slot);
      slot = slot + 1 < AHEAD ? slot + 1 : 0;
    }
  }
  if (ring) cp_async_wait<0>();
  return true;
}

// PLAIN: nothing follows the product but a bias.
template <int MODE, typename T, int ROWS, int AHEAD, bool TWO, bool PLAIN, typename Join>
__device__ __forceinline__ bool store_tile(const ProductParams& p, uint32_t taddr, uint32_t second,
                                           int part, int parts, int n_valid, int64_t row0, int f0,
                                           int g, bool zeros, uint8_t* stg, int lane, Join join) {
  constexpr bool kMore = MODE == kProductForward && !PLAIN;
  if constexpr (kMore) {
    if (p.preact != nullptr || p.residual != nullptr)
      return store_chunks<MODE, T, 16, true, true, AHEAD, TWO>(
          p, taddr, second, part, parts, n_valid, row0, f0, g, zeros, stg, lane, join);
  }
  return store_chunks<MODE, T, ROWS, false, kMore, AHEAD, TWO>(
      p, taddr, second, part, parts, n_valid, row0, f0, g, zeros, stg, lane, join);
}

}  // namespace product
}  // namespace moe
