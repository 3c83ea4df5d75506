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

// Activations and their slopes in fp32.  gelu uses erfc, whose relative error
// stays small in the negative tail where 1 + erf cancels; gelu_tanh is
// 0.5 (1 + tanh u) = sigmoid(2 u), for the same reason.
constexpr float kSqrtHalf = 0.70710678118654752f;
constexpr float kInvSqrt2Pi = 0.39894228040143268f;
constexpr float kTanhScale = 0.79788456080286536f;  // sqrt(2 / pi)
constexpr float kTanhCubic = 0.044715f;

__device__ __forceinline__ float sigmoid(float z) { return 1.0f / (1.0f + __expf(-z)); }

__device__ __forceinline__ float activate(float z, int act) {
  switch (act) {
    case MOE_ACT_RELU:
      return z < 0.f ? 0.f : z;  // NaN stays NaN
    case MOE_ACT_SILU:
      return z / (1.0f + __expf(-z));
    case MOE_ACT_GELU:
      return 0.5f * z * erfcf(-z * kSqrtHalf);
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
    case MOE_ACT_GELU:
      return 0.5f * erfcf(-z * kSqrtHalf) + z * kInvSqrt2Pi * __expf(-0.5f * z * z);
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
  __device__ __forceinline__ int count(int g) const { return row0[g + 1] - row0[g]; }
};

constexpr int group_table_bytes(int groups) { return 2 * (groups + 1) * 4; }

__device__ __forceinline__ GroupTable build_group_table(int* mem, const int* offsets, int groups,
                                                        int rows, int unit) {
  GroupTable t{mem, mem + groups + 1};
  if (offsets == nullptr) {
    if (threadIdx.x == 0) {
      t.row0[0] = 0;
      t.row0[1] = rows;
      t.block_start[0] = 0;
      t.block_start[1] = (rows + unit - 1) / unit;
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

// Row blocks per ordering chunk: inside a group, chunks of 4 row blocks run
// feature-major, so a weight tile's readers follow one another and the
// chunk's rows stay in L2 across its weight tiles.
constexpr int kChunk = 4;

template <int MODE, int BM>
__device__ __forceinline__ Tile decode(const ProductParams& p, const GroupTable& t, int w) {
  Tile r;
  const int f_tiles = (p.feats + BM - 1) / BM;
  int local, blocks, in_chunk_first;
  if (MODE == kProductDw) {
    blocks = (p.cols + p.bn - 1) / p.bn;
    const int per_group = f_tiles * blocks;
    r.g = w / per_group;
    local = w - r.g * per_group;
  } else {
    // tiles before group g: block_start[g] * f_tiles
    const int b = w / f_tiles;
    r.g = group_of_block(t, p.groups, b);
    local = w - t.block_start[r.g] * f_tiles;
    blocks = t.block_start[r.g + 1] - t.block_start[r.g];
  }
  const int per_chunk = f_tiles * kChunk;
  const int c = local / per_chunk;
  const int rem = local - c * per_chunk;
  in_chunk_first = c * kChunk;
  const int in_chunk = min(kChunk, blocks - in_chunk_first);
  const int ft = rem / in_chunk;
  const int nb = in_chunk_first + (rem - ft * in_chunk);
  r.f0 = ft * BM;
  if (MODE == kProductDw) {
    r.j0 = nb * p.bn;
    r.n_valid = min(p.bn, p.cols - r.j0);
    r.c0 = t.row0[r.g];
    r.depth = t.count(r.g);
  } else {
    r.j0 = t.row0[r.g] + nb * p.bn;
    r.n_valid = min(p.bn, t.count(r.g) - nb * p.bn);
    r.c0 = 0;
    r.depth = p.depth;
  }
  return r;
}

// One finished value: the forward adds the bias, keeps z if asked, applies
// the activation and adds the residual; rounded once to the output type.
template <int MODE, typename T>
__device__ __forceinline__ void finish_value(const ProductParams& p, int64_t row, int feat,
                                             float bias, float v) {
  if (MODE == kProductForward) {
    v += bias;
    if (p.preact != nullptr) static_cast<T*>(p.preact)[row * p.ld_preact + feat] = from_f32<T>(v);
    v = activate(v, p.act);
    if (p.residual != nullptr)
      v += to_f32<T>(static_cast<const T*>(p.residual)[row * p.ld_residual + feat]);
  }
  static_cast<T*>(p.out)[row * p.ld_out + feat] = from_f32<T>(v);
}

template <typename T>
constexpr bool is_bf16() {
  return __is_same(T, __nv_bfloat16);
}

}  // namespace product
}  // namespace moe
