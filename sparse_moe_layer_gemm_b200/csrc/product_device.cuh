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

}  // namespace product
}  // namespace moe
