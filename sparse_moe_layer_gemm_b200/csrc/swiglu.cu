// SwiGLU of the experts as an operator of its own, forward and backward:
//   a = min(gate, L), v = clip(up, -L, L)  (L = 0: gate, up)
//   out  = s * silu(a) * v
//   dgate = dout * s * v * silu'(a) where gate <= L, else 0
//   dup   = dout * s * silu(a) where |up| <= L, else 0
//   ds    = sum over the row of dout * silu(a) * v
// with s the row's gate weight (1 without).  6 bytes per element forward, 10
// backward at 16 bits: bound by memory.  One CTA per row at a time, 16 bytes
// per thread and access where the rows allow it; the row's sum is added per
// thread, over the warp, then over the warps in order, in fp32.
#include <algorithm>

#include "moe_internal.h"
#include "product_device.cuh"

namespace moe {

namespace {

using namespace product;

constexpr int kMaxThreads = 256;

template <typename T, int V>
struct alignas(sizeof(T) * V) Pack {
  T v[V];
};

template <typename T>
__device__ __forceinline__ float exp_of(float x) { return __expf(x); }
template <>
__device__ __forceinline__ float exp_of<float>(float x) { return expf(x); }

// NaN passes both clamps, as it passes the plain formula.
__device__ __forceinline__ float clamp_gate(float g, float L) { return L > 0.f && g > L ? L : g; }
__device__ __forceinline__ float clamp_up(float u, float L) {
  return L > 0.f ? (u > L ? L : (u < -L ? -L : u)) : u;
}

template <typename T, int V>
__global__ void __launch_bounds__(kMaxThreads) swiglu_kernel(const SwigluParams p) {
  pdl_wait();
  int r0 = 0, r1 = p.rows;
  if (p.offsets != nullptr) {
    r0 = min(max(p.offsets[0], 0), p.rows);
    r1 = min(max(p.offsets[p.groups], 0), p.rows);
  }
  for (int64_t row = static_cast<int64_t>(r0) + blockIdx.x; row < r1; row += gridDim.x) {
    const T* gate = static_cast<const T*>(p.gate) + row * p.ld_gate;
    const T* up = static_cast<const T*>(p.up) + row * p.ld_up;
    T* out = static_cast<T*>(p.out) + row * p.ld_out;
    const float s = p.scale != nullptr ? p.scale[row] : 1.f;
    for (int c = threadIdx.x * V; c < p.cols; c += blockDim.x * V) {
      const Pack<T, V> g = *reinterpret_cast<const Pack<T, V>*>(gate + c);
      const Pack<T, V> u = *reinterpret_cast<const Pack<T, V>*>(up + c);
      Pack<T, V> o;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float a = clamp_gate(to_f32<T>(g.v[i]), p.limit);
        const float b = clamp_up(to_f32<T>(u.v[i]), p.limit);
        o.v[i] = from_f32<T>(s * (a / (1.0f + exp_of<T>(-a))) * b);
      }
      *reinterpret_cast<Pack<T, V>*>(out + c) = o;
    }
  }
}

template <typename T, int V>
__global__ void __launch_bounds__(kMaxThreads) swiglu_backward_kernel(const SwigluParams p) {
  __shared__ float sums[kMaxThreads / 32];
  pdl_wait();
  int r0 = 0, r1 = p.rows;
  if (p.offsets != nullptr) {
    r0 = min(max(p.offsets[0], 0), p.rows);
    r1 = min(max(p.offsets[p.groups], 0), p.rows);
  }
  const float L = p.limit;
  for (int64_t row = static_cast<int64_t>(r0) + blockIdx.x; row < r1; row += gridDim.x) {
    const T* gate = static_cast<const T*>(p.gate) + row * p.ld_gate;
    const T* up = static_cast<const T*>(p.up) + row * p.ld_up;
    const T* dout = static_cast<const T*>(p.dout) + row * p.ld_dout;
    T* dgate = static_cast<T*>(p.dgate) + row * p.ld_dgate;
    T* dup = static_cast<T*>(p.dup) + row * p.ld_dup;
    const float s = p.scale != nullptr ? p.scale[row] : 1.f;
    float acc = 0.f;
    for (int c = threadIdx.x * V; c < p.cols; c += blockDim.x * V) {
      const Pack<T, V> g = *reinterpret_cast<const Pack<T, V>*>(gate + c);
      const Pack<T, V> u = *reinterpret_cast<const Pack<T, V>*>(up + c);
      const Pack<T, V> d = *reinterpret_cast<const Pack<T, V>*>(dout + c);
      Pack<T, V> dg, du;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float gf = to_f32<T>(g.v[i]), uf = to_f32<T>(u.v[i]), df = to_f32<T>(d.v[i]);
        const float a = clamp_gate(gf, L), b = clamp_up(uf, L);
        const float sg = 1.0f / (1.0f + exp_of<T>(-a));
        const float silu = a * sg;
        acc += df * silu * b;
        const float dgv = df * s * b * sg * (1.0f + a * (1.0f - sg));
        const float duv = df * s * silu;
        dg.v[i] = from_f32<T>(L > 0.f && gf > L ? 0.f : dgv);
        du.v[i] = from_f32<T>(L > 0.f && fabsf(uf) > L ? 0.f : duv);
      }
      *reinterpret_cast<Pack<T, V>*>(dgate + c) = dg;
      *reinterpret_cast<Pack<T, V>*>(dup + c) = du;
    }
    if (p.dscale != nullptr) {
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, d);
      if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = acc;
      __syncthreads();
      if (threadIdx.x == 0) {
        float v = 0.f;
        for (int i = 0; i < static_cast<int>(blockDim.x >> 5); ++i) v += sums[i];
        p.dscale[row] = v;
      }
      __syncthreads();
    }
  }
}

// elements per access: 16 bytes where every row of every tensor starts at a
// 16-byte boundary and the row length is a multiple, else one
template <typename T>
bool vec_ok(const SwigluParams& p, bool backward) {
  constexpr int V = 16 / sizeof(T);
  auto ok = [](const void* q, int64_t ld) {
    return reinterpret_cast<uintptr_t>(q) % 16 == 0 && ld % V == 0;
  };
  if (p.cols % V != 0 || !ok(p.gate, p.ld_gate) || !ok(p.up, p.ld_up)) return false;
  if (!backward) return ok(p.out, p.ld_out);
  return ok(p.dout, p.ld_dout) && ok(p.dgate, p.ld_dgate) && ok(p.dup, p.ld_dup);
}

template <typename T>
cudaError_t run(const SwigluParams& p, bool backward, cudaStream_t st) {
  constexpr int V = 16 / sizeof(T);
  const bool vec = vec_ok<T>(p, backward);
  const int pieces = (p.cols + (vec ? V : 1) - 1) / (vec ? V : 1);
  const int threads = std::min(kMaxThreads, (pieces + 31) / 32 * 32);
  const dim3 grid(static_cast<unsigned>(std::min(p.rows, 1 << 20)));
  if (backward)
    return vec ? launch_pdl(swiglu_backward_kernel<T, V>, grid, dim3(threads), 0, st, p)
               : launch_pdl(swiglu_backward_kernel<T, 1>, grid, dim3(threads), 0, st, p);
  return vec ? launch_pdl(swiglu_kernel<T, V>, grid, dim3(threads), 0, st, p)
             : launch_pdl(swiglu_kernel<T, 1>, grid, dim3(threads), 0, st, p);
}

cudaError_t dispatch(int dtype, const SwigluParams& p, bool backward, cudaStream_t st) {
  if (dtype == MOE_F32) return run<float>(p, backward, st);
  if (dtype == MOE_BF16) return run<__nv_bfloat16>(p, backward, st);
  return run<__half>(p, backward, st);
}

}  // namespace

cudaError_t launch_swiglu(int dtype, const SwigluParams& p, cudaStream_t st) {
  return dispatch(dtype, p, false, st);
}

cudaError_t launch_swiglu_backward(int dtype, const SwigluParams& p, cudaStream_t st) {
  return dispatch(dtype, p, true, st);
}

}  // namespace moe
