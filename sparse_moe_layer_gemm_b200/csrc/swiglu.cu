// SwiGLU of the experts as an operator of its own, forward and backward:
//   a = min(gate, L), v = clip(up, -L, L)  (L = 0: gate, up)
//   out  = s * silu(a) * v
//   dgate = dout * s * v * silu'(a) where gate <= L, else 0
//   dup   = dout * s * silu(a) where |up| <= L, else 0
//   ds    = sum over the row of dout * silu(a) * v
// with s the row's gate weight (1 without).  6 bytes per element forward, 10
// backward at 16 bits: bound by memory.
//
// A team of one or eight warps takes a row at a time, 16 bytes per lane and
// access where every row starts at a 16-byte boundary: one warp per row from
// kManyRows rows on (32768 x 1280 bf16 with clamp and scale: 41 us forward, 66
// backward, 6.2 and 6.35 TB/s; one CTA per row took 58 and 95), a whole CTA
// per row below, where the row's length is what takes time.  The instructions
// count too: the sigmoid is one ex2, one rcp and two more, the clamps min and
// max with NaN (with the library's expf and division 49 and 86 us).  The row's
// sum is added per lane, over the warp, then over the warps in order, in fp32:
// the same on every run.  For 16-bit tensors its terms too take the approximate
// sigmoid, a few units of 2^-23 of each term off (dscale of 32768 x 1280 rows
// 1.4e-7 from the definition, the plain formula in fp32 1.1e-7); fp32 tensors
// take the exact ones.
#include <algorithm>

#include "moe_internal.h"
#include "product_device.cuh"

namespace moe {

namespace {

using namespace product;

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kManyRows = 1024;

template <typename T, int V>
struct alignas(sizeof(T) * V) Pack {
  T v[V];
};

// 4 sigmoid(x); fp32 rows take the exact division and exponential.
template <typename T>
__device__ __forceinline__ float sigmoid4_of(float x) { return sigmoid_times_4(x); }
template <>
__device__ __forceinline__ float sigmoid4_of<float>(float x) { return 4.0f / (1.0f + expf(-x)); }

// NaN passes the clamps, as it passes the plain formula.
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ void row_range(const SwigluParams& p, int* r0, int* r1) {
  *r0 = 0;
  *r1 = p.rows;
  if (p.offsets != nullptr) {
    *r0 = min(max(p.offsets[0], 0), p.rows);
    *r1 = min(max(p.offsets[p.groups], 0), p.rows);
  }
}

// TEAM: warps per row.  U accesses of each tensor under way per lane.
template <typename T, int V, int TEAM, int U, bool CLAMP>
__global__ void __launch_bounds__(kThreads, V == 1 ? 3 : 6) swiglu_kernel(const SwigluParams p) {
  pdl_wait();
  pdl_trigger();
  int r0, r1;
  row_range(p, &r0, &r1);
  const float L = p.limit;
  constexpr int kStep = 32 * TEAM * V;  // columns per access of the team
  const int team = static_cast<int>(threadIdx.x) / (32 * TEAM);
  const int lane = static_cast<int>(threadIdx.x) % (32 * TEAM);
  constexpr int kTeams = kWarps / TEAM;
  for (int64_t row = r0 + static_cast<int64_t>(blockIdx.x) * kTeams + team; row < r1;
       row += static_cast<int64_t>(gridDim.x) * kTeams) {
    const T* gate = static_cast<const T*>(p.gate) + row * p.ld_gate;
    const T* up = static_cast<const T*>(p.up) + row * p.ld_up;
    T* out = static_cast<T*>(p.out) + row * p.ld_out;
    const float s = p.scale != nullptr ? p.scale[row] : 1.f;
    for (int c0 = lane * V; c0 < p.cols; c0 += U * kStep) {
      Pack<T, V> g[U], u[U];
#pragma unroll
      for (int k = 0; k < U; ++k)
        if (c0 + k * kStep < p.cols) {
          g[k] = *reinterpret_cast<const Pack<T, V>*>(gate + c0 + k * kStep);
          u[k] = *reinterpret_cast<const Pack<T, V>*>(up + c0 + k * kStep);
        }
#pragma unroll
      for (int k = 0; k < U; ++k)
        if (c0 + k * kStep < p.cols) {
          Pack<T, V> o;
#pragma unroll
          for (int i = 0; i < V; ++i) {
            float a = to_f32<T>(g[k].v[i]), b = to_f32<T>(u[k].v[i]);
            if (CLAMP) {
              a = min_nan(a, L);
              b = max_nan(min_nan(b, L), -L);
            }
            o.v[i] = from_f32<T>(s * b * (0.25f * a * sigmoid4_of<T>(a)));
          }
          *reinterpret_cast<Pack<T, V>*>(out + c0 + k * kStep) = o;
        }
    }
  }
}

template <typename T, int V, int TEAM, int U, bool CLAMP>
__global__ void __launch_bounds__(kThreads, V == 1 ? 3 : 6) swiglu_backward_kernel(const SwigluParams p) {
  __shared__ float sums[kWarps];
  pdl_wait();
  pdl_trigger();
  int r0, r1;
  row_range(p, &r0, &r1);
  const float L = p.limit;
  constexpr int kStep = 32 * TEAM * V;
  const int team = static_cast<int>(threadIdx.x) / (32 * TEAM);
  const int lane = static_cast<int>(threadIdx.x) % (32 * TEAM);
  constexpr int kTeams = kWarps / TEAM;
  for (int64_t row = r0 + static_cast<int64_t>(blockIdx.x) * kTeams + team; row < r1;
       row += static_cast<int64_t>(gridDim.x) * kTeams) {
    const T* gate = static_cast<const T*>(p.gate) + row * p.ld_gate;
    const T* up = static_cast<const T*>(p.up) + row * p.ld_up;
    const T* dout = static_cast<const T*>(p.dout) + row * p.ld_dout;
    T* dgate = static_cast<T*>(p.dgate) + row * p.ld_dgate;
    T* dup = static_cast<T*>(p.dup) + row * p.ld_dup;
    const float s = p.scale != nullptr ? p.scale[row] : 1.f;
    float acc = 0.f;
    for (int c0 = lane * V; c0 < p.cols; c0 += U * kStep) {
      Pack<T, V> g[U], u[U], d[U];
#pragma unroll
      for (int k = 0; k < U; ++k)
        if (c0 + k * kStep < p.cols) {
          g[k] = *reinterpret_cast<const Pack<T, V>*>(gate + c0 + k * kStep);
          u[k] = *reinterpret_cast<const Pack<T, V>*>(up + c0 + k * kStep);
          d[k] = *reinterpret_cast<const Pack<T, V>*>(dout + c0 + k * kStep);
        }
#pragma unroll
      for (int k = 0; k < U; ++k)
        if (c0 + k * kStep < p.cols) {
          Pack<T, V> dg, du;
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const float gf = to_f32<T>(g[k].v[i]), uf = to_f32<T>(u[k].v[i]);
            const float df = to_f32<T>(d[k].v[i]);
            float a = gf, b = uf;
            if (CLAMP) {
              a = min_nan(gf, L);
              b = max_nan(min_nan(uf, L), -L);
            }
            const float sg = 0.25f * sigmoid4_of<T>(a);
            const float dsg = df * sg;
            const float dsilu = dsg * a;
            acc = fmaf(dsilu, b, acc);
            float dgv = dsg * s * b * fmaf(a, 1.0f - sg, 1.0f);
            float duv = dsilu * s;
            if (CLAMP) {
              dgv = gf > L ? 0.f : dgv;
              duv = fabsf(uf) > L ? 0.f : duv;
            }
            dg.v[i] = from_f32<T>(dgv);
            du.v[i] = from_f32<T>(duv);
          }
          *reinterpret_cast<Pack<T, V>*>(dgate + c0 + k * kStep) = dg;
          *reinterpret_cast<Pack<T, V>*>(dup + c0 + k * kStep) = du;
        }
    }
    if (p.dscale != nullptr) {
      __syncwarp();
#pragma unroll
      for (int m = 16; m > 0; m >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, m);
      if (TEAM == 1) {
        if (lane == 0) p.dscale[row] = acc;
      } else {
        if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = acc;
        __syncthreads();
        if (threadIdx.x == 0) {
          float v = 0.f;
#pragma unroll
          for (int i = 0; i < kWarps; ++i) v += sums[i];
          p.dscale[row] = v;
        }
        __syncthreads();
      }
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

template <typename T, int V, int TEAM, bool CLAMP>
cudaError_t launch_clamp(const SwigluParams& p, bool backward, cudaStream_t st) {
  // of 16-byte accesses one per tensor is under way in a lane, and registers are
  // held to 6 CTAs per SM (32768 x 1280 with clamp and scale: backward 66 us so,
  // 78 at 3 CTAs, 109 with two accesses per tensor); of one element, 8
  constexpr int U = V == 1 ? 8 : 1;
  constexpr int kTeams = kWarps / TEAM;
  const dim3 grid(static_cast<unsigned>(std::min((p.rows + kTeams - 1) / kTeams, 1 << 20)));
  return backward ? launch_pdl(swiglu_backward_kernel<T, V, TEAM, U, CLAMP>, grid, dim3(kThreads),
                               0, st, p)
                  : launch_pdl(swiglu_kernel<T, V, TEAM, U, CLAMP>, grid, dim3(kThreads), 0, st, p);
}

template <typename T, int V, int TEAM>
cudaError_t launch(const SwigluParams& p, bool backward, cudaStream_t st) {
  return p.limit > 0.f ? launch_clamp<T, V, TEAM, true>(p, backward, st)
                       : launch_clamp<T, V, TEAM, false>(p, backward, st);
}

template <typename T>
cudaError_t run(const SwigluParams& p, bool backward, cudaStream_t st) {
  constexpr int V = 16 / sizeof(T);
  const bool many = p.rows >= kManyRows;
  if (vec_ok<T>(p, backward))
    return many ? launch<T, V, 1>(p, backward, st) : launch<T, V, kWarps>(p, backward, st);
  return many ? launch<T, 1, 1>(p, backward, st) : launch<T, 1, kWarps>(p, backward, st);
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
