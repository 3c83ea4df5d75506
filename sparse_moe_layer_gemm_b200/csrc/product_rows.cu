// Row kernels of the products' backward pass: dz = dout * act'(preact), the
// bias gradient's column sums, and the aligned copies of operands whose
// strides the TMA cannot address.  All of them move bytes; the arithmetic is
// fp32.
#include <algorithm>

#include "moe_internal.h"
#include "product_device.cuh"

namespace moe {

namespace {

using namespace product;

constexpr int kPackThreads = 256;

// One CTA per row of any of the operands.
__global__ void __launch_bounds__(kPackThreads) pack_rows_kernel(const PackParams p) {
  pdl_wait();
  int64_t row = blockIdx.x;
  int i = 0;
  while (row >= p.op[i].groups * p.op[i].rows) row -= p.op[i].groups * p.op[i].rows, ++i;
  const PackOperand& o = p.op[i];
  const int64_t g = row / o.rows;
  const uint16_t* s = static_cast<const uint16_t*>(o.src) + g * o.group_stride + (row - g * o.rows) * o.ld;
  uint16_t* d = static_cast<uint16_t*>(o.dst) + row * o.ld_dst;
  constexpr int U = 4;  // loads under way per thread
  for (int c = threadIdx.x; c < o.cols; c += U * kPackThreads) {
    uint16_t v[U];
#pragma unroll
    for (int k = 0; k < U; ++k)
      if (c + k * kPackThreads < o.cols) v[k] = s[c + k * kPackThreads];
#pragma unroll
    for (int k = 0; k < U; ++k)
      if (c + k * kPackThreads < o.cols) d[c + k * kPackThreads] = v[k];
  }
}

constexpr int kGradThreads = 256;          // 8 warps: rows of a chunk are dealt to them
constexpr int kGradWarps = kGradThreads / 32;
constexpr int kVec = 8;                    // elements per 16-byte access
constexpr int kGradCols = 32 * kVec;       // columns per CTA

template <typename T>
struct alignas(16) Vec {
  T v[kVec];
};

// One CTA: 64 rows of one group x 256 columns, or with `direct` all rows of
// the group.  The column sums are added in fp32, per warp over its rows, then
// over the warps in order; direct: they are the group's and go to db at once.
// VEC: every row starts at a 16-byte boundary and cols % 8 == 0.  Each lane
// keeps U rows' loads under way.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kGradThreads) row_grad_kernel(const RowGradParams p) {
  extern __shared__ int tab_mem[];
  __shared__ float sums[kGradWarps][kGradCols];
  pdl_wait();
  const GroupTable tab = build_group_table(tab_mem, p.offsets, p.groups, p.rows, kRowChunk);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int col_blocks = (p.cols + kGradCols - 1) / kGradCols;
  const int total = (p.direct ? p.groups : tab.block_start[p.groups]) * col_blocks;
  const T* dout = static_cast<const T*>(p.dout);
  const T* preact = static_cast<const T*>(p.preact);
  T* dz = static_cast<T*>(p.dz);
  constexpr int U = VEC ? 4 : 2;
  for (int w = blockIdx.x; w < total; w += gridDim.x) {
    const int chunk = w / col_blocks;  // (direct: the group)
    const int c0 = (w - chunk * col_blocks) * kGradCols;
    const int g = p.direct ? chunk : group_of_block(tab, p.groups, chunk);
    const int first = p.direct ? 0 : (chunk - tab.block_start[g]) * kRowChunk;
    const int n = p.direct ? tab.count(g) : min(kRowChunk, tab.count(g) - first);
    const int64_t row0 = static_cast<int64_t>(tab.row0[g]) + first;
    float acc[kVec] = {};
    // column of element i of this lane: contiguous pieces, or 32 apart
    const int col = VEC ? c0 + lane * kVec : c0 + lane;
    if (col < p.cols) {
      for (int r = warp; r < n; r += U * kGradWarps) {
        if (VEC) {
          Vec<T> d[U], z[U];
#pragma unroll
          for (int k = 0; k < U; ++k)
            if (r + k * kGradWarps < n) {
              const int64_t row = row0 + r + k * kGradWarps;
              d[k] = *reinterpret_cast<const Vec<T>*>(dout + row * p.ld_dout + col);
              if (preact != nullptr)
                z[k] = *reinterpret_cast<const Vec<T>*>(preact + row * p.ld_preact + col);
            }
#pragma unroll
          for (int k = 0; k < U; ++k)
            if (r + k * kGradWarps < n) {
              if (preact != nullptr) {
#pragma unroll
                for (int i = 0; i < kVec; ++i) {
                  const float v =
                      to_f32<T>(d[k].v[i]) * activation_slope(to_f32<T>(z[k].v[i]), p.act);
                  acc[i] += v;
                  d[k].v[i] = from_f32<T>(v);
                }
                *reinterpret_cast<Vec<T>*>(dz + (row0 + r + k * kGradWarps) * p.ld_dz + col) = d[k];
              } else {
#pragma unroll
                for (int i = 0; i < kVec; ++i) acc[i] += to_f32<T>(d[k].v[i]);
              }
            }
        } else {
          T d[U][kVec], z[U][kVec];
#pragma unroll
          for (int k = 0; k < U; ++k)
#pragma unroll
            for (int i = 0; i < kVec; ++i)
              if (r + k * kGradWarps < n && col + 32 * i < p.cols) {
                const int64_t row = row0 + r + k * kGradWarps;
                d[k][i] = dout[row * p.ld_dout + col + 32 * i];
                if (preact != nullptr) z[k][i] = preact[row * p.ld_preact + col + 32 * i];
              }
#pragma unroll
          for (int k = 0; k < U; ++k)
#pragma unroll
            for (int i = 0; i < kVec; ++i)
              if (r + k * kGradWarps < n && col + 32 * i < p.cols) {
                const int64_t row = row0 + r + k * kGradWarps;
                float v = to_f32<T>(d[k][i]);
                if (preact != nullptr) {
                  v *= activation_slope(to_f32<T>(z[k][i]), p.act);
                  dz[row * p.ld_dz + col + 32 * i] = from_f32<T>(v);
                }
                acc[i] += v;
              }
        }
      }
    }
    if (p.db != nullptr) {
#pragma unroll
      for (int i = 0; i < kVec; ++i) sums[warp][VEC ? lane * kVec + i : lane + 32 * i] = acc[i];
      __syncthreads();
      const int c = c0 + threadIdx.x;
      if (c < p.cols) {
        float v = 0.f;
#pragma unroll
        for (int i = 0; i < kGradWarps; ++i) v += sums[i][threadIdx.x];
        if (p.direct)
          static_cast<T*>(p.db)[static_cast<int64_t>(g) * p.cols + c] = from_f32<T>(v);
        else
          p.partial[static_cast<int64_t>(chunk) * p.cols + c] = v;
      }
      __syncthreads();
    }
  }
}

// db[g][c] for 32 columns per CTA: warp k adds chunks k, k + 8, ..., then the
// warps' sums are added in order and rounded once.
template <typename T>
__global__ void __launch_bounds__(kGradThreads) bias_grad_kernel(const RowGradParams p) {
  extern __shared__ int tab_mem[];
  __shared__ float sums[kGradWarps][32];
  pdl_wait();
  const GroupTable tab = build_group_table(tab_mem, p.offsets, p.groups, p.rows, kRowChunk);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int col_blocks = (p.cols + 31) / 32;
  for (int w = blockIdx.x; w < p.groups * col_blocks; w += gridDim.x) {
    const int g = w / col_blocks;
    const int c = (w - g * col_blocks) * 32 + lane;
    const int n = tab.block_start[g + 1] - tab.block_start[g];
    float v = 0.f;
    if (c < p.cols) {
      const float* s = p.partial + static_cast<int64_t>(tab.block_start[g]) * p.cols + c;
#pragma unroll 8
      for (int i = warp; i < n; i += kGradWarps) v += s[static_cast<int64_t>(i) * p.cols];
    }
    sums[warp][lane] = v;
    __syncthreads();
    if (warp == 0 && c < p.cols) {
      v = 0.f;
#pragma unroll
      for (int i = 0; i < kGradWarps; ++i) v += sums[i][lane];
      static_cast<T*>(p.db)[static_cast<int64_t>(g) * p.cols + c] = from_f32<T>(v);
    }
    __syncthreads();
  }
}

bool rows_aligned(const void* p, int64_t ld) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % kVec == 0;
}

template <typename T>
cudaError_t row_grad(const RowGradParams& p, int num_sms, cudaStream_t st) {
  const size_t tab = group_table_bytes(p.groups);
  const bool vec = p.cols % kVec == 0 && rows_aligned(p.dout, p.ld_dout) &&
                   (p.preact == nullptr ||
                    (rows_aligned(p.preact, p.ld_preact) && rows_aligned(p.dz, p.ld_dz)));
  const int64_t items = static_cast<int64_t>(p.direct ? p.groups
                                                      : row_grad_chunks(p.rows, p.groups) + 1) *
                        ((p.cols + kGradCols - 1) / kGradCols);
  const int grid = static_cast<int>(std::min<int64_t>(items, 6 * num_sms));
  cudaError_t e;
  if (vec)
    e = launch_pdl(row_grad_kernel<T, true>, dim3(grid), dim3(kGradThreads), tab, st, p);
  else
    e = launch_pdl(row_grad_kernel<T, false>, dim3(grid), dim3(kGradThreads), tab, st, p);
  if (e != cudaSuccess || p.db == nullptr || p.direct) return e;
  const int64_t outs = static_cast<int64_t>(p.groups) * ((p.cols + 31) / 32);
  return launch_pdl(bias_grad_kernel<T>, dim3(static_cast<int>(std::min<int64_t>(outs, 4 * num_sms))),
                    dim3(kGradThreads), tab, st, p);
}

}  // namespace

cudaError_t launch_pack_rows(const PackParams& p, cudaStream_t st) {
  int64_t rows = 0;
  for (const PackOperand& o : p.op) rows += o.groups * o.rows;
  if (rows == 0) return cudaSuccess;
  if (rows > INT32_MAX) return cudaErrorInvalidValue;
  return launch_pdl(pack_rows_kernel, dim3(static_cast<unsigned>(rows)), dim3(kPackThreads), 0, st,
                    p);
}

cudaError_t launch_row_grad(bool bf16, const RowGradParams& p, int num_sms, cudaStream_t st) {
  return bf16 ? row_grad<__nv_bfloat16>(p, num_sms, st) : row_grad<__half>(p, num_sms, st);
}

}  // namespace moe
