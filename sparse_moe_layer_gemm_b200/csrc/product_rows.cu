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

__global__ void pack_rows_kernel(const uint16_t* src, int64_t ld, int64_t group_stride,
                                 int64_t rows, int cols, uint16_t* dst, int64_t ld_dst) {
  pdl_wait();
  const int64_t row = blockIdx.x;
  const int64_t g = row / rows;
  const uint16_t* s = src + g * group_stride + (row - g * rows) * ld;
  uint16_t* d = dst + row * ld_dst;
  for (int c = threadIdx.x; c < cols; c += kPackThreads) d[c] = s[c];
}

constexpr int kGradThreads = 256;          // 8 warps: rows of a chunk are dealt to them
constexpr int kGradWarps = kGradThreads / 32;
constexpr int kVec = 8;                    // elements per 16-byte access
constexpr int kGradCols = 32 * kVec;       // columns per CTA

template <typename T>
struct alignas(16) Vec {
  T v[kVec];
};

// One CTA: 128 rows of one group x 256 columns.  The column sums of the chunk
// are added in fp32, per warp over its rows, then over the warps in order.
// VEC: every row starts at a 16-byte boundary and cols % 8 == 0.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kGradThreads) row_grad_kernel(const RowGradParams p) {
  extern __shared__ int tab_mem[];
  __shared__ float sums[kGradWarps][kGradCols];
  pdl_wait();
  const GroupTable tab = build_group_table(tab_mem, p.offsets, p.groups, p.rows, kRowChunk);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int col_blocks = (p.cols + kGradCols - 1) / kGradCols;
  const int total = tab.block_start[p.groups] * col_blocks;
  const T* dout = static_cast<const T*>(p.dout);
  const T* preact = static_cast<const T*>(p.preact);
  T* dz = static_cast<T*>(p.dz);
  for (int w = blockIdx.x; w < total; w += gridDim.x) {
    const int chunk = w / col_blocks;
    const int c0 = (w - chunk * col_blocks) * kGradCols;
    const int g = group_of_block(tab, p.groups, chunk);
    const int first = (chunk - tab.block_start[g]) * kRowChunk;
    const int n = min(kRowChunk, tab.count(g) - first);
    const int64_t row0 = static_cast<int64_t>(tab.row0[g]) + first;
    float acc[kVec] = {};
    // column of element i of this lane: contiguous pieces, or 32 apart
    const int col = VEC ? c0 + lane * kVec : c0 + lane;
    if (col < p.cols) {
      for (int r = warp; r < n; r += kGradWarps) {
        const int64_t row = row0 + r;
        if (VEC) {
          Vec<T> d = *reinterpret_cast<const Vec<T>*>(dout + row * p.ld_dout + col);
          if (preact != nullptr) {
            const Vec<T> z = *reinterpret_cast<const Vec<T>*>(preact + row * p.ld_preact + col);
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
              const float v = to_f32<T>(d.v[i]) * activation_slope(to_f32<T>(z.v[i]), p.act);
              acc[i] += v;
              d.v[i] = from_f32<T>(v);
            }
            *reinterpret_cast<Vec<T>*>(dz + row * p.ld_dz + col) = d;
          } else {
#pragma unroll
            for (int i = 0; i < kVec; ++i) acc[i] += to_f32<T>(d.v[i]);
          }
        } else {
#pragma unroll
          for (int i = 0; i < kVec; ++i) {
            const int c = col + 32 * i;
            if (c < p.cols) {
              float v = to_f32<T>(dout[row * p.ld_dout + c]);
              if (preact != nullptr) {
                v *= activation_slope(to_f32<T>(preact[row * p.ld_preact + c]), p.act);
                dz[row * p.ld_dz + c] = from_f32<T>(v);
              }
              acc[i] += v;
            }
          }
        }
      }
    }
    if (p.partial != nullptr) {
#pragma unroll
      for (int i = 0; i < kVec; ++i) sums[warp][VEC ? lane * kVec + i : lane + 32 * i] = acc[i];
      __syncthreads();
      const int c = c0 + threadIdx.x;
      if (c < p.cols) {
        float v = 0.f;
#pragma unroll
        for (int i = 0; i < kGradWarps; ++i) v += sums[i][threadIdx.x];
        p.partial[static_cast<int64_t>(chunk) * p.cols + c] = v;
      }
      __syncthreads();
    }
  }
}

// db[g][c]: the chunks' sums added in order, rounded once.
template <typename T>
__global__ void __launch_bounds__(kGradThreads) bias_grad_kernel(const RowGradParams p) {
  extern __shared__ int tab_mem[];
  pdl_wait();
  const GroupTable tab = build_group_table(tab_mem, p.offsets, p.groups, p.rows, kRowChunk);
  const int col_blocks = (p.cols + kGradThreads - 1) / kGradThreads;
  for (int w = blockIdx.x; w < p.groups * col_blocks; w += gridDim.x) {
    const int g = w / col_blocks;
    const int c = (w - g * col_blocks) * kGradThreads + threadIdx.x;
    if (c >= p.cols) continue;
    const float* s = p.partial + static_cast<int64_t>(tab.block_start[g]) * p.cols + c;
    const int n = tab.block_start[g + 1] - tab.block_start[g];
    float v = 0.f;
#pragma unroll 8
    for (int i = 0; i < n; ++i) v += s[static_cast<int64_t>(i) * p.cols];
    static_cast<T*>(p.db)[static_cast<int64_t>(g) * p.cols + c] = from_f32<T>(v);
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
  const int64_t items = static_cast<int64_t>(row_grad_chunks(p.rows, p.groups) + 1) *
                        ((p.cols + kGradCols - 1) / kGradCols);
  const int grid = static_cast<int>(std::min<int64_t>(items, 6 * num_sms));
  cudaError_t e;
  if (vec)
    e = launch_pdl(row_grad_kernel<T, true>, dim3(grid), dim3(kGradThreads), tab, st, p);
  else
    e = launch_pdl(row_grad_kernel<T, false>, dim3(grid), dim3(kGradThreads), tab, st, p);
  if (e != cudaSuccess || p.db == nullptr) return e;
  const int64_t outs = static_cast<int64_t>(p.groups) * ((p.cols + kGradThreads - 1) / kGradThreads);
  return launch_pdl(bias_grad_kernel<T>, dim3(static_cast<int>(std::min<int64_t>(outs, 4 * num_sms))),
                    dim3(kGradThreads), tab, st, p);
}

}  // namespace

cudaError_t launch_pack_rows(const void* src, int64_t ld, int64_t group_stride, int groups,
                             int64_t rows, int cols, void* dst, int64_t ld_dst, cudaStream_t st) {
  return launch_pdl(pack_rows_kernel, dim3(static_cast<unsigned>(groups * rows)), dim3(kPackThreads),
                    0, st, static_cast<const uint16_t*>(src), ld, group_stride, rows, cols,
                    static_cast<uint16_t*>(dst), ld_dst);
}

cudaError_t launch_row_grad(bool bf16, const RowGradParams& p, int num_sms, cudaStream_t st) {
  return bf16 ? row_grad<__nv_bfloat16>(p, num_sms, st) : row_grad<__half>(p, num_sms, st);
}

}  // namespace moe
