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

// One row of any of the operands, by a warp.
__device__ __forceinline__ void pack_row(const PackParams& p, int64_t row, int lane) {
  int i = 0;
  while (i < 3 && row >= p.op[i].groups * p.op[i].rows) {
    row -= p.op[i].groups * p.op[i].rows;
    ++i;
  }
  if (i == 3) return;
  const PackOperand& o = p.op[i];
  const int64_t g = row / o.rows;
  // (offsets that decrease are raised by the products: no such group has rows either)
  if (o.offsets != nullptr && o.offsets[g + 1] <= o.offsets[g]) return;
  const uint16_t* s = static_cast<const uint16_t*>(o.src) + g * o.group_stride + (row - g * o.rows) * o.ld;
  uint16_t* d = static_cast<uint16_t*>(o.dst) + row * o.ld_dst;
  constexpr int U = 8;  // loads under way per lane
  for (int c = lane; c < o.cols; c += U * 32) {
    uint16_t v[U];
#pragma unroll
    for (int k = 0; k < U; ++k)
      if (c + k * 32 < o.cols) v[k] = s[c + k * 32];
#pragma unroll
    for (int k = 0; k < U; ++k)
      if (c + k * 32 < o.cols) d[c + k * 32] = v[k];
  }
}

__global__ void __launch_bounds__(kPackThreads) pack_rows_kernel(const PackParams p) {
  pdl_wait();
  pack_row(p, static_cast<int64_t>(blockIdx.x) * (kPackThreads / 32) + (threadIdx.x >> 5),
           threadIdx.x & 31);
}

// CTAs for the copies: a warp per row
int64_t pack_ctas(const PackParams& p) {
  int64_t rows = 0;
  for (const PackOperand& o : p.op) rows += o.groups * o.rows;
  constexpr int kPer = kPackThreads / 32;
  return (rows + kPer - 1) / kPer;
}

constexpr int kGradThreads = kPackThreads;  // 8 warps: rows of a chunk are dealt to them
constexpr int kGradWarps = kGradThreads / 32;
constexpr int kVec = 8;                    // elements per 16-byte access
// Forms of the dz kernel: 16-byte pieces; single elements, eight per row and
// lane 32 apart; or two, for outputs of few CTAs whatever their alignment (77
// rows x 776 with gelu_tanh, db alone: 9.2 us in 16-byte pieces, 4.8 so).
constexpr int kFormVec = 0, kFormWide = 1, kFormNarrow = 2;
template <int FORM>
constexpr int kLaneCols = FORM == kFormNarrow ? 2 : kVec;

template <typename T>
struct alignas(16) Vec {
  T v[kVec];
};

// One CTA: `chunk` rows of one group x 256 columns (narrow form: 64), or with
// `direct` all rows of the group.  The column sums are added in fp32, per warp
// over its rows, then over the warps in order; direct: they are the group's and
// go to db at once.  The vector form needs every row at a 16-byte boundary and
// cols % 8 == 0.  Each lane keeps U rows' loads under way; with an activation
// (ACT, else dz = dout) the slope's registers leave room for one row of eight.
// The first copy_ctas CTAs copy misaligned operands instead.
template <typename T, int FORM, bool ACT>
__global__ void __launch_bounds__(kGradThreads, 4) row_grad_kernel(const RowGradParams p) {
  constexpr bool VEC = FORM == kFormVec;
  constexpr int E = kLaneCols<FORM>;
  constexpr int U = FORM == kFormVec ? (ACT ? 1 : 4) : FORM == kFormWide ? (ACT ? 1 : 2) : (ACT ? 4 : 8);
  constexpr int kCols = 32 * E;
  extern __shared__ int tab_mem[];
  __shared__ alignas(16) float sums[kGradWarps][kCols];
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (blockIdx.x < p.copy_ctas) {
    pack_row(p.copies, static_cast<int64_t>(blockIdx.x) * kGradWarps + warp, lane);
    return;
  }
  const GroupTable tab = build_group_table(tab_mem, p.offsets, p.groups, p.rows, p.chunk);
  const int col_blocks = (p.cols + kCols - 1) / kCols;
  const int total = (p.direct ? p.groups : tab.block_start[p.groups]) * col_blocks;
  const T* dout = static_cast<const T*>(p.dout);
  const T* preact = static_cast<const T*>(p.preact);
  T* dz = static_cast<T*>(p.dz);
  for (int w = blockIdx.x - p.copy_ctas; w < total; w += gridDim.x - p.copy_ctas) {
    const int chunk = w / col_blocks;  // (direct: the group)
    const int c0 = (w - chunk * col_blocks) * kCols;
    const int g = p.direct ? chunk : group_of_block(tab, p.groups, chunk);
    const int first = p.direct ? 0 : (chunk - tab.block_start[g]) * p.chunk;
    const int n = p.direct ? tab.count(g) : min(p.chunk, tab.count(g) - first);
    const int64_t row0 = static_cast<int64_t>(tab.row0[g]) + first;
    float acc[E] = {};
    const int col = VEC ? c0 + lane * kVec : c0 + lane;
    if (col < p.cols) {
      for (int r = warp; r < n; r += U * kGradWarps) {
        // the rows' values, loaded before the first is used
        Vec<T> dv[U], zv[U];
#pragma unroll
        for (int k = 0; k < U; ++k) {
          const int64_t row = row0 + min(r + k * kGradWarps, n - 1);
          const T* d = dout + row * p.ld_dout + col;
          const T* z = preact + row * p.ld_preact + col;
          if (VEC) {
            dv[k] = *reinterpret_cast<const Vec<T>*>(d);
            if (ACT) zv[k] = *reinterpret_cast<const Vec<T>*>(z);
          } else {
#pragma unroll
            for (int i = 0; i < E; ++i)
              if (col + 32 * i < p.cols) {
                dv[k].v[i] = d[32 * i];
                if (ACT) zv[k].v[i] = z[32 * i];
              }
          }
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
          if (r + k * kGradWarps < n) {
            T* out = dz + (row0 + r + k * kGradWarps) * p.ld_dz + col;
            float v[E];
#pragma unroll
            for (int i = 0; i < E; ++i) v[i] = to_f32<T>(dv[k].v[i]);
            if (ACT) {
              float s[E];
#pragma unroll
              for (int i = 0; i < E; ++i) s[i] = to_f32<T>(zv[k].v[i]);
              slope_all(s, p.act);
#pragma unroll
              for (int i = 0; i < E; ++i) v[i] *= s[i];
            }
#pragma unroll
            for (int i = 0; i < E; ++i) {
              if (VEC || col + 32 * i < p.cols) acc[i] += v[i];
              // (a bf16 dz is never scaled)
              dv[k].v[i] = from_f32<T>(is_bf16<T>() ? v[i] : v[i] * p.dz_scale);
              if (!VEC && dz != nullptr && col + 32 * i < p.cols) out[32 * i] = dv[k].v[i];
            }
            if (VEC && dz != nullptr) *reinterpret_cast<Vec<T>*>(out) = dv[k];
          }
        }
      }
    }
    if (p.db != nullptr) {
      if (VEC) {
#pragma unroll
        for (int i = 0; i < E; i += 4)
          *reinterpret_cast<float4*>(&sums[warp][lane * kVec + i]) =
              make_float4(acc[i], acc[i + 1], acc[i + 2], acc[i + 3]);
      } else {
#pragma unroll
        for (int i = 0; i < E; ++i) sums[warp][lane + 32 * i] = acc[i];
      }
      __syncthreads();
      const int c = c0 + threadIdx.x;
      if (threadIdx.x < kCols && c < p.cols) {
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
  begin_ordered(p.order);
  pdl_trigger();
  const GroupTable tab = build_group_table(tab_mem, p.offsets, p.groups, p.rows, p.chunk);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int col_blocks = (p.cols + 31) / 32;
  for (int w = blockIdx.x; w < p.groups * col_blocks; w += gridDim.x) {
    const int g = w / col_blocks;
    const int c = (w - g * col_blocks) * 32 + lane;
    const int n = tab.block_start[g + 1] - tab.block_start[g];
    float v = 0.f;
    if (c < p.cols) {
      const float* s = p.partial + static_cast<int64_t>(tab.block_start[g]) * p.cols + c;
#pragma unroll 16
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
  end_ordered(p.order);
}

bool rows_aligned(const void* p, int64_t ld) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % kVec == 0;
}

template <typename T>
cudaError_t row_grad(const RowGradParams& p0, int num_sms, cudaStream_t st) {
  RowGradParams p = p0;
  const int64_t copies = pack_ctas(p.copies);
  if (copies > INT32_MAX / 2) return cudaErrorInvalidValue;
  p.copy_ctas = static_cast<unsigned>(copies);
  const size_t tab = group_table_bytes(p.groups);
  const bool vec = p.cols % kVec == 0 && rows_aligned(p.dout, p.ld_dout) &&
                   (p.preact == nullptr || rows_aligned(p.preact, p.ld_preact)) &&
                   (p.dz == nullptr || rows_aligned(p.dz, p.ld_dz));
  const int64_t units =
      p.direct ? p.groups : static_cast<int64_t>(row_grad_chunks(p.rows, p.groups, p.chunk)) + 1;
  auto items = [&](int form) {
    const int cols = 32 * (form == kFormNarrow ? 2 : kVec);
    return units * ((p.cols + cols - 1) / cols);
  };
  const int form = items(kFormWide) < (vec ? 1 : 2) * num_sms ? kFormNarrow
                   : vec                                     ? kFormVec
                                                             : kFormWide;
  const dim3 grid(p.copy_ctas + static_cast<unsigned>(std::min<int64_t>(items(form), 4 * num_sms)));
  auto go = [&](auto kernel) { return launch_pdl(kernel, grid, dim3(kGradThreads), tab, st, p); };
  if (p.preact != nullptr)
    return form == kFormVec    ? go(row_grad_kernel<T, kFormVec, true>)
           : form == kFormWide ? go(row_grad_kernel<T, kFormWide, true>)
                               : go(row_grad_kernel<T, kFormNarrow, true>);
  return form == kFormVec    ? go(row_grad_kernel<T, kFormVec, false>)
         : form == kFormWide ? go(row_grad_kernel<T, kFormWide, false>)
                             : go(row_grad_kernel<T, kFormNarrow, false>);
}

template <typename T>
cudaError_t bias_grad(const RowGradParams& p, int num_sms, cudaStream_t st) {
  const int64_t outs = static_cast<int64_t>(p.groups) * ((p.cols + 31) / 32);
  return launch_pdl(bias_grad_kernel<T>, dim3(static_cast<int>(std::min<int64_t>(outs, 4 * num_sms))),
                    dim3(kGradThreads), group_table_bytes(p.groups), st, p);
}

}  // namespace

cudaError_t launch_pack_rows(const PackParams& p, cudaStream_t st) {
  const int64_t ctas = pack_ctas(p);
  if (ctas == 0) return cudaSuccess;
  if (ctas > INT32_MAX) return cudaErrorInvalidValue;
  return launch_pdl(pack_rows_kernel, dim3(static_cast<unsigned>(ctas)), dim3(kPackThreads), 0, st,
                    p);
}

cudaError_t launch_row_grad(bool bf16, const RowGradParams& p, int num_sms, cudaStream_t st) {
  return bf16 ? row_grad<__nv_bfloat16>(p, num_sms, st) : row_grad<__half>(p, num_sms, st);
}

cudaError_t launch_bias_grad(bool bf16, const RowGradParams& p, int num_sms, cudaStream_t st) {
  return bf16 ? bias_grad<__nv_bfloat16>(p, num_sms, st) : bias_grad<__half>(p, num_sms, st);
}

}  // namespace moe
