// Internal interface of the stand-alone products (linear, grouped_linear and
// their gradients): what products_api.cu fills in for the kernels of
// product_gemm.cu and product_rows.cu.  Not installed, not part of the ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace moe {

// One kernel computes all three products, as out[j][f] = sum_c A[f][c] B[j][c]
// (features f on the MMA's M side and the accumulator's lanes, so a warp's
// lanes write consecutive outputs; rows j on its N side, 16 at a time, so a
// tile with few rows costs little):
//   forward  A = W_g^T (features = N, read MN-major from W [K, N]), B = x,  c = K
//   dx       A = W_g   (features = K, read K-major),                B = dz, c = N
//   dw       A = dz^T  (features = N, MN-major), B = x^T (MN-major, j = K),
//            c = the group's rows
constexpr int kProductForward = 0;
constexpr int kProductDx = 1;
constexpr int kProductDw = 2;

constexpr int kProductMaxGroups = 1024;
constexpr int kProductBM = 128;     // features per CTA tile
constexpr int kProductMaxBN = 128;  // rows per one-CTA tile (a multiple of 16)
constexpr int kProductMaxSplit = 8;

// Division of 0 <= n < 2^31 by a divisor known on the host.
struct FastDiv {
  uint32_t mul, shift, d;
};
inline FastDiv fast_div(uint32_t d) {
  uint32_t s = 0;
  while ((1ull << s) < d) ++s;
  return {static_cast<uint32_t>(((1ull << 32) * ((1ull << s) - d)) / d + 1), s, d};
}

// A product, a bias gradient and SwiGLU let their successor in the stream start
// (pdl_trigger) once they have waited for their predecessor and allocated their
// tensor memory; the successor sets itself up below them and waits for their end
// before it touches a tensor.  (An allocation of the successor's that came first
// would wait with it for good.)  Calls in a row, 32 rows 1280 -> 4096: 7.7 us
// each without, 6.8 so.  Not so the row pass, whose registers the products' CTAs
// would take (4096 x 4096 x 1280 gradients 97.2 us a pass for 96.1).
//
// The kernels of one backward call run one after another, but some do not need
// the one before: dw runs beside dx, the bias gradient beside both.  Such a
// kernel (late_wait) does not wait for what it reads: the row pass's dz, copies
// and partial sums.  It relies on the call's first product, which precedes it in
// the stream and lets it start only after all of its own CTAs have waited for
// the row pass to complete with its memory visible (pdl_wait before
// pdl_trigger); a kernel of another host thread's call that comes between them
// in the stream either waits itself or was let start by one that did.  So a
// call's first product is never late_wait.  Such a kernel waits for its
// predecessor only before it ends, so that what follows it in the stream follows
// both.
struct LaunchOrder {
  bool late_wait;
};

struct ProductParams {
  LaunchOrder order;
  const int* offsets;  // [groups + 1] first row of each group; nullptr: one group of all rows
  int groups;          // >= 1
  int rows;            // rows of x / dz that exist
  int feats;           // F: features of the output
  int cols;            // dw: J, the output's rows per group; else unused
  int depth;           // contraction length (forward K, dx N; dw: unused)
  int bn;              // rows per tile, a multiple of 16
  int box_rows;        // rows of map b's box (forward, dx)
  int chunk;           // row blocks per ordering chunk
  int stages, subs;    // pipeline slots, sub-slots of 64 steps in each
  // forward: the weights' map walks 64-element chunks in a dimension of its own,
  // so that one load brings both chunks of a CTA's 128 features (else one each;
  // 4096 x 4096 -> 11264 248 us against 258; dw gained nothing from it)
  bool wide_a;
  int split;           // CTAs, or pairs, of a cluster sharing one tile's contraction
  // of the tile order, filled in at launch: feature tiles, row blocks per group
  // and their rows (dw: even parts rounded up to 32), and divisions by the tiles
  // of a group (dw) or of a row block, and by those of an ordering chunk
  int f_tiles, dw_blocks, dw_rows;
  FastDiv by_group, by_chunk;
  float out_scale;     // dx, dw in fp16: 1 / dz_scale
  void* out;
  int64_t ld_out;      // elements between output rows
  const void* bias;    // [groups, feats] or nullptr
  const void* residual;
  int64_t ld_residual;
  void* preact;
  int64_t ld_preact;
  int act;             // moe_activation_t
  // elements per access that the rows' alignment allows: 8 (and feats a multiple
  // of 8), 2 or 1
  int width_out, width_residual, width_preact;
  int* status;         // device status word
};

// Fills in the tile order for tiles of bm features; returns the most tiles the
// launch can have (a ragged problem's count is known on the device only).
inline int64_t product_tile_order(int mode, int bm, ProductParams* p) {
  p->f_tiles = (p->feats + bm - 1) / bm;
  p->dw_blocks = mode == kProductDw ? (p->cols + p->bn - 1) / p->bn : 0;
  if (mode == kProductDw) {
    const int even = ((p->cols + p->dw_blocks - 1) / p->dw_blocks + 31) / 32 * 32;
    p->dw_rows = even < p->bn ? even : p->bn;
  }
  p->by_group = fast_div(static_cast<uint32_t>(p->f_tiles * (mode == kProductDw ? p->dw_blocks : 1)));
  p->by_chunk = fast_div(static_cast<uint32_t>(p->f_tiles * p->chunk));
  int64_t blocks;
  if (mode == kProductDw)
    blocks = static_cast<int64_t>(p->groups) * p->dw_blocks;
  else if (p->offsets == nullptr)
    blocks = (p->rows + p->bn - 1) / p->bn;
  else
    blocks = p->rows / p->bn + p->groups < p->rows ? p->rows / p->bn + p->groups : p->rows;
  return blocks * p->f_tiles;
}

struct ProductMaps {
  CUtensorMap a, b;
};

cudaError_t launch_product(int mode, bool bf16, const ProductMaps& m, const ProductParams& p,
                           int num_sms, cudaStream_t st);
// Fills in the pipeline's slots; returns the dynamic shared memory, 0 if it does
// not fit.
size_t product_slots(int mode, ProductParams* p);
size_t product_pair_slots(int mode, ProductParams* p);

// The same on CTA pairs (product_pair.cu): tiles of 256 features x bn rows, up
// to 256 with one accumulator per tile, up to 512 with two of half the rows;
// map b's box has half of an accumulator's rows (dw: 64 steps, as for one CTA).
constexpr int kProductPairMaxBN = 512;
constexpr int kProductPairMaxSplit = 4;
constexpr int product_pair_half(int bn, int unit) {
  return bn <= 256 ? bn : (bn / 2 + unit - 1) / unit * unit;
}
cudaError_t launch_product_pair(int mode, bool bf16, const ProductMaps& m, const ProductParams& p,
                                int num_sms, cudaStream_t st);

// one-time per-device kernel attributes (dynamic shared memory limits)
cudaError_t product_configure_device();
// CTAs in clusters of that size that fit the device at once, one per SM
cudaError_t product_cluster_room(int cluster, int* ctas);
cudaError_t product_pair_configure_device();

// Row kernels (product_rows.cu).
// Copies of operands with rows of ld_dst elements, all in one launch (groups 0:
// no operand).
struct PackOperand {
  const void* src;
  int64_t ld, group_stride;
  int64_t groups, rows;
  int cols;
  void* dst;
  int64_t ld_dst;
  const int* offsets;  // not nullptr: groups of no rows are left out
};
struct PackParams {
  PackOperand op[3];
};
cudaError_t launch_pack_rows(const PackParams& p, cudaStream_t st);

struct RowGradParams {
  LaunchOrder order;   // of the bias gradient's launch
  PackParams copies;   // made in the same launch as dz
  unsigned copy_ctas;  // (filled in at launch)
  const void* dout;
  int64_t ld_dout;
  const void* preact;  // nullptr: dz = dout
  int64_t ld_preact;
  void* dz;            // nullptr: not written
  int64_t ld_dz;
  // dz is stored times this: 1/2 in fp16, since slopes reach 1.13 and |dout| fp16's
  // largest value (dz would be infinite where dx and dw are not), else 1.  A power
  // of two, taken back exactly in the products' fp32 sums; it costs the steps of
  // 2^-24 below 2^-13, which become 2^-23.
  float dz_scale;
  const int* offsets;
  int groups, rows, cols;
  int act;
  void* db;            // [groups, cols] or nullptr
  // db of few rows: a CTA sums all rows of a group, in the one launch; else each
  // CTA sums a chunk of rows into partial [chunks, cols] and a second launch
  // adds the chunks
  bool direct;
  int chunk;           // rows of a chunk, see row_grad_chunk
  float* partial;
};
// Up to here a CTA walks its group's rows alone: 16 rows per warp at most.
constexpr int kRowDirect = 128;
inline size_t row_grad_chunks(int rows, int groups, int chunk) {
  return static_cast<size_t>(rows) / chunk + static_cast<size_t>(groups);
}
// Rows of a chunk: 128 where that makes enough work for the device, else 32.
inline int row_grad_chunk(int rows, int groups, int cols) {
  return row_grad_chunks(rows, groups, 128) * ((cols + 255) / 256) >= 512 ? 128 : 32;
}
// dz = dout * act'(preact), and db (direct) or its partial sums from dz in fp32
cudaError_t launch_row_grad(bool bf16, const RowGradParams& p, int num_sms, cudaStream_t st);
// db from the partial sums
cudaError_t launch_bias_grad(bool bf16, const RowGradParams& p, int num_sms, cudaStream_t st);

// SwiGLU (swiglu.cu)
struct SwigluParams {
  const void *gate, *up, *dout;
  int64_t ld_gate, ld_up, ld_dout;
  void *out, *dgate, *dup;
  int64_t ld_out, ld_dgate, ld_dup;
  const float* scale;  // [rows] or nullptr
  float* dscale;       // [rows] or nullptr
  const int* offsets;  // rows outside [offsets[0], offsets[groups]) are left alone
  int groups, rows, cols;
  float limit;
};
cudaError_t launch_swiglu(int dtype, const SwigluParams& p, cudaStream_t st);
cudaError_t launch_swiglu_backward(int dtype, const SwigluParams& p, cudaStream_t st);

}  // namespace moe
