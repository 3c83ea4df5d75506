// C ABI of the stand-alone operators (moe_linear*, moe_swiglu*): argument
// checks, tensor maps, the choice of tile and split, the workspace.
#include <algorithm>
#include <cmath>
#include <cudaTypedefs.h>

#include "api_util.h"
#include "moe_internal.h"
#include "products.h"

namespace moe {
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();
}

namespace {

using namespace moe;

constexpr int kMaxRows = 1 << 24;
constexpr int kMaxFeatures = 65536;
constexpr int64_t kMaxStride = (1LL << 31) - 1;
constexpr size_t kWsAlign = 256;
constexpr int kMaxDevices = 64;

size_t ws_round(size_t v) { return (v + kWsAlign - 1) / kWsAlign * kWsAlign; }

// The kernels' status word of each device (set by a bounded wait that gave up).
__device__ int g_product_status;

// CTAs of clusters of 1, 2, 4 and 8 that fit the device at once, one per SM.
struct Room {
  int ctas[4];
  int of(int cluster) const { return ctas[cluster >= 8 ? 3 : cluster >= 4 ? 2 : cluster - 1]; }
  int sms() const { return ctas[0]; }
};

// The current device's status word and room, looked up once per device and
// host thread (and again if a device reset gave the device another context),
// with the kernels' attributes set.
int device_of(Room* room, int** status) {
  struct Entry {
    unsigned long long ctx = 0;
    Room room{};
    int* status = nullptr;
  };
  static thread_local Entry cache[kMaxDevices];
  int dev = -1;
  MOE_CUDA(cudaGetDevice(&dev));
  if (dev < 0 || dev >= kMaxDevices) return MOE_ERR_UNSUPPORTED;
  Entry& e = cache[dev];
  CUcontext ctx = nullptr;
  unsigned long long id = 0;
  static thread_local PFN_cuCtxGetCurrent_v4000 get_ctx = nullptr;
  static thread_local PFN_cuCtxGetId_v12000 get_id = nullptr;
  if (get_ctx == nullptr || get_id == nullptr) {
    cudaDriverEntryPointQueryResult q;
    void *a = nullptr, *b = nullptr;
    MOE_CUDA(cudaGetDriverEntryPointByVersion("cuCtxGetCurrent", &a, 12000, cudaEnableDefault, &q));
    MOE_CUDA(cudaGetDriverEntryPointByVersion("cuCtxGetId", &b, 12000, cudaEnableDefault, &q));
    if (a == nullptr || b == nullptr) return MOE_ERR_CUDA;
    get_ctx = reinterpret_cast<PFN_cuCtxGetCurrent_v4000>(a);
    get_id = reinterpret_cast<PFN_cuCtxGetId_v12000>(b);
  }
  const bool have = get_ctx(&ctx) == CUDA_SUCCESS && ctx != nullptr &&
                    get_id(ctx, &id) == CUDA_SUCCESS;
  if (e.status == nullptr || !have || id != e.ctx) {
    void* p = nullptr;
    MOE_CUDA(cudaGetSymbolAddress(&p, g_product_status));
    MOE_CUDA(cudaDeviceGetAttribute(&e.room.ctas[0], cudaDevAttrMultiProcessorCount, dev));
    MOE_CUDA(product_configure_device());
    for (int i = 1; i < 4; ++i) MOE_CUDA(product_cluster_room(1 << i, &e.room.ctas[i]));
    MOE_CUDA(product_pair_configure_device());
    e.status = static_cast<int*>(p);
    if (get_ctx(&ctx) != CUDA_SUCCESS || ctx == nullptr || get_id(ctx, &id) != CUDA_SUCCESS)
      return MOE_ERR_CUDA;
    e.ctx = id;
  }
  *room = e.room;
  *status = e.status;
  return MOE_OK;
}

// A 16-bit operand [groups][rows][cols] with its strides, 128-byte swizzle,
// out-of-range elements read as zero.
//  wide = false: (cols, rows, groups), box 64 columns (128 bytes) x box_rows;
//  wide = true:  (64, rows, cols / 64, groups), box 64 x box_rows x 2 chunks,
//                cols a multiple of 64 (so every element lies in the tensor).
// Without groups (group_stride 0) that dimension is left out.
bool encode(CUtensorMap* m, bool bf16, const void* base, int64_t cols, int64_t rows,
            int64_t groups, int64_t ld, int64_t group_stride, int box_rows, bool wide) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  if (enc == nullptr) return false;
  cuuint64_t dim[4], stride[3];
  cuuint32_t box[4], n = 0;
  auto add = [&](int64_t d, int b, int64_t s) {  // s: bytes from one index to the next
    dim[n] = static_cast<cuuint64_t>(d);
    box[n] = static_cast<cuuint32_t>(b);
    if (n > 0) stride[n - 1] = static_cast<cuuint64_t>(s);
    ++n;
  };
  add(wide ? 64 : cols, 64, 2);
  add(rows, box_rows, ld * 2);
  if (wide) add(cols / 64, 2, 128);
  if (group_stride > 0) add(groups, 1, group_stride * 2);
  cuuint32_t estr[4] = {1, 1, 1, 1};
  return enc(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, n,
             const_cast<void*>(base), dim, stride, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool tma_ready(const void* p, int64_t ld, int64_t group_stride) {
  return aligned(p, 16) && ld % 8 == 0 && group_stride % 8 == 0;
}

// Elements per access to the rows of a 16-bit matrix.
int row_width(const void* p, int64_t ld, int64_t cols) {
  if (aligned(p, 16) && ld % 8 == 0 && cols % 8 == 0) return 8;
  return aligned(p, 4) && ld % 2 == 0 ? 2 : 1;
}

// A matrix in memory: rows of `cols` bytes, `ld` bytes apart.
struct Block {
  const void* p;
  int64_t rows, cols, ld;
};
Block block(const void* p, int64_t rows, int64_t cols, int64_t ld, int el = 2) {
  return {p, rows, cols * el, ld * el};
}
Block flat(const void* p, int64_t n, int el = 2) { return {p, 1, n * el, n * el}; }

// Whether two matrices share bytes: their extents meet, and they are not
// columns apart in rows of the same stride (slices of one tensor).
bool overlap(const Block& x, const Block& y) {
  if (x.p == nullptr || y.p == nullptr || x.rows <= 0 || y.rows <= 0) return false;
  const uintptr_t a = reinterpret_cast<uintptr_t>(x.p), b = reinterpret_cast<uintptr_t>(y.p);
  const uintptr_t a1 = a + static_cast<uintptr_t>((x.rows - 1) * x.ld + x.cols);
  const uintptr_t b1 = b + static_cast<uintptr_t>((y.rows - 1) * y.ld + y.cols);
  if (a >= b1 || b >= a1) return false;
  // a single row lies in rows of any stride (it may cross two of them)
  const int64_t ld = x.rows > 1 ? x.ld : y.ld;
  if ((x.rows > 1 && y.rows > 1 && x.ld != y.ld) || x.cols > ld || y.cols > ld) return true;
  // y starts d bytes into a row of x's
  int64_t d = static_cast<int64_t>(b - a) % ld;
  if (d < 0) d += ld;
  return !(d >= x.cols && ld - d >= y.cols);
}

bool stride_ok(int64_t ld, int64_t cols) { return ld >= cols && ld <= kMaxStride; }

int check_config(const moe_linear_config_t* c) {
  if (c == nullptr || c->rows < 0 || c->in_features < 1 || c->out_features < 1 || c->groups < 0 ||
      c->activation < MOE_ACT_NONE || c->activation > MOE_ACT_GELU_TANH)
    return MOE_ERR_INVALID_ARG;
  if (c->dtype < MOE_F32 || c->dtype > MOE_F16) return MOE_ERR_INVALID_ARG;
  if (c->dtype != MOE_BF16 && c->dtype != MOE_F16) return MOE_ERR_UNSUPPORTED;
  if (c->rows > kMaxRows || c->in_features > kMaxFeatures || c->out_features > kMaxFeatures ||
      c->groups > kProductMaxGroups)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// W's own checks: strides, and the elements it spans
int check_w(const moe_linear_config_t* c, const void* w, int64_t ld, int64_t gs, Block* r) {
  if (w == nullptr || !aligned(w, 2) || !stride_ok(ld, c->out_features)) return MOE_ERR_INVALID_ARG;
  const int64_t K = c->in_features, G = c->groups;
  *r = block(w, K, c->out_features, ld);
  if (G > 1) {
    if (gs < (K - 1) * ld + c->out_features) return MOE_ERR_INVALID_ARG;
    if (gs > (1LL << 38)) return MOE_ERR_UNSUPPORTED;
    // groups whole rows apart are more rows; else everything from first to last
    *r = gs % ld == 0 ? block(w, (G - 1) * (gs / ld) + K, c->out_features, ld)
                      : flat(w, (G - 1) * gs + (K - 1) * ld + c->out_features);
  }
  return MOE_OK;
}

int check_forward(const moe_linear_config_t* c, const moe_linear_args_t* a) {
  int r = check_config(c);
  if (r != MOE_OK) return r;
  if (a == nullptr) return MOE_ERR_INVALID_ARG;
  if (c->rows == 0) return MOE_OK;
  const int64_t R = c->rows, K = c->in_features, N = c->out_features;
  Block w{};
  if (a->x == nullptr || a->out == nullptr || (c->groups > 0) != (a->offsets != nullptr) ||
      !stride_ok(a->ld_x, K) || !stride_ok(a->ld_out, N) ||
      (a->residual != nullptr && !stride_ok(a->ld_residual, N)) ||
      (a->preact != nullptr && !stride_ok(a->ld_preact, N)))
    return MOE_ERR_INVALID_ARG;
  if (!aligned(a->x, 2) || !aligned(a->out, 2) || !aligned(a->bias, 2) ||
      !aligned(a->residual, 2) || !aligned(a->preact, 2) || !aligned(a->offsets, 4))
    return MOE_ERR_INVALID_ARG;
  if ((r = check_w(c, a->w, a->ld_w, a->group_stride_w, &w)) != MOE_OK) return r;
  const Block x = block(a->x, R, K, a->ld_x), out = block(a->out, R, N, a->ld_out);
  const Block pre = block(a->preact, R, N, a->ld_preact);
  const Block res = block(a->residual, R, N, a->ld_residual);
  const Block bias = flat(a->bias, std::max(1, c->groups) * N);
  const bool in_place = a->residual == a->out && a->ld_residual == a->ld_out;
  for (const Block& o : {out, pre})
    if (overlap(o, x) || overlap(o, w) || overlap(o, bias)) return MOE_ERR_INVALID_ARG;
  if (overlap(out, pre) || overlap(pre, res) || (overlap(out, res) && !in_place))
    return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

int check_backward(const moe_linear_config_t* c, const moe_linear_grads_t* a) {
  int r = check_config(c);
  if (r != MOE_OK) return r;
  if (a == nullptr) return MOE_ERR_INVALID_ARG;
  const int64_t R = c->rows, K = c->in_features, N = c->out_features;
  const int64_t G = std::max(1, c->groups);
  if (!aligned(a->dw, 2) || !aligned(a->dbias, 2) || !aligned(a->dx, 2)) return MOE_ERR_INVALID_ARG;
  if (R == 0) return MOE_OK;
  if (a->dout == nullptr || !aligned(a->dout, 2) || !stride_ok(a->ld_dout, N) ||
      (c->groups > 0) != (a->offsets != nullptr) || !aligned(a->offsets, 4) ||
      (c->activation != MOE_ACT_NONE) != (a->preact != nullptr) || !aligned(a->preact, 2) ||
      (a->preact != nullptr && !stride_ok(a->ld_preact, N)) ||
      (a->dx != nullptr && !stride_ok(a->ld_dx, K)) ||
      (a->dw != nullptr && (a->x == nullptr || !aligned(a->x, 2) || !stride_ok(a->ld_x, K))))
    return MOE_ERR_INVALID_ARG;
  Block w{};
  if (a->dx != nullptr && (r = check_w(c, a->w, a->ld_w, a->group_stride_w, &w)) != MOE_OK) return r;
  const Block in[4] = {block(a->dout, R, N, a->ld_dout), w, block(a->preact, R, N, a->ld_preact),
                       block(a->dw != nullptr ? a->x : nullptr, R, K, a->ld_x)};
  const Block out[3] = {block(a->dx, R, K, a->ld_dx), flat(a->dw, G * K * N),
                        flat(a->dbias, G * N)};
  for (int i = 0; i < 3; ++i) {
    for (const Block& v : in)
      if (overlap(out[i], v)) return MOE_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return MOE_ERR_INVALID_ARG;
  }
  return MOE_OK;
}

int64_t padded(int64_t cols) { return (cols + 7) / 8 * 8; }
size_t copy_bytes(int64_t rows, int64_t cols) {
  return ws_round(static_cast<size_t>(rows) * static_cast<size_t>(padded(cols)) * 2);
}

struct ForwardWs {
  bool copy_x, copy_w;
  size_t x, w, total;
};
int64_t group_stride(const moe_linear_config_t* c, int64_t gs, int64_t ld) {
  return c->groups > 1 ? gs : ld * c->in_features;
}
ForwardWs forward_ws(const moe_linear_config_t* c, const moe_linear_args_t* a) {
  ForwardWs w{};
  if (c->rows == 0) return w;
  w.copy_x = !tma_ready(a->x, a->ld_x, 0);
  w.copy_w = !tma_ready(a->w, a->ld_w, group_stride(c, a->group_stride_w, a->ld_w));
  w.x = w.total;
  if (w.copy_x) w.total += copy_bytes(c->rows, c->in_features);
  w.w = w.total;
  if (w.copy_w)
    w.total += copy_bytes(static_cast<int64_t>(std::max(1, c->groups)) * c->in_features,
                          c->out_features);
  return w;
}

struct BackwardWs {
  bool copy_x, copy_w, copy_dout, make_dz;
  size_t x, w, dz, partial, total;
};
BackwardWs backward_ws(const moe_linear_config_t* c, const moe_linear_grads_t* a) {
  BackwardWs w{};
  if (c->rows == 0) return w;
  const int G = std::max(1, c->groups);
  const bool products = a->dx != nullptr || a->dw != nullptr;
  w.make_dz = c->activation != MOE_ACT_NONE && products;
  w.copy_dout = c->activation == MOE_ACT_NONE && products && !tma_ready(a->dout, a->ld_dout, 0);
  w.copy_x = a->dw != nullptr && !tma_ready(a->x, a->ld_x, 0);
  w.copy_w = a->dx != nullptr &&
             !tma_ready(a->w, a->ld_w, group_stride(c, a->group_stride_w, a->ld_w));
  w.x = w.total;
  if (w.copy_x) w.total += copy_bytes(c->rows, c->in_features);
  w.w = w.total;
  if (w.copy_w)
    w.total += copy_bytes(static_cast<int64_t>(G) * c->in_features, c->out_features);
  w.dz = w.total;
  if (w.make_dz || w.copy_dout) w.total += copy_bytes(c->rows, c->out_features);
  w.partial = w.total;
  if (a->dbias != nullptr && c->rows > kRowDirect)
    w.total += ws_round(row_grad_chunks(c->rows, G, row_grad_chunk(c->rows, G, c->out_features)) *
                        static_cast<size_t>(c->out_features) * 4);
  return w;
}

int check_ws(const void* ws, size_t have, size_t need) {
  if (need == 0) return MOE_OK;
  return ws == nullptr || !aligned(ws, kWsAlign) || have < need ? MOE_ERR_WORKSPACE : MOE_OK;
}

struct Operand {
  const void* p;
  int64_t ld, gs;
};

// Tile, split and order of a product.
struct Choice {
  bool pair;
  int bn, split, chunk;
};

// What the choice goes by: features, `groups` groups of `mean` rows (dw:
// output rows) each, of differing sizes if ragged, and blocks64 slots of 64
// contraction steps per tile.
struct Shape {
  int64_t feats, groups, mean, blocks64;
  bool ragged, dw, epilogue;  // epilogue: more than a bias
  int width;                  // of the output's accesses, see row_width
  int a_lines, b_lines;       // L2 lines per 128 bytes of an operand's rows: 1 or 2
};
// Rows that do not start at 128 bytes take two lines per 128 bytes (132 rows
// 4904 -> 4624: 34 us on tiles that L2's delivery bounds, 4864 -> 4608 18).
int lines(const Operand& o) { return aligned(o.p, 128) && o.ld % 64 == 0 ? 1 : 2; }

// Row blocks of bn rows over all groups; a ragged group fills half of its last
// one on average.
int64_t row_blocks(const Shape& q, int64_t bn) {
  if (!q.ragged) return q.groups * ((q.mean + bn - 1) / bn);
  return (q.groups * q.mean + bn - 1) / bn + q.groups / 2;
}

// Nanoseconds, as measured on one B200 with weights from L2 (graphs of calls in
// a row), of one slot of 64 contraction steps.  A few CTAs alone are bound by
// what their MMA warps issue; many by what L2 delivers, 16 bytes a picosecond.
// One CTA, 128 features x bn rows: 16 CTAs take 132, 128, 154, 163 ns per slot at
// bn = 16, 32, 64, 128, 128 CTAs 160 at 16 rows, 210 at 64, 258 at 128.
int64_t l2_ns(const Shape& q, int64_t ctas, int b_rows) {
  return ctas * (kProductBM * q.a_lines + b_rows * q.b_lines) * 128 / 16000;
}
int64_t one_cta_slot_ns(const Shape& q, int bn, int64_t ctas) {
  const int alone = bn <= 32 ? 132 : bn <= 64 ? 154 : 162;
  return std::max<int64_t>(alone, l2_ns(q, ctas, bn));
}
// A CTA pair, 256 features: 262 ns per slot up to 224 rows and 280 at 256 for a
// few pairs; on all SMs 360 at 256 rows (23 us per wave of 64 slots), 330 at
// 224, 310 at 208 and below.  With two accumulators of half the rows 43 us per
// wave at 512 rows, 28 at 320, and 4.6 us more per tile, since its epilogue
// overlaps the next tile less (1280 -> 4096 at 4096 rows: 33 us with one, 42
// with two; 4096 -> 1280, where two accumulators make one wave of what else is
// two: 36 us and 40 forward, 33 and 39 for dx, 35 and 44 for dw).
int64_t pair_slot_ns(const Shape& q, int bn, int64_t ctas, int num_sms) {
  const int64_t l2 = l2_ns(q, ctas, bn / 2);
  if (bn > 256) return std::max<int64_t>(440 + std::max(0, bn - 320) * 240 / 192, l2);
  const int all = bn >= 240 ? 360 : bn >= 224 ? 330 : 310;
  return std::max<int64_t>({bn >= 240 ? 280 : 265, all * ctas / num_sms, l2});
}
constexpr int kPairTileNs = 500, kPairTwoTileNs = 4600;
// What a call takes beside its slots and epilogues.
constexpr int kOneCtaNs = 3700, kPairNs = 4500;
// Nanoseconds of a tile's epilogue, the least that a tile takes (dw of few rows
// per group: 48 x 3588 x 744 103 us in one-CTA tiles of 128 rows, 36 x 4096 x
// 1280 117 us in pair tiles of 256); twice that where rows are not at 16 bytes.
// With the above, intercepts over the contraction's length: 4.2 us on one-CTA
// tiles of 16 rows, 5.3 at 128, 7.8 on pair tiles at 256.
int one_cta_epilogue_ns(int bn) { return 500 + 13 * bn; }
int pair_epilogue_ns(int bn) { return 700 + 10 * bn; }
// Joining a split tile (intercepts over the contraction's length: 64 rows 4096
// features 4.6 us unsplit, 5.0 in 2 parts, 6.2 in 4; 128 rows 5.3, 6.1, 7.3; one
// tile of 64 rows 4.2, 4.6, 5.1, 5.6 in 1, 2, 4, 8; pairs at 192 and 256 rows 1.9
// and 2.5 in 4 parts).
int one_cta_join_ns(int split, int rows) {
  return split == 2 ? 500 + 5 * rows : (split == 4 ? 1000 : 1300) + 8 * rows;
}
int pair_join_ns(int split, int rows) { return split == 2 ? 700 + 7 * rows : 1100 + 5 * rows; }

Choice choose(const Shape& q, const Room& room) {
  const int num_sms = room.sms();
  Choice best{false, 0, 1, 1};
  const int slow = q.width == 8 ? 1 : 2;
  int64_t best_ns = 0;
  auto offer = [&](bool pair, int bn, int split, int64_t ns) {
    if (best.bn == 0 || ns < best_ns) {
      best = {pair, bn, split, 1};
      best_ns = ns;
    }
  };
  auto slots = [&](int split) { return (q.blocks64 + split - 1) / split; };
  const int64_t f1 = (q.feats + kProductBM - 1) / kProductBM;
  for (int bn = 16; bn <= kProductMaxBN; bn *= 2) {
    if (bn > 16 && bn >= 2 * q.mean) break;
    const int rows = static_cast<int>(std::min<int64_t>(bn, q.mean));
    const int64_t tiles = f1 * row_blocks(q, bn);
    for (int split = 1; split <= kProductMaxSplit; split *= 2) {
      if (split > 1 && (tiles * split > room.of(split) || split > q.blocks64)) break;
      const int64_t ctas = std::min<int64_t>(tiles * split, num_sms);
      const int64_t ns = slots(split) * one_cta_slot_ns(q, bn, ctas);
      const int64_t end = slow * one_cta_epilogue_ns(bn);
      const int64_t waves = (tiles + num_sms - 1) / num_sms;
      offer(false, bn, split,
            kOneCtaNs + (split > 1 ? ns + one_cta_join_ns(split, rows) + end
                                   : waves * std::max(ns, end) + std::min(ns, end)));
    }
  }
  const int64_t f2 = (q.feats + 2 * kProductBM - 1) / (2 * kProductBM);
  // dw's rows per tile are multiples of 32, see product_pair.cu.  A longer epilogue
  // costs two accumulators' poorer overlap more, and takes one (4096 -> 11264 with
  // gelu: 272 us with two, 254 with one; without it 251 and 242).
  const int step = q.dw ? 32 : 16;
  for (int bn = q.epilogue ? 256 : kProductPairMaxBN; bn >= 128 && q.mean > 64; bn -= step) {
    const int rows = static_cast<int>(std::min<int64_t>(bn, q.mean));
    const int64_t tiles = f2 * row_blocks(q, bn);
    const int64_t waves = (tiles + num_sms / 2 - 1) / (num_sms / 2);
    for (int split = 1; split <= (q.dw || bn > 256 ? 1 : kProductPairMaxSplit); split *= 2) {
      // (an uneven deal of the chunks of 16 rows sends more than the slots hold)
      if (split > 1 && (2 * tiles * split > room.of(2 * split) || split > q.blocks64 ||
                        bn % (16 * split) != 0))
        break;
      const int64_t ctas = std::min<int64_t>(2 * tiles * split, num_sms);
      const int64_t ns = slots(split) * pair_slot_ns(q, bn, ctas, num_sms);
      const int64_t end = slow * pair_epilogue_ns(std::min(bn, 256));
      const int64_t tile = bn <= 256 ? kPairTileNs : slow * kPairTwoTileNs;
      offer(true, bn, split,
            kPairNs + (split > 1 ? ns + pair_join_ns(split, rows) + end
                                 : waves * (std::max(ns, bn <= 256 ? end : slow * pair_epilogue_ns(bn)) +
                                            tile) + std::min(ns, end)));
    }
  }
  // a chunk's rows stay in L2 across its weight tiles: up to 32 MB of them
  // (4096 x 4096 -> 11264: 259 us with 8 blocks, 274 with 4; its dx, with rows
  // of 22 KB, 254 with 2 and 272 with 8)
  const int64_t block_bytes = static_cast<int64_t>(best.bn) * q.blocks64 * 128;
  best.chunk = static_cast<int>(std::min<int64_t>(16, std::max<int64_t>(1, (32 << 20) / block_bytes)));
  return best;
}

// Groups that can have rows, and their mean size.
void filled(const int32_t* offsets, int64_t groups, int64_t rows, int64_t* n, int64_t* mean) {
  *n = offsets == nullptr ? 1 : std::min(groups, rows);
  *mean = (rows + *n - 1) / *n;
}

int box_rows(const Choice& ch, int rows) {
  return ch.pair ? product_pair_half(ch.bn, 16) / 2 : std::min(ch.bn, rows);
}

cudaError_t launch_any(const Choice& ch, int mode, bool bf16, const ProductMaps& m,
                       const ProductParams& p, int sms, cudaStream_t st) {
  return ch.pair ? launch_product_pair(mode, bf16, m, p, sms, st)
                 : launch_product(mode, bf16, m, p, sms, st);
}

// The choice for one of the products and its place in the parameters.
void take(const Shape& q, const Room& room, ProductParams* p, Choice* ch) {
  *ch = choose(q, room);
  p->bn = ch->bn;
  p->box_rows = box_rows(*ch, p->rows);
  p->chunk = ch->chunk;
  p->split = ch->split;
}

Choice choose_forward(const moe_linear_config_t* c, const moe_linear_args_t* a, const Operand& x,
                      const Operand& w, const Room& room, ProductParams* p) {
  const int64_t K = c->in_features, N = c->out_features;
  p->offsets = a->offsets;
  p->groups = std::max(1, c->groups);
  p->rows = c->rows;
  p->feats = c->out_features;
  p->depth = c->in_features;
  p->out = a->out;
  p->ld_out = a->ld_out;
  p->bias = a->bias;
  p->residual = a->residual;
  p->ld_residual = a->ld_residual;
  p->preact = a->preact;
  p->ld_preact = a->ld_preact;
  p->act = c->activation;
  p->width_out = row_width(a->out, a->ld_out, N);
  p->width_residual = row_width(a->residual, a->ld_residual, N);
  p->width_preact = row_width(a->preact, a->ld_preact, N);
  p->wide_a = N % 64 == 0;
  int64_t n_groups, mean;
  filled(a->offsets, p->groups, c->rows, &n_groups, &mean);
  const bool epilogue =
      c->activation != MOE_ACT_NONE || a->residual != nullptr || a->preact != nullptr;
  Choice ch;
  take({N, n_groups, mean, (K + 63) / 64, n_groups > 1, false, epilogue, p->width_out, lines(w),
        lines(x)}, room, p, &ch);
  return ch;
}

Choice choose_dx(const moe_linear_config_t* c, const moe_linear_grads_t* a, const Operand& dz,
                 const Operand& w, const Room& room, ProductParams* p) {
  const int64_t K = c->in_features, N = c->out_features;
  p->offsets = a->offsets;
  p->groups = std::max(1, c->groups);
  p->rows = c->rows;
  p->feats = c->in_features;
  p->depth = c->out_features;
  p->out = a->dx;
  p->ld_out = a->ld_dx;
  p->width_out = row_width(a->dx, a->ld_dx, K);
  int64_t n_groups, mean;
  filled(a->offsets, p->groups, c->rows, &n_groups, &mean);
  Choice ch;
  take({K, n_groups, mean, (N + 63) / 64, n_groups > 1, false, false, p->width_out, lines(w),
        lines(dz)}, room, p, &ch);
  return ch;
}

Choice choose_dw(const moe_linear_config_t* c, const moe_linear_grads_t* a, const Operand& dz,
                 const Operand& x, const Room& room, ProductParams* p) {
  const int64_t K = c->in_features, N = c->out_features;
  p->offsets = a->offsets;
  p->groups = std::max(1, c->groups);
  p->rows = c->rows;
  p->feats = c->out_features;
  p->cols = c->in_features;
  p->depth = 0;
  p->out = a->dw;
  p->ld_out = N;
  p->width_out = row_width(a->dw, N, N);
  const int64_t steps = std::max<int64_t>(1, (c->rows / p->groups + 63) / 64);
  Choice ch;
  take({N, p->groups, K, steps, false, true, false, p->width_out, lines(dz), lines(x)}, room, p, &ch);
  return ch;
}

int report(int mode, const Choice& ch, ProductParams* p, moe_linear_tiles_t* t) {
  if ((ch.pair ? product_pair_slots(mode, p) : product_slots(mode, p)) == 0) return MOE_ERR_CUDA;
  *t = {ch.pair ? 1 : 0, ch.bn, ch.pair && ch.bn > 256 ? 2 : 1, ch.split, p->stages, 64 * p->subs};
  return MOE_OK;
}

// Turns *o into its copy at dst with 16-byte aligned rows.  With offsets the
// weights of groups without rows are left out.
PackOperand aligned_copy(Operand* o, int64_t groups, int64_t rows, int64_t cols, void* dst,
                         const int32_t* offsets = nullptr) {
  const int64_t ld = padded(cols);
  const PackOperand c{o->p, o->ld, o->gs, groups, rows, static_cast<int>(cols), dst, ld, offsets};
  *o = {dst, ld, groups > 1 || o->gs > 0 ? ld * rows : 0};
  return c;
}

}  // namespace

extern "C" {

int moe_linear_config_check(const moe_linear_config_t* cfg) { return check_config(cfg); }

int moe_linear_workspace_size(const moe_linear_config_t* cfg, const moe_linear_args_t* args,
                              size_t* bytes) {
  if (bytes == nullptr) return MOE_ERR_INVALID_ARG;
  const int r = check_forward(cfg, args);
  if (r != MOE_OK) return r;
  *bytes = forward_ws(cfg, args).total;
  return MOE_OK;
}

int moe_linear_backward_workspace_size(const moe_linear_config_t* cfg,
                                       const moe_linear_grads_t* grads, size_t* bytes) {
  if (bytes == nullptr) return MOE_ERR_INVALID_ARG;
  const int r = check_backward(cfg, grads);
  if (r != MOE_OK) return r;
  *bytes = backward_ws(cfg, grads).total;
  return MOE_OK;
}

int moe_linear(const moe_linear_config_t* c, const moe_linear_args_t* a, void* workspace,
               size_t ws_bytes, void* stream) {
  int r = check_forward(c, a);
  if (r != MOE_OK) return r;
  if (c->rows == 0) return MOE_OK;
  const ForwardWs ws = forward_ws(c, a);
  if ((r = check_ws(workspace, ws_bytes, ws.total)) != MOE_OK) return r;
  Room room{};
  int* status = nullptr;
  if ((r = device_of(&room, &status)) != MOE_OK) return r;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint8_t* base = static_cast<uint8_t*>(workspace);
  const int64_t R = c->rows, K = c->in_features, N = c->out_features;
  const int G = std::max(1, c->groups);
  const bool bf16 = c->dtype == MOE_BF16;
  Operand x{a->x, a->ld_x, 0}, w{a->w, a->ld_w, group_stride(c, a->group_stride_w, a->ld_w)};
  PackParams pack{};
  if (ws.copy_x) pack.op[0] = aligned_copy(&x, 1, R, K, base + ws.x);
  if (ws.copy_w) pack.op[1] = aligned_copy(&w, G, K, N, base + ws.w, a->offsets);
  MOE_CUDA(launch_pack_rows(pack, st));
  ProductParams p{};
  const Choice ch = choose_forward(c, a, x, w, room, &p);
  p.status = status;
  ProductMaps m;
  if (!encode(&m.a, bf16, w.p, N, K, G, w.ld, w.gs, 64, p.wide_a) ||
      !encode(&m.b, bf16, x.p, K, R, 1, x.ld, 0, p.box_rows, false))
    return MOE_ERR_CUDA;
  MOE_CUDA(launch_any(ch, kProductForward, bf16, m, p, room.sms(), st));
  return MOE_OK;
}

int moe_linear_backward(const moe_linear_config_t* c, const moe_linear_grads_t* a,
                        void* workspace, size_t ws_bytes, void* stream) {
  int r = check_backward(c, a);
  if (r != MOE_OK) return r;
  const BackwardWs ws = backward_ws(c, a);
  if ((r = check_ws(workspace, ws_bytes, ws.total)) != MOE_OK) return r;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int64_t R = c->rows, K = c->in_features, N = c->out_features;
  const int G = std::max(1, c->groups);
  const bool bf16 = c->dtype == MOE_BF16;
  if (R == 0) {
    if (a->dw != nullptr) MOE_CUDA(cudaMemsetAsync(a->dw, 0, static_cast<size_t>(G) * K * N * 2, st));
    if (a->dbias != nullptr) MOE_CUDA(cudaMemsetAsync(a->dbias, 0, static_cast<size_t>(G) * N * 2, st));
    return MOE_OK;
  }
  Room room{};
  int* status = nullptr;
  if ((r = device_of(&room, &status)) != MOE_OK) return r;
  uint8_t* base = static_cast<uint8_t*>(workspace);
  Operand x{a->x, a->ld_x, 0}, w{a->w, a->ld_w, group_stride(c, a->group_stride_w, a->ld_w)};
  Operand dz{a->dout, a->ld_dout, 0};
  const bool products = a->dx != nullptr || a->dw != nullptr;
  const bool row_pass = ws.make_dz || a->dbias != nullptr;
  const bool joins = a->dbias != nullptr && c->rows > kRowDirect;  // a launch of its own adds db
  // copies and dz in one launch, then dx, then dw beside it, then db beside both
  PackParams pack{};
  if (ws.copy_dout && !row_pass) pack.op[0] = aligned_copy(&dz, 1, R, N, base + ws.dz);
  if (ws.copy_w) pack.op[1] = aligned_copy(&w, G, K, N, base + ws.w, a->offsets);
  if (ws.copy_x) pack.op[2] = aligned_copy(&x, 1, R, K, base + ws.x);
  RowGradParams q{};
  if (!row_pass) {
    MOE_CUDA(launch_pack_rows(pack, st));
  } else {
    q.copies = pack;
    q.dout = a->dout;
    q.ld_dout = a->ld_dout;
    q.preact = a->preact;
    q.ld_preact = a->ld_preact;
    q.dz = ws.make_dz || ws.copy_dout ? base + ws.dz : nullptr;
    q.ld_dz = padded(N);
    q.dz_scale = ws.make_dz && !bf16 ? 0.5f : 1.f;
    q.offsets = a->offsets;
    q.groups = G;
    q.rows = c->rows;
    q.cols = c->out_features;
    q.act = c->activation;
    q.db = a->dbias;
    q.direct = a->dbias != nullptr && !joins;
    q.chunk = row_grad_chunk(c->rows, G, c->out_features);
    q.partial = reinterpret_cast<float*>(base + ws.partial);
    MOE_CUDA(launch_row_grad(bf16, q, room.sms(), st));
    if (q.dz != nullptr) dz = {base + ws.dz, padded(N), 0};
  }
  ProductParams p{};
  p.status = status;
  p.out_scale = ws.make_dz && !bf16 ? 2.f : 1.f;
  ProductMaps m;
  if (a->dx != nullptr) {
    const Choice ch = choose_dx(c, a, dz, w, room, &p);
    if (!encode(&m.a, bf16, w.p, N, K, G, w.ld, w.gs, kProductBM, false) ||
        !encode(&m.b, bf16, dz.p, N, R, 1, dz.ld, 0, p.box_rows, false))
      return MOE_ERR_CUDA;
    p.order = {false};
    MOE_CUDA(launch_any(ch, kProductDx, bf16, m, p, room.sms(), st));
  }
  if (a->dw != nullptr) {
    const Choice ch = choose_dw(c, a, dz, x, room, &p);
    if (!encode(&m.a, bf16, dz.p, N, R, 1, dz.ld, 0, 64, false) ||
        !encode(&m.b, bf16, x.p, K, R, 1, x.ld, 0, 64, false))
      return MOE_ERR_CUDA;
    p.order = {a->dx != nullptr};
    MOE_CUDA(launch_any(ch, kProductDw, bf16, m, p, room.sms(), st));
  }
  if (joins) {
    q.order = {products};
    MOE_CUDA(launch_bias_grad(bf16, q, room.sms(), st));
  }
  return MOE_OK;
}

int moe_linear_tiles(const moe_linear_config_t* c, const moe_linear_args_t* a,
                     moe_linear_tiles_t* tiles) {
  if (tiles == nullptr) return MOE_ERR_INVALID_ARG;
  int r = check_forward(c, a);
  if (r != MOE_OK) return r;
  *tiles = {};
  if (c->rows == 0) return MOE_OK;
  Room room{};
  int* status = nullptr;
  if ((r = device_of(&room, &status)) != MOE_OK) return r;
  Operand x{a->x, a->ld_x, 0}, w{a->w, a->ld_w, group_stride(c, a->group_stride_w, a->ld_w)};
  // (a workspace starts at 256 bytes, as its parts do)
  const ForwardWs ws = forward_ws(c, a);
  if (ws.copy_x) x = {nullptr, padded(c->in_features), 0};
  if (ws.copy_w) w = {nullptr, padded(c->out_features), 0};
  ProductParams p{};
  const Choice ch = choose_forward(c, a, x, w, room, &p);
  return report(kProductForward, ch, &p, tiles);
}

int moe_linear_backward_tiles(const moe_linear_config_t* c, const moe_linear_grads_t* a,
                              moe_linear_tiles_t* dx, moe_linear_tiles_t* dw) {
  if (dx == nullptr || dw == nullptr) return MOE_ERR_INVALID_ARG;
  int r = check_backward(c, a);
  if (r != MOE_OK) return r;
  *dx = *dw = {};
  if (c->rows == 0) return MOE_OK;
  Room room{};
  int* status = nullptr;
  if ((r = device_of(&room, &status)) != MOE_OK) return r;
  Operand x{a->x, a->ld_x, 0}, w{a->w, a->ld_w, group_stride(c, a->group_stride_w, a->ld_w)};
  Operand dz{a->dout, a->ld_dout, 0};
  const BackwardWs ws = backward_ws(c, a);
  if (ws.copy_x) x = {nullptr, padded(c->in_features), 0};
  if (ws.copy_w) w = {nullptr, padded(c->out_features), 0};
  if (ws.make_dz || ws.copy_dout) dz = {nullptr, padded(c->out_features), 0};
  ProductParams p{};
  if (a->dx != nullptr) {
    const Choice ch = choose_dx(c, a, dz, w, room, &p);
    if ((r = report(kProductDx, ch, &p, dx)) != MOE_OK) return r;
  }
  if (a->dw != nullptr) {
    const Choice ch = choose_dw(c, a, dz, x, room, &p);
    if ((r = report(kProductDw, ch, &p, dw)) != MOE_OK) return r;
  }
  return MOE_OK;
}

int moe_linear_get_device_error(int* device_err) {
  Room room{};
  int* status = nullptr;
  if (device_err == nullptr) return MOE_ERR_INVALID_ARG;
  const int r = device_of(&room, &status);
  if (r != MOE_OK) return r;
  MOE_CUDA(cudaDeviceSynchronize());
  MOE_CUDA(cudaMemcpy(device_err, status, sizeof(int), cudaMemcpyDeviceToHost));
  if (*device_err == 0) return MOE_OK;
  MOE_CUDA(cudaMemset(status, 0, sizeof(int)));
  return MOE_ERR_DEVICE_TIMEOUT;
}

}  // extern "C"

namespace {

int check_swiglu(const moe_swiglu_config_t* c) {
  if (c == nullptr || c->rows < 0 || c->width < 1 || c->groups < 0 || !std::isfinite(c->limit) ||
      c->limit < 0.f || c->dtype < MOE_F32 || c->dtype > MOE_F16)
    return MOE_ERR_INVALID_ARG;
  if (c->dtype == MOE_FP8_E4M3 || c->rows > kMaxRows || c->width > kMaxFeatures ||
      c->groups > kProductMaxGroups)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// an output may be one of the inputs (the same rows, read before written by
// the thread that writes them) or apart from it
bool apart_or_same(const Block& o, const Block& i) {
  return (o.p == i.p && o.ld == i.ld) || !overlap(o, i);
}

}  // namespace

extern "C" {

int moe_swiglu(const moe_swiglu_config_t* c, const void* gate, int64_t ld_gate, const void* up,
               int64_t ld_up, const float* scale, const int32_t* offsets, void* out,
               int64_t ld_out, void* stream) {
  const int r = check_swiglu(c);
  if (r != MOE_OK) return r;
  if (c->rows == 0) return MOE_OK;
  const int el = c->dtype == MOE_F32 ? 4 : 2;
  const int64_t R = c->rows, W = c->width;
  if (gate == nullptr || up == nullptr || out == nullptr || !aligned(gate, el) ||
      !aligned(up, el) || !aligned(out, el) || !aligned(scale, 4) || !aligned(offsets, 4) ||
      !stride_ok(ld_gate, W) || !stride_ok(ld_up, W) || !stride_ok(ld_out, W) ||
      (c->groups > 0) != (offsets != nullptr) ||
      !apart_or_same(block(out, R, W, ld_out, el), block(gate, R, W, ld_gate, el)) ||
      !apart_or_same(block(out, R, W, ld_out, el), block(up, R, W, ld_up, el)) ||
      overlap(block(out, R, W, ld_out, el), flat(scale, R, 4)))
    return MOE_ERR_INVALID_ARG;
  SwigluParams p{};
  p.gate = gate;
  p.ld_gate = ld_gate;
  p.up = up;
  p.ld_up = ld_up;
  p.out = out;
  p.ld_out = ld_out;
  p.scale = scale;
  p.offsets = offsets;
  p.groups = c->groups;
  p.rows = c->rows;
  p.cols = c->width;
  p.limit = c->limit;
  MOE_CUDA(launch_swiglu(c->dtype, p, static_cast<cudaStream_t>(stream)));
  return MOE_OK;
}

int moe_swiglu_backward(const moe_swiglu_config_t* c, const void* dout, int64_t ld_dout,
                        const void* gate, int64_t ld_gate, const void* up, int64_t ld_up,
                        const float* scale, const int32_t* offsets, void* dgate, int64_t ld_dgate,
                        void* dup, int64_t ld_dup, float* dscale, void* stream) {
  const int r = check_swiglu(c);
  if (r != MOE_OK) return r;
  if (c->rows == 0) return MOE_OK;
  const int el = c->dtype == MOE_F32 ? 4 : 2;
  const int64_t R = c->rows, W = c->width;
  if (dout == nullptr || gate == nullptr || up == nullptr || dgate == nullptr || dup == nullptr ||
      !aligned(dout, el) || !aligned(gate, el) || !aligned(up, el) || !aligned(dgate, el) ||
      !aligned(dup, el) || !aligned(scale, 4) || !aligned(dscale, 4) || !aligned(offsets, 4) ||
      !stride_ok(ld_dout, W) || !stride_ok(ld_gate, W) || !stride_ok(ld_up, W) ||
      !stride_ok(ld_dgate, W) || !stride_ok(ld_dup, W) || (c->groups > 0) != (offsets != nullptr))
    return MOE_ERR_INVALID_ARG;
  const Block in[3] = {block(dout, R, W, ld_dout, el), block(gate, R, W, ld_gate, el),
                       block(up, R, W, ld_up, el)};
  const Block outs[2] = {block(dgate, R, W, ld_dgate, el), block(dup, R, W, ld_dup, el)};
  const Block sc = flat(scale, R, 4), ds = flat(dscale, R, 4);
  for (const Block& o : outs) {
    for (const Block& i : in)
      if (!apart_or_same(o, i)) return MOE_ERR_INVALID_ARG;
    if (overlap(o, sc) || overlap(o, ds)) return MOE_ERR_INVALID_ARG;
  }
  for (const Block& i : in)
    if (overlap(i, ds)) return MOE_ERR_INVALID_ARG;
  if (overlap(outs[0], outs[1]) || overlap(ds, sc)) return MOE_ERR_INVALID_ARG;
  SwigluParams p{};
  p.gate = gate;
  p.ld_gate = ld_gate;
  p.up = up;
  p.ld_up = ld_up;
  p.dout = dout;
  p.ld_dout = ld_dout;
  p.dgate = dgate;
  p.ld_dgate = ld_dgate;
  p.dup = dup;
  p.ld_dup = ld_dup;
  p.scale = scale;
  p.dscale = dscale;
  p.offsets = offsets;
  p.groups = c->groups;
  p.rows = c->rows;
  p.cols = c->width;
  p.limit = c->limit;
  MOE_CUDA(launch_swiglu_backward(c->dtype, p, static_cast<cudaStream_t>(stream)));
  return MOE_OK;
}

}  // extern "C"
