// C ABI of the operators around the attention (declared in
// include/wsattn.h): argument checks, work split, tensor maps and launches.
#include <cmath>
#include <cstring>
#include <new>

#include "ops.h"

using wsattn::GemmParams;
using wsattn::QkParams;
using wsattn::QkPart;
using wsattn::RotTable;

struct wsattn_rotary_s {
  RotTable table;
};

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t round8(int64_t a) { return (a + 7) / 8 * 8; }
size_t up256(size_t x) { return (x + 255) / 256 * 256; }
int dtype_size(int dtype) { return dtype == WSATTN_FP32 ? 4 : 2; }
bool dtype_ok(int dtype) { return dtype >= WSATTN_BF16 && dtype <= WSATTN_FP32; }

int sm_count() {
  static int sms[wsattn::kMaxDevices] = {};
  const int dev = wsattn::current_device();
  if (dev < 0) return 0;
  if (!sms[dev] &&
      cudaDeviceGetAttribute(&sms[dev], cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    sms[dev] = 0;
  return sms[dev];
}

// ------------------------------------------------------------- head views

// The smallest strides that keep a view's elements apart, whatever the order
// of its dimensions.
bool apart(const wsattn_heads* v, int batch, int64_t n, int dim) {
  int64_t size[3] = {batch, v->heads, n};
  int64_t stride[3] = {v->stride_b, v->stride_h, v->stride_n};
  for (int i = 0; i < 3; ++i)
    for (int j = i + 1; j < 3; ++j)
      if (stride[j] < stride[i]) {
        const int64_t s = stride[i], z = size[i];
        stride[i] = stride[j];
        size[i] = size[j];
        stride[j] = s;
        size[j] = z;
      }
  int64_t extent = dim;
  for (int i = 0; i < 3; ++i) {
    if (size[i] <= 1) continue;
    if (stride[i] < extent || stride[i] > (INT64_MAX - extent) / size[i]) return false;
    extent = stride[i] * (size[i] - 1) + extent;
  }
  return true;
}

bool view_ok(const wsattn_heads* v, int esize) {
  if (!v || v->heads < 1 || v->stride_b < 0 || v->stride_h < 0 || v->stride_n < 0) return false;
  return (reinterpret_cast<uintptr_t>(v->data) & static_cast<uintptr_t>(esize - 1)) == 0;
}

// Every row of the view starts on a 16-byte boundary.
bool view_vec(const wsattn_heads* v, int batch, int64_t n, int esize) {
  const int64_t per = 16 / esize;
  return aligned16(v->data) && (batch <= 1 || v->stride_b % per == 0) &&
         (v->heads <= 1 || v->stride_h % per == 0) && (n <= 1 || v->stride_n % per == 0);
}

QkPart part_of(const wsattn_heads* in, const wsattn_heads* out, int norm, int turn,
               const void* weight) {
  QkPart p;
  std::memset(&p, 0, sizeof(p));
  p.io.in = in->data;
  p.io.out = out->data;
  p.io.ib = in->stride_b;
  p.io.in_ = in->stride_n;
  p.io.ih = in->stride_h;
  p.io.ob = out->stride_b;
  p.io.on = out->stride_n;
  p.io.oh = out->stride_h;
  p.io.heads = in->heads;
  p.norm = norm;
  p.turn = turn;
  p.weight = weight;
  return p;
}

// Lanes per head row, rows per CTA, and the heads that a warp walks for one
// token: all of a part's, or a half, a quarter ... until there are enough work
// items (a CTA's tokens times a group of heads).  Forward: one group size for
// all parts (a CTA is an item), want_items of them.  Backward: each part its
// own, 32 items a CTA as long as a warp keeps more than 12 heads (an item costs
// its angles, one and a half heads' time), and 8 items with fewer.
// False: more items than an int counts.
bool split_work(QkParams* p, int64_t rows, int64_t ctas, bool back) {
  const bool equal = !back;
  const int pieces = p->rot.pairs / 8;
  p->lanes_log2 = 0;
  while ((1 << p->lanes_log2) < pieces) ++p->lanes_log2;
  p->rows = rows;
  const int per_cta = wsattn::kQkThreads / 32 * (32 >> p->lanes_log2);
  p->row_blocks = cdiv(rows, per_cta);
  int gh[3] = {1, 1, 1}, most = 1;
  for (int i = 0; i < p->parts; ++i) {
    gh[i] = p->part[i].io.heads;
    if (gh[i] > most) most = gh[i];
  }
  if (equal) gh[0] = gh[1] = gh[2] = most;
  const int counted = equal || p->parts < 2 ? p->parts : 2;  // the backward's copies go apart
  auto groups = [&] {
    int64_t n = 0;
    for (int i = 0; i < counted; ++i) n += cdiv(p->part[i].io.heads, gh[i]);
    return n;
  };
  while (true) {
    int k = 0;
    for (int i = 1; i < counted; ++i)
      if (gh[i] > gh[k]) k = i;
    const int64_t want = !back ? ctas : gh[k] > 12 ? 32 * ctas : 8 * ctas;
    if (p->row_blocks * groups() >= want || gh[k] <= (back ? 4 : 1)) break;
    const int less = (gh[k] + 1) / 2;
    if (equal) gh[0] = gh[1] = gh[2] = less;
    else gh[k] = less;
  }
  p->groups = 0;
  for (int i = 0; i < p->parts; ++i) {
    p->part[i].group0 = p->groups;
    p->part[i].group_heads = gh[i];
    p->part[i].groups = static_cast<int>(cdiv(p->part[i].io.heads, gh[i]));
    p->groups += p->part[i].groups;
  }
  return p->row_blocks <= INT32_MAX / p->groups;
}

// Rows (batch times tokens) then fit 64 bits.
bool tokens_ok(int64_t n_tokens) { return n_tokens >= 0 && n_tokens <= INT32_MAX; }
bool positions_ok(const float* positions, int64_t pos_stride_b) {
  return pos_stride_b >= 0 && (reinterpret_cast<uintptr_t>(positions) & 3u) == 0;
}

// CTAs of the backward pass: fixed upper bound, so that the workspace does
// not depend on the device.
constexpr int kMaxBackCtas = 1024;

// ------------------------------------------------------------------ linear

struct Operand {
  const void* ptr;
  int64_t ld;  // elements
};

bool rows_vec(const void* p, int64_t ld, int64_t rows, int64_t cols, int esize) {
  const int64_t per = 16 / esize;
  return aligned16(p) && (rows <= 1 || ld % per == 0) && cols % per == 0;
}
// TMA reads rows of any length, but each must start on 16 bytes.
bool tma_rows(const void* p, int64_t ld, int64_t rows) {
  return aligned16(p) && (rows <= 1 || ld % 8 == 0);
}

bool encode(CUtensorMap* m, CUtensorMapDataType type, int esize, const void* ptr, int64_t inner,
            int64_t outer, int64_t ld, int box_inner, int box_outer) {
  PFN_cuTensorMapEncodeTiled_v12000 fn = wsattn::tensor_map_encoder();
  if (!fn) return false;
  // a single row's stride is never used, but must be a valid one
  const int64_t per = 16 / esize;
  if (outer <= 1) ld = (inner + per - 1) / per * per;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(outer)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * esize};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(box_inner), static_cast<cuuint32_t>(box_outer)};
  const cuuint32_t es[2] = {1, 1};
  return fn(m, type, 2, const_cast<void*>(ptr), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Product {
  int dtype;
  bool out_f32;
  Operand p, q;  // rows and columns of the output
  bool p_mn, q_mn;
  int64_t R;
  int C, K;
  const void* bias;
  const void* res;
  int64_t ldr;
  void* out;
  int64_t ldo;
  void* pre;
  int64_t ldp;
  int act;
  // column sums to add on the side (db null: none)
  const float* part;
  int parts;
  float* db;
  int db_cols;
};

// The kernel's parameters for one product under a tiling; false: a tensor
// map could not be made, or the sizes exceed an int's range of tiles.
bool fill(const Product& g, const wsattn::GemmShape& shape, void* partial, GemmParams* out) {
  GemmParams& prm = *out;
  const CUtensorMapDataType type = g.dtype == WSATTN_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                          : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  const int esize = g.out_f32 ? 4 : 2;
  const int rows_p = shape.pair_cols ? 128 : shape.bn;
  const int rows_q = shape.pair_cols ? shape.pair_cols / 2 : wsattn::kTileCols;
  auto operand = [&](CUtensorMap* m, const Operand& o, bool mn, int64_t own, int box) {
    return mn ? encode(m, type, 2, o.ptr, own, g.K, o.ld, 64, wsattn::kGemmK)
              : encode(m, type, 2, o.ptr, g.K, own, o.ld, wsattn::kGemmK, box);
  };
  if (!operand(&prm.tm_p, g.p, g.p_mn, g.R, rows_p) || !operand(&prm.tm_q, g.q, g.q_mn, g.C, rows_q))
    return false;
  prm.status = wsattn::op_status_ptr();
  if (!prm.status) return false;
  prm.R = g.R;
  prm.C = g.C;
  prm.K = g.K;
  prm.p_mn = g.p_mn;
  prm.q_mn = g.q_mn;
  prm.bias = g.bias;
  prm.res = g.res;
  prm.ldr = g.ldr;
  prm.out = g.out;
  prm.ldo = g.ldo;
  prm.pre = g.pre;
  prm.ldp = g.ldp;
  prm.act = g.act;
  prm.part = g.part;
  prm.ldpart = g.db_cols;
  prm.parts = g.parts;
  prm.db = g.db;
  prm.db_cols = g.db_cols;
  prm.bias_vec = g.bias && aligned16(g.bias);
  prm.res_vec = g.res && rows_vec(g.res, g.ldr, g.R, g.C, esize);
  prm.out_vec = tma_rows(g.out, g.out_f32 ? 2 * g.ldo : g.ldo, g.R);
  prm.pre_vec = g.pre && tma_rows(g.pre, g.ldp, g.R);
  int64_t tr, tc;
  if (shape.pair_cols) {
    tr = cdiv(g.R, wsattn::kPairRows);
    tc = cdiv(g.C, shape.pair_cols);
    auto tma_cols = [&](bool rows_ok, int size) {
      return !rows_ok ? 0 : g.C % (16 / size) == 0 ? g.C : g.C / (128 / size) * (128 / size);
    };
    prm.out_tma = tma_cols(prm.out_vec, esize);
    prm.pre_tma = tma_cols(prm.pre_vec && !g.out_f32, 2);
    prm.edge_tile = prm.out_vec && g.C % (16 / esize) ? static_cast<int>(tc) - 1 : -1;
    if (prm.out_tma && !encode(&prm.tm_out, g.out_f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : type, esize,
                               g.out, g.C, g.R, g.ldo, 128 / esize, 32))
      return false;
    if (prm.pre_tma && !encode(&prm.tm_pre, type, 2, g.pre, g.C, g.R, g.ldp, 64, 32))
      return false;
  } else {
    tr = cdiv(g.R, shape.bn);
    tc = cdiv(g.C, wsattn::kTileCols);
    prm.bn = shape.bn;
    // a ring of about 96 KB: two CTAs fit an SM
    prm.stages = 96 / (16 + shape.bn / 8);
  }
  prm.tiles_r = static_cast<int>(tr);
  prm.tiles_c = static_cast<int>(tc);
  prm.split = shape.split;
  prm.whole_tiles = shape.split > 1 ? shape.whole : static_cast<int>(tr * tc);
  prm.partial = static_cast<float*>(partial);
  return tr * tc <= INT32_MAX;
}

// partial: scratch of shape.bytes(g.R, g.C).
int run_product(const Product& g, const wsattn::GemmShape& shape, int sms, void* partial,
                cudaStream_t s) {
  wsattn::PairParams pp;
  std::memset(&pp, 0, sizeof(pp));
  if (!fill(g, shape, partial, &pp.g[0])) return WSATTN_ERR_CUDA;
  const cudaError_t e =
      shape.pair_cols ? wsattn::launch_gemm_pair(&pp, g.dtype, g.out_f32, shape.pair_cols, sms, s)
                      : wsattn::launch_gemm_tile(pp.g[0], g.dtype, g.out_f32, s);
  return e == cudaSuccess ? WSATTN_OK : WSATTN_ERR_CUDA;
}

// Both in one launch; g carries the column sums.
int run_together(const Product& g, const Product& h, int sms, cudaStream_t s) {
  const wsattn::GemmShape shape{256, 0, 1, 0};
  const bool g_first = g.K >= h.K;
  wsattn::PairParams pp;
  std::memset(&pp, 0, sizeof(pp));
  Product first = g_first ? g : h;
  first.part = g.part;
  first.parts = g.parts;
  first.db = g.db;
  first.db_cols = g.db_cols;
  if (!fill(first, shape, nullptr, &pp.g[0]) ||
      !fill(g_first ? h : g, shape, nullptr, &pp.g[1]))
    return WSATTN_ERR_CUDA;
  return wsattn::launch_gemm_pair(&pp, g.dtype, g.out_f32, 256, sms, s) == cudaSuccess
             ? WSATTN_OK
             : WSATTN_ERR_CUDA;
}

// A job of the pack pass (rows = 0: none).
wsattn::PackJob pack_job(const void* src, int64_t lds, int64_t rows, int cols, void* dst) {
  wsattn::PackJob j;
  std::memset(&j, 0, sizeof(j));
  j.src = src;
  j.lds = lds;
  j.rows = rows;
  j.cols = cols;
  j.dst = dst;
  j.ldd = round8(cols);
  return j;
}

// Scratch of one operand copied to aligned rows.
size_t packed_bytes(int64_t rows, int64_t cols) {
  return up256(static_cast<size_t>(rows) * static_cast<size_t>(round8(cols)) * 2);
}

constexpr int64_t kMaxRows = (int64_t(1) << 31) - 512;

bool linear_args_ok(const wsattn_linear_args* a) {
  if (!a || a->m < 0 || a->m > kMaxRows || a->n < 1 || a->k < 1 || a->n > (1 << 30) ||
      a->k > (1 << 30))
    return false;
  if (a->activation < WSATTN_ACT_NONE || a->activation > WSATTN_ACT_SILU) return false;
  if (a->x_heads < 0 || (a->x_heads == 0 && a->ldx < a->k) || a->ldw < a->k || a->ldo < a->n ||
      (a->residual && a->ldr < a->n) || (a->preact && a->ldp < a->n))
    return false;
  if (a->x_heads > 0) {
    if (a->k % a->x_heads || a->k / a->x_heads % 8) return false;
    if (a->m > 0 && (a->x_tokens < 1 || a->m % a->x_tokens)) return false;
  }
  return true;
}
bool half_type(int dtype) { return dtype == WSATTN_BF16 || dtype == WSATTN_FP16; }
bool elem_aligned(const void* p, int esize) {
  return (reinterpret_cast<uintptr_t>(p) & static_cast<uintptr_t>(esize - 1)) == 0;
}

wsattn::GemmShape linear_shape(const wsattn_linear_args* a) {
  double ns = 0.0;
  return wsattn::choose_gemm(a->m, a->n, a->k, false, &ns);
}

size_t linear_ws(const wsattn_linear_args* a, const wsattn::GemmShape& shape) {
  size_t b = 0;
  if (a->m == 0) return 0;
  if (a->x_heads > 0 || !tma_rows(a->x, a->ldx, a->m)) b += packed_bytes(a->m, a->k);
  if (!tma_rows(a->w, a->ldw, a->n)) b += packed_bytes(a->n, a->k);
  return b + shape.bytes(a->m, a->n);
}

bool grad_args_ok(const wsattn_linear_grad_args* a) {
  if (!a || a->m < 0 || a->m > kMaxRows || a->n < 1 || a->k < 1 || a->n > (1 << 30) ||
      a->k > (1 << 30))
    return false;
  if (a->activation < WSATTN_ACT_NONE || a->activation > WSATTN_ACT_SILU) return false;
  if (a->ldd < a->n || a->ldx < a->k || a->ldw < a->k || (a->preact && a->ldp < a->n) ||
      (a->dx && a->lddx < a->k) || (a->dw && a->lddw < a->k))
    return false;
  return true;
}

// Rows of dout per CTA of the dact pass: about 608 CTAs (four an SM, a
// constant, so that the workspace does not depend on the device), at least 32
// rows each (the partial sums stay small).
int dact_rows(int64_t m, int n) {
  const int64_t cols = cdiv(n, wsattn::kDactCols);
  int64_t blocks = cdiv(608, cols);
  int64_t rows = cdiv(m, blocks < 1 ? 1 : blocks);
  rows = (rows + 31) / 32 * 32;
  if (cdiv(m, rows) > 65535) rows = (cdiv(m, 65535) + 31) / 32 * 32;
  return static_cast<int>(rows);
}

struct GradPlan {
  bool act, dz, pack_x, pack_w;
  bool together;  // both products in one launch
  wsattn::GemmShape shape_w, shape_x;
  size_t dz_bytes, part_bytes, x_bytes, w_bytes, tile_bytes;
  int rows_per_block, row_blocks;
  size_t total() const { return dz_bytes + part_bytes + x_bytes + w_bytes + tile_bytes; }
};

GradPlan plan_grad(const wsattn_linear_grad_args* a) {
  GradPlan g;
  std::memset(&g, 0, sizeof(g));
  if (a->m == 0) return g;
  const bool products = a->dx || a->dw;
  g.act = a->activation != WSATTN_ACT_NONE;
  g.dz = products && (g.act || !tma_rows(a->dout, a->ldd, a->m));
  g.pack_x = a->dw && !tma_rows(a->x, a->ldx, a->m);
  g.pack_w = a->dx && !tma_rows(a->w, a->ldw, a->n);
  g.rows_per_block = dact_rows(a->m, a->n);
  g.row_blocks = static_cast<int>(cdiv(a->m, g.rows_per_block));
  if (g.dz) g.dz_bytes = packed_bytes(a->m, a->n);
  if (a->db) g.part_bytes = up256(sizeof(float) * static_cast<size_t>(g.row_blocks) * a->n);
  if (g.pack_x) g.x_bytes = packed_bytes(a->m, a->k);
  if (g.pack_w) g.w_bytes = packed_bytes(a->n, a->k);
  double nw = 0.0, nx = 0.0;
  if (a->dw) g.shape_w = wsattn::choose_gemm(a->n, a->k, static_cast<int>(a->m), true, &nw);
  if (a->dx) g.shape_x = wsattn::choose_gemm(a->m, a->k, a->n, false, &nx);
  g.together = a->dw && a->dx &&
               wsattn::pair_time_of_two(a->n, a->k, static_cast<int>(a->m), a->m, a->k, a->n) <
                   nw + nx;
  if (!g.together) {  // one after the other, through the same partial tiles
    const size_t bw = a->dw ? g.shape_w.bytes(a->n, a->k) : 0;
    const size_t bx = a->dx ? g.shape_x.bytes(a->m, a->k) : 0;
    g.tile_bytes = bw > bx ? bw : bx;
  }
  return g;
}

}  // namespace

extern "C" {

int wsattn_rotary_plan(int head_dim, int axes, const int32_t* pair_axis, const double* pair_freq,
                       int interleaved, wsattn_rotary_t* out) {
  if (!out) return WSATTN_ERR_BAD_ARG;
  *out = nullptr;
  if (!pair_axis || !pair_freq || axes < 1 || axes > wsattn::kRotMaxAxes || interleaved < 0 ||
      interleaved > 1)
    return WSATTN_ERR_BAD_ARG;
  if (head_dim < 16 || head_dim % 16 || head_dim > 2 * wsattn::kRotMaxPairs)
    return WSATTN_ERR_UNSUPPORTED;
  const int pairs = head_dim / 2;
  for (int i = 0; i < pairs; ++i)
    if (pair_axis[i] < 0 || pair_axis[i] >= axes || !std::isfinite(pair_freq[i]) ||
        std::fabs(pair_freq[i]) > 1e30)
      return WSATTN_ERR_BAD_ARG;
  wsattn_rotary_s* r = new (std::nothrow) wsattn_rotary_s();
  if (!r) return WSATTN_ERR_NO_MEMORY;
  std::memset(&r->table, 0, sizeof(r->table));
  const double two_pi = 6.283185307179586476925286766559;
  for (int i = 0; i < pairs; ++i) {
    const double turns = pair_freq[i] / two_pi;
    r->table.hi[i] = static_cast<float>(turns);
    r->table.lo[i] = static_cast<float>(turns - static_cast<double>(r->table.hi[i]));
    r->table.axis[i] = static_cast<uint8_t>(pair_axis[i]);
  }
  r->table.pairs = pairs;
  r->table.axes = axes;
  r->table.interleaved = interleaved;
  *out = r;
  return WSATTN_OK;
}

int wsattn_rotary_destroy(wsattn_rotary_t rot) {
  delete rot;
  return WSATTN_OK;
}

int wsattn_rotary(wsattn_rotary_t rot, int dtype, int batch, int64_t n_tokens,
                  const wsattn_heads* x, const float* positions, int64_t pos_stride_b, int inverse,
                  const wsattn_heads* y, void* stream) {
  if (!rot || !dtype_ok(dtype) || batch < 0 || !tokens_ok(n_tokens) || inverse < 0 || inverse > 1)
    return WSATTN_ERR_BAD_ARG;
  const int esize = dtype_size(dtype), dim = 2 * rot->table.pairs;
  if (!view_ok(x, esize) || !view_ok(y, esize) || x->heads != y->heads ||
      !positions_ok(positions, pos_stride_b) || !apart(y, batch, n_tokens, dim))
    return WSATTN_ERR_BAD_ARG;
  const int64_t rows = static_cast<int64_t>(batch) * n_tokens;
  if (rows == 0) return WSATTN_OK;
  if (!x->data || !y->data || !positions) return WSATTN_ERR_BAD_ARG;
  const int sms = sm_count();
  if (!sms) return WSATTN_ERR_CUDA;
  QkParams p;
  std::memset(&p, 0, sizeof(p));
  p.rot = rot->table;
  p.parts = 1;
  p.part[0] = part_of(x, y, 0, inverse ? -1 : 1, nullptr);
  p.pos = positions;
  p.pos_b = pos_stride_b;
  p.tokens = n_tokens;
  p.status = wsattn::op_status_ptr();
  if (!p.status) return WSATTN_ERR_CUDA;
  if (!split_work(&p, rows, 6LL * sms, false)) return WSATTN_ERR_BAD_ARG;
  const bool vec = view_vec(x, batch, n_tokens, esize) && view_vec(y, batch, n_tokens, esize);
  return wsattn::launch_qk_forward(p, dtype, vec, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? WSATTN_OK
             : WSATTN_ERR_CUDA;
}

int wsattn_qknorm(wsattn_rotary_t rot, int dtype, int batch, int64_t n_tokens,
                  const wsattn_heads* q, const wsattn_heads* k, const wsattn_heads* v,
                  const void* q_weight, const void* k_weight, int weight_dtype, float eps,
                  const float* positions, int64_t pos_stride_b, const wsattn_heads* q_out,
                  const wsattn_heads* k_out, const wsattn_heads* v_out, void* stream) {
  if (!rot || !dtype_ok(dtype) || batch < 0 || !tokens_ok(n_tokens) || !(eps >= 0.f) ||
      !std::isfinite(eps) || (weight_dtype != dtype && weight_dtype != WSATTN_FP32) || (!v) != (!v_out))
    return WSATTN_ERR_BAD_ARG;
  const int esize = dtype_size(dtype), dim = 2 * rot->table.pairs;
  const wsattn_heads* in[3] = {q, k, v};
  const wsattn_heads* out[3] = {q_out, k_out, v_out};
  const int parts = v ? 3 : 2;
  const int64_t rows = static_cast<int64_t>(batch) * n_tokens;
  bool vec = true;
  for (int i = 0; i < parts; ++i) {
    if (!view_ok(in[i], esize) || !view_ok(out[i], esize) || in[i]->heads != out[i]->heads ||
        !apart(out[i], batch, n_tokens, dim))
      return WSATTN_ERR_BAD_ARG;
    if (rows && (!in[i]->data || !out[i]->data)) return WSATTN_ERR_BAD_ARG;
    vec = vec && view_vec(in[i], batch, n_tokens, esize) && view_vec(out[i], batch, n_tokens, esize);
  }
  const int wsize = dtype_size(weight_dtype);
  if (!positions_ok(positions, pos_stride_b) || !elem_aligned(q_weight, wsize) ||
      !elem_aligned(k_weight, wsize))
    return WSATTN_ERR_BAD_ARG;
  if (rows == 0) return WSATTN_OK;
  if (!positions) return WSATTN_ERR_BAD_ARG;
  const int sms = sm_count();
  if (!sms) return WSATTN_ERR_CUDA;
  QkParams p;
  std::memset(&p, 0, sizeof(p));
  p.rot = rot->table;
  p.parts = parts;
  for (int i = 0; i < parts; ++i)
    p.part[i] = part_of(in[i], out[i], i < 2, i < 2, i == 0 ? q_weight : i == 1 ? k_weight : nullptr);
  p.weight_f32 = weight_dtype == WSATTN_FP32;
  p.eps = eps;
  p.pos = positions;
  p.pos_b = pos_stride_b;
  p.tokens = n_tokens;
  p.status = wsattn::op_status_ptr();
  if (!p.status) return WSATTN_ERR_CUDA;
  if (!split_work(&p, rows, 6LL * sms, false)) return WSATTN_ERR_BAD_ARG;
  return wsattn::launch_qk_forward(p, dtype, vec, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? WSATTN_OK
             : WSATTN_ERR_CUDA;
}

int wsattn_qknorm_backward_workspace(wsattn_rotary_t rot, size_t* bytes) {
  if (!rot || !bytes) return WSATTN_ERR_BAD_ARG;
  *bytes = sizeof(float) * 2 * kMaxBackCtas * 2 * static_cast<size_t>(rot->table.pairs);
  return WSATTN_OK;
}

int wsattn_qknorm_backward(wsattn_rotary_t rot, int dtype, int batch, int64_t n_tokens,
                           const wsattn_heads* dq_out, const wsattn_heads* dk_out,
                           const wsattn_heads* dv_out, const wsattn_heads* q,
                           const wsattn_heads* k, const void* q_weight, const void* k_weight,
                           int weight_dtype, float eps, const float* positions,
                           int64_t pos_stride_b, const wsattn_heads* dq, const wsattn_heads* dk,
                           const wsattn_heads* dv, float* dq_weight, float* dk_weight,
                           void* workspace, size_t workspace_bytes, void* stream) {
  if (!rot || !dtype_ok(dtype) || batch < 0 || !tokens_ok(n_tokens) || !(eps >= 0.f) ||
      !std::isfinite(eps) || (weight_dtype != dtype && weight_dtype != WSATTN_FP32) ||
      (!dv_out) != (!dv))
    return WSATTN_ERR_BAD_ARG;
  const int esize = dtype_size(dtype), dim = 2 * rot->table.pairs;
  const wsattn_heads* in[3] = {dq_out, dk_out, dv_out};
  const wsattn_heads* out[3] = {dq, dk, dv};
  const wsattn_heads* x[2] = {q, k};
  const int parts = dv ? 3 : 2;
  const int64_t rows = static_cast<int64_t>(batch) * n_tokens;
  bool vec = true;
  for (int i = 0; i < parts; ++i) {
    if (!view_ok(in[i], esize) || !view_ok(out[i], esize) || in[i]->heads != out[i]->heads ||
        !apart(out[i], batch, n_tokens, dim))
      return WSATTN_ERR_BAD_ARG;
    if (rows && (!in[i]->data || !out[i]->data)) return WSATTN_ERR_BAD_ARG;
    vec = vec && view_vec(in[i], batch, n_tokens, esize) && view_vec(out[i], batch, n_tokens, esize);
    if (i < 2) {
      if (!view_ok(x[i], esize) || x[i]->heads != in[i]->heads || (rows && !x[i]->data))
        return WSATTN_ERR_BAD_ARG;
      vec = vec && view_vec(x[i], batch, n_tokens, esize);
    }
  }
  const int wsize = dtype_size(weight_dtype);
  const bool gains = dq_weight || dk_weight;
  size_t need = 0;
  wsattn_qknorm_backward_workspace(rot, &need);
  if (!positions_ok(positions, pos_stride_b) || !elem_aligned(q_weight, wsize) ||
      !elem_aligned(k_weight, wsize) || !elem_aligned(dq_weight, 4) || !elem_aligned(dk_weight, 4) ||
      (gains && rows && (!workspace || !aligned16(workspace) || workspace_bytes < need)))
    return WSATTN_ERR_BAD_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (rows == 0) {
    if ((dq_weight && cudaMemsetAsync(dq_weight, 0, sizeof(float) * dim, s) != cudaSuccess) ||
        (dk_weight && cudaMemsetAsync(dk_weight, 0, sizeof(float) * dim, s) != cudaSuccess))
      return WSATTN_ERR_CUDA;
    return WSATTN_OK;
  }
  if (!positions) return WSATTN_ERR_BAD_ARG;
  const int sms = sm_count();
  if (!sms) return WSATTN_ERR_CUDA;
  QkParams p;
  std::memset(&p, 0, sizeof(p));
  p.rot = rot->table;
  p.parts = parts;
  for (int i = 0; i < parts; ++i) {
    p.part[i] = part_of(in[i], out[i], i < 2, i < 2 ? -1 : 0,
                        i == 0 ? q_weight : i == 1 ? k_weight : nullptr);
    if (i < 2) {
      p.part[i].x = x[i]->data;
      p.part[i].xb = x[i]->stride_b;
      p.part[i].xn = x[i]->stride_n;
      p.part[i].xh = x[i]->stride_h;
    }
  }
  p.weight_f32 = weight_dtype == WSATTN_FP32;
  p.eps = eps;
  p.pos = positions;
  p.pos_b = pos_stride_b;
  p.tokens = n_tokens;
  p.status = wsattn::op_status_ptr();
  if (!p.status) return WSATTN_ERR_CUDA;
  p.dw_part = gains ? static_cast<float*>(workspace) : nullptr;
  int64_t blocks = static_cast<int64_t>(sms) * wsattn::kQkBackCtasPerSm;
  if (blocks > kMaxBackCtas) blocks = kMaxBackCtas;
  if (!split_work(&p, rows, blocks, true)) return WSATTN_ERR_BAD_ARG;
  // no CTA without work of its own
  const int64_t items =
      p.row_blocks * static_cast<int64_t>(p.part[0].groups + p.part[1].groups);
  if (blocks > items) blocks = items;
  return wsattn::launch_qk_backward(p, dtype, vec, static_cast<int>(blocks), dq_weight, dk_weight,
                                    s) == cudaSuccess
             ? WSATTN_OK
             : WSATTN_ERR_CUDA;
}

int wsattn_linear_workspace(const wsattn_linear_args* args, size_t* bytes) {
  if (!bytes || !linear_args_ok(args)) return WSATTN_ERR_BAD_ARG;
  *bytes = args->m ? linear_ws(args, linear_shape(args)) : 0;
  return WSATTN_OK;
}

int wsattn_linear(const wsattn_linear_args* a, void* workspace, size_t workspace_bytes,
                  void* stream) {
  if (!linear_args_ok(a)) return WSATTN_ERR_BAD_ARG;
  if (!half_type(a->dtype) || (a->out_dtype != a->dtype && a->out_dtype != WSATTN_FP32))
    return WSATTN_ERR_UNSUPPORTED;
  if (a->m == 0) return WSATTN_OK;
  const int osize = dtype_size(a->out_dtype);
  if (!a->x || !a->w || !a->out || !elem_aligned(a->w, 2) || !elem_aligned(a->bias, 2) ||
      !elem_aligned(a->preact, 2) || !elem_aligned(a->residual, osize) ||
      !elem_aligned(a->out, osize) || (a->x_heads > 0 ? !aligned16(a->x) : !elem_aligned(a->x, 2)))
    return WSATTN_ERR_BAD_ARG;
  const wsattn::GemmShape shape = linear_shape(a);
  const size_t need = linear_ws(a, shape);
  if (need && (!workspace || !aligned16(workspace) || workspace_bytes < need))
    return WSATTN_ERR_BAD_ARG;
  const int sms = sm_count();
  if (!sms) return WSATTN_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  Product g;
  std::memset(&g, 0, sizeof(g));
  g.dtype = a->dtype;
  g.out_f32 = a->out_dtype == WSATTN_FP32;
  g.p = Operand{a->x, a->ldx};
  g.q = Operand{a->w, a->ldw};
  wsattn::PackJob jx = pack_job(nullptr, 0, 0, 8, nullptr), jw = jx;
  if (a->x_heads > 0 || !tma_rows(a->x, a->ldx, a->m)) {
    jx = pack_job(a->x, a->ldx, a->m, a->k, ws);
    jx.f32_heads = a->x_heads;
    jx.tokens = a->x_tokens;
    g.p = Operand{ws, jx.ldd};
    ws += packed_bytes(a->m, a->k);
  }
  if (!tma_rows(a->w, a->ldw, a->n)) {
    jw = pack_job(a->w, a->ldw, a->n, a->k, ws);
    g.q = Operand{ws, jw.ldd};
    ws += packed_bytes(a->n, a->k);
  }
  if (wsattn::launch_pack(a->dtype, jx, jw, s) != cudaSuccess) return WSATTN_ERR_CUDA;
  g.R = a->m;
  g.C = a->n;
  g.K = a->k;
  g.bias = a->bias;
  g.res = a->residual;
  g.ldr = a->ldr;
  g.out = a->out;
  g.ldo = a->ldo;
  g.pre = a->preact;
  g.ldp = a->ldp;
  g.act = a->activation;
  return run_product(g, shape, sms, ws, s);
}

int wsattn_linear_backward_workspace(const wsattn_linear_grad_args* args, size_t* bytes) {
  if (!bytes || !grad_args_ok(args)) return WSATTN_ERR_BAD_ARG;
  *bytes = plan_grad(args).total();
  return WSATTN_OK;
}

int wsattn_linear_backward(const wsattn_linear_grad_args* a, void* workspace,
                           size_t workspace_bytes, void* stream) {
  if (!grad_args_ok(a)) return WSATTN_ERR_BAD_ARG;
  if (!half_type(a->dtype)) return WSATTN_ERR_UNSUPPORTED;
  if (!elem_aligned(a->dout, 2) || !elem_aligned(a->x, 2) || !elem_aligned(a->w, 2) ||
      !elem_aligned(a->preact, 2) || !elem_aligned(a->dx, 2) || !elem_aligned(a->dw, 2) ||
      !elem_aligned(a->db, 4))
    return WSATTN_ERR_BAD_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (a->m == 0) {
    if ((a->dw && cudaMemset2DAsync(a->dw, 2 * a->lddw, 0, 2 * static_cast<size_t>(a->k), a->n,
                                    s) != cudaSuccess) ||
        (a->db && cudaMemsetAsync(a->db, 0, sizeof(float) * a->n, s) != cudaSuccess))
      return WSATTN_ERR_CUDA;
    return WSATTN_OK;
  }
  if (!a->dout || (a->dw && !a->x) || (a->dx && !a->w) ||
      (a->activation != WSATTN_ACT_NONE && !a->preact))
    return WSATTN_ERR_BAD_ARG;
  const GradPlan plan = plan_grad(a);
  if (plan.total() && (!workspace || !aligned16(workspace) || workspace_bytes < plan.total()))
    return WSATTN_ERR_BAD_ARG;
  const int sms = sm_count();
  if (!sms) return WSATTN_ERR_CUDA;
  char* ws = static_cast<char*>(workspace);
  char* ws_dz = ws;
  char* ws_part = ws_dz + plan.dz_bytes;
  char* ws_x = ws_part + plan.part_bytes;
  char* ws_w = ws_x + plan.x_bytes;
  char* ws_tiles = ws_w + plan.w_bytes;
  Operand dz{a->dout, a->ldd}, x{a->x, a->ldx}, w{a->w, a->ldw};
  wsattn::DactParams d;
  std::memset(&d, 0, sizeof(d));
  if (plan.dz || a->db) {
    d.dout = a->dout;
    d.ldd = a->ldd;
    d.pre = plan.act ? a->preact : nullptr;
    d.ldp = a->ldp;
    d.dz = plan.dz ? ws_dz : nullptr;
    d.ldz = round8(a->n);
    d.part = a->db ? reinterpret_cast<float*>(ws_part) : nullptr;
    d.ldpart = a->n;
    d.rows = a->m;
    d.cols = a->n;
    d.act = a->activation;
    d.rows_per_block = plan.rows_per_block;
    d.row_blocks = plan.row_blocks;
    d.vec = rows_vec(a->dout, a->ldd, a->m, a->n, 2) &&
            (!d.pre || rows_vec(a->preact, a->ldp, a->m, a->n, 2));
    if (wsattn::launch_dact(d, a->dtype, s) != cudaSuccess) return WSATTN_ERR_CUDA;
    if (a->db && !a->dx && !a->dw)
      return wsattn::launch_sum_parts(d, a->db, s) == cudaSuccess ? WSATTN_OK : WSATTN_ERR_CUDA;
    if (plan.dz) dz = Operand{ws_dz, d.ldz};
  }
  wsattn::PackJob jx = pack_job(nullptr, 0, 0, 8, nullptr), jw = jx;
  if (plan.pack_x) {
    jx = pack_job(a->x, a->ldx, a->m, a->k, ws_x);
    x = Operand{ws_x, jx.ldd};
  }
  if (plan.pack_w) {
    jw = pack_job(a->w, a->ldw, a->n, a->k, ws_w);
    w = Operand{ws_w, jw.ldd};
  }
  if (wsattn::launch_pack(a->dtype, jx, jw, s) != cudaSuccess) return WSATTN_ERR_CUDA;
  Product gw, gx;
  std::memset(&gw, 0, sizeof(gw));
  gw.dtype = a->dtype;
  gx = gw;
  // dw[n, k] = sum over rows of dz[., n] x[., k]
  gw.p = dz;
  gw.p_mn = true;
  gw.q = x;
  gw.q_mn = true;
  gw.R = a->n;
  gw.C = a->k;
  gw.K = static_cast<int>(a->m);
  gw.out = a->dw;
  gw.ldo = a->lddw;
  // dx[m, k] = sum over features of dz[m, .] w[., k]
  gx.p = dz;
  gx.q = w;
  gx.q_mn = true;
  gx.R = a->m;
  gx.C = a->k;
  gx.K = a->n;
  gx.out = a->dx;
  gx.ldo = a->lddx;
  Product& side = a->dw ? gw : gx;  // the first product launched
  side.part = d.part;
  side.parts = d.row_blocks;
  side.db = a->db;
  side.db_cols = a->n;
  if (plan.together) return run_together(gw, gx, sms, s);
  int rc = WSATTN_OK;
  if (a->dw) rc = run_product(gw, plan.shape_w, sms, ws_tiles, s);
  if (a->dx && rc == WSATTN_OK) rc = run_product(gx, plan.shape_x, sms, ws_tiles, s);
  return rc;
}

int wsattn_op_status(void* stream) {
  int* w = wsattn::op_status_ptr();
  if (!w) return WSATTN_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int st = 0;
  if (cudaMemcpyAsync(&st, w, sizeof(int), cudaMemcpyDeviceToHost, s) != cudaSuccess ||
      cudaStreamSynchronize(s) != cudaSuccess)
    return WSATTN_ERR_CUDA;
  if (st == 0) return WSATTN_OK;
  // the bits reported here and no others: one that another stream's kernel sets
  // meanwhile is left for the next query
  if (wsattn::launch_clear_status(w, st, s) != cudaSuccess ||
      cudaStreamSynchronize(s) != cudaSuccess)
    return WSATTN_ERR_CUDA;
  return (st & wsattn::kStatusBounds) ? WSATTN_ERR_BOUNDS : WSATTN_ERR_TIMEOUT;
}

}  // extern "C"
