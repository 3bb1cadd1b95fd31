// Internal declarations of the operators around the attention: rotary
// positions, query/key norms and linear products.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.h"

namespace wsattn {

// ------------------------------------------------ rotary positions, norms
constexpr int kRotMaxPairs = 128;  // head_dim <= 256
constexpr int kRotMaxAxes = 4;

// Per-pair turning rates, passed to the kernels by value.  A pair turns by
// pos[axis] * (hi + lo) revolutions: freq / 2 pi split into two floats, so
// that the product keeps 48 bits and far positions lose nothing.
struct alignas(16) RotTable {
  float hi[kRotMaxPairs];
  float lo[kRotMaxPairs];
  uint8_t axis[kRotMaxPairs];
  int pairs;        // head_dim / 2
  int axes;         // columns of the positions
  int interleaved;  // pairs (2p, 2p + 1), else (p, p + head_dim / 2)
};

struct HeadsPtr {
  const void* in;
  void* out;
  int64_t ib, in_, ih;  // input strides in elements: batch, token, head
  int64_t ob, on, oh;   // output strides
  int heads;
};

// One of the three parts (q, k, v) of a pass over a projection's heads.
struct QkPart {
  HeadsPtr io;           // forward: x -> y; backward: dy -> dx
  const void* x;         // backward: the forward's input (norm only)
  int64_t xb, xn, xh;
  const void* weight;    // gain [D], or null
  int norm;              // RMS norm over the head
  int turn;              // 1 turns, -1 turns back, 0 leaves the angles alone
  int group0;            // first head group of this part
  int groups;
  int group_heads;       // heads a warp walks for one token
};

struct QkParams {
  RotTable rot;
  QkPart part[3];
  int parts;
  int weight_f32;        // gains are fp32, else of the tensors' type
  float eps;
  const float* pos;      // [N, axes] or [B, N, axes]
  int64_t pos_b;         // batch stride of pos (0: shared)
  int64_t tokens;        // N
  int64_t rows;          // B * N
  int64_t row_blocks;    // ceil(rows / rows per CTA)
  int lanes_log2;        // lanes of one head row: 2^lanes_log2 >= D / 16
  int groups;            // head groups of all parts together
  float* dw_part;        // backward: [2][blocks][D] partial gain gradients, or null
  int* status;           // device status word (debug build: bounds checks)
};

// dtype: WSATTN_BF16, WSATTN_FP16 or WSATTN_FP32.  vec: every row starts on a
// 16-byte boundary.
cudaError_t launch_qk_forward(const QkParams& p, int dtype, bool vec, cudaStream_t s);
cudaError_t launch_qk_backward(const QkParams& p, int dtype, bool vec, int blocks, float* dwq,
                               float* dwk, cudaStream_t s);
constexpr int kQkThreads = 256;
// CTAs of the backward pass per SM (its register budget).
constexpr int kQkBackCtasPerSm = 2;

// -------------------------------------------------------- linear products
// out[R, C] = residual + act(P Q^T + bias): P holds the rows, Q the columns,
// both with the contraction of length K along one of their two dimensions.
constexpr int kGemmK = 64;        // contraction per pipeline stage
constexpr int kPairRows = 256;    // rows of a CTA pair's tile
constexpr int kTileCols = 128;    // columns of a single CTA's tile

struct GemmParams {
  CUtensorMap tm_p;    // P: box {64, rows} over [R, K], or {64, 64} over [K, R] (p_mn)
  CUtensorMap tm_q;    // Q likewise
  CUtensorMap tm_out;  // out [R, C], box {128 bytes, 32 rows}, 128-byte swizzle
  CUtensorMap tm_pre;  // preact, the same
  int64_t R;
  int C, K;
  int p_mn, q_mn;      // the operand's own dimension is the contiguous one
  const void* bias;    // [C] or null
  const void* res;     // [R, C], row stride ldr, or null
  int64_t ldr;
  void* out;
  int64_t ldo;
  void* pre;           // P Q^T + bias, or null
  int64_t ldp;
  int act;
  int bias_vec, res_vec, out_vec, pre_vec;  // 16-byte accesses hold
  int tiles_r, tiles_c;
  int split;           // parts of the contraction: the CTAs of a cluster (single-CTA
                       // tiles), or of the pair kernel's last tiles
  // CTA pairs
  int whole_tiles;     // tiles before those that are split
  float* partial;      // [(tiles - whole_tiles) * split][256][256]
  // TMA writes units of 16 bytes, and the one that the last column ends in
  // whole, zeros behind it: columns that it stores (up to the last whole staging
  // chunk then), and the column tile that holds the rest (-1: none)
  int out_tma, pre_tma, edge_tile;
  // single-CTA tiles
  int bn;              // rows of a tile (the MMA's N)
  int stages;
  int* status;         // device status word (bit set on an expired wait)
  // the bias gradient: column sums of the slope pass's partial rows, added by
  // warps that have nothing else to do meanwhile (db null: none)
  const float* part;   // [parts, ldpart]
  int64_t ldpart;
  int parts, db_cols;
  float* db;
};

// One launch of the CTA-pair kernel: one product, or two with the same types
// (a and b) whose tiles it deals out together (tiles_b = 0: only a).
struct PairParams {
  GemmParams g[2];
  int tiles_a, tiles_b;
  // a's tiles go round the pairs first; the pairs that get one less take
  // `head_rounds` rounds of b's tiles meanwhile, then all of them the rest
  int head_rounds;
};

// How a product is tiled.
struct GemmShape {
  int pair_cols;  // columns of a CTA pair's tile (256 or 128), 0: single-CTA tiles
  int bn;         // single-CTA tiles: rows per tile
  int split;      // CTAs per tile; pairs: parts of each tile behind `whole`
  int whole;      // pairs: tiles that are not split
  // Scratch for the partial tiles.
  size_t bytes(int64_t R, int C) const {
    if (!pair_cols || split < 2) return 0;
    const int64_t tiles = ((R + kPairRows - 1) / kPairRows) * ((C + pair_cols - 1) / pair_cols);
    return static_cast<size_t>(tiles - whole) * split * kPairRows * pair_cols * sizeof(float);
  }
};
// Tilings are chosen for 152 SMs whatever the device has (they stay right on
// any), so that a workspace's size needs no device.
constexpr int kTilingSms = 152;
GemmShape choose_gemm(int64_t R, int C, int K, bool p_mn, double* ns);
// Estimated nanoseconds of two products in one launch of the pair kernel.
double pair_time_of_two(int64_t Ra, int Ca, int Ka, int64_t Rb, int Cb, int Kb);

size_t pair_smem_bytes(int pair_cols);
size_t tile_smem_bytes(int bn, int stages);
// 16-bit operands of type `dtype`; out and residual of that type or fp32.
// tiles_a, tiles_b and head_rounds are set here.
cudaError_t launch_gemm_pair(PairParams* p, int dtype, bool out_f32, int pair_cols, int sms,
                             cudaStream_t s);
cudaError_t launch_gemm_tile(const GemmParams& p, int dtype, bool out_f32, cudaStream_t s);

// Device status word of the operators that have no plan (one per device, in
// the library's image; its address is looked up once per device).
int* op_status_ptr();
// Clears the bits `seen` of a status word.
cudaError_t launch_clear_status(int* word, int seen, cudaStream_t s);

// Copies [rows, cols] matrices with any row stride and alignment to rows of
// `ldd` elements (a multiple of 8), up to two in one launch; f32_heads > 0
// (the first one only): src is fp32 [rows / tokens, heads, tokens,
// cols / heads] and is rounded to dtype.
struct PackJob {
  const void* src;
  int64_t lds;
  int64_t rows;  // 0: nothing to copy
  int cols;
  void* dst;
  int64_t ldd;
  int f32_heads;
  int64_t tokens;
};
cudaError_t launch_pack(int dtype, const PackJob& a, const PackJob& b, cudaStream_t s);

// dz = dout * act'(preact) (dz null: not stored) and, in parts, its column
// sums: part [row_blocks, ldpart].
struct DactParams {
  const void* dout;
  int64_t ldd;
  const void* pre;  // null: act'(.) = 1
  int64_t ldp;
  void* dz;
  int64_t ldz;
  float* part;      // null: no sums
  int64_t ldpart;
  int64_t rows;
  int cols;
  int act;
  int rows_per_block;
  int row_blocks;
  int vec;          // dout and preact rows start on 16-byte boundaries
};
cudaError_t launch_dact(const DactParams& p, int dtype, cudaStream_t s);
// db = sums of part's rows (where no product does it on the side).
cudaError_t launch_sum_parts(const DactParams& p, float* db, cudaStream_t s);
constexpr int kDactCols = 256;

}  // namespace wsattn
