// Passes over memory beside the linear products, and how a product is tiled.
//
//   pack   rows of any stride and alignment, or the attention's fp32
//          [B, H, N, D], to 16-bit rows that TMA can read
//   dact   dz = dout * act'(preact) with its column sums (the bias gradient)
//
// Both round an operand of a product to 16 bits, because the tensor cores' full
// rate is for 16-bit operands: a second 16-bit term for what the rounding drops
// would double a product that is the operator's whole time.  The attention's
// output was itself made from 16-bit probabilities and values; dz costs dx and
// dw a second rounding (2.3e-3 relative in bf16 against 1.7e-3 of one, an eighth
// of that in fp16).  The bias gradient sums the unrounded dz.
#include "epilogue.cuh"
#include "ptx.cuh"

namespace wsattn {
namespace {

using namespace ptx;

// 8 values a thread, read element by element: the sources of this pass are
// those whose rows start on no common boundary.
__device__ __forceinline__ void pack_rows(const PackJob& j, int64_t i) {
  const int64_t per = j.ldd / 8, r = i / per;
  if (r >= j.rows) return;
  const int c = static_cast<int>(i - r * per) * 8;
  const uint16_t* q = static_cast<const uint16_t*>(j.src) + r * j.lds + c;
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e)
    w[e] = (c + 2 * e < j.cols ? q[2 * e] : 0u) | (c + 2 * e + 1 < j.cols ? q[2 * e + 1] : 0u) << 16;
  *reinterpret_cast<uint4*>(static_cast<uint16_t*>(j.dst) + r * j.ldd + c) =
      make_uint4(w[0], w[1], w[2], w[3]);
}

// fp32 [B, H, N, D] -> rows (b, n) of H * D, rounded once.  A thread takes 8
// values of one head row (D is a multiple of 8): 16 bytes out, 32 in.
template <typename T>
__device__ __forceinline__ void pack_heads(const PackJob& j, int64_t i) {
  const int per = j.cols / 8, dim = j.cols / j.f32_heads;
  const int64_t r = i / per;
  if (r >= j.rows) return;
  const int64_t b = r / j.tokens, n = r - b * j.tokens;
  const int c = static_cast<int>(i - r * per) * 8, h = c / dim, d = c - h * dim;
  const float4* q = reinterpret_cast<const float4*>(
      static_cast<const float*>(j.src) + ((b * j.f32_heads + h) * j.tokens + n) * dim + d);
  const float4 x = q[0], y = q[1];
  *reinterpret_cast<uint4*>(static_cast<T*>(j.dst) + r * j.ldd + c) =
      make_uint4(pack_pair(x.x, x.y, T()), pack_pair(x.z, x.w, T()), pack_pair(y.x, y.y, T()),
                 pack_pair(y.z, y.w, T()));
}

template <typename T>
__global__ void __launch_bounds__(256) pack_kernel(const PackJob a, const PackJob b,
                                                   int64_t blocks_a) {
  griddep_wait();
  griddep_launch_dependents();
  const bool first = blockIdx.x < blocks_a;
  const int64_t i = (blockIdx.x - (first ? 0 : blocks_a)) * 256 + threadIdx.x;
  if (!first) pack_rows(b, i);
  else if (a.f32_heads > 0) pack_heads<T>(a, i);
  else pack_rows(a, i);
}

template <bool VEC>
__device__ __forceinline__ uint4 load_raw8(const void* base, int64_t ld, int64_t r, int c, int cols) {
  const uint16_t* q = static_cast<const uint16_t*>(base) + r * ld + c;
  if constexpr (VEC) {
    return *reinterpret_cast<const uint4*>(q);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      w[e] = (c + 2 * e < cols ? q[2 * e] : 0u) | (c + 2 * e + 1 < cols ? q[2 * e + 1] : 0u) << 16;
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// CTA (x, y): 256 columns of rows [y * rows_per_block, ...); a warp takes
// every eighth row, a lane 8 columns of it, two rows' loads in flight.
// Bound by HBM (dout and preact in, dz out).  The sums stay in fp32
// registers (of the unrounded dz), then go through shared memory in the
// order of the warps.
template <typename T, bool VEC, int ACT>
__global__ void __launch_bounds__(256, 4) dact_kernel(DactParams p) {
  constexpr int U = 2;
  __shared__ float red[8][kDactCols];
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  const int c = static_cast<int>(blockIdx.x) * kDactCols + 8 * lane;
  const int64_t r0 = static_cast<int64_t>(blockIdx.y) * p.rows_per_block;
  const int64_t r1 = min(p.rows, r0 + p.rows_per_block);
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  griddep_wait();
  griddep_launch_dependents();
  if (c < p.cols) {
    for (int64_t r = r0 + warp; r < r1; r += 8 * U) {
      uint4 gw[U], zw[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const bool on = r + 8 * u < r1;
        gw[u] = on ? load_raw8<VEC>(p.dout, p.ldd, r + 8 * u, c, p.cols) : make_uint4(0, 0, 0, 0);
        if (ACT != WSATTN_ACT_NONE)
          zw[u] = on ? load_raw8<VEC>(p.pre, p.ldp, r + 8 * u, c, p.cols) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint32_t g[4] = {gw[u].x, gw[u].y, gw[u].z, gw[u].w};
        const uint32_t z[4] = {zw[u].x, zw[u].y, zw[u].z, zw[u].w};
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float2 d = unpack_pair(g[i], T());
          if (ACT != WSATTN_ACT_NONE) {
            // rounded here, so that the sums are the same with and without dz
            const float2 y = unpack_pair(clamp_pair(z[i], T()), T());
            d.x = __fmul_rn(d.x, act_slope<ACT>(y.x));
            d.y = __fmul_rn(d.y, act_slope<ACT>(y.y));
          }
          acc[2 * i] += d.x;
          acc[2 * i + 1] += d.y;
          o[i] = pack_pair(d.x, d.y, T());
        }
        if (p.dz && r + 8 * u < r1)
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.dz) + (r + 8 * u) * p.ldz + c) =
              make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
  }
  if (!p.part) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) red[warp][8 * lane + i] = acc[i];
  __syncthreads();
  float t = 0.f;
#pragma unroll
  for (int w = 0; w < 8; ++w) t += red[w][threadIdx.x];
  const int cc = static_cast<int>(blockIdx.x) * kDactCols + static_cast<int>(threadIdx.x);
  if (cc < p.cols) p.part[static_cast<int64_t>(blockIdx.y) * p.ldpart + cc] = t;
}

__global__ void __launch_bounds__(128) sum_parts(const float* __restrict__ part, int64_t ldpart,
                                                 int parts, int cols, float* __restrict__ out) {
  griddep_wait();
  griddep_launch_dependents();
  const int c = 128 * static_cast<int>(blockIdx.x) + static_cast<int>(threadIdx.x);
  if (c < cols) out[c] = sum_column(part, ldpart, parts, c);
}

template <typename T, bool VEC>
cudaError_t dact_t(const DactParams& p, cudaStream_t s) {
  const dim3 grid((p.cols + kDactCols - 1) / kDactCols, p.row_blocks);
  const int act = p.pre ? p.act : WSATTN_ACT_NONE;
  auto run = [&](void (*kernel)(DactParams)) {
    return launch_dependent(kernel, grid, dim3(256), 0, s, p);
  };
  if (act == WSATTN_ACT_GELU) return run(dact_kernel<T, VEC, WSATTN_ACT_GELU>);
  if (act == WSATTN_ACT_GELU_TANH) return run(dact_kernel<T, VEC, WSATTN_ACT_GELU_TANH>);
  if (act == WSATTN_ACT_SILU) return run(dact_kernel<T, VEC, WSATTN_ACT_SILU>);
  return run(dact_kernel<T, VEC, WSATTN_ACT_NONE>);
}

__device__ int g_op_status;

__global__ void clear_status(int* word, int seen) { atomicAnd(word, ~seen); }

}  // namespace

int* op_status_ptr() {
  static int* ptr[kMaxDevices] = {};
  const int dev = current_device();
  if (dev < 0) return nullptr;
  if (!ptr[dev]) {
    void* a = nullptr;
    if (cudaGetSymbolAddress(&a, g_op_status) != cudaSuccess) return nullptr;
    ptr[dev] = static_cast<int*>(a);
  }
  return ptr[dev];
}

cudaError_t launch_clear_status(int* word, int seen, cudaStream_t s) {
  clear_status<<<1, 1, 0, s>>>(word, seen);
  return cudaGetLastError();
}

cudaError_t launch_pack(int dtype, const PackJob& a, const PackJob& b, cudaStream_t s) {
  auto blocks = [](const PackJob& j) { return (j.rows * (j.ldd / 8) + 255) / 256; };
  const int64_t na = blocks(a), nb = blocks(b);
  if (na + nb == 0) return cudaSuccess;
  if (na + nb > INT32_MAX) return cudaErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(na + nb));
  return dtype == WSATTN_BF16
             ? launch_dependent(pack_kernel<__nv_bfloat16>, grid, dim3(256), 0, s, a, b, na)
             : launch_dependent(pack_kernel<__half>, grid, dim3(256), 0, s, a, b, na);
}

cudaError_t launch_dact(const DactParams& p, int dtype, cudaStream_t s) {
  if (dtype == WSATTN_BF16)
    return p.vec ? dact_t<__nv_bfloat16, true>(p, s) : dact_t<__nv_bfloat16, false>(p, s);
  return p.vec ? dact_t<__half, true>(p, s) : dact_t<__half, false>(p, s);
}

cudaError_t launch_sum_parts(const DactParams& p, float* db, cudaStream_t s) {
  return launch_dependent(sum_parts, dim3((p.cols + 127) / 128), dim3(128), 0, s,
                          static_cast<const float*>(p.part), p.ldpart, p.row_blocks, p.cols, db);
}

// Estimated time of each tiling in nanoseconds; the least one wins.  The
// constants are fitted to the timings of every tiling at 60 to 90 shapes (1 to
// 20000 rows, 64 to 5120 columns and values, all three orders of the
// operands, back to back with operands from HBM): the tiling taken is then
// within 2.5 % of the best one on average, 1.25 at worst.
//   pair   a 64-wide step of a 256-column tile takes 290 ns (the MMAs alone
//          270 at full clocks), of a 128-column tile 269, for half the MMAs: its
//          24 KB a CTA come at 89 KB a microsecond, less than the 110 of the
//          256-column tile's 32 KB, so L2's rate is not what it waits for (six
//          slices in flight at their latency may be; not measured apart); a tile
//          1.2 or 0.65 us beside its steps, and the first loads and the last
//          epilogue are seen once
//   tile   a step of a CTA takes the time of its bytes at 134 KB a
//          microsecond and SM, shared by two CTAs, or 200 ns; a row of the
//          tile 45 ns of epilogue, and the cluster's exchange 800 ns
constexpr double kPairStart256 = 4000.0, kPairTile256 = 1200.0, kPairStep256 = 290.0,
                 kPairStart128 = 3500.0, kPairTile128 = 650.0, kPairStep128 = 269.0;

GemmShape choose_gemm(int64_t R, int C, int K, bool p_mn, double* ns) {
  constexpr int sms = kTilingSms;
  const int64_t ksteps = (K + kGemmK - 1) / kGemmK;
  GemmShape best{256, 0, 1, 0};
  double best_t = 1e300;
  auto cdiv = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
  auto consider = [&](double t, const GemmShape& s) {
    if (t < best_t) {
      best_t = t;
      best = s;
    }
  };
  const double steps = static_cast<double>(ksteps);
  for (int bn = 256; bn >= 128; bn -= 128) {
    const double waves = static_cast<double>(cdiv(cdiv(R, kPairRows) * cdiv(C, bn), sms / 2));
    consider(bn == 256 ? kPairStart256 + waves * (steps * kPairStep256 + kPairTile256)
                       : kPairStart128 + waves * (steps * kPairStep128 + kPairTile128),
             GemmShape{bn, 0, 1, 0});
  }
  // pairs whose last round is split: parts of at least 8 steps, one a pair.
  // The partial tiles and the second kernel cost 4 us and 100 ns a part
  // (dw of 5120 x 5120 over 21952 rows, 400 tiles: 690 us whole, 634 with the
  // last 20 in 3 parts each; 1024 x 5120: 223 and 140), so not below 2^33
  // multiply-adds, where that is what it could save
  const int64_t tiles = cdiv(R, kPairRows) * cdiv(C, 256), pairs = sms / 2;
  const int64_t rest = tiles % pairs;
  if (rest > 0 && static_cast<double>(R) * C * K >= 8589934592.0) {
    int64_t parts = pairs / rest;
    if (parts > ksteps / 8) parts = ksteps / 8;
    if (parts > 16) parts = 16;
    if (parts >= 2 && tiles <= INT32_MAX)
      consider(kPairStart256 + static_cast<double>(tiles / pairs) * (steps * kPairStep256 + kPairTile256) +
                   static_cast<double>(cdiv(ksteps, parts)) * kPairStep256 + 4000.0 +
                   100.0 * static_cast<double>(rest * parts),
               GemmShape{256, 0, static_cast<int>(parts), static_cast<int>(tiles - rest)});
  }
  // SMs that clusters of `split` CTAs reach (the occupancy query's answer for
  // one CTA an SM): they stay within a GPC, whose SMs need not divide evenly
  static const struct { int split, of_152; } kSplits[] = {
      {1, 152}, {2, 152}, {3, 138}, {4, 144}, {8, 120}};
  for (int bn = 16; bn <= 128; bn *= 2) {
    if (p_mn && bn < 64) continue;
    if (bn > 16 && bn / 2 >= R && !(p_mn && bn == 64)) continue;
    const double rows = static_cast<double>(R < bn ? R : bn);
    for (const auto& sp : kSplits) {
      if (sp.split > ksteps) break;
      const int64_t ctas = cdiv(R, bn) * cdiv(C, kTileCols) * sp.split;
      const int64_t reach = static_cast<int64_t>(sms) * sp.of_152 / 152;
      const double waves = static_cast<double>(cdiv(ctas, 2 * reach));
      const double per_sm = ctas > reach ? 2.0 : 1.0;
      const double bytes = per_sm * (16.0 + bn / 8.0) * 7.45, least = 203.0 + 1.6 * bn;
      const double t = (sp.split > 1 ? 800.0 : 0.0) +
                       waves * (static_cast<double>(cdiv(ksteps, sp.split)) *
                                    (bytes > least ? bytes : least) +
                                3170.0 + 13.7 * rows * per_sm / sp.split + 44.7 * rows);
      consider(t, GemmShape{0, bn, sp.split, 0});
    }
  }
  *ns = best_t;
  return best;
}

double pair_time_of_two(int64_t Ra, int Ca, int Ka, int64_t Rb, int Cb, int Kb) {
  constexpr int64_t pairs = kTilingSms / 2;
  auto cdiv = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
  if (Ka < Kb) return pair_time_of_two(Rb, Cb, Kb, Ra, Ca, Ka);
  // the steps of a mixed launch take 8 % longer than one product's own (its
  // pairs walk through L2 at different places)
  auto tile_ns = [&](int K) {
    return static_cast<double>(cdiv(K, kGemmK)) * 1.08 * kPairStep256 + kPairTile256;
  };
  const int64_t na = cdiv(Ra, kPairRows) * cdiv(Ca, 256), nb = cdiv(Rb, kPairRows) * cdiv(Cb, 256);
  const double la = tile_ns(Ka), lb = tile_ns(Kb);
  // the pairs' loads as the kernel deals the tiles out
  const int64_t full = na / pairs, rest = na % pairs;
  double t;
  if (rest == 0) {
    t = static_cast<double>(full) * la + static_cast<double>(cdiv(nb, pairs)) * lb;
  } else {
    const int64_t others = pairs - rest, head = cdiv(cdiv(Ka, kGemmK), cdiv(Kb, kGemmK));
    const int64_t left = nb > head * others ? nb - head * others : 0;
    const int64_t rounds = left / pairs, extra = left % pairs;
    const int64_t first = left > 0 ? head : cdiv(nb, others);
    const double t1 = static_cast<double>(full + 1) * la +
                      static_cast<double>(rounds + (extra > 0)) * lb;
    const double t2 = static_cast<double>(full) * la +
                      static_cast<double>(first + rounds + (extra > rest)) * lb;
    t = t1 > t2 ? t1 : t2;
  }
  return kPairStart256 + t;
}

}  // namespace wsattn
