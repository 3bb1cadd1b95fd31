// Forward pass of a block's norms (norm.cuh has the formulas).
//
// Bound by HBM: x and the residual are read once, hidden and out written once.
// The vectors come from the L1 cache (many rows share them).  Rows of up to 1024 columns
// take a warp each, four to a CTA; wider ones a CTA of up to 12 warps.
//
// 43904 x 5120 bf16, gate, residual, scale and shift: 302 us, 5.95 TB/s (a copy of as
// many bytes takes 262); without the vectors 257.  What counts is how many rows are on
// their way: with five CTAs an SM of 64 registers a thread (some values spilled) it is
// 302, with 80 registers and fewer CTAs 357, with 56 registers 357 too, with the vectors
// held in registers ahead of the reductions (100 registers) 410.
#include "norm.cuh"

namespace wsattn {
namespace {

using namespace norm;

constexpr int kRowsPerCta = 4;  // rows of one warp

template <typename T, typename R, int V, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB) norm_forward_kernel(const __grid_constant__ NormParams p) {
  __shared__ float red[kReducerFloats];
  Reducer rd{red, p.warps, 0};
  const int threads = 32 * p.warps;
  const int team = threadIdx.x / threads, lane = threadIdx.x - team * threads;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (p.warps == 1 ? kRowsPerCta : 1) + team;
  griddep_wait();
  griddep_launch_dependents();
  if (row >= p.m) return;  // a whole warp, or (wide rows) no thread
  const int n = p.n;
  const bool vec = p.vec != 0;
  const float inv_n = 1.f / static_cast<float>(n);
  const int64_t g = row / p.group;
  const bool ok = WSATTN_BOUNDS(p.status, g < p.groups && threads * V * 8 >= n && p.warps <= 12);
  if (!ok) return;

  Raw8<T> xr[V];
  Raw8<R> rr[V];
#pragma unroll
  for (int j = 0; j < V; ++j)
    xr[j] = load_raw(static_cast<const T*>(p.x) + row * p.ldx, n, column(lane, threads, j), vec);
  if (p.res) {
#pragma unroll
    for (int j = 0; j < V; ++j)
      rr[j] = load_raw(static_cast<const R*>(p.res) + row * p.ldr, n, column(lane, threads, j), vec);
  }
  Pairs h[V];
#pragma unroll
  for (int j = 0; j < V; ++j) unpack(xr[j], h[j]);

  // h becomes std(h); elements behind the row's end stay zero
  auto standardise = [&](int kind) {
    uint64_t t;
    if (kind == WSATTN_NORM_LAYER) {
      t = f2_pack(0.f, 0.f);
#pragma unroll
      for (int j = 0; j < V; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) t = f2_add(t, h[j][i]);
      float2 v = f2_unpack(t);
      float s[1] = {v.x + v.y};
      row_sums(rd, s);
      const float mean = s[0] * inv_n;
      const uint64_t m2 = f2_pack(-mean, -mean);
#pragma unroll
      for (int j = 0; j < V; ++j) {
#pragma unroll
        for (int i = 0; i < 4; ++i) h[j][i] = f2_add(h[j][i], m2);
        trim(h[j], column(lane, threads, j), n);
      }
    }
    t = f2_pack(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) t = f2_fma(h[j][i], h[j][i], t);
    const float2 v = f2_unpack(t);
    float q[1] = {v.x + v.y};
    row_sums(rd, q);
    const float r = rsqrtf(fmaf(q[0], inv_n, p.eps));
    const uint64_t r2 = f2_pack(r, r);
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) h[j][i] = f2_mul(h[j][i], r2);
  };
  auto times = [&](const void* v, int64_t at, int f32) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      Pairs f;
      vector8<T>(v, at, f32, n, column(lane, threads, j), vec, f);
#pragma unroll
      for (int i = 0; i < 4; ++i) h[j][i] = f2_mul(h[j][i], f[i]);
    }
  };

  if (p.post != WSATTN_NORM_NONE) {
    standardise(p.post);
    if (p.post_weight) times(p.post_weight, 0, p.weight_f32);
  }
  if (p.gate) times(p.gate, g * p.ldg, p.mod_f32);
  if (p.res) {
    const uint64_t s2 = f2_pack(p.res_scale, p.res_scale);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      Pairs f;
      unpack(rr[j], f);
#pragma unroll
      for (int i = 0; i < 4; ++i) h[j][i] = f2_fma(s2, f[i], h[j][i]);
    }
  }
  if (p.hidden) {
#pragma unroll
    for (int j = 0; j < V; ++j)
      store8(static_cast<R*>(p.hidden) + row * p.ldh, n, column(lane, threads, j), vec, h[j]);
  }
  if (!p.out) return;
  standardise(p.norm);
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int c = column(lane, threads, j);
    Pairs f;
    if (p.weight) {
      vector8<T>(p.weight, 0, p.weight_f32, n, c, vec, f);
#pragma unroll
      for (int i = 0; i < 4; ++i) h[j][i] = f2_mul(h[j][i], f[i]);
    }
    if (p.bias) {
      vector8<T>(p.bias, 0, p.weight_f32, n, c, vec, f);
#pragma unroll
      for (int i = 0; i < 4; ++i) h[j][i] = f2_add(h[j][i], f[i]);
    }
    if (p.scale) {
      vector8<T>(p.scale, g * p.lds, p.mod_f32, n, c, vec, f);
#pragma unroll
      for (int i = 0; i < 4; ++i) h[j][i] = f2_fma(h[j][i], f[i], h[j][i]);
    }
    if (p.shift) {
      vector8<T>(p.shift, g * p.ldf, p.mod_f32, n, c, vec, f);
#pragma unroll
      for (int i = 0; i < 4; ++i) h[j][i] = f2_add(h[j][i], f[i]);
    }
    store8(static_cast<T*>(p.out) + row * p.ldo, n, c, vec, h[j]);
  }
}

template <typename T, typename R>
cudaError_t forward(const NormParams& p, int v, cudaStream_t s) {
  const int64_t grid = p.warps == 1 ? (p.m + kRowsPerCta - 1) / kRowsPerCta : p.m;
  const dim3 g(static_cast<unsigned>(grid)), b(32 * p.warps * (p.warps == 1 ? kRowsPerCta : 1));
  switch (v) {
    case 1: return launch_dependent(norm_forward_kernel<T, R, 1, 128, 8>, g, b, 0, s, p);
    case 2: return launch_dependent(norm_forward_kernel<T, R, 2, 160, 7>, g, b, 0, s, p);
    default:
      if (p.warps <= 6) return launch_dependent(norm_forward_kernel<T, R, 4, 192, 5>, g, b, 0, s, p);
      return launch_dependent(norm_forward_kernel<T, R, 4, 384, 2>, g, b, 0, s, p);
  }
}

}  // namespace

// A warp a row as long as four pieces a thread hold it; then two pieces a thread
// for CTAs of up to five warps (n = 2048: 72 us against 76, 2560: 90 against 103),
// and four for wider rows (5120: 302 against 309; 4096: the same).
static int norm_forward_width(int n) {
  return n <= 256 ? 1 : n <= 512 ? 2 : n <= 1024 ? 4 : n <= 2560 ? 2 : 4;
}

cudaError_t launch_norm_forward(const NormParams& q, int dtype, bool f32, cudaStream_t s) {
  NormParams p = q;
  const int v = norm_forward_width(p.n);
  p.warps = (p.n + 256 * v - 1) / (256 * v);
  switch (dtype) {
    case WSATTN_BF16:
      return f32 ? forward<__nv_bfloat16, float>(p, v, s) : forward<__nv_bfloat16, __nv_bfloat16>(p, v, s);
    case WSATTN_FP16:
      return f32 ? forward<__half, float>(p, v, s) : forward<__half, __half>(p, v, s);
    default: return forward<float, float>(p, v, s);
  }
}

}  // namespace wsattn
