// Gradients of a block's norms: how the work is shared, the sums over the shares,
// and the fp32 kernels (norm_back.cuh has the pass over the rows).
#include "norm_back.cuh"

namespace wsattn {
namespace {

using namespace norm;

// Sums over the shares: row y < groups of the grid finishes that group's
// vectors (unless one share held it all), row `groups` the [n] gradients; the
// grid's rows count from `first`.
// Thread (c, k) of a CTA takes column c and shares k, k + 32, ..., and the 32
// sums are added in order.
__global__ void __launch_bounds__(1024) norm_finish_kernel(const __grid_constant__ NormParams p,
                                                           int dtype, int64_t first) {
  __shared__ float red[3][32][33];
  const int n = p.n, c = 32 * blockIdx.x + threadIdx.x;
  const int64_t g = first + blockIdx.y;
  const bool single = g == p.groups;
  griddep_wait();
  int64_t u0 = 0, u1 = p.units - 1;
  const int64_t gs = g * p.group;
  if (!single) {
    if (!p.part) return;
    const int64_t ge = gs + p.group < p.m ? gs + p.group : p.m;
    u0 = share_of(p, gs);
    u1 = share_of(p, ge - 1);
    if (u0 == u1) return;
  } else if (!p.wpart) {
    return;
  }
  float s[3] = {0.f, 0.f, 0.f};
  if (c < n)
    for (int64_t u = u0 + threadIdx.y; u <= u1; u += 4 * 32) {
      float v[4][3];  // four shares' loads in flight
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int64_t ux = u + 32 * x;
        const float* from = single ? p.wpart + ux * 3 * n
                                   : p.part + (ux * 2 + (gs < share_begin(p, ux) ? 0 : 1)) * 3 * n;
#pragma unroll
        for (int k = 0; k < 3; ++k) v[x][k] = ux <= u1 ? from[k * n + c] : 0.f;
      }
#pragma unroll
      for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int k = 0; k < 3; ++k) s[k] += v[x][k];
    }
#pragma unroll
  for (int k = 0; k < 3; ++k) red[k][threadIdx.y][threadIdx.x] = s[k];
  __syncthreads();
  if (threadIdx.y != 0 || c >= n) return;
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    s[k] = 0.f;
    for (int i = 0; i < 32; ++i) s[k] += red[k][i][threadIdx.x];
  }
  if (single) {
    if (p.dweight) p.dweight[c] = s[0];
    if (p.dbias) p.dbias[c] = s[1];
    if (p.dpost) p.dpost[c] = s[2];
    return;
  }
  auto value = [&](const void* v, float other) {
    if (!v) return other;
    if (p.weight_f32) return static_cast<const float*>(v)[c];
    return dtype == WSATTN_BF16 ? to_f32(static_cast<const __nv_bfloat16*>(v)[c])
                                 : to_f32(static_cast<const __half*>(v)[c]);
  };
  if (p.dscale) p.dscale[g * n + c] = fmaf(s[1], value(p.bias, 0.f), s[0] * value(p.weight, 1.f));
  if (p.dshift) p.dshift[g * n + c] = s[1];
  if (p.dgate) p.dgate[g * n + c] = s[2] * value(p.post_weight, 1.f);
}

}  // namespace

int norm_backward_units(int64_t m, int n) {
  const int64_t most = static_cast<int64_t>(kTilingSms) * back_shape(n).per_sm;
  const int64_t want = (m + 3) / 4;  // rows enough to be worth the sums they leave
  return static_cast<int>(want < most ? want : most);
}

cudaError_t launch_norm_backward(const NormParams& p, int dtype, bool f32, cudaStream_t s) {
  cudaError_t e;
  switch (dtype) {
    case WSATTN_BF16: e = norm_backward_bf16(p, f32, s); break;
    case WSATTN_FP16: e = norm_backward_fp16(p, f32, s); break;
    default: e = norm_backward_f32(p, s);
  }
  const bool shared = p.part && !p.whole;
  if (e != cudaSuccess || (!shared && !p.wpart)) return e;
  // where every share ends with a group, only the [n] gradients are left
  const int64_t first = shared ? 0 : p.groups, rows = p.groups - first + (p.wpart ? 1 : 0);
  return launch_dependent(norm_finish_kernel,
                          dim3((p.n + 31) / 32, static_cast<unsigned>(rows)), dim3(32, 32), 0, s, p,
                          dtype, first);
}

cudaError_t norm_backward_f32(const NormParams& p, cudaStream_t s) { return norm::backward<float, float>(p, s); }

}  // namespace wsattn
