// Gradients of the attention to an encoder's states.  A warp takes a query, or
// a key.
#include "epilogue.cuh"

namespace wsattn {
namespace {

using namespace ptx;

template <typename T>
__device__ __forceinline__ const T* row_of(const CrossView& v, int64_t b, int64_t h, int64_t i) {
  return static_cast<const T*>(v.data) + b * v.sb + h * v.sh + i * v.sn;
}
__device__ __forceinline__ int keys_of(const CrossParams& p, int b) {
  return p.lengths ? max(0, min(p.lengths[b], p.m)) : p.m;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
template <typename T>
__device__ __forceinline__ void load4(const T* p, int dim, float (&f)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int c = 32 * i + (threadIdx.x & 31);
    f[i] = c < dim ? to_f32(p[c]) : 0.f;
  }
}
template <typename T>
__device__ __forceinline__ void store4(const T* p, int dim, const float (&f)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int c = 32 * i + (threadIdx.x & 31);
    if (c < dim) const_cast<T*>(p)[c] = from_f32<T>(f[i]);
  }
}
__device__ __forceinline__ float dot(const float (&a)[4], const float (&b)[4]) {
  return warp_sum(a[0] * b[0] + a[1] * b[1] + a[2] * b[2] + a[3] * b[3]);
}

template <typename T>
__global__ void __launch_bounds__(128) cross_dq_kernel(const __grid_constant__ CrossParams p) {
  griddep_wait();
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 4 + threadIdx.x / 32;
  if (row >= static_cast<int64_t>(p.batch) * p.heads * p.n) return;
  const int i = static_cast<int>(row % p.n);
  const int h = static_cast<int>(row / p.n % p.heads), b = static_cast<int>(row / p.n / p.heads);
  const int e = h / (p.heads / p.kv_heads), len = keys_of(p, b);
  float q[4], d[4], o[4], dq[4] = {0.f, 0.f, 0.f, 0.f};
  load4(row_of<T>(p.q, b, h, i), p.dim, q);
  load4(row_of<T>(p.dout, b, h, i), p.dim, d);
  load4(row_of<T>(p.o, b, h, i), p.dim, o);
  const float delta = dot(d, o), lse = p.lse[row];
  for (int j = 0; j < len; ++j) {
    float k[4], v[4];
    load4(row_of<T>(p.k, b, e, j), p.dim, k);
    load4(row_of<T>(p.v, b, e, j), p.dim, v);
    const float ds = expf(dot(q, k) * p.scale - lse) * (dot(d, v) - delta) * p.scale;
#pragma unroll
    for (int c = 0; c < 4; ++c) dq[c] += ds * k[c];
  }
  store4(row_of<T>(p.dq, b, h, i), p.dim, dq);
}

template <typename T>
__global__ void __launch_bounds__(128) cross_dkv_kernel(const __grid_constant__ CrossParams p) {
  griddep_wait();
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 4 + threadIdx.x / 32;
  if (row >= static_cast<int64_t>(p.batch) * p.kv_heads * p.m) return;
  const int j = static_cast<int>(row % p.m);
  const int e = static_cast<int>(row / p.m % p.kv_heads), b = static_cast<int>(row / p.m / p.kv_heads);
  const int r = p.heads / p.kv_heads;
  float k[4], v[4], dk[4] = {0.f, 0.f, 0.f, 0.f}, dv[4] = {0.f, 0.f, 0.f, 0.f};
  if (j < keys_of(p, b)) {
    load4(row_of<T>(p.k, b, e, j), p.dim, k);
    load4(row_of<T>(p.v, b, e, j), p.dim, v);
    for (int h = e * r; h < e * r + r; ++h)
      for (int i = 0; i < p.n; ++i) {
        float q[4], d[4], o[4];
        load4(row_of<T>(p.q, b, h, i), p.dim, q);
        load4(row_of<T>(p.dout, b, h, i), p.dim, d);
        load4(row_of<T>(p.o, b, h, i), p.dim, o);
        const float w = expf(dot(q, k) * p.scale - p.lse[(static_cast<int64_t>(b) * p.heads + h) * p.n + i]);
        const float ds = w * (dot(d, v) - dot(d, o)) * p.scale;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          dk[c] += ds * q[c];
          dv[c] += w * d[c];
        }
      }
  }
  if (p.dk.data) store4(row_of<T>(p.dk, b, e, j), p.dim, dk);
  if (p.dv.data) store4(row_of<T>(p.dv, b, e, j), p.dim, dv);
}

template <typename F>
cudaError_t by_rows(F* kernel, const CrossParams& p, int64_t rows, cudaStream_t s) {
  return launch_dependent(kernel, dim3(static_cast<unsigned>((rows + 3) / 4)), dim3(128), 0, s, p);
}

}  // namespace

cudaError_t launch_cross_backward(const CrossParams& p, int dtype, cudaStream_t s) {
  const int64_t rows = static_cast<int64_t>(p.batch) * p.heads * p.n;
  const int64_t keys = static_cast<int64_t>(p.batch) * p.kv_heads * p.m;
  cudaError_t e = cudaSuccess;
  if (p.dq.data && rows)
    e = dtype == WSATTN_BF16 ? by_rows(cross_dq_kernel<__nv_bfloat16>, p, rows, s)
                             : by_rows(cross_dq_kernel<__half>, p, rows, s);
  if (e != cudaSuccess || !keys || (!p.dk.data && !p.dv.data)) return e;
  return dtype == WSATTN_BF16 ? by_rows(cross_dkv_kernel<__nv_bfloat16>, p, keys, s)
                              : by_rows(cross_dkv_kernel<__half>, p, keys, s);
}

}  // namespace wsattn
