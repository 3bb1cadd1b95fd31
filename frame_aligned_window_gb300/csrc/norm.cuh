// Norms of a block: the end of one part (its norm, gate and residual) and the
// start of the next (norm, weight, scale and shift) in one pass over the rows.
//
//   u = x, or std(x) * post_weight             std(t) = (t - mean) r, r = 1 / sqrt(var + eps)
//   h = res_scale * residual + gate * u        (rms: no mean, var = mean of squares)
//   y = (std(h) * weight + bias) (1 + scale) + shift
//
// A row is read once and stays in registers: a thread holds V pieces of eight
// columns, `warps` warps a row.  Means come first and squares of deviations
// after them (two reductions of the row), so that a row whose mean is far from
// zero loses nothing; all of it in fp32, rounded once where it is stored.
#pragma once

#include "epilogue.cuh"

namespace wsattn {
namespace norm {

using namespace ptx;

// Eight columns as raw words.
template <typename T>
struct Raw8 {
  uint4 a;
};
template <>
struct Raw8<float> {
  uint4 a, b;
};

// First column of a thread's piece j: eight neighbours, neighbouring threads
// side by side.
__device__ __forceinline__ int column(int lane, int threads, int j) {
  return 8 * (lane + threads * j);
}

__device__ __forceinline__ uint32_t bits_of(float v) { return __float_as_uint(v); }
__device__ __forceinline__ uint32_t bits_of(__nv_bfloat16 v) { return __bfloat16_as_ushort(v); }
__device__ __forceinline__ uint32_t bits_of(__half v) { return __half_as_ushort(v); }

// Columns c .. c + 7 of a row of n, zeros behind its end; element by element
// where rows do not start on 16 bytes or n is no multiple of eight.
template <typename T>
__device__ __forceinline__ Raw8<T> load_raw(const T* row, int n, int c, bool vec) {
  Raw8<T> r;
  r.a = make_uint4(0, 0, 0, 0);
  if constexpr (sizeof(T) == 4) r.b = r.a;
  if (vec) {
    if (c < n) {
      r.a = *reinterpret_cast<const uint4*>(row + c);
      if constexpr (sizeof(T) == 4) r.b = *reinterpret_cast<const uint4*>(row + c + 4);
    }
  } else {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = c + i < n ? bits_of(row[c + i]) : 0u;
    if constexpr (sizeof(T) == 4) {
      r.a = make_uint4(w[0], w[1], w[2], w[3]);
      r.b = make_uint4(w[4], w[5], w[6], w[7]);
    } else {
      r.a = make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16);
    }
  }
  return r;
}
// Eight columns as four fp32 pairs (the arithmetic is on pairs: half the
// instructions of single values).
typedef uint64_t Pairs[4];
__device__ __forceinline__ void unpack(const Raw8<float>& r, Pairs& f) {
  f[0] = f2_pack(__uint_as_float(r.a.x), __uint_as_float(r.a.y));
  f[1] = f2_pack(__uint_as_float(r.a.z), __uint_as_float(r.a.w));
  f[2] = f2_pack(__uint_as_float(r.b.x), __uint_as_float(r.b.y));
  f[3] = f2_pack(__uint_as_float(r.b.z), __uint_as_float(r.b.w));
}
template <typename T>
__device__ __forceinline__ void unpack(const Raw8<T>& r, Pairs& f) {
  const uint32_t w[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = unpack_pair(w[i], T());
    f[i] = f2_pack(v.x, v.y);
  }
}
__device__ __forceinline__ void fill(Pairs& f, float v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = f2_pack(v, v);
}
// Columns behind the row's end (n) become zero.
__device__ __forceinline__ void trim(Pairs& f, int c, int n) {
  if (c + 8 <= n) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = f2_unpack(f[i]);
    f[i] = f2_pack(c + 2 * i < n ? v.x : 0.f, c + 2 * i + 1 < n ? v.y : 0.f);
  }
}

template <typename T>
__device__ __forceinline__ void store8(T* row, int n, int c, bool vec, const Pairs& f) {
  const float2 a = f2_unpack(f[0]), b = f2_unpack(f[1]), d = f2_unpack(f[2]), e = f2_unpack(f[3]);
  if (vec) {
    if (c >= n) return;
    if constexpr (sizeof(T) == 4) {
      *reinterpret_cast<float4*>(row + c) = make_float4(a.x, a.y, b.x, b.y);
      *reinterpret_cast<float4*>(row + c + 4) = make_float4(d.x, d.y, e.x, e.y);
    } else {
      *reinterpret_cast<uint4*>(row + c) =
          make_uint4(pack_pair(a.x, a.y, T()), pack_pair(b.x, b.y, T()), pack_pair(d.x, d.y, T()),
                     pack_pair(e.x, e.y, T()));
    }
  } else {
    const float v[8] = {a.x, a.y, b.x, b.y, d.x, d.y, e.x, e.y};
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < n) row[c + i] = from_f32<T>(v[i]);
  }
}

// Columns c .. c + 7 of a vector (gate, weight, ...) of fp32 values or of T.
template <typename T>
__device__ __forceinline__ void vector8(const void* v, int64_t at, bool f32, int n, int c, bool vec,
                                        Pairs& f) {
  const float* pf = static_cast<const float*>(v) + at + c;
  const T* pt = static_cast<const T*>(v) + at + c;
  if (!vec) {
    float t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = c + i >= n ? 0.f : f32 ? pf[i] : to_f32(pt[i]);
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = f2_pack(t[2 * i], t[2 * i + 1]);
    return;
  }
  Raw8<float> r;
  r.a = r.b = make_uint4(0, 0, 0, 0);
  if (f32 || sizeof(T) == 4) {
    if (c < n) {
      r.a = *reinterpret_cast<const uint4*>(pf);
      r.b = *reinterpret_cast<const uint4*>(pf + 4);
    }
    unpack(r, f);
  } else {
    Raw8<T> q;
    q.a = r.a;
    if (c < n) q.a = *reinterpret_cast<const uint4*>(pt);
    unpack(q, f);
  }
}

// Sums of K values over a row's warps; every thread gets them.  Two buffers in
// turn: one barrier a reduction.
struct Reducer {
  float* buf;  // [2][kMaxSums][32]
  int warps, parity;
};
constexpr int kMaxSums = 4;
constexpr int kReducerFloats = 2 * kMaxSums * 32;
template <int K>
__device__ __forceinline__ void row_sums(Reducer& r, float (&v)[K]) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
  if (r.warps == 1) return;
  float* b = r.buf + r.parity * kMaxSums * 32;
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  if (lane == 0)
#pragma unroll
    for (int k = 0; k < K; ++k) b[k * 32 + warp] = v[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < K; ++k) {
    v[k] = lane < r.warps ? b[k * 32 + lane] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
  }
  r.parity ^= 1;
}

}  // namespace norm
}  // namespace wsattn
