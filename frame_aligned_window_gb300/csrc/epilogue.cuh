// Activations, 16-bit pairs and what the epilogues of the linear products and
// their gradients share.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ops.h"
#include "ptx.cuh"

namespace wsattn {

// Activations and their slopes in fp32, on the approximate exponential and
// reciprocal of the special-function unit (each within 2^-22 relative, and the
// exponential's argument u within 2^-21 of itself): 2^-18 + 2^-21 |u| relative
// in all, |u| being |z| (silu), z^2 / 2 (gelu) or the tanh form's 2 u; what is
// below 2^-126 counts as zero.  That is far below the rounding of a stored
// 16-bit value, and not above what the product itself is off by in an fp32
// output (two truncations of 2^-23 for each 16 values of the contraction), at a
// third of the instructions of the exact functions, which the epilogue of a
// short contraction would wait for.
//
// logistic(x) = 1 / (1 + exp(-x)), from t = -x log2(e)
__device__ __forceinline__ float logistic_log2(float t) {
  return ptx::rcp_approx(1.f + ptx::ex2_approx(t));
}

// tanh form of gelu: 0.5 z (1 + tanh u) = z logistic(2 u), u = sqrt(2/pi) (z + 0.044715 z^3);
// -2 u log2(e):
__device__ __forceinline__ float gelu_log2(float z, float zz) {
  return z * fmaf(-0.10294323967f, zz, -2.30220819814f);
}

// The normal distribution function, and e = exp(-z^2 / 2), which its density
// shares.  For z <= 0 it is e times (erfc(x) exp(x^2)) / 2 with x = |z| / sqrt 2,
// which a polynomial of degree 7 in t = 1 / (1 + 3 x / 8) without a constant
// term fits with a relative error below 1.2e-6 (least squares, reweighted
// towards the largest error, over x in [0, 9.4]; the first coefficient makes
// the value at 0 exactly 1/2).  So the far negative side, where 1 + erf would
// cancel, keeps its relative precision, at a third of the instructions of
// erff and expf.
__device__ __forceinline__ float normal_cdf(float z, float& e) {
  const float t = ptx::rcp_approx(fmaf(0.26516504294496f, fabsf(z), 1.f));
  e = ptx::ex2_approx(z * z * -0.72134752044448f);
  float h = fmaf(t, -0.06712194532f, 0.192492038f);
  h = fmaf(t, h, -0.06275060028f);
  h = fmaf(t, h, 0.1400828362f);
  h = fmaf(t, h, 0.08388032764f);
  h = fmaf(t, h, 0.1077397019f);
  h = fmaf(t, h, 0.1056776494f);
  h *= t * e;
  return z < 0.f ? h : 1.f - h;
}

template <int ACT>
__device__ __forceinline__ float act_value(float z) {
  if (ACT == WSATTN_ACT_GELU) {
    float e;
    return z * normal_cdf(z, e);
  }
  if (ACT == WSATTN_ACT_GELU_TANH) return z * logistic_log2(gelu_log2(z, z * z));
  if (ACT == WSATTN_ACT_SILU) return z * logistic_log2(z * -1.44269504088896f);
  return z;
}

// Slope for |z| <= 1000 (clamp_pair): beyond, it is 0 or 1 as at the ends.
template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
  if (ACT == WSATTN_ACT_GELU) {
    float e;
    const float c = normal_cdf(z, e);
    return fmaf(z * 0.39894228040143f, e, c);
  }
  if (ACT == WSATTN_ACT_GELU_TANH) {
    const float zz = z * z;
    const float s = logistic_log2(gelu_log2(z, zz));
    return fmaf(s * (1.f - s) * z, fmaf(0.2140644488178f, zz, 1.5957691216057f), s);
  }
  if (ACT == WSATTN_ACT_SILU) {
    const float s = logistic_log2(z * -1.44269504088896f);
    return s * fmaf(z, 1.f - s, 1.f);
  }
  return 1.f;
}

__device__ __forceinline__ float act_any(int act, float z) {
  switch (act) {
    case WSATTN_ACT_GELU: return act_value<WSATTN_ACT_GELU>(z);
    case WSATTN_ACT_GELU_TANH: return act_value<WSATTN_ACT_GELU_TANH>(z);
    case WSATTN_ACT_SILU: return act_value<WSATTN_ACT_SILU>(z);
    default: return z;
  }
}

// 16-bit pairs <-> fp32
__device__ __forceinline__ float2 unpack_pair(uint32_t w, __nv_bfloat16) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ float2 unpack_pair(uint32_t w, __half) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
__device__ __forceinline__ uint32_t pack_pair(float lo, float hi, __nv_bfloat16) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t pack_pair(float lo, float hi, __half) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// Pre-activations held to +-1000 (exact in both types) before their slope is
// taken: past 65504 rounding to fp16 made them infinite where the forward pass
// was finite, and a slope's 0 * infinity would be a NaN.  A NaN stays one.  Two
// at a time: the sums of 21952 x 5120 behind the tanh form take 79 us with it
// and without, 86 when each fp32 value is held by itself.
__device__ __forceinline__ uint32_t clamp_pair(uint32_t w, __nv_bfloat16) {
  const __nv_bfloat162 v = __hmax2_nan(
      __hmin2_nan(*reinterpret_cast<const __nv_bfloat162*>(&w), __float2bfloat162_rn(1000.f)),
      __float2bfloat162_rn(-1000.f));
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t clamp_pair(uint32_t w, __half) {
  const __half2 v =
      __hmax2_nan(__hmin2_nan(*reinterpret_cast<const __half2*>(&w), __float2half2_rn(1000.f)),
                  __float2half2_rn(-1000.f));
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <typename O>
__device__ __forceinline__ O from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

template <typename T>
struct IsHalf {
  static constexpr bool value = false;
};
template <>
struct IsHalf<__half> {
  static constexpr bool value = true;
};

// Waits of these kernels are bounded (about one second); an expired one sets
// a status bit and the CTA's abort flag, and every role then leaves.
constexpr long long kGemmWaitLimit = 1LL << 31;
// The wait for a tile's accumulator spans its contraction, of up to 2^31 values
// (a weight gradient's rows): 32 cycles more for each, of which it takes 10.
// Formed where a wait has become slow: the epilogue has no registers to spare.
__device__ __forceinline__ long long accumulator_limit(int values) {
  return kGemmWaitLimit + (static_cast<long long>(values) << 5);
}

struct GemmShared {
  uint32_t stages;  // shared-memory address of the operand ring
  uint32_t bars;
  volatile int* abort_flag;
  int* status;
};

// Column c of the partial rows, summed in a fixed order (eight interleaved
// sums, loads in flight together, then those in order).
__device__ __forceinline__ float sum_column(const float* part, int64_t ld, int parts, int c) {
  float a[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int i = 0; i < parts; i += 8) {
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = i + j < parts ? part[(i + j) * ld + c] : 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) a[j] += v[j];
  }
  float s = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) s += a[j];
  return s;
}
// Thread `first` of `n` in all takes columns first, first + n, ...
__device__ __forceinline__ void side_sums(const GemmParams& p, int first, int n) {
  if (!p.db) return;
  for (int c = first; c < p.db_cols; c += n) p.db[c] = sum_column(p.part, p.ldpart, p.parts, c);
}

}  // namespace wsattn
