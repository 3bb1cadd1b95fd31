// What the epilogues of the linear products and their gradients share.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ops.h"

namespace wsattn {

// Activations and their slopes in fp32.  The logistic function is formed
// with the fast exponential and division: their error (a few 2^-22 relative)
// is far below the rounding of the stored 16-bit value.
__device__ __forceinline__ float logistic(float x) { return __fdividef(1.f, 1.f + __expf(-x)); }

// tanh form of gelu: 0.5 z (1 + tanh u) = z logistic(2 u), u = sqrt(2/pi) (z + 0.044715 z^3)
__device__ __forceinline__ float gelu_2u(float z) {
  return z * fmaf(0.0713548162726f, z * z, 1.5957691216057f);
}

template <int ACT>
__device__ __forceinline__ float act_value(float z) {
  if (ACT == WSATTN_ACT_GELU) return 0.5f * z * (1.f + erff(z * 0.70710678118655f));
  if (ACT == WSATTN_ACT_GELU_TANH) return z * logistic(gelu_2u(z));
  if (ACT == WSATTN_ACT_SILU) return z * logistic(z);
  return z;
}

template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
  if (ACT == WSATTN_ACT_GELU)
    return fmaf(z * 0.39894228040143f, __expf(-0.5f * z * z),
                0.5f * (1.f + erff(z * 0.70710678118655f)));
  if (ACT == WSATTN_ACT_GELU_TANH) {
    // past |z| = 1000, s (1 - s) is zero: the square is kept finite for it
    const float s = logistic(gelu_2u(z));
    return fmaf(s * (1.f - s) * z, fmaf(0.2140644488178f, fminf(z * z, 1e6f), 1.5957691216057f), s);
  }
  if (ACT == WSATTN_ACT_SILU) {
    const float s = logistic(z);
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

struct GemmShared {
  uint32_t stages;  // shared-memory address of the operand ring
  uint32_t bars;
  volatile int* abort_flag;
  int* status;
};

}  // namespace wsattn
