// What the argument checks of the operators share: alignment, types and
// [batch, heads, N, head_dim] views.
#pragma once

#include <cstdint>

#include "ops.h"

namespace wsattn {
namespace args {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int64_t round8(int64_t a) { return (a + 7) / 8 * 8; }
inline size_t up256(size_t x) { return (x + 255) / 256 * 256; }
inline int dtype_size(int dtype) { return dtype == WSATTN_FP32 ? 4 : 2; }
inline bool dtype_ok(int dtype) { return dtype >= WSATTN_BF16 && dtype <= WSATTN_FP32; }

inline bool half_type(int dtype) { return dtype == WSATTN_BF16 || dtype == WSATTN_FP16; }
inline bool elem_aligned(const void* p, int esize) {
  return (reinterpret_cast<uintptr_t>(p) & static_cast<uintptr_t>(esize - 1)) == 0;
}

inline int sm_count() {
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
inline bool apart(const wsattn_heads* v, int batch, int64_t n, int dim) {
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

inline bool view_ok(const wsattn_heads* v, int esize) {
  if (!v || v->heads < 1 || v->stride_b < 0 || v->stride_h < 0 || v->stride_n < 0) return false;
  return (reinterpret_cast<uintptr_t>(v->data) & static_cast<uintptr_t>(esize - 1)) == 0;
}

// Every row of the view starts on a 16-byte boundary.
inline bool view_vec(const wsattn_heads* v, int batch, int64_t n, int esize) {
  const int64_t per = 16 / esize;
  return aligned16(v->data) && (batch <= 1 || v->stride_b % per == 0) &&
         (v->heads <= 1 || v->stride_h % per == 0) && (n <= 1 || v->stride_n % per == 0);
}

}  // namespace args
}  // namespace wsattn
