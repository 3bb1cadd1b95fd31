// Rotary positions on several axes, alone or in one pass with the per-head
// RMS norm of queries and keys, and their gradients.
//
//   forward   y = R_a (g * x r),          r = 1 / sqrt(mean_d x_d^2 + eps)
//   backward  h = R_-a dy,  u = g * h,  xh = x r
//             dx = r (u - xh mean_d(u xh)),   dg = sum over rows of h * xh
//
// R_a turns pair p of a head by a_p = pos[axis(p)] * freq(p).  The norm and
// the gain act on a whole head row and the turn on pairs of it, so one read
// of x and one write of y is all the traffic there has to be: the passes are
// bound by HBM (the angles come from the positions, 4 bytes per token and
// axis, not from a table of D values per token).
//
// Work split: 2^l lanes (the least power of two that covers D / 16) hold one
// head row, 16 elements a lane in 16-byte pieces, the same ones of each half
// of the head: element e of the first half and e + D/2 then sit in one thread,
// which serves both pair layouts without an exchange.  A lane group keeps one
// token and walks its heads: sine and cosine are formed once for all heads
// of q (or k), the loads of several heads are in flight together, and the
// lane groups of a warp hold neighbouring tokens, so that the packed
// [B, H, N, D] side is written in runs of whole lines.  A launch with few
// tokens splits the heads into groups until every SM has warps.
//
// Angles: pos * (freq / 2 pi) is an fp32 product with its exact error term
// and a second float of the rate; the whole revolutions are dropped before
// the sum is rounded.  That rounding is 2^-25 of a turn at most.  What grows
// with the angle of t turns: the rate's second float is off by 2^-48 |t|, the
// sum of error term and second product (2^-23 |t| in size) by 2^-47 |t|, the
// rate in 64 bits by 2^-52 |t|; together below 2^-46 |t| (2^-32 of a turn at
// position 70000 and one radian a step, where an fp32 angle would be off by
// 2^-9 radians).  Measured up to 2^47 turns: 2^-48 |t|.
#pragma once

#include "epilogue.cuh"

namespace wsattn {
namespace qk {

using namespace ptx;

template <typename T>
struct Half8;  // 8 elements as raw words
template <>
struct Half8<float> {
  uint4 a, b;
};
template <>
struct Half8<__nv_bfloat16> {
  uint4 a;
};
template <>
struct Half8<__half> {
  uint4 a;
};

__device__ __forceinline__ uint32_t elem_bits(float v) { return __float_as_uint(v); }
__device__ __forceinline__ uint32_t elem_bits(__nv_bfloat16 v) { return __bfloat16_as_ushort(v); }
__device__ __forceinline__ uint32_t elem_bits(__half v) { return __half_as_ushort(v); }

// Raw 8-element load; VEC: 16-byte loads, else element by element (rows that
// start on any element).
template <bool VEC>
__device__ __forceinline__ Half8<float> load8(const float* p, int step) {
  const float* q = p + step;
  Half8<float> r;
  if (VEC) {
    r.a = *reinterpret_cast<const uint4*>(p);
    r.b = *reinterpret_cast<const uint4*>(q);
  } else {
    r.a = make_uint4(elem_bits(p[0]), elem_bits(p[1]), elem_bits(p[2]), elem_bits(p[3]));
    r.b = make_uint4(elem_bits(q[0]), elem_bits(q[1]), elem_bits(q[2]), elem_bits(q[3]));
  }
  return r;
}
template <bool VEC, typename T>
__device__ __forceinline__ Half8<T> load8(const T* p, int) {
  Half8<T> r;
  if (VEC) {
    r.a = *reinterpret_cast<const uint4*>(p);
  } else {
    r.a = make_uint4(elem_bits(p[0]) | elem_bits(p[1]) << 16, elem_bits(p[2]) | elem_bits(p[3]) << 16,
                     elem_bits(p[4]) | elem_bits(p[5]) << 16, elem_bits(p[6]) | elem_bits(p[7]) << 16);
  }
  return r;
}

__device__ __forceinline__ void unpack8(const Half8<float>& r, float* f) {
  const uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i]);
}
template <typename T>
__device__ __forceinline__ void unpack8(const Half8<T>& r, float* f) {
  const uint32_t w[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = unpack_pair(w[i], T());
    f[2 * i] = v.x;
    f[2 * i + 1] = v.y;
  }
}

template <bool VEC>
__device__ __forceinline__ void store8(float* p, int step, const float* f) {
  float* q = p + step;
  if (VEC) {
    *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
    *reinterpret_cast<float4*>(q) = make_float4(f[4], f[5], f[6], f[7]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = f[i];
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = f[4 + i];
  }
}
template <bool VEC, typename T>
__device__ __forceinline__ void store8(T* p, int, const float* f) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = pack_pair(f[2 * i], f[2 * i + 1], T());
  if (VEC) {
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    uint16_t* u = reinterpret_cast<uint16_t*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      u[2 * i] = static_cast<uint16_t>(w[i]);
      u[2 * i + 1] = static_cast<uint16_t>(w[i] >> 16);
    }
  }
}

// The lane's place in its head row: eight elements of each half of the head,
// in 16 bits elements [8c, 8c + 8), in fp32 [4c, 4c + 4) of the half's first
// half and of its second (either way neighbouring lanes touch neighbouring
// 16 bytes).
struct Lane {
  int c;
  bool on;   // the lane holds a piece (D / 16 need not be a power of two)
  int half;  // D / 2
  int off;   // its first element
  int step;  // fp32: from its first four elements to its second
};

template <typename T, int LG>
__device__ __forceinline__ Lane make_lane(const RotTable& t) {
  Lane ln;
  ln.c = threadIdx.x & ((1 << LG) - 1);
  ln.half = t.pairs;
  ln.on = 16 * ln.c < 2 * t.pairs;
  ln.off = (sizeof(T) == 4 ? 4 : 8) * ln.c;
  ln.step = t.pairs / 2;
  return ln;
}
// Element (of the head) that the lane's i-th value is.
template <typename T>
__device__ __forceinline__ int lane_element(const Lane& ln, int i) {
  const int in_half = sizeof(T) == 4 ? (i & 4 ? ln.step : 0) + (i & 3) : i & 7;
  return (i < 8 ? 0 : ln.half) + ln.off + in_half;
}

// Row (of B * N) -> batch element and token.
__device__ __forceinline__ void split_row(const QkParams& p, int64_t row, int64_t& b, int64_t& n) {
  if (p.rows <= INT32_MAX) {
    const uint32_t q = static_cast<uint32_t>(row) / static_cast<uint32_t>(p.tokens);
    b = q;
    n = static_cast<uint32_t>(row) - q * static_cast<uint32_t>(p.tokens);
  } else {
    b = row / p.tokens;
    n = row - b * p.tokens;
  }
}

// The rates of a lane's eight pairs, in the order in which turn16 takes them.
// They are read from the kernel's parameters through generic addresses:
// indexed reads of constant memory would go lane by lane.
struct Rates {
  float hi[8], lo[8];
  uint32_t axis[8];
};
// N consecutive pairs from p0 on
template <int N>
__device__ __forceinline__ void read_rates(const RotTable* g, int p0, float* hi, float* lo,
                                           uint32_t* axis) {
  if constexpr (N == 4) {
    const float4 h = *reinterpret_cast<const float4*>(g->hi + p0);
    const float4 l = *reinterpret_cast<const float4*>(g->lo + p0);
    const uint32_t a = *reinterpret_cast<const uint32_t*>(g->axis + p0);
    hi[0] = h.x, hi[1] = h.y, hi[2] = h.z, hi[3] = h.w;
    lo[0] = l.x, lo[1] = l.y, lo[2] = l.z, lo[3] = l.w;
#pragma unroll
    for (int i = 0; i < 4; ++i) axis[i] = a >> (8 * i) & 255u;
  } else {
    const float2 h = *reinterpret_cast<const float2*>(g->hi + p0);
    const float2 l = *reinterpret_cast<const float2*>(g->lo + p0);
    const uint32_t a = *reinterpret_cast<const uint16_t*>(g->axis + p0);
    hi[0] = h.x, hi[1] = h.y;
    lo[0] = l.x, lo[1] = l.y;
    axis[0] = a & 255u, axis[1] = a >> 8;
  }
}
template <typename T>
__device__ __forceinline__ Rates lane_rates(const RotTable& t, const Lane& ln) {
  const RotTable* g = &t;
  asm volatile("" : "+l"(g));  // an address like any other from here on
  Rates r;
  if (!t.interleaved) {  // pair e: elements e and e + D / 2
    const int second = sizeof(T) == 4 ? ln.off + ln.step : ln.off + 4;
    read_rates<4>(g, ln.off, r.hi, r.lo, r.axis);
    read_rates<4>(g, second, r.hi + 4, r.lo + 4, r.axis + 4);
  } else if constexpr (sizeof(T) == 4) {  // pair e / 2: elements e and e + 1
#pragma unroll
    for (int k = 0; k < 4; ++k)
      read_rates<2>(g, (ln.off + k * ln.step) / 2, r.hi + 2 * k, r.lo + 2 * k, r.axis + 2 * k);
  } else {
    read_rates<4>(g, ln.off / 2, r.hi, r.lo, r.axis);
    read_rates<4>(g, (ln.half + ln.off) / 2, r.hi + 4, r.lo + 4, r.axis + 4);
  }
  return r;
}

template <typename T>
__device__ __forceinline__ void lane_angles(const RotTable& t, const Lane& ln, const float* pos,
                                            float sign, float (&cs)[8], float (&sn)[8]) {
  float x[kRotMaxAxes];
#pragma unroll
  for (int a = 0; a < kRotMaxAxes; ++a) x[a] = a < t.axes ? pos[a] : 0.f;
  const Rates r = lane_rates<T>(t, ln);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float w = r.hi[i], wl = r.lo[i];
    const uint32_t a = r.axis[i];
    const float v = a < 2 ? (a == 0 ? x[0] : x[1]) : (a == 2 ? x[2] : x[3]);
    const float hi = v * w;
    const float err = fmaf(v, w, -hi);
    const float frac = (hi - rintf(hi)) + fmaf(v, wl, err);
    float s, c;
    sincospif(2.f * frac, &s, &c);
    cs[i] = c;
    sn[i] = sign * s;
  }
}

// Turns the lane's 16 elements (x: 8 of each half) in place.
__device__ __forceinline__ void turn16(float (&x)[16], const float (&cs)[8], const float (&sn)[8],
                                       bool interleaved) {
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = x[2 * i], b = x[2 * i + 1];
      x[2 * i] = fmaf(a, cs[i], -b * sn[i]);
      x[2 * i + 1] = fmaf(a, sn[i], b * cs[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = x[i], b = x[8 + i];
      x[i] = fmaf(a, cs[i], -b * sn[i]);
      x[8 + i] = fmaf(a, sn[i], b * cs[i]);
    }
  }
}

// Sum over the 2^LG lanes of a head row (every lane gets it).
template <int LG>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = 1 << LG >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The lane's gains, from E values laid out as its T elements are.
template <typename E, typename T>
__device__ __forceinline__ void gain16(const void* weight, const Lane& ln, float (&w)[16]) {
  const E* g = static_cast<const E*>(weight) + ln.off;
  // fp32 gains of 16-bit heads: eight in a row
  const int step = sizeof(T) == 4 ? ln.step : 4;
  if ((reinterpret_cast<uintptr_t>(weight) & 15u) == 0) {
    unpack8(load8<true>(g, step), w);
    unpack8(load8<true>(g + ln.half, step), w + 8);
  } else {
    unpack8(load8<false>(g, step), w);
    unpack8(load8<false>(g + ln.half, step), w + 8);
  }
}
template <typename T>
__device__ __forceinline__ void load_gain(const QkParams& p, const QkPart& part, const Lane& ln,
                                          float (&w)[16]) {
#pragma unroll
  for (int i = 0; i < 16; ++i) w[i] = 1.f;
  if (!part.weight || !ln.on) return;
  if (p.weight_f32) gain16<float, T>(part.weight, ln, w);
  else gain16<T, T>(part.weight, ln, w);
}

template <bool VEC>
__device__ __forceinline__ void store_raw8(float* p, int step, const Half8<float>& r) {
  float f[8];
  unpack8(r, f);
  store8<VEC>(p, step, f);
}
template <bool VEC, typename T>
__device__ __forceinline__ void store_raw8(T* p, int, const Half8<T>& r) {
  if (VEC) {
    *reinterpret_cast<uint4*>(p) = r.a;
  } else {
    const uint32_t w[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
    uint16_t* u = reinterpret_cast<uint16_t*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      u[2 * i] = static_cast<uint16_t>(w[i]);
      u[2 * i + 1] = static_cast<uint16_t>(w[i] >> 16);
    }
  }
}

// Copies a lane's share of `heads` head rows (v: neither norm nor turn).
template <typename T, bool VEC>
__device__ __forceinline__ void copy_heads(const T* src, int64_t sstep, T* dst, int64_t dstep,
                                           int heads, const Lane& ln) {
  constexpr int U = sizeof(T) == 4 ? 2 : 4;
  for (int h = 0; h < heads; h += U) {
    Half8<T> r0[U], r1[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (h + u < heads) {
        r0[u] = load8<VEC>(src + u * sstep, ln.step);
        r1[u] = load8<VEC>(src + u * sstep + ln.half, ln.step);
      }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (h + u < heads) {
        store_raw8<VEC>(dst + u * dstep, ln.step, r0[u]);
        store_raw8<VEC>(dst + u * dstep + ln.half, ln.step, r1[u]);
      }
    src += U * sstep;
    dst += U * dstep;
  }
}

// Calls F<T, VEC, LG> for the lanes of a head row.
#define WSATTN_BY_LANES(F, T, VEC)                  \
  switch (p.lanes_log2) {                           \
    case 0: return F<T, VEC, 0>(p, grid, s);        \
    case 1: return F<T, VEC, 1>(p, grid, s);        \
    case 2: return F<T, VEC, 2>(p, grid, s);        \
    case 3: return F<T, VEC, 3>(p, grid, s);        \
    default: return F<T, VEC, 4>(p, grid, s);       \
  }

}  // namespace qk
}  // namespace wsattn
