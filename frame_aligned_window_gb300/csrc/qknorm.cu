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
// head row, 16 elements a lane in two 16-byte pieces, one from each half of
// the head: element e of the first half and e + D/2 then sit in one thread,
// which serves both pair layouts without an exchange.  A lane group keeps one
// token and walks its heads: sine and cosine are formed once for all heads
// of q (or k), the loads of several heads are in flight together, and the
// lane groups of a warp hold neighbouring tokens, so that the packed
// [B, H, N, D] side is written in runs of whole lines.  A launch with few
// tokens splits the heads into groups until every SM has warps.
//
// Angles: pos * (freq / 2 pi) is an fp32 product with its exact error term
// and a second float of the rate; the whole revolutions are dropped before
// the sum is rounded, so the fraction of a turn is good to 2^-25 at any
// position (an fp32 angle at position 70000 would be off by 2^-9).
#include "ops.h"
#include "ptx.cuh"

namespace wsattn {
namespace {

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

__device__ __forceinline__ void words2(uint32_t w, float& lo, float& hi, __nv_bfloat16) {
  lo = __uint_as_float(w << 16);
  hi = __uint_as_float(w & 0xFFFF0000u);
}
__device__ __forceinline__ void words2(uint32_t w, float& lo, float& hi, __half) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
  lo = f.x;
  hi = f.y;
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi, __nv_bfloat16) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi, __half) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ uint32_t elem_bits(float v) { return __float_as_uint(v); }
__device__ __forceinline__ uint32_t elem_bits(__nv_bfloat16 v) { return __bfloat16_as_ushort(v); }
__device__ __forceinline__ uint32_t elem_bits(__half v) { return __half_as_ushort(v); }

// Raw 8-element load; VEC: 16-byte loads, else element by element (rows that
// start on any element).
template <bool VEC>
__device__ __forceinline__ Half8<float> load8(const float* p) {
  Half8<float> r;
  if (VEC) {
    r.a = *reinterpret_cast<const uint4*>(p);
    r.b = *reinterpret_cast<const uint4*>(p + 4);
  } else {
    r.a = make_uint4(elem_bits(p[0]), elem_bits(p[1]), elem_bits(p[2]), elem_bits(p[3]));
    r.b = make_uint4(elem_bits(p[4]), elem_bits(p[5]), elem_bits(p[6]), elem_bits(p[7]));
  }
  return r;
}
template <bool VEC, typename T>
__device__ __forceinline__ Half8<T> load8(const T* p) {
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
  for (int i = 0; i < 4; ++i) words2(w[i], f[2 * i], f[2 * i + 1], T());
}

template <bool VEC>
__device__ __forceinline__ void store8(float* p, const float* f) {
  if (VEC) {
    *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(f[4], f[5], f[6], f[7]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = f[i];
  }
}
template <bool VEC, typename T>
__device__ __forceinline__ void store8(T* p, const float* f) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = pack2(f[2 * i], f[2 * i + 1], T());
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

// The lane's place in its head row and the angles of its eight pairs.
struct Lane {
  int c;        // piece: elements [8c, 8c + 8) of each half of the head
  bool on;      // the lane holds a piece (D / 16 need not be a power of two)
  int half;     // D / 2
};

// Pair i (0..7) of a lane: interleaved, pairs 4c .. 4c+3 of the first half
// and D/4 + 4c .. of the second; split, pairs 8c .. 8c+7.
__device__ __forceinline__ int pair_index(const RotTable& t, const Lane& ln, int i) {
  if (!t.interleaved) return 8 * ln.c + i;
  return (i < 4 ? 0 : ln.half / 2) + 4 * ln.c + (i & 3);
}

__device__ __forceinline__ void lane_angles(const RotTable& t, const Lane& ln, const float* pos,
                                            float sign, float (&cs)[8], float (&sn)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int p = pair_index(t, ln, i);
    const float x = pos[t.axis[p]];
    const float hi = x * t.hi[p];
    const float err = fmaf(x, t.hi[p], -hi);
    const float frac = (hi - rintf(hi)) + fmaf(x, t.lo[p], err);
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

// Sum over the 2^lg lanes of a head row (every lane gets it).
__device__ __forceinline__ float row_sum(float v, int lg) {
  for (int o = 1 << lg >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <typename T>
__device__ __forceinline__ void load_gain(const QkParams& p, const QkPart& part, const Lane& ln,
                                          float (&w)[16]) {
#pragma unroll
  for (int i = 0; i < 16; ++i) w[i] = 1.f;
  if (!part.weight || !ln.on) return;
  for (int i = 0; i < 16; ++i) {
    const int e = (i < 8 ? 0 : ln.half) + 8 * ln.c + (i & 7);
    w[i] = p.weight_f32 ? static_cast<const float*>(part.weight)[e]
                        : static_cast<float>(static_cast<const T*>(part.weight)[e]);
  }
}

// Heads whose loads are in flight together.
template <typename T>
constexpr int kUnroll = sizeof(T) == 4 ? 2 : 4;

template <typename T, bool VEC>
__global__ void __launch_bounds__(kQkThreads) qk_forward_kernel(const __grid_constant__ QkParams p) {
  constexpr int U = kUnroll<T>;
  const int lane = threadIdx.x & 31;
  const int lg = p.lanes_log2;
  Lane ln;
  ln.c = lane & ((1 << lg) - 1);
  ln.half = p.rot.pairs;
  ln.on = 16 * ln.c < 2 * p.rot.pairs;
  const int g = static_cast<int>(blockIdx.x % p.groups);
  const int64_t rb = blockIdx.x / p.groups;
  const int per_warp = 32 >> lg;
  const int64_t row = (rb * (kQkThreads / 32) + threadIdx.x / 32) * per_warp + (lane >> lg);
  const bool active = row < p.rows && ln.on;
  int pi = 0;
  while (pi + 1 < p.parts && g >= p.part[pi + 1].group0) ++pi;
  const QkPart& part = p.part[pi];
  const int h0 = (g - part.group0) * p.group_heads;
  const int h1 = min(part.io.heads, h0 + p.group_heads);
  const int64_t b = active ? row / p.tokens : 0, n = active ? row - b * p.tokens : 0;
  const T* src = static_cast<const T*>(part.io.in) + b * part.io.ib + n * part.io.in_ + 8 * ln.c;
  T* dst = static_cast<T*>(part.io.out) + b * part.io.ob + n * part.io.on + 8 * ln.c;

  float cs[8], sn[8], w[16];
  if (part.turn && active)
    lane_angles(p.rot, ln, p.pos + b * p.pos_b + n * p.rot.axes, static_cast<float>(part.turn), cs,
                sn);
  load_gain<T>(p, part, ln, w);
  const float inv_d = 0.5f / static_cast<float>(p.rot.pairs);

  for (int h = h0; h < h1; h += U) {
    Half8<T> r0[U], r1[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (active && h + u < h1) {
        const T* q = src + (h + u) * part.io.ih;
        r0[u] = load8<VEC>(q);
        r1[u] = load8<VEC>(q + ln.half);
      } else {
        r0[u] = Half8<T>{};
        r1[u] = Half8<T>{};
      }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float x[16];
      unpack8(r0[u], x);
      unpack8(r1[u], x + 8);
      if (part.norm) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) ss = fmaf(x[i], x[i], ss);
        const float r = 1.f / sqrtf(fmaf(row_sum(ss, lg), inv_d, p.eps));
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] *= r * w[i];
      }
      if (part.turn) turn16(x, cs, sn, p.rot.interleaved != 0);
      if (active && h + u < h1) {
        T* q = dst + (h + u) * part.io.oh;
        store8<VEC>(q, x);
        store8<VEC>(q + ln.half, x + 8);
      }
    }
  }
}

// Backward.  Persistent: the work items (rows of one CTA, one head group) of
// q and k form one list, the group the slow index, of which each CTA takes a
// contiguous share; then the same for v's copies.  A CTA's share of the gain
// gradients stays in registers until its part changes, and one partial row
// per CTA and part goes to global memory: the sums have a fixed order.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kQkThreads, kQkBackCtasPerSm)
    qk_backward_kernel(const __grid_constant__ QkParams p) {
  constexpr int U = sizeof(T) == 4 ? 1 : 2;
  __shared__ float red[kQkThreads / 32][2 * kRotMaxPairs];
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  const int lg = p.lanes_log2;
  Lane ln;
  ln.c = lane & ((1 << lg) - 1);
  ln.half = p.rot.pairs;
  ln.on = 16 * ln.c < 2 * p.rot.pairs;
  const int per_warp = 32 >> lg;
  const float inv_d = 0.5f / static_cast<float>(p.rot.pairs);
  const int D = 2 * p.rot.pairs;
  float acc[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) acc[i] = 0.f;

  // adds the CTA's gain gradient of part pi and writes its partial row
  auto flush = [&](int pi) {
    if (!p.dw_part || pi > 1) return;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      for (int o = 1 << lg; o < 32; o <<= 1) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
      if (lane < (1 << lg) && ln.on) red[warp][(i < 8 ? 0 : ln.half) + 8 * ln.c + (i & 7)] = acc[i];
      acc[i] = 0.f;
    }
    __syncthreads();
    float* out = p.dw_part + (static_cast<int64_t>(pi) * gridDim.x + blockIdx.x) * D;
    for (int d = threadIdx.x; d < D; d += kQkThreads) {
      float t = 0.f;
      for (int v = 0; v < kQkThreads / 32; ++v) t += red[v][d];
      out[d] = t;
    }
    __syncthreads();
  };

  // the groups of parts [a, z) share the work of one pass over the list
  auto pass = [&](int a, int z) {
    const int g0 = p.part[a].group0;
    const int64_t items = static_cast<int64_t>(p.part[z - 1].group0 + p.part[z - 1].groups - g0) *
                          p.row_blocks;
    const int64_t i1 = items * (blockIdx.x + 1) / gridDim.x;
    int64_t i = items * blockIdx.x / gridDim.x;
    int pi = a;
    float w[16];
    bool have_w = false;
    for (; i < i1; ++i) {
      const int g = g0 + static_cast<int>(i / p.row_blocks);
      const int64_t rb = i % p.row_blocks;
      while (pi + 1 < z && g >= p.part[pi + 1].group0) {
        flush(pi++);
        have_w = false;
      }
      const QkPart& part = p.part[pi];
      if (!have_w) load_gain<T>(p, part, ln, w);
      have_w = true;
      const int h0 = (g - part.group0) * p.group_heads;
      const int h1 = min(part.io.heads, h0 + p.group_heads);
      const int64_t row = (rb * (kQkThreads / 32) + warp) * per_warp + (lane >> lg);
      const bool active = row < p.rows && ln.on;
      const int64_t b = active ? row / p.tokens : 0, n = active ? row - b * p.tokens : 0;
      const T* gy = static_cast<const T*>(part.io.in) + b * part.io.ib + n * part.io.in_ + 8 * ln.c;
      const T* xs = static_cast<const T*>(part.x) + b * part.xb + n * part.xn + 8 * ln.c;
      T* dx = static_cast<T*>(part.io.out) + b * part.io.ob + n * part.io.on + 8 * ln.c;
      // idle lanes hold zeros and join the row sums: no turn there
      float cs[8] = {}, sn[8] = {};
      if (part.turn && active)
        lane_angles(p.rot, ln, p.pos + b * p.pos_b + n * p.rot.axes,
                    static_cast<float>(part.turn), cs, sn);
      for (int h = h0; h < h1; h += U) {
        Half8<T> g0r[U], g1r[U], x0r[U], x1r[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const bool on = active && h + u < h1;
          g0r[u] = on ? load8<VEC>(gy + (h + u) * part.io.ih) : Half8<T>{};
          g1r[u] = on ? load8<VEC>(gy + (h + u) * part.io.ih + ln.half) : Half8<T>{};
          if (part.norm) {
            x0r[u] = on ? load8<VEC>(xs + (h + u) * part.xh) : Half8<T>{};
            x1r[u] = on ? load8<VEC>(xs + (h + u) * part.xh + ln.half) : Half8<T>{};
          }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const bool on = active && h + u < h1;
          float gr[16];
          unpack8(g0r[u], gr);
          unpack8(g1r[u], gr + 8);
          if (part.turn) turn16(gr, cs, sn, p.rot.interleaved != 0);
          if (part.norm) {
            float x[16];
            unpack8(x0r[u], x);
            unpack8(x1r[u], x + 8);
            float ss = 0.f, dot = 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              ss = fmaf(x[i], x[i], ss);
              dot = fmaf(gr[i] * w[i], x[i], dot);
            }
            // idle lanes and rows hold zeros; an all-zero row keeps r finite
            // through eps, and with eps = 0 its own NaN stays its own
            const float r = 1.f / sqrtf(fmaf(row_sum(ss, lg), inv_d, p.eps));
            const float m = row_sum(dot, lg) * inv_d * r * r;
            if (on) {
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                acc[i] = fmaf(gr[i], x[i] * r, acc[i]);
                gr[i] = r * fmaf(-x[i], m, gr[i] * w[i]);
              }
            }
          }
          if (on) {
            store8<VEC>(dx + (h + u) * part.io.oh, gr);
            store8<VEC>(dx + (h + u) * part.io.oh + ln.half, gr + 8);
          }
        }
      }
    }
    // partial rows of the parts this CTA did not reach are zero
    for (; pi < z; ++pi) flush(pi);
  };
  griddep_launch_dependents();
  pass(0, 2);
  if (p.parts > 2) pass(2, 3);
}

// Gain gradients from the partial rows: CTA (x, y) takes 32 columns of part
// y; thread (c, g) adds rows g, g + 32, ... and the 32 sums are added in order.
__global__ void __launch_bounds__(1024) qk_reduce_gain(const float* __restrict__ parts, int blocks,
                                                       int D, float* dwq, float* dwk) {
  __shared__ float red[32][33];
  griddep_wait();
  const int c = 32 * blockIdx.x + threadIdx.x;
  const float* src = parts + static_cast<int64_t>(blockIdx.y) * blocks * D;
  float t = 0.f;
  if (c < D)
    for (int i = threadIdx.y; i < blocks; i += 32) t += src[static_cast<int64_t>(i) * D + c];
  red[threadIdx.y][threadIdx.x] = t;
  __syncthreads();
  if (threadIdx.y == 0 && c < D) {
    float s = 0.f;
    for (int i = 0; i < 32; ++i) s += red[i][threadIdx.x];
    float* out = blockIdx.y ? dwk : dwq;
    if (out) out[c] = s;
  }
}

template <typename T>
cudaError_t forward_t(const QkParams& p, bool vec, cudaStream_t s) {
  const int64_t grid = p.row_blocks * p.groups;
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  if (vec)
    qk_forward_kernel<T, true><<<static_cast<unsigned>(grid), kQkThreads, 0, s>>>(p);
  else
    qk_forward_kernel<T, false><<<static_cast<unsigned>(grid), kQkThreads, 0, s>>>(p);
  return cudaGetLastError();
}

template <typename T>
cudaError_t backward_t(const QkParams& p, bool vec, int blocks, cudaStream_t s) {
  if (vec)
    qk_backward_kernel<T, true><<<blocks, kQkThreads, 0, s>>>(p);
  else
    qk_backward_kernel<T, false><<<blocks, kQkThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_qk_forward(const QkParams& p, int dtype, bool vec, cudaStream_t s) {
  if (dtype == WSATTN_BF16) return forward_t<__nv_bfloat16>(p, vec, s);
  if (dtype == WSATTN_FP16) return forward_t<__half>(p, vec, s);
  return forward_t<float>(p, vec, s);
}

cudaError_t launch_qk_backward(const QkParams& p, int dtype, bool vec, int blocks, float* dwq,
                               float* dwk, cudaStream_t s) {
  cudaError_t e;
  if (dtype == WSATTN_BF16)
    e = backward_t<__nv_bfloat16>(p, vec, blocks, s);
  else if (dtype == WSATTN_FP16)
    e = backward_t<__half>(p, vec, blocks, s);
  else
    e = backward_t<float>(p, vec, blocks, s);
  if (e != cudaSuccess || !p.dw_part) return e;
  const int D = 2 * p.rot.pairs;
  return launch_dependent(qk_reduce_gain, dim3((D + 31) / 32, 2), dim3(32, 32), 0, s,
                          static_cast<const float*>(p.dw_part), blocks, D, dwq, dwk);
}

}  // namespace wsattn
